// Attention to states of another length in fp32, forward and backward, on
// mma.sync: tiles of 64 rows x 64 keys, a warp 16 rows (dk, dv: 16 keys).
//
// A factor is split into the nearest tf32 number and the rest, and a product taken
// as three (high x high, high x low, low x high), which leaves 2^-22 of each term;
// sums are fp32.  Logits come out of the product in the layout in which the next
// one takes its left operand, if that one's k index tig (tig + 4) stands for column
// 2 tig (2 tig + 1): nothing passes shared memory but the tiles.  What bounds it is
// the issue of the splits and of the reads of right operands (about 2.5
// instructions beside each matrix instruction) and, where there is one tile an SM, the
// chain from one to the next.  (On the fp32 units, with 16 sums a thread, a backward pass
// of 2 x 8 / 2 heads, 333 x 1000 ragged rows, took 158 us, so 78; a forward pass of
// 4 x 4 heads, 37 x 777, 19.7 and 14.8.)
#include "sfa_cross.cuh"

namespace sfa {

constexpr int kTileN = kF32Tile;
constexpr int kPitch = 68;  // floats a line: lines 4 banks apart, so both reads of right operands are free of conflicts
constexpr int kThreads32 = 128;

// A number of infinite or overflowing products: split, its parts' products are
// infinities of either sign.  Below it sums of 64 products stay finite.
__device__ __forceinline__ bool huge(float x) { return fabsf(x) >= 0x1p60f; }

struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
  Split s;
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(s.hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(s.lo) : "f"(x - __uint_as_float(s.hi)));
  return s;
}
__device__ __forceinline__ void mma_tf32(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Left operand of 16 rows x 64 dims: row gid and gid + 8, dims tig + 4 i.
struct Left {
  static constexpr int kUnroll = 8;
  float x[2][16];
  // rows: those of this lane, nullptr for zeros
  __device__ __forceinline__ void load(const float* lo, const float* hi, int tig) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[0][i] = lo ? lo[tig + 4 * i] : 0.0f;
      x[1][i] = hi ? hi[tig + 4 * i] : 0.0f;
    }
  }
  __device__ __forceinline__ bool plain() const {
    bool y = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) y |= huge(x[0][i]) || huge(x[1][i]);
    return y;
  }
  // step s: rows gid, gid + 8 of k tig, then of k tig + 4
  __device__ __forceinline__ void step(int s, Split* a) const {
    a[0] = split(x[0][2 * s]);
    a[1] = split(x[1][2 * s]);
    a[2] = split(x[0][2 * s + 1]);
    a[3] = split(x[1][2 * s + 1]);
  }
};
// The same in a tile, from row `row` of it on.
struct LeftTile {
  static constexpr int kUnroll = 2;
  const float* at;
  __device__ __forceinline__ LeftTile(const float* tile, int row, int gid, int tig) : at(tile + (row + gid) * kPitch + tig) {}
  __device__ __forceinline__ void step(int s, Split* a) const {
    a[0] = split(at[8 * s]);
    a[1] = split(at[8 * kPitch + 8 * s]);
    a[2] = split(at[8 * s + 4]);
    a[3] = split(at[8 * kPitch + 8 * s + 4]);
  }
};

// c[n] = this warp's 16 rows times rows 8 n + .. of a tile (N of them from n0 on).
// High parts and the rest are added up apart, so that two short chains run side by side.
template <int N, typename L>
__device__ __forceinline__ void rows_product(float (*c)[4], const L& q, const float* tile, int n0, int gid, int tig) {
  float d[N][4];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] = d[n][e] = 0.0f;
#pragma unroll L::kUnroll
  for (int s = 0; s < 8; ++s) {
    Split a[4], b[N][2];
    q.step(s, a);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float* const row = tile + (8 * (n0 + n) + gid) * kPitch + 8 * s + tig;
      b[n][0] = split(row[0]);
      b[n][1] = split(row[4]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(c[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[n][0].hi, b[n][1].hi);
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(d[n], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[n][0].hi, b[n][1].hi);
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(d[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[n][0].lo, b[n][1].lo);
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] += d[n][e];
}
// o[j] += p (16 rows x rows 8 n + .. of a tile, as a product left it) times those rows'
// dims 8 j + ...  Each such product is added by itself: the matrix unit cuts its sums off
// where an addition rounds, which over a thousand rows would show (2e-6).
__device__ __forceinline__ void dims_product(float (*o)[4], const float* p, const float* tile, int n, int gid, int tig) {
  const Split a[4] = {split(p[0]), split(p[2]), split(p[1]), split(p[3])};
  const float* const row = tile + (8 * n + 2 * tig) * kPitch + gid;
#pragma unroll
  for (int j0 = 0; j0 < 8; j0 += 4) {
    Split b[4][2];
    float t[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b[j][0] = split(row[8 * (j0 + j)]);
      b[j][1] = split(row[kPitch + 8 * (j0 + j)]);
      t[j][0] = t[j][1] = t[j][2] = t[j][3] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) mma_tf32(t[j], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[j][0].hi, b[j][1].hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) mma_tf32(t[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].lo, b[j][1].lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) mma_tf32(t[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].hi, b[j][1].hi);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j0 + j][e] += t[j][e];
  }
}

// Tiles that hold huge numbers are multiplied as they are, by the following two.
// c[n] as rows_product's, of left(h, d): this lane's row gid (h = 0) or gid + 8, dim d.
template <int N, typename F>
__device__ __forceinline__ void rows_plain(float (*c)[4], const F& left, const float* tile, int n0, int tig) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* const row = tile + (8 * (n0 + n) + 2 * tig + (e & 1)) * kPitch;
      float y = 0.0f;
#pragma unroll 1
      for (int d = 0; d < kD; ++d) y = fmaf(left(e >> 1, d), row[d], y);
      c[n][e] = y;
    }
}
// o += as dims_product's.
__device__ __forceinline__ void dims_plain(float (*o)[4], const float* p, const float* tile, int n, int gid, int tig) {
#pragma unroll 1
  for (int key = 0; key < 8; ++key) {
    const int from = 4 * gid + (key >> 1);
    const float lo = __shfl_sync(0xffffffffu, key & 1 ? p[1] : p[0], from), hi = __shfl_sync(0xffffffffu, key & 1 ? p[3] : p[2], from);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = fmaf(e < 2 ? lo : hi, tile[(8 * n + key) * kPitch + 8 * c + 2 * tig + (e & 1)], o[c][e]);
  }
}

// 64 rows into a tile: row(r) gives row r's address, or nullptr for zeros.  Sixteen
// lanes a row.  Whether this thread met a huge number.
template <typename F>
__device__ __forceinline__ bool load_tile(float* tile, const F& row) {
  const int c = (threadIdx.x & 15) * 4;
  bool plain = false;
#pragma unroll
  for (int r = threadIdx.x >> 4; r < kTileN; r += kThreads32 / 16) {
    const float* const p = row(r);
    const float4 x = p ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    plain |= huge(x.x) || huge(x.y) || huge(x.z) || huge(x.w);
    *reinterpret_cast<float4*>(tile + r * kPitch + c) = x;
  }
  return plain;
}

// ---- forward: a CTA has 64 rows of a (sequence, KV head) and a split of its keys
__global__ void __launch_bounds__(kThreads32) cross_fwd_kernel(const CrossArgs a) {
  __shared__ __align__(16) float Ks[kTileN * kPitch];
  __shared__ __align__(16) float Vs[kTileN * kPitch];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int rows = a.G * a.Tq, tiles = (rows + kTileN - 1) / kTileN;
  uint32_t x = blockIdx.x;
  const int s = x % a.splits;
  x /= a.splits;
  const int r0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = x % a.Hkv, b = x / a.Hkv;
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kF32Keys, a.splits, s, k0, k1);
  if (r0 >= (int64_t)nq * a.G) k1 = k0;  // no query in the tile
  auto query = [&](int h) {
    const int r = r0 + 16 * warp + gid + 8 * h, t = r / a.G, head = kvh * a.G + (r - t * a.G);
    return r < rows && t < nq ? static_cast<const float*>(a.q) + b * a.qs.b + head * a.qs.h + t * a.qs.t : nullptr;
  };
  auto query_dim = [&](int h, int d) {
    const float* const row = query(h);
    return row ? row[d] : 0.0f;
  };
  Left q;
  q.load(query(0), query(1), tig);
  const bool q_plain = q.plain();
  const float* const kp = static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h;
  const float* const vp = static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h;
  float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // of rows gid, gid + 8 (l: this lane's keys)
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
  for (int j0 = k0; j0 < k1; j0 += kTileN) {
    __syncthreads();  // the last tile has been read
    bool plain = load_tile(Ks, [&](int r) { return j0 + r < k1 ? kp + (int64_t)(j0 + r) * a.ks.t : nullptr; });
    plain |= load_tile(Vs, [&](int r) { return j0 + r < k1 ? vp + (int64_t)(j0 + r) * a.vs.t : nullptr; });
    plain = __syncthreads_or(plain || q_plain);
    // 32 keys at a time, in a loop: where there are few tiles, fetching this code costs as
    // much as running it
#pragma unroll 1
    for (int n0 = 0; n0 < kTileN / 8 && j0 + 8 * n0 < k1; n0 += kF32Keys / 8) {
      float p[4][4];
      if (plain)
        rows_plain<4>(p, query_dim, Ks, n0, tig);
      else
        rows_product<4>(p, q, Ks, n0, gid, tig);
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[n][e] = j0 + 8 * (n0 + n) + 2 * tig + (e & 1) < k1 ? p[n][e] * kLogitScale : -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], p[n][e]);
        }
      float sh[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const float to = fmaxf(m[h], top[h]);
        sh[h] = shift_of(to);
        const float corr = exp2f(m[h] - sh[h]);  // 0 on the first keys
        m[h] = to;
        l[h] *= corr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][2 * h] *= corr;
          o[j][2 * h + 1] *= corr;
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[n][e] = exp2f(p[n][e] - sh[e >> 1]);
          l[e >> 1] += p[n][e];
        }
        if (plain)
          dims_plain(o, p[n], Vs, n0 + n, gid, tig);
        else
          dims_product(o, p[n], Vs, n0 + n, gid, tig);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const int r = r0 + 16 * warp + gid + 8 * h;
    if (r >= rows) continue;
    const bool none = k1 <= k0 || r / a.G >= nq;
    const int64_t row = a.row(b, kvh, r);
    if (a.parts) {
      const int64_t at = s * a.rows + row;
      if (!none)
#pragma unroll
        for (int j = 0; j < 8; ++j) store2(a.part_o + at * kD + 8 * j + 2 * tig, o[j][2 * h], o[j][2 * h + 1]);
      if (tig == 0) a.part_ml[at] = none ? make_float2(-INFINITY, -1.0f) : make_float2(m[h], l[h]);
    } else {
      const float inv = 1.0f / l[h];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        store2(static_cast<float*>(a.o) + row * kD + 8 * j + 2 * tig, none ? 0.0f : o[j][2 * h] * inv, none ? 0.0f : o[j][2 * h + 1] * inv);
      if (a.lse && tig == 0) a.lse[row] = none ? -INFINITY : (m[h] + log2f(l[h])) * kLn2;
    }
  }
}

// ---- backward
// dq: a CTA has 64 rows and a split of their keys.
//   ds = p (dO v - delta), dq = sum ds k / 8
__device__ __forceinline__ void cross_dq(const CrossArgs& a, float* sm, uint32_t x) {
  float *const Ks = sm, *const Vs = sm + kTileN * kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int rows = a.G * a.Tq, tiles = (rows + kTileN - 1) / kTileN;
  const int s = x % a.splits;
  x /= a.splits;
  const int r0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = x % a.Hkv, b = x / a.Hkv;
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kTileN, a.splits, s, k0, k1);
  if (r0 >= (int64_t)nq * a.G) k1 = k0;
  auto query = [&](int h) {
    const int r = r0 + 16 * warp + gid + 8 * h, t = r / a.G, head = kvh * a.G + (r - t * a.G);
    return r < rows && t < nq ? static_cast<const float*>(a.q) + b * a.qs.b + head * a.qs.h + t * a.qs.t : nullptr;
  };
  auto grad = [&](int h) {
    const int r = r0 + 16 * warp + gid + 8 * h;
    return r < rows && r / a.G < nq ? static_cast<const float*>(a.dO) + a.row(b, kvh, r) * kD : nullptr;
  };
  auto query_dim = [&](int h, int d) {
    const float* const row = query(h);
    return row ? row[d] : 0.0f;
  };
  auto grad_dim = [&](int h, int d) {
    const float* const row = grad(h);
    return row ? row[d] : 0.0f;
  };
  Left q, g;
  q.load(query(0), query(1), tig);
  g.load(grad(0), grad(1), tig);
  const bool q_plain = q.plain() || g.plain();
  float2 st[2];
  bool counts[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * warp + gid + 8 * h;
    counts[h] = r < rows && r / a.G < nq;
    st[h] = counts[h] ? a.stat[a.row(b, kvh, r)] : make_float2(0.0f, 0.0f);
  }
  const float* const kp = static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h;
  const float* const vp = static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h;
  float dq[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) dq[j][e] = 0.0f;
  for (int j0 = k0; j0 < k1; j0 += kTileN) {
    __syncthreads();
    bool plain = load_tile(Ks, [&](int r) { return j0 + r < k1 ? kp + (int64_t)(j0 + r) * a.ks.t : nullptr; });
    plain |= load_tile(Vs, [&](int r) { return j0 + r < k1 ? vp + (int64_t)(j0 + r) * a.vs.t : nullptr; });
    plain = __syncthreads_or(plain || q_plain);
#pragma unroll 1
    for (int n = 0; n < 8; n += 2) {
      float p[2][4], dp[2][4];
      if (plain) {
        rows_plain<2>(p, query_dim, Ks, n, tig);
        rows_plain<2>(dp, grad_dim, Vs, n, tig);
      } else {
        rows_product<2>(p, q, Ks, n, gid, tig);
        rows_product<2>(dp, g, Vs, n, gid, tig);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool there = j0 + 8 * (n + i) + 2 * tig + (e & 1) < k1 && counts[e >> 1];
          p[i][e] = there ? exp2f(fmaf(p[i][e], kLogitScale, -st[e >> 1].x)) * (dp[i][e] - st[e >> 1].y) : 0.0f;
        }
        if (plain)
          dims_plain(dq, p[i], Ks, n + i, gid, tig);
        else
          dims_product(dq, p[i], Ks, n + i, gid, tig);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * warp + gid + 8 * h;
    if (r >= rows) continue;
    const bool none = !counts[h];  // (its sums were of zeros times keys, NaN where a key is no number)
    const int64_t row = a.row(b, kvh, r);
    float* const out = a.parts ? a.part_a + (s * a.rows + row) * kD : static_cast<float*>(a.dq) + row * kD;
#pragma unroll
    for (int j = 0; j < 8; ++j) store2(out + 8 * j + 2 * tig, none ? 0.0f : 0.125f * dq[j][2 * h], none ? 0.0f : 0.125f * dq[j][2 * h + 1]);
  }
}

// dk, dv: a CTA has 64 keys and a split of the rows that attend them.
//   dv = sum p dO, dk = sum ds q / 8
__device__ __forceinline__ void cross_dkv(const CrossArgs& a, float* sm, uint32_t x) {
  float *const Qs = sm, *const Ds = sm + kTileN * kPitch, *const Ks = sm + 2 * kTileN * kPitch, *const Vs = sm + 3 * kTileN * kPitch;
  __shared__ float2 stat[kTileN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int tiles = (a.Tk + kTileN - 1) / kTileN;
  const int s = x % a.splits;
  x /= a.splits;
  const int j0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = x % a.Hkv, b = x / a.Hkv;
  const int nq = a.queries(b), nk = a.keys(b), rows = a.G * nq;
  int b0, b1;
  split_keys(j0 < nk ? rows : 0, kTileN, a.splits, s, b0, b1);
  const float* const kp = static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h;
  const float* const vp = static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h;
  bool k_plain = false;
  if (b0 < b1) {
    k_plain |= load_tile(Ks, [&](int r) { return j0 + r < nk ? kp + (int64_t)(j0 + r) * a.ks.t : nullptr; });
    k_plain |= load_tile(Vs, [&](int r) { return j0 + r < nk ? vp + (int64_t)(j0 + r) * a.vs.t : nullptr; });
  }
  auto key_dim = [&](int h, int d) { return Ks[(16 * warp + gid + 8 * h) * kPitch + d]; };
  auto value_dim = [&](int h, int d) { return Vs[(16 * warp + gid + 8 * h) * kPitch + d]; };
  const LeftTile k(Ks, 16 * warp, gid, tig), v(Vs, 16 * warp, gid, tig);
  float dk[8][4], dv[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[j][e] = dv[j][e] = 0.0f;
  for (int r0 = b0; r0 < b1; r0 += kTileN) {
    __syncthreads();
    auto query = [&](int i) {
      const int r = r0 + i, t = r / a.G, head = kvh * a.G + (r - t * a.G);
      return r < b1 ? static_cast<const float*>(a.q) + b * a.qs.b + head * a.qs.h + t * a.qs.t : nullptr;
    };
    bool plain = load_tile(Qs, query);
    plain |= load_tile(Ds, [&](int i) { return r0 + i < b1 ? static_cast<const float*>(a.dO) + a.row(b, kvh, r0 + i) * kD : nullptr; });
    if (threadIdx.x < kTileN) {
      const int r = r0 + threadIdx.x;
      stat[threadIdx.x] = r < b1 ? a.stat[a.row(b, kvh, r)] : make_float2(0.0f, 0.0f);
    }
    plain = __syncthreads_or(plain || k_plain);
#pragma unroll 1
    for (int n = 0; n < 8; n += 2) {
      float p[2][4], dp[2][4];  // [key][row]
      if (plain) {
        rows_plain<2>(p, key_dim, Qs, n, tig);
        rows_plain<2>(dp, value_dim, Ds, n, tig);
      } else {
        rows_product<2>(p, k, Qs, n, gid, tig);
        rows_product<2>(dp, v, Ds, n, gid, tig);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 8 * (n + i) + 2 * tig + (e & 1);
          const float2 st = stat[r];
          const bool there = r0 + r < b1;
          p[i][e] = there ? exp2f(fmaf(p[i][e], kLogitScale, -st.x)) : 0.0f;
          dp[i][e] = there ? p[i][e] * (dp[i][e] - st.y) : 0.0f;
        }
        if (plain) {
          dims_plain(dv, p[i], Ds, n + i, gid, tig);
          dims_plain(dk, dp[i], Qs, n + i, gid, tig);
        } else {
          dims_product(dv, p[i], Ds, n + i, gid, tig);
          dims_product(dk, dp[i], Qs, n + i, gid, tig);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = j0 + 16 * warp + gid + 8 * h;
    if (j >= a.Tk) continue;
    const bool none = j >= nk;  // (its probabilities were of a row of zeros)
    const int64_t row = ((int64_t)b * a.Hkv + kvh) * a.Tk + j, at = a.parts ? (int64_t)s * a.B * a.Hkv * a.Tk + row : row;
    float *const ok = (a.parts ? a.part_a : static_cast<float*>(a.dk)) + at * kD, *const ov = (a.parts ? a.part_b : static_cast<float*>(a.dv)) + at * kD;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      store2(ok + 8 * c + 2 * tig, none ? 0.0f : 0.125f * dk[c][2 * h], none ? 0.0f : 0.125f * dk[c][2 * h + 1]);
      store2(ov + 8 * c + 2 * tig, none ? 0.0f : dv[c][2 * h], none ? 0.0f : dv[c][2 * h + 1]);
    }
  }
}

// Both, which wait for nothing of one another, in one launch, so that their last CTAs fill
// the SMs together (2 x 8 / 2 heads, 333 x 1000 ragged rows: 78 us, 97 one behind the other):
// the first n0 CTAs are kv's.
constexpr size_t kBwdSmemBytes = 4 * kTileN * kPitch * sizeof(float);
__global__ void __launch_bounds__(kThreads32, 3) cross_bwd_kernel(const CrossArgs q, const CrossArgs kv, uint32_t n0) {
  extern __shared__ __align__(16) float sm[];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x < n0)
    cross_dkv(kv, sm, blockIdx.x);
  else
    cross_dq(q, sm, blockIdx.x - n0);
}

static unsigned tiles_grid(const CrossArgs& a, int rows) { return (unsigned)((int64_t)a.B * a.Hkv * ((rows + kTileN - 1) / kTileN) * a.splits); }

int launch_cross_fwd_f32(const CrossArgs& a, void* stream) {
  LaunchTimer tm(SFA_KERNEL_CROSS_FWD, stream);
  const cudaError_t e = launch_pdl(cross_fwd_kernel, dim3(tiles_grid(a, a.G * a.Tq)), dim3(kThreads32), 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}
int launch_cross_bwd_f32(const CrossArgs& q, const CrossArgs& kv, void* stream) {
  const unsigned n0 = tiles_grid(kv, kv.Tk);
  LaunchTimer tm(SFA_KERNEL_CROSS_BWD_KV, stream);
  cudaError_t e = cudaFuncSetAttribute(cross_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBwdSmemBytes);
  if (e == cudaSuccess)
    e = launch_pdl(cross_bwd_kernel, dim3(n0 + tiles_grid(q, q.G * q.Tq)), dim3(kThreads32), kBwdSmemBytes, (cudaStream_t)stream, q, kv, n0);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
