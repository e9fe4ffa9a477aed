// Few rows over many keys: the step of a decoder over an encoder's states, and
// the own rows of the sequences behind a shared prefix.
//
// Every key and value is read once for the rows of its KV head and used for a few
// multiplications a row: memory bounds it.  All sums are fp32; no shared memory but
// for the join of a CTA's four warps and of a cluster's CTAs.
//
// fp32: eight lanes hold a key, 8 dims each, so a warp reads four whole rows at a time
// straight into registers; a row's products are summed over the eight lanes by halving
// exchanges that leave row r's logit in lane r (7 shuffles for 8 rows, not 24).
//
// bf16: up to 16 rows are the left operand of mma.sync, keys and then values the right
// one, in the order in which lanes read whole 16-byte pieces: which dims a k index of
// the logits' product stands for, and which dim a column of the outputs' is, is free as
// long as both operands agree.  Logits come out of the product as probabilities go into
// the next, values need one byte permutation a register (two keys' numbers of a dim
// side by side).  Probabilities are rounded to bf16 for their product.  (The fp32
// kernel on bf16 rows took 62 us for 500 sequences of up to 700 rows of 16 / 2 heads.)
#include <type_traits>

#include "sfa_cross.cuh"

namespace sfa {

constexpr int kStreamWarps = 4;

// Sums of acc[0 .. NR) over the eight lanes of a key; lane l gets row l mod NR's.
template <int NR>
__device__ __forceinline__ float sum_rows(float* acc, int lane) {
#pragma unroll
  for (int bit = 4, n = NR; bit > 0; bit >>= 1) {
    if (n > bit) {  // rows' halves are exchanged: n -> n / 2 (bit is n / 2 then)
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i)
        if (i < n / 2) {
          const float mine = up ? acc[i + n / 2] : acc[i], other = up ? acc[i] : acc[i + n / 2];
          acc[i] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
        }
      n /= 2;
    } else {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (i < n) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], bit);
    }
  }
  return acc[0];
}

// The warps' sums of a CTA's rows, R of them, [warp][row][64] and (m, l), to parts
// or to o and lse; in a cluster, whose CTAs have a split each, rank by rank a row.
template <typename TIO, int R>
__device__ __forceinline__ void stream_out(const CrossArgs& a, float (*so)[R][kD], float2 (*sml)[R], int b, int kvh, int r0, int s, int nq, bool keys) {
  const int rows = a.G * a.Tq, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = 2 * lane;
  for (int r = warp; r < R; r += kStreamWarps) {
    if (r0 + r >= rows) break;
    const int t = (r0 + r) / a.G;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) mm = fmaxf(mm, sml[w][r].x);
    const float sh = shift_of(mm);
    float ll = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) {
      const float f = exp2f(sml[w][r].x - sh);
      ll = fmaf(f, sml[w][r].y, ll);
      y0 = fmaf(f, so[w][r][d], y0);
      y1 = fmaf(f, so[w][r][d + 1], y1);
    }
    const int64_t row = a.row(b, kvh, r0 + r);
    const bool none = t >= nq || !keys;
    if (a.parts) {
      const int64_t at = s * a.rows + row;
      if (!none) store2(a.part_o + at * kD + d, y0, y1);
      if (d == 0) a.part_ml[at] = none ? make_float2(-INFINITY, -1.0f) : make_float2(mm, ll);
    } else if (a.cluster) {
      __syncwarp();  // (the row is this warp's alone)
      so[0][r][d] = y0;
      so[0][r][d + 1] = y1;
      if (d == 0) sml[0][r] = none ? make_float2(-INFINITY, -1.0f) : make_float2(mm, ll);
    } else {
      const float inv = 1.0f / ll;
      store2(static_cast<TIO*>(a.o) + row * kD + d, none ? 0.0f : y0 * inv, none ? 0.0f : y1 * inv);
      if (a.lse && d == 0) a.lse[row] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  }
  if (!a.cluster) return;
  cluster_sync();
  for (int r = s + a.splits * warp; r < R; r += a.splits * kStreamWarps) {
    if (r0 + r >= rows) break;
    float m[kClusterSplits], l[kClusterSplits], y0[kClusterSplits], y1[kClusterSplits], mm = -INFINITY;
#pragma unroll
    for (int c = 0; c < kClusterSplits; ++c) {
      const bool there = c < a.splits;  // (else this CTA's own, for nothing)
      const int rank = there ? c : s;
      m[c] = cluster_read(&sml[0][r].x, rank);
      l[c] = cluster_read(&sml[0][r].y, rank);
      y0[c] = cluster_read(&so[0][r][d], rank);
      y1[c] = cluster_read(&so[0][r][d + 1], rank);
      if (!there) l[c] = -1.0f;
      if (there) mm = fmaxf(mm, m[c]);
    }
    const float sh = shift_of(mm);
    float ll = 0.0f, z0 = 0.0f, z1 = 0.0f;
    bool any = false;
#pragma unroll
    for (int c = 0; c < kClusterSplits; ++c)
      if (!(l[c] < 0.0f)) {
        const float f = exp2f(m[c] - sh);
        any = true;
        ll = fmaf(f, l[c], ll);
        z0 = fmaf(f, y0[c], z0);
        z1 = fmaf(f, y1[c], z1);
      }
    const int64_t row = a.row(b, kvh, r0 + r);
    const float inv = 1.0f / ll;
    store2(static_cast<TIO*>(a.o) + row * kD + d, any ? z0 * inv : 0.0f, any ? z1 * inv : 0.0f);
    if (a.lse && d == 0) a.lse[row] = any ? (mm + log2f(ll)) * kLn2 : -INFINITY;
  }
  cluster_sync();  // until all have read
}

// The CTA's sequence, KV head, first row and split.
struct StreamUnit {
  int b, kvh, r0, s;
};
__device__ __forceinline__ StreamUnit stream_unit(const CrossArgs& a, int R, uint32_t x) {
  const int groups = (a.G * a.Tq + R - 1) / R;
  StreamUnit u;
  u.s = x % a.splits;
  x /= a.splits;
  u.r0 = (int)(x % groups) * R;
  x /= groups;
  u.kvh = x % a.Hkv;
  u.b = x / a.Hkv;
  return u;
}

// TWO calls in one launch, which wait for nothing of one another: the first n0 CTAs are
// a0's, the others a1's.  (A decode step of 4 sequences behind 1000 rows: 16.1 us in two
// launches, so 11.8.)
template <bool TWO>
struct StreamCall {
  const bool second;
  const CrossArgs a;
  const uint32_t x;
  __device__ __forceinline__ StreamCall(const CrossArgs& a0, const CrossArgs& a1, uint32_t n0)
      : second(TWO && blockIdx.x >= n0), a(second ? a1 : a0), x(second ? blockIdx.x - n0 : blockIdx.x) {}
};

constexpr int kMmaStep = 16;  // keys a warp takes at a time; the next ones are under way meanwhile

template <typename TQ, bool TWO>
__global__ void __launch_bounds__(32 * kStreamWarps) cross_stream_mma_kernel(const CrossArgs a0, const CrossArgs a1, uint32_t n0) {
  constexpr int PARTS = sizeof(TQ) == 4 ? 2 : 1;  // of a query: fp32 ones as two bf16 numbers
  __shared__ float so[kStreamWarps][16][kD];
  __shared__ float2 sml[kStreamWarps][16];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const StreamCall<TWO> call(a0, a1, n0);
  const CrossArgs& a = call.a;
  const StreamUnit u = stream_unit(a, 16, call.x);
  const int nq = a.queries(u.b), nk = a.keys(u.b);
  int k0, k1;
  split_keys(nk, kMmaStep, a.splits, u.s, k0, k1);

  // queries: rows gid and gid + 8, dims 16 tig .. 16 tig + 15; k indexes 2 tig, 2 tig + 1,
  // 2 tig + 8, 2 tig + 9 of step s are dims 16 tig + 4 s .. 4 s + 3
  uint32_t q[PARTS][4][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = u.r0 + gid + 8 * h, t = r / a.G, head = u.kvh * a.G + (r - t * a.G);
    float x[16];
    if (r < a.G * a.Tq && t < nq) {
      const TQ* row = static_cast<const TQ*>(a.q) + u.b * a.qs.b + head * a.qs.h + t * a.qs.t + 16 * tig;
      load8(row, x);
      load8(row + 8, x + 8);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float x0 = x[4 * s + 2 * c], x1 = x[4 * s + 2 * c + 1];
        const uint32_t hi = pack_bf16(x0, x1);
        q[0][s][2 * c + h] = hi;
        if (PARTS == 2) {
          const float2 f = unpack_bf16(hi);
          q[PARTS - 1][s][2 * c + h] = pack_bf16(x0 - f.x, x1 - f.y);
        }
      }
  }
  const bf16* const kp = static_cast<const bf16*>(a.k) + u.b * a.ks.b + u.kvh * a.ks.h + 16 * tig;
  const bf16* const vp = static_cast<const bf16*>(a.v) + u.b * a.vs.b + u.kvh * a.vs.h + 8 * gid;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // of rows gid, gid + 8 (l: this lane's keys)
  float o[8][4];  // [j]: row gid dims 16 tig + j, 16 tig + 8 + j, the same of row gid + 8
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

  struct Rows {
    uint4 k[2][2], v[2][2];  // key 8 n + gid: both halves of its 32 bytes; keys 8 n + 2 tig, + 1
  };
  auto load = [&](Rows& x, int base) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = base + 8 * n + gid;
      const uint4* row = reinterpret_cast<const uint4*>(kp + (int64_t)j * a.ks.t);
      x.k[n][0] = j < k1 ? row[0] : make_uint4(0, 0, 0, 0);
      x.k[n][1] = j < k1 ? row[1] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = base + 8 * n + 2 * tig + h;
        x.v[n][h] = j < k1 ? *reinterpret_cast<const uint4*>(vp + (int64_t)j * a.vs.t) : make_uint4(0, 0, 0, 0);
      }
  };
  auto take = [&](const Rows& x, int base) {
    float c[2][4];  // [n]: rows gid (0, 1) and gid + 8 (2, 3), keys 8 n + 2 tig, + 1
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) c[n][e] = 0.0f;
      const uint32_t kr[8] = {x.k[n][0].x, x.k[n][0].y, x.k[n][0].z, x.k[n][0].w, x.k[n][1].x, x.k[n][1].y, x.k[n][1].z, x.k[n][1].w};
#pragma unroll
      for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_bf16(c[n], q[p][s], kr[2 * s], kr[2 * s + 1]);
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (base + 8 * n + 2 * tig + (e & 1) >= k1) c[n][e] = -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], c[n][e]);
      }
    // (a lane's own maxima: a row's four lanes exchange theirs only where one has grown)
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const float to = fmaxf(m[h], top[h]), corr = ex2((m[h] - shift_of(to)) * kLogitScale);
        m[h] = to;
        l[h] *= corr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][2 * h] *= corr;
          o[j][2 * h + 1] *= corr;
        }
      }
    }
    const float sh[2] = {shift_of(m[0]), shift_of(m[1])};
    uint32_t p[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = ex2((c[n][2 * h] - sh[h]) * kLogitScale), p1 = ex2((c[n][2 * h + 1] - sh[h]) * kLogitScale);
        l[h] += p0 + p1;
        p[n][h] = pack_bf16(p0, p1);
      }
    const uint32_t pa[4] = {p[0][0], p[0][1], p[1][0], p[1][1]};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
      auto word = [&](const uint4& w) { return (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w; };
      mma_bf16(o[j], pa, __byte_perm(word(x.v[0][0]), word(x.v[0][1]), sel), __byte_perm(word(x.v[1][0]), word(x.v[1][1]), sel));
    }
  };
  constexpr int kNext = kMmaStep * kStreamWarps;
  Rows r0, r1;
  int base = k0 + warp * kMmaStep;
  if (base < k1) load(r0, base);
  for (; base < k1; base += 2 * kNext) {
    if (base + kNext < k1) load(r1, base + kNext);
    take(r0, base);
    if (base + kNext >= k1) break;
    if (base + 2 * kNext < k1) load(r0, base + 2 * kNext);
    take(r1, base + kNext);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    float* const row = &so[warp][gid + 8 * h][16 * tig];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(row + j) = make_float4(o[j][2 * h], o[j + 1][2 * h], o[j + 2][2 * h], o[j + 3][2 * h]);
      *reinterpret_cast<float4*>(row + 8 + j) = make_float4(o[j][2 * h + 1], o[j + 1][2 * h + 1], o[j + 2][2 * h + 1], o[j + 3][2 * h + 1]);
    }
    if (tig == 0) sml[warp][gid + 8 * h] = make_float2(m[h] == -INFINITY ? m[h] : m[h] * kLogitScale, l[h]);
  }
  __syncthreads();
  stream_out<bf16, 16>(a, so, sml, u.b, u.kvh, u.r0, u.s, nq, k1 > k0);
}

template <int NR, bool TWO>
__global__ void __launch_bounds__(32 * kStreamWarps) cross_stream_kernel(const CrossArgs a0, const CrossArgs a1, uint32_t n0) {
  constexpr int U = 2;          // keys a lane takes at a time
  constexpr int kStep = 4 * U;  // keys a warp takes at a time
  __shared__ float so[kStreamWarps][NR][kD];
  __shared__ float2 sml[kStreamWarps][NR];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kg = lane >> 3, d8 = (lane & 7) * 8;
  const StreamCall<TWO> call(a0, a1, n0);
  const CrossArgs& a = call.a;
  const int rows = a.G * a.Tq;
  const StreamUnit unit = stream_unit(a, NR, call.x);
  const int s = unit.s, r0 = unit.r0, kvh = unit.kvh, b = unit.b;
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kStep, a.splits, s, k0, k1);

  float q[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int t = (r0 + r) / a.G, h = kvh * a.G + (r0 + r - t * a.G);
    if (r0 + r < rows && t < nq) {
      load8(static_cast<const float*>(a.q) + b * a.qs.b + h * a.qs.h + t * a.qs.t + d8, q[r]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[r][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q[r][e] *= kLogitScale;
  }
  const float* kp = static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h + d8;
  const float* vp = static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h + d8;
  float m = -INFINITY, l = 0.0f;  // of row lane mod NR
  float o[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) o[r][e] = 0.0f;

  for (int base = k0 + warp * kStep; base < k1; base += kStep * kStreamWarps) {
    float kf[U][8], vf[U][8], p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + 4 * u + kg;
      const int64_t at = j < k1 ? j : k0;  // (a row that is there)
      load8(kp + at * a.ks.t, kf[u]);
      load8(vp + at * a.vs.t, vf[u]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y = fmaf(q[r][e], kf[u][e], y);
        acc[r] = y;
      }
      p[u] = sum_rows<NR>(acc, lane);
      if (base + 4 * u + kg >= k1) p[u] = -INFINITY;
      top = fmaxf(top, p[u]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (__any_sync(0xffffffffu, top > m)) {
      const float mn = fmaxf(m, top), corr = exp2f(m - shift_of(mn));
      l *= corr;
      m = mn;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float c = __shfl_sync(0xffffffffu, corr, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] *= c;
      }
    }
    const float sh = shift_of(m);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = base + 4 * u + kg < k1;
      p[u] = exp2f(p[u] - sh);
      l += p[u];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float pr = __shfl_sync(0xffffffffu, p[u], (lane & 24) | r);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] = there ? fmaf(pr, vf[u][e], o[r][e]) : o[r][e];
      }
    }
  }
  // the warp's four keys, then the warps
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (lane < NR) sml[warp][lane] = make_float2(m, l);
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 8);
      o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 16);
    }
  if (kg == 0)
#pragma unroll
    for (int r = 0; r < NR; ++r) st_smem8(&so[warp][r][d8], o[r]);
  __syncthreads();
  stream_out<float, NR>(a, so, sml, b, kvh, r0, s, nq, k1 > k0);
}

// Parts of each row to o and lse, a warp a row.  pos (of sequences whose rows
// are queries' heads, Tq = 1): a position outside [0, T) leaves a zero row.
template <int S, typename TIO>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossArgs a, const int32_t* pos, int T) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.rows, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  int n = a.splits;
  if (pos) {
    const int p = pos[row / a.Hq];
    if (p < 0 || p >= T) n = 0;
  }
  join_row<S, TIO>(a, row, n, lane, [&](int i) { return a.part_ml[i * rows + row]; }, [&](int i) { return a.part_o + (i * rows + row) * kD; });
}

int launch_cross_join(const CrossArgs& a, int dtype, const int32_t* pos, int pos_T, void* stream) {
  const int64_t rows = a.rows;
  const dim3 grid((unsigned)((rows + 7) / 8));
  cudaStream_t st = (cudaStream_t)stream;
  LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
  constexpr int F = kFewParts / 4;
  const bool few = a.splits <= kFewParts;
  auto* f = dtype == SFA_BF16 ? (few ? cross_join_kernel<F, bf16> : cross_join_kernel<8, bf16>)
                              : (few ? cross_join_kernel<F, float> : cross_join_kernel<8, float>);
  const cudaError_t e = launch_pdl(f, grid, dim3(256), 0, st, a, pos, pos_T);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

static unsigned stream_grid(const CrossArgs& a, int R) { return (unsigned)((int64_t)a.B * a.Hkv * ((a.G * a.Tq + R - 1) / R) * a.splits); }

template <bool TWO>
static int launch_stream(const CrossArgs& a0, const CrossArgs& a1, bool q32, int dtype, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const int rows = a0.G * a0.Tq, nr = rows == 1 ? 1 : rows == 2 ? 2 : rows <= 4 ? 4 : 8, R = dtype == SFA_BF16 ? 16 : nr;
  const unsigned n0 = stream_grid(a0, R);
  const dim3 grid(n0 + (TWO ? stream_grid(a1, R) : 0)), block(32 * kStreamWarps);
  using Q16 = std::conditional_t<TWO, float, bf16>;  // (two: of fp32 queries always)
  auto* f = dtype == SFA_BF16 ? (q32 ? cross_stream_mma_kernel<float, TWO> : cross_stream_mma_kernel<Q16, TWO>)
            : nr == 1         ? cross_stream_kernel<1, TWO>
            : nr == 2         ? cross_stream_kernel<2, TWO>
            : nr == 4         ? cross_stream_kernel<4, TWO>
                              : cross_stream_kernel<8, TWO>;
  LaunchTimer tm(SFA_KERNEL_CROSS_FWD, stream);
  const cudaError_t e = !TWO && a0.cluster ? launch_pdl_cluster(f, grid, block, (unsigned)a0.splits, 0, st, a0, a1, n0)
                                           : launch_pdl(f, grid, block, 0, st, a0, a1, n0);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int launch_cross_stream(const CrossArgs& a, bool q32, int dtype, void* stream) { return launch_stream<false>(a, a, q32, dtype, stream); }
int launch_cross_stream_two(const CrossArgs& a, const CrossArgs& b, int dtype, void* stream) { return launch_stream<true>(a, b, true, dtype, stream); }

}  // namespace sfa
