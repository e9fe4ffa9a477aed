// Attention of query rows over the paged 4-bit cache.
//
// Keys are the rows of a tensor-core tile: S^T = K Q^T (16 keys x 8 query
// heads a product), softmax statistics per column in fp32, O^T += V^T P.  All
// heads of a KV head are columns of the same tile, so a cache row is read and
// dequantised once for the whole group.  What keeps it exact:
//  * keys and values are whole f16 numbers (code * scale);
//  * the query, rotated in fp32, is scaled by a power of two to its own row's
//    size and split into two f16 parts (22 bits), whose products go to one
//    fp32 accumulator: logits are good to fp32's last bits;
//  * probabilities are rounded to f16 (2^-12 of each) for the values' product;
//    fp32 outputs add a second product with what that rounding dropped;
//  * the softmax sum is taken in fp32 from the unrounded probabilities.
#include <math.h>

#include <algorithm>

#include "sfa_kv4.cuh"
#include "sfa_launch.cuh"

namespace sfa {

// Probabilities are kept times 2^kPShift: f16's smallest steps then lie 2^-36
// below the largest probability of a column.
constexpr float kPShift = 12.0f;

// The group's queries of one row as B fragments: lane (g, t) holds dims
// 16t .. 16t + 15 of head 8 nt + g, in the order the keys' codes come in.
template <int NT>
struct QFrag {
  uint32_t hi[NT][8], lo[NT][8];
  float c[NT][2];  // logit of accumulator (heads 2t, 2t + 1), log2 units

  // row: q + the group's first head; heads from G on are zero columns.
  template <typename TIO>
  __device__ __forceinline__ void load(const TIO* row, int G, const float2* rope, int pos, float scale, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = 8 * nt + g;
      float x[16], y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.0f;
      if (head < G) {
        load8(row + head * kD + 16 * t, x);
        load8(row + head * kD + 16 * t + 8, x + 8);
        if (rope) {  // the pair of dim j is j +- 32
          load8(row + head * kD + 16 * (t ^ 2), y);
          load8(row + head * kD + 16 * (t ^ 2) + 8, y + 8);
#pragma unroll
          for (int c8 = 0; c8 < 16; c8 += 8) {
            float cs[8], sn[8];
            load_rope8(rope, pos, 16 * (t & 1) + c8, cs, sn);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c8 + e] = x[c8 + e] * cs[e] + (t < 2 ? -y[c8 + e] : y[c8 + e]) * sn[e];
          }
        }
      }
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^(8 - exponent of the largest): its parts then reach f16's 2^-24 steps
      // 2^-33 below it
      const int ex = min(max((int)(__float_as_uint(m) >> 23), 9), 253);
      const float f = __uint_as_float((uint32_t)(254 - ex) << 23) * 256.0f;
      const float back = __uint_as_float((uint32_t)ex << 23) * (scale * 0.00390625f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[2 * e] * f, b = x[2 * e + 1] * f;
        hi[nt][e] = pack_f16(a, b);
        const float2 r = unpack_f16(hi[nt][e]);
        lo[nt][e] = pack_f16(a - r.x, b - r.y);
      }
      c[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      c[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
  }
};

// Keys g and g + 8 of a tile: 16 codes and the scale of dims 16t .. 16t + 15
// each.  s[nt] = accumulators of keys (g, g, g + 8, g + 8) x heads (2t, 2t + 1).
template <int NT>
__device__ __forceinline__ void key_products(const QFrag<NT>& q, uint2 ka, uint2 kb, uint32_t sa, uint32_t sb, float (*s)[4]) {
  const uint32_t fa = e4m3x2_f16x2(sa * 0x101u), fb = e4m3x2_f16x2(sb * 0x101u);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const uint32_t wa = (ks < 2 ? ka.x : ka.y) >> (16 * (ks & 1)), wb = (ks < 2 ? kb.x : kb.y) >> (16 * (ks & 1));
    const uint32_t a[4] = {hmul2(e2m1x2_f16x2(wa & 255u), fa), hmul2(e2m1x2_f16x2(wb & 255u), fb),
                           hmul2(e2m1x2_f16x2((wa >> 8) & 255u), fa), hmul2(e2m1x2_f16x2((wb >> 8) & 255u), fb)};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16(s[nt], a, q.hi[nt][2 * ks], q.hi[nt][2 * ks + 1]);
      mma_f16(s[nt], a, q.lo[nt][2 * ks], q.lo[nt][2 * ks + 1]);
    }
  }
}

// Values of keys 2t, 2t + 1, 2t + 8, 2t + 9: codes of dims 8g .. 8g + 7 and the
// scales of their block (bytes, first key first).  o[nt][mt] = accumulators of
// dims (8g + 2 mt, 8g + 2 mt + 1) x heads (2t, 2t + 1).
template <int NT, bool EXACT>
__device__ __forceinline__ void value_products(const uint32_t* w, uint32_t scales, const float (*p)[4], float (*o)[4][4]) {
  uint32_t b0[NT], b1[NT], l0[NT], l1[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t x0 = pack_f16(p[nt][0], p[nt][1]), x1 = pack_f16(p[nt][2], p[nt][3]);
    b0[nt] = movmatrix_t(x0);
    b1[nt] = movmatrix_t(x1);
    if (EXACT) {
      const float2 r0 = unpack_f16(x0), r1 = unpack_f16(x1);
      l0[nt] = movmatrix_t(pack_f16(p[nt][0] - r0.x, p[nt][1] - r0.y));
      l1[nt] = movmatrix_t(pack_f16(p[nt][2] - r1.x, p[nt][3] - r1.y));
    }
  }
  const uint32_t fab = e4m3x2_f16x2(scales & 0xffffu), fcd = e4m3x2_f16x2(scales >> 16);
  // bytes that hold one dim of two keys: even dims, then odd dims
  const uint32_t lo4 = 0x0f0f0f0fu;
  const uint32_t eab = (w[0] & lo4) | ((w[1] << 4) & ~lo4), oab = ((w[0] >> 4) & lo4) | (w[1] & ~lo4);
  const uint32_t ecd = (w[2] & lo4) | ((w[3] << 4) & ~lo4), ocd = ((w[2] >> 4) & lo4) | (w[3] & ~lo4);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const uint32_t a[4] = {hmul2(e2m1x2_f16x2((eab >> (8 * mt)) & 255u), fab), hmul2(e2m1x2_f16x2((oab >> (8 * mt)) & 255u), fab),
                           hmul2(e2m1x2_f16x2((ecd >> (8 * mt)) & 255u), fcd), hmul2(e2m1x2_f16x2((ocd >> (8 * mt)) & 255u), fcd)};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16(o[nt][mt], a, b0[nt], b1[nt]);
      if (EXACT) mma_f16(o[nt][mt], a, l0[nt], l1[nt]);
    }
  }
}

// One online-softmax step over a tile's logits (log2 units times c, -inf for
// absent keys): p = 2^(s - m + kPShift), o and l rescaled when m grows.
template <int NT>
__device__ __forceinline__ void softmax_step(const QFrag<NT>& q, float (*s)[4], bool va, bool vb, float (*m)[2], float (*l)[2],
                                             float (*o)[4][4]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = va ? s[nt][e] * q.c[nt][e] : -INFINITY, y = vb ? s[nt][2 + e] * q.c[nt][e] : -INFINITY;
      float mx = fmaxf(x, y);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      if (mx > m[nt][e]) {
        const float corr = ex2(m[nt][e] - mx);  // 0 on the first keys
        m[nt][e] = mx;
        l[nt][e] *= corr;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          o[nt][mt][e] *= corr;
          o[nt][mt][2 + e] *= corr;
        }
      }
      const float ref = m[nt][e] == -INFINITY ? 0.0f : m[nt][e] - kPShift;  // no key yet: 2^-inf = 0
      x = ex2(x - ref);
      y = ex2(y - ref);
      l[nt][e] += x + y;
      s[nt][e] = x;
      s[nt][2 + e] = y;
    }
}

// What a warp holds of its columns when it has seen its keys.
template <int NT>
struct Acc {
  float m[NT][2], l[NT][2], o[NT][4][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
    }
  }
  // l over all the warp's keys (the lanes' keys are added in a fixed order)
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][e] = x;
      }
  }
};

// One head's output row (dims 8g .. 8g + 7 of lane (g, t)) and log-sum-exp.
// l = 0: no keys, a zero row and -inf.
template <typename TIO>
__device__ __forceinline__ void write_head(const Kv4Args& a, int64_t n, int head, int g, const float* x, float m, float l) {
  float y[8];
  const float inv = l == 0.0f ? 0.0f : a.vscale / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = l == 0.0f ? 0.0f : x[e] * inv;
  store8(static_cast<TIO*>(a.o) + (n * a.Hq + head) * kD + 8 * g, y);
  if (a.lse && g == 0) a.lse[n * a.Hq + head] = l == 0.0f ? -INFINITY : (m - kPShift) * kLn2 + logf(l);
}

// ---------------------------------------------------------------- gather

// Any offset list, one (row, KV head) a group of `warps` warps: lanes look up
// their keys' pages, tiles of 16 keys go round the group's warps, and the
// group's partial results meet in shared memory.  Bounded by latency (row map,
// block table, cache row: three dependent loads) at decode sizes and by the
// gathered sectors (32 + 32 + 32 bytes a key) at prompt sizes.
constexpr int kGatherWarps = 4;

template <typename TIO, int NT>
__global__ void __launch_bounds__(32 * kGatherWarps)
    kv4_gather_kernel(const Kv4Args a, const __grid_constant__ Plan P, int warps) {
  constexpr bool kExact = sizeof(TIO) == 4;
  extern __shared__ float part[];  // [kGatherWarps][8 NT][66]
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int mine = warp % warps;
  const int64_t unit = (int64_t)blockIdx.x * (kGatherWarps / warps) + warp / warps;
  const int64_t n = unit / a.Hkv;
  const int h = (int)(unit - n * a.Hkv), G = 1 << a.lgG, S = 1 << a.lgS;
  pdl_wait();
  int r = 0, pos = -1;
  const bool live = n < a.N && kv4_row(a, (int)n, lane, r, pos);
  if (live && (pos < -1 || (pos < 0 && a.cu_q) || pos >= (a.max_pages << a.lgS) || (a.rope && pos >= a.rope_T))) {
    if (lane == 0) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
    pos = -1;
  }
  Acc<NT> acc;
  acc.clear();
  if (live && pos >= 0) {
    QFrag<NT> q;
    q.load(static_cast<const TIO*>(a.q) + n * a.q_stride + h * G * kD, G, a.rope, pos, 0.125f * kLog2e * a.kscale, lane);
    const int32_t* trow = a.table + (int64_t)r * a.max_pages;
    const int Wt = min(P.W, pos);
    int nr = 0;
    while (nr < P.n && P.c[nr] <= pos) ++nr;
    const int nk = Wt + 1 + nr;
    for (int j0 = 16 * mine; j0 < nk; j0 += 16 * warps) {
      const int j = j0 + (lane & 15);
      int slot = -1;
      if (j < nk) {
        const int p = pos - (j <= Wt ? j : P.c[j - Wt - 1]);
        const int page = trow[p >> a.lgS];
        if (page >= 0 && page < a.n_pages)
          slot = (page << a.lgS) + (p & (S - 1));
        else
          record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
      }
      auto block = [&](int sl) { return a.cache + ((int64_t)(sl >> a.lgS) * a.Hkv + h) * (kKv4Row * S); };
      const int ia = __shfl_sync(0xffffffffu, slot, g), ib = __shfl_sync(0xffffffffu, slot, g + 8);
      uint2 ka = make_uint2(0, 0), kb = ka;
      uint32_t sa = 0, sb = 0, w[4] = {0, 0, 0, 0}, vs = 0;
      if (ia >= 0) {
        const uint8_t* b = block(ia);
        ka = *reinterpret_cast<const uint2*>(b + 32 * (ia & (S - 1)) + 8 * t);
        sa = b[64 * S + 8 * (ia & (S - 1)) + t];
      }
      if (ib >= 0) {
        const uint8_t* b = block(ib);
        kb = *reinterpret_cast<const uint2*>(b + 32 * (ib & (S - 1)) + 8 * t);
        sb = b[64 * S + 8 * (ib & (S - 1)) + t];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int iv = __shfl_sync(0xffffffffu, slot, 2 * t + (e & 1) + 8 * (e >> 1));
        if (iv >= 0) {
          const uint8_t* b = block(iv);
          w[e] = *reinterpret_cast<const uint32_t*>(b + 32 * S + 32 * (iv & (S - 1)) + 4 * g);
          vs |= (uint32_t)b[64 * S + 8 * (iv & (S - 1)) + 4 + (g >> 1)] << (8 * e);
        }
      }
      float s[NT][4];
      key_products(q, ka, kb, sa, sb, s);
      softmax_step(q, s, ia >= 0, ib >= 0, acc.m, acc.l, acc.o);
      value_products<NT, kExact>(w, vs, s, acc.o);
    }
  }
  acc.close();
  if (warps == 1) {
    if (live)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * nt + 2 * t + e;
          float x[8];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            x[2 * mt] = acc.o[nt][mt][e];
            x[2 * mt + 1] = acc.o[nt][mt][2 + e];
          }
          if (head < G) write_head<TIO>(a, n, h * G + head, g, x, acc.m[nt][e], acc.l[nt][e]);
        }
    return;
  }
  // [warp][head][m, l, 64 dims]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* w = part + (warp * 8 * NT + 8 * nt + 2 * t + e) * 66;
      if (g == 0) {
        w[0] = acc.m[nt][e];
        w[1] = acc.l[nt][e];
      }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
        *reinterpret_cast<float2*>(w + 2 + 8 * g + 2 * mt) = make_float2(acc.o[nt][mt][e], acc.o[nt][mt][2 + e]);
    }
  __syncthreads();
  if (!live) return;
  // lanes 8 i .. 8 i + 7 of the group's warp w join head 4 w + i, and so on
  for (int head = 4 * mine + (lane >> 3); head < G; head += 4 * warps) {
    const float* w = part + ((warp - mine) * 8 * NT + head) * 66;
    const int d = lane & 7;
    float m = -INFINITY, l = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int i = 0; i < warps; ++i) m = fmaxf(m, w[i * 8 * NT * 66]);
    for (int i = 0; i < warps; ++i) {
      const float* wi = w + i * 8 * NT * 66;
      if (wi[1] == 0.0f) continue;
      const float f = ex2(wi[0] - m);
      l += wi[1] * f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += wi[2 + 8 * d + e] * f;
    }
    write_head<TIO>(a, n, h * G + head, d, x, m, l);
  }
}

template <typename TIO, int NT>
static cudaError_t gather(const Kv4Args& a, const Plan& p, int warps, cudaStream_t s) {
  const int64_t units = (int64_t)a.N * a.Hkv;
  const int per = kGatherWarps / warps;
  const size_t smem = warps > 1 ? (size_t)kGatherWarps * 8 * NT * 66 * sizeof(float) : 0;
  return launch_pdl(kv4_gather_kernel<TIO, NT>, dim3((unsigned)((units + per - 1) / per)), dim3(32 * kGatherWarps), smem, s, a, p, warps);
}

size_t kv4_attend_workspace(const Kv4Args&, const Plan&, int) { return 0; }

int launch_kv4_attend(const Kv4Args& a, const Plan& p, int dtype, void*, void* stream) {
  if (a.N == 0) return SFA_OK;
  const int tiles = (int)std::min<int64_t>(((int64_t)p.W + 1 + p.n + 15) / 16, ((int64_t)a.max_pages << a.lgS) / 16);
  const int warps = tiles <= 2 ? 1 : tiles <= 4 ? 2 : 4;
  const int G = 1 << a.lgG;
  cudaStream_t s = (cudaStream_t)stream;
  LaunchTimer tm(SFA_KERNEL_KV4_ATTEND, stream);
  cudaError_t e;
  if (dtype == SFA_BF16)
    e = G <= 8 ? gather<bf16, 1>(a, p, warps, s) : G == 16 ? gather<bf16, 2>(a, p, warps, s) : gather<bf16, 4>(a, p, warps, s);
  else
    e = G <= 8 ? gather<float, 1>(a, p, warps, s) : G == 16 ? gather<float, 2>(a, p, warps, s) : gather<float, 4>(a, p, warps, s);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
