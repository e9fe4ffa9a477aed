// Attention of query rows over the paged 4-bit cache.
//
// Keys are the rows of a tensor-core tile: S^T = K Q^T (16 keys x 8 query
// heads a product), softmax statistics per column in fp32, O^T += V^T P.  All
// heads of a KV head are columns of the same tile, so a cache row is read and
// dequantised once for the whole group.  What keeps it exact:
//  * keys and values are whole f16 numbers (code * scale);
//  * the query, rotated in fp32, is scaled by a power of two to its own row's
//    size (and by the mantissa of kscale log2(e) / 8) and split into two f16
//    parts (22 bits), whose products go to one fp32 accumulator: logits, a power
//    of two times that, are good to fp32's last bits;
//  * what is added to a logit before 2^x is rounded so that the result cannot
//    pass the largest that the kernel reckons with, however large logits are;
//  * probabilities are rounded to f16 (2^-12 of each) for the values' product;
//    fp32 outputs add a second product with what that rounding dropped;
//  * the softmax sum is taken in fp32 from the unrounded probabilities.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "sfa_kv4_stream.cuh"
#include "sfa_launch.cuh"

namespace sfa {

// Queries as B fragments: column c is head c mod G of row c / G; lane (g, t)
// holds dims 16t .. 16t + 15 of column 8 nt + g, in the order the keys' codes
// come in.
// One column tile: 8 B registers of high and 8 of low parts; returns the factor
// that takes the accumulator of column g to its logit (log2 units).  base: the first head of the first row; p: the position of this
// lane's column, below 0 for a zero column.
template <typename TIO>
__device__ __forceinline__ float load_queries(const TIO* base, int64_t stride, int lgG, int p, const float2* rope, float qmul, int qexp, int nt,
                                              int lane, uint32_t* hi, uint32_t* lo) {
  const int g = lane >> 2, t = lane & 3, col = 8 * nt + g;
  const TIO* row = base + (col >> lgG) * stride + (col & ((1 << lgG) - 1)) * kD;
  float x[16], y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.0f;
  if (p >= 0) {
    load8(row + 16 * t, x);
    load8(row + 16 * t + 8, x + 8);
    if (rope) {  // the pair of dim j is j +- 32
      load8(row + 16 * (t ^ 2), y);
      load8(row + 16 * (t ^ 2) + 8, y + 8);
#pragma unroll
      for (int c8 = 0; c8 < 16; c8 += 8) {
        float cs[8], sn[8];
        load_rope8(rope, p, 16 * (t & 1) + c8, cs, sn);
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
  const float f = __uint_as_float((uint32_t)(254 - ex) << 23) * 256.0f * qmul;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = x[2 * e] * f, b = x[2 * e + 1] * f;
    hi[e] = pack_f16(a, b);
    const float2 r = unpack_f16(hi[e]);
    lo[e] = pack_f16(a - r.x, b - r.y);
  }
  return logit_factor(ex, qexp);
}

// All of them in registers, 16 a column tile.
template <int NT>
struct QFrag {
  uint32_t hi[NT][8], lo[NT][8];
  float c[NT][2];  // logit of accumulator (heads 2t, 2t + 1), log2 units

  // at: position of column 8 nt + lane / 4
  template <typename TIO, typename AT>
  __device__ __forceinline__ void load(const TIO* base, int64_t stride, int lgG, AT at, const float2* rope, float qmul, int qexp, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float back = load_queries(base, stride, lgG, at(8 * nt + (lane >> 2)), rope, qmul, qexp, nt, lane, hi[nt], lo[nt]);
      c[nt][0] = __shfl_sync(0xffffffffu, back, 8 * (lane & 3));
      c[nt][1] = __shfl_sync(0xffffffffu, back, 8 * (lane & 3) + 4);
    }
  }
  // the B registers of step ks, columns nt: two of high parts, two of low ones
  __device__ __forceinline__ uint4 b(int ks, int nt) const {
    return make_uint4(hi[nt][2 * ks], hi[nt][2 * ks + 1], lo[nt][2 * ks], lo[nt][2 * ks + 1]);
  }
};

// The same in shared memory, for all of a CTA's warps: 64 registers a lane less
// with four column tiles, which is what lets two CTAs share an SM.
template <int NT>
struct QShared {
  uint32_t frag;  // shared address of this lane's: [step][column tile][lane]
  float c[NT][2];
  // (volatile: read where it is used, not kept in the registers that it is here to save)
  __device__ __forceinline__ uint4 b(int ks, int nt) const {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(frag + (ks * NT + nt) * 512));
    return v;
  }
};

// Keys g and g + 8 of a tile: 16 codes and the scale of dims 16t .. 16t + 15
// each.  s[nt] = accumulators of keys (g, g, g + 8, g + 8) x heads (2t, 2t + 1).
template <int NT, typename Q>
__device__ __forceinline__ void key_products(const Q& q, uint2 ka, uint2 kb, uint32_t sa, uint32_t sb, float (*s)[4]) {
  const uint32_t fa = e4m3x2_f16x2(sa * 0x101u), fb = e4m3x2_f16x2(sb * 0x101u);
  uint32_t xa[8], xb[8];
  e2m1x8_f16(ka.x, xa);
  e2m1x8_f16(ka.y, xa + 4);
  e2m1x8_f16(kb.x, xb);
  e2m1x8_f16(kb.y, xb + 4);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const uint32_t a[4] = {hmul2(xa[2 * ks], fa), hmul2(xb[2 * ks], fb), hmul2(xa[2 * ks + 1], fa), hmul2(xb[2 * ks + 1], fb)};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 b = q.b(ks, nt);
      mma_f16(s[nt], a, b.x, b.y);
      mma_f16(s[nt], a, b.z, b.w);
    }
  }
}

// Values of keys 2t, 2t + 1, 2t + 8, 2t + 9: codes of dims 8g .. 8g + 7 and the
// scales of their block (bytes of two keys each, the first in the low one).  o[nt][mt] = accumulators of
// dims (8g + 2 mt, 8g + 2 mt + 1) x heads (2t, 2t + 1).
template <int NT, bool EXACT>
__device__ __forceinline__ void value_products(const uint32_t* w, uint32_t sab, uint32_t scd, const float (*p)[4], float (*o)[4][4]) {
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
  const uint32_t fab = e4m3x2_f16x2(sab), fcd = e4m3x2_f16x2(scd);
  // bytes that hold one dim of two keys: even dims, then odd dims
  const uint32_t lo4 = 0x0f0f0f0fu;
  uint32_t x[4][4];
  e2m1x8_f16((w[0] & lo4) | ((w[1] << 4) & ~lo4), x[0]);
  e2m1x8_f16(((w[0] >> 4) & lo4) | (w[1] & ~lo4), x[1]);
  e2m1x8_f16((w[2] & lo4) | ((w[3] << 4) & ~lo4), x[2]);
  e2m1x8_f16(((w[2] >> 4) & lo4) | (w[3] & ~lo4), x[3]);
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const uint32_t a[4] = {hmul2(x[0][mt], fab), hmul2(x[1][mt], fab), hmul2(x[2][mt], fcd), hmul2(x[3][mt], fcd)};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16(o[nt][mt], a, b0[nt], b1[nt]);
      if (EXACT) mma_f16(o[nt][mt], a, l0[nt], l1[nt]);
    }
  }
}

// One online-softmax step over two tiles' logits (log2 units times c, -inf for
// absent keys: there(nt, e, i) says whether column 8 nt + 2 t + e attends key g
// of the first tile (i = 0), g + 8 (1), g and g + 8 of the second (2, 3)):
// p = 2^(s - m + kPShift), o and l rescaled when m grows.
template <int NT, typename THERE>
__device__ __forceinline__ void softmax_step(const QFrag<NT>& q, float (*s)[NT][4], THERE there, float (*m)[2], float (*l)[2],
                                             float (*o)[4][4]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = there(nt, e, i) ? s[i >> 1][nt][2 * (i & 1) + e] * q.c[nt][e] : -INFINITY;
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
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
      const float ref = m[nt][e] == -INFINITY ? 0.0f : __fsub_ru(m[nt][e], kPShift);  // no key yet: 2^-inf = 0
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = ex2(x[i] - ref);
        s[i >> 1][nt][2 * (i & 1) + e] = x[i];
      }
      l[nt][e] += (x[0] + x[1]) + (x[2] + x[3]);
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

// ---------------------------------------------------------------- gather

// Any offset list, one (row, KV head) a group of `warps` warps: lanes look up
// their keys' pages, pairs of 16-key tiles go round the group's warps, and the
// group's partial results meet in shared memory.  Bounded by latency (row map,
// block table, cache row: three dependent loads) at decode sizes (32 rows of 23
// keys, 8 / 2 heads: 4.3 us) and by its instructions at prompt sizes (7807 rows
// of 19 keys, 8 / 2 heads: 24 us, 2070 warp instructions a row pair and KV head at
// 2 a clock; the query's rotation and split are 250 of them).  The offsets
// beyond the window are taken to shared memory once a CTA, which walks over
// units: read where they come in, by as many addresses as lanes, they were
// replayed for every tile.
constexpr int kGatherWarps = 4;
constexpr uint32_t kNone = 0xffffffffu;

// PACK: 8 / G consecutive rows share a warp's columns.  Their keys follow one
// another in the tiles, and a key of another row counts as absent: what a row
// costs besides its keys (its query, its outputs) is paid once for all of them,
// and tiles fill up (7807 rows of 19 keys, 8 / 2 heads: 28 us a row a warp, 24
// so; 12800 rows, 4 / 4 heads: 84 and 49).
//
// CLUSTER: a (row, KV head) is a cluster of 8 CTAs, 32 warps, whose results meet
// through distributed shared memory: a few rows over some thousands of keys in
// one launch without a workspace.
enum GatherKind { kOne, kPack, kCluster };
constexpr int kClusterCtas = 8;

// A cluster a (row, KV head), where all of them fit the card at once: 1 row of
// 1000 keys, 8 / 2 heads 8.4 -> 6.4 us against the streaming kernel and its join,
// 38 rows 11.3 -> 9.1, 4 requests of 6 to 9 rows 14.3 -> 9.2.  Up to 512 keys four
// warps are no slower (7.0 and 6.4 us, 8.7 and 9.0); in two waves it loses
// (64 rows: 12.5 and 15.5 us; four CTAs an SM, two with more than 8 heads a KV
// head: 64 rows of 16 / 1 heads 14.1 and 20.2).
static bool clustered(const Kv4Args& a, int64_t keys) {
  return keys > 512 && (int64_t)a.N * a.Hkv * kClusterCtas <= (a.lgG > 3 ? 2 : 4) * kSMs;
}

struct GatherRows {
  int rows;        // 8 / G with PACK, else 1
  int keys;        // most keys of a row
  uint32_t magic;  // 2^32 / keys, rounded up: a key's row without a division
};

template <typename TIO, int NT, GatherKind KIND>
__global__ void __launch_bounds__(32 * kGatherWarps, NT == 1 ? 5 : 1)
    kv4_gather_kernel(const Kv4Args a, const __grid_constant__ Plan P, int warps, const GatherRows gr) {
  constexpr bool kExact = sizeof(TIO) == 4, PACK = KIND == kPack;
  __shared__ int rung[kMaxRungs];
  extern __shared__ float part[];  // [kGatherWarps][8 NT][66]
  __shared__ float joined[KIND == kCluster ? 8 * NT : 1][66];  // the CTA's (m, l, 64 sums) of a head
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  // this warp among those of its (row, KV head)
  const int rank = KIND == kCluster ? blockIdx.x % kClusterCtas : 0;
  const int mine = KIND == kCluster ? rank * kGatherWarps + warp : warp % warps;
  const int G = 1 << a.lgG, S = 1 << a.lgS;
  for (int i = threadIdx.x; i < P.n; i += 32 * kGatherWarps) rung[i] = P.c[i];
  pdl_wait();
  __syncthreads();
  const int nrow = PACK ? gr.rows : 1;
  const int units = (PACK ? (a.N + nrow - 1) / nrow : a.N) * a.Hkv;  // (N * Hkv <= 2^27)
  const int per = KIND == kCluster ? 1 : kGatherWarps / warps;
  const int begin = KIND == kCluster ? blockIdx.x / kClusterCtas : blockIdx.x * per;
  const int stride = KIND == kCluster ? gridDim.x / kClusterCtas : gridDim.x * per;
  for (int first = begin; first < units; first += stride) {
    const int unit = KIND == kCluster ? first : first + warp / warps;
    const int nu = (int)((uint32_t)unit / (uint32_t)a.Hkv), h = unit - nu * a.Hkv;
    const int n = nu * nrow;
    // lane i: row n + i, its request, position (-1: no keys) and keys
    int r = 0, pos = -1, nk = 0;
    bool live = false;
    if (!PACK) {
      live = n < a.N && kv4_row(a, n, lane, r, pos);
    } else {
      int r1 = 0, p1 = -1, end = 0;
      for (int i = 0; i < nrow; ++i) {  // rows of one request stand side by side
        bool l1 = n + i < a.N;
        if (l1 && a.cu_q && i > 0 && n + i < end) {
          ++p1;
        } else {
          l1 = l1 && kv4_row(a, n + i, lane, r1, p1);
          end = l1 && a.cu_q ? a.cu_q[r1 + 1] : 0;
        }
        if (lane == i) {
          r = r1;
          pos = p1;
          live = l1;
        }
      }
    }
    if (live && (pos < -1 || (pos < 0 && a.cu_q) || pos >= (a.max_pages << a.lgS) || (a.rope && pos >= a.rope_T))) {
      if (PACK || lane == 0) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
      pos = -1;
    }
    if (!live) pos = -1;
    for (int i = 0; i < nrow; ++i) {
      const int p = PACK ? __shfl_sync(0xffffffffu, pos, i) : pos;
      int nr = 0;  // rungs that reach a row
      for (int k = 0; k < P.n; k += 32) nr += __popc(__ballot_sync(0xffffffffu, k + lane < P.n && rung[k + lane] <= p));
      if (!PACK || lane == i) nk = p < 0 ? 0 : min(P.W, p) + 1 + nr;
    }
    const uint32_t alive = PACK ? __ballot_sync(0xffffffffu, live) : live ? 1u : 0u;
    // this lane's columns (two a column tile) belong to row (8 nt + 2 t + e) / G
    Acc<NT> acc;
    acc.clear();
    const int most = PACK ? gr.keys * nrow : nk;
    if (PACK ? __any_sync(0xffffffffu, nk > 0) : nk > 0) {
      QFrag<NT> q;
      auto at = [&](int col) {
        const int p = PACK ? __shfl_sync(0xffffffffu, pos, col >> a.lgG) : pos;
        return PACK || col < G ? p : -1;
      };
      q.load(static_cast<const TIO*>(a.q) + n * a.q_stride + h * G * kD, a.q_stride, a.lgG, at, a.rope, a.qmul, a.qexp, lane);
      for (int j0 = 32 * mine; j0 < most; j0 += 32 * (KIND == kCluster ? kClusterCtas * kGatherWarps : warps)) {
        // lane i: key i of two tiles, its code row (in 32 bytes from the cache's begin) and its scales
        int j = j0 + lane, kr = 0;
        if (PACK) {
          kr = (int)__umulhi((uint32_t)j, gr.magic);
          j -= kr * gr.keys;
        }
        const int kpos = PACK ? __shfl_sync(0xffffffffu, pos, kr & 7) : pos;
        const int knk = PACK ? __shfl_sync(0xffffffffu, nk, kr & 7) : nk;
        const int kreq = PACK ? __shfl_sync(0xffffffffu, r, kr & 7) : r;
        uint32_t row = kNone;
        uint2 sc = make_uint2(0, 0);
        if (kr < nrow && j < knk) {
          const int Wt = min(P.W, kpos), p = kpos - (j <= Wt ? j : rung[j - Wt - 1]);
          const int page = a.table[(int64_t)kreq * a.max_pages + (p >> a.lgS)], in = p & (S - 1);
          if (page >= 0 && page < a.n_pages) {
            const uint32_t first_row = ((uint32_t)page * a.Hkv + h) * (uint32_t)(9 * S / 4);
            row = first_row + in;
            sc = *reinterpret_cast<const uint2*>(a.cache + (uint64_t)first_row * 32 + 64 * S + 8 * in);
          } else {
            record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
          }
        }
        if (PACK) {  // a NaN value block reaches its own row's columns, and no others (0 * NaN would)
          uint32_t nan = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if ((sc.y >> (8 * b) & 127u) == 127u) nan |= 1u << b;
          uint32_t with = __ballot_sync(0xffffffffu, nan != 0);
          if (with) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (nan >> b & 1) sc.y &= ~(255u << (8 * b));
            for (; with; with &= with - 1) {
              const int k = __ffs(with) - 1;
              const uint32_t kn = __shfl_sync(0xffffffffu, nan, k);
              const int of = __shfl_sync(0xffffffffu, kr, k);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (kn >> (g >> 1) & 1 && of == (2 * t + e) >> a.lgG)
#pragma unroll
                  for (int mt = 0; mt < 4; ++mt) acc.o[0][mt][e] = acc.o[0][mt][2 + e] = __int_as_float(0x7fffffff);
            }
          }
        }
        const bool two = most - j0 > 16;  // (uniform) the second tile has keys
        float s[2][NT][4];
        uint32_t w[2][4], vs[2][4];
        int there = 0, of[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !two) break;
          const int g0 = 16 * i + g;
          const uint32_t ra = __shfl_sync(0xffffffffu, row, g0), rb = __shfl_sync(0xffffffffu, row, g0 + 8);
          const uint32_t sa = __shfl_sync(0xffffffffu, sc.x, g0) >> (8 * t) & 255u;
          const uint32_t sb = __shfl_sync(0xffffffffu, sc.x, g0 + 8) >> (8 * t) & 255u;
          uint2 ka = make_uint2(0, 0), kb = ka;
          if (ra != kNone) ka = *reinterpret_cast<const uint2*>(a.cache + (uint64_t)ra * 32 + 8 * t);
          if (rb != kNone) kb = *reinterpret_cast<const uint2*>(a.cache + (uint64_t)rb * 32 + 8 * t);
          there |= (ra != kNone) << (2 * i) | (rb != kNone) << (2 * i + 1);
          if (PACK) {
            of[2 * i] = (int)__umulhi((uint32_t)(j0 + g0), gr.magic);
            of[2 * i + 1] = (int)__umulhi((uint32_t)(j0 + g0 + 8), gr.magic);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int from = 16 * i + 2 * t + (e & 1) + 8 * (e >> 1);
            const uint32_t rv = __shfl_sync(0xffffffffu, row, from);
            vs[i][e] = __shfl_sync(0xffffffffu, sc.y, from) >> (8 * (g >> 1)) & 255u;
            w[i][e] = rv == kNone ? 0u : *reinterpret_cast<const uint32_t*>(a.cache + (uint64_t)rv * 32 + 32 * S + 4 * g);
          }
          key_products<NT>(q, ka, kb, sa, sb, s[i]);
        }
        softmax_step(
            q, s, [&](int, int e, int i) { return (there >> i & 1) && (!PACK || of[i] == (2 * t + e) >> a.lgG); }, acc.m, acc.l, acc.o);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (i == 0 || two) value_products<NT, kExact>(w[i], vs[i][0] | vs[i][1] << 8, vs[i][2] | vs[i][3] << 8, s[i], acc.o);
      }
    }
    acc.close();
    if (KIND != kCluster && warps == 1) {
      if (alive)
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
            const int of = PACK ? head >> a.lgG : 0;
            if (PACK ? alive >> of & 1 : head < G)
              write_head<TIO>(a, n + of, h * G + (PACK ? head & (G - 1) : head), g, x, acc.m[nt][e], acc.l[nt][e]);
          }
      continue;
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
    // lanes 8 i .. 8 i + 7 of the group's warp w join head 4 w + i, and so on
    const int team = KIND == kCluster ? kGatherWarps : warps, member = KIND == kCluster ? warp : mine, d = lane & 7;
    for (int head = 4 * member + (lane >> 3); live && head < G; head += 4 * team) {
      const float* w = part + ((warp - member) * 8 * NT + head) * 66;
      float m = -INFINITY, l = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int i = 0; i < team; ++i) m = fmaxf(m, w[i * 8 * NT * 66]);
      for (int i = 0; i < team; ++i) {
        const float* wi = w + i * 8 * NT * 66;
        if (wi[1] == 0.0f) continue;
        const float f = wi[0] == -INFINITY ? 0.0f : ex2(wi[0] - m);
        l += wi[1] * f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += wi[2 + 8 * d + e] * f;
      }
      if (KIND != kCluster) {
        write_head<TIO>(a, n, h * G + head, d, x, m, l);
        continue;
      }
      if (d == 0) {
        joined[head][0] = m;
        joined[head][1] = l;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) joined[head][2 + 8 * d + e] = x[e];
    }
    if (KIND != kCluster) {
      __syncthreads();  // the buffer is filled again by the next unit
      continue;
    }
    cluster_sync();
    // CTA `rank` joins heads rank, rank + 8, ..: a warp a head, eight dims a lane
    for (int head = rank + kClusterCtas * warp; live && head < G; head += kClusterCtas * kGatherWarps) {
      float m[kClusterCtas], M = -INFINITY, l = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kClusterCtas; ++c) {
        m[c] = cluster_read(&joined[head][0], c);
        M = fmaxf(M, m[c]);
      }
#pragma unroll
      for (int c = 0; c < kClusterCtas; ++c) {
        const float f = m[c] == -INFINITY ? 0.0f : ex2(m[c] - M);
        l = fmaf(cluster_read(&joined[head][1], c), f, l);
        if (lane < 8)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(cluster_read(&joined[head][2 + 8 * lane + e], c), f, x[e]);
      }
      if (lane < 8) write_head<TIO>(a, n, h * G + head, lane, x, M, l);
    }
    cluster_sync();  // until all have read, before the next unit or the end
  }
}

template <typename TIO, int NT, GatherKind KIND>
static cudaError_t gather(const Kv4Args& a, const Plan& p, int warps, const GatherRows& gr, cudaStream_t s) {
  const int64_t units = (int64_t)((a.N + gr.rows - 1) / gr.rows) * a.Hkv;
  const int per = kGatherWarps / warps;
  const size_t smem = KIND == kCluster || warps > 1 ? (size_t)kGatherWarps * 8 * NT * 66 * sizeof(float) : 0;
  if (KIND == kCluster)
    return launch_pdl_cluster(kv4_gather_kernel<TIO, NT, KIND>, dim3((unsigned)(units * kClusterCtas)), dim3(32 * kGatherWarps),
                              kClusterCtas, smem, s, a, p, warps, gr);
  const int64_t ctas = std::min<int64_t>((units + per - 1) / per, kSMs * 16);
  return launch_pdl(kv4_gather_kernel<TIO, NT, KIND>, dim3((unsigned)ctas), dim3(32 * kGatherWarps), smem, s, a, p, warps, gr);
}

template <typename TIO, GatherKind KIND>
static cudaError_t gather_nt(const Kv4Args& a, const Plan& p, int warps, const GatherRows& gr, cudaStream_t s) {
  const int G = 1 << a.lgG;
  return G > 16  ? gather<TIO, 4, KIND>(a, p, warps, gr, s)
         : G > 8 ? gather<TIO, 2, KIND>(a, p, warps, gr, s)
                 : gather<TIO, 1, KIND>(a, p, warps, gr, s);
}

template <typename TIO>
static cudaError_t gather_any(const Kv4Args& a, const Plan& p, cudaStream_t s) {
  const int64_t keys = std::min<int64_t>((int64_t)p.W + 1 + p.n, (int64_t)a.max_pages << a.lgS), units = (int64_t)a.N * a.Hkv;
  const int tiles = (int)((keys + 15) / 16), G = 1 << a.lgG;
  GatherRows gr = {1, (int)keys, 0};
  if (clustered(a, keys)) return gather_nt<TIO, kCluster>(a, p, kGatherWarps, gr, s);
  // up to a wave of warps: a row's keys go round several, for its latency; beyond, what counts is work
  const int64_t wave = kSMs * 5 * kGatherWarps;
  const bool many = units > wave;
  // Rows side by side while that leaves more than a wave of warps' work, up to 128 keys (16000 rows of 19, 97,
  // 193 keys, 8 / 2 heads: 46 us and 59 a row a warp, 118 and 125, 206 and 201; 2 / 2 heads 33 and 56, 111 and
  // 121, 215 and 196); below it, where few warps end the call, up to 16 (3200 rows of 9, 33, 129 keys: 12.0 and
  // 13.1, 18.6 and 18.4, 43 and 36; 2 / 2 heads 11.6 and 12.4, 23 and 18, 68 and 35)
  if (G < 8 && many && keys <= (units * G / 8 * 4 > 5 * wave ? 128 : 16)) {
    gr.rows = 8 / G;
    gr.keys = std::max(2, gr.keys);  // (2^32 / 1 would not fit)
    gr.magic = (uint32_t)(((1ull << 32) + gr.keys - 1) / gr.keys);  // exact up to 8 * 4096 keys
    return gather<TIO, 1, kPack>(a, p, 1, gr, s);
  }
  return gather_nt<TIO, kOne>(a, p, many || tiles <= 2 ? 1 : tiles <= 4 ? 2 : 4, gr, s);  // two tiles a step
}

// ---------------------------------------------------------------- stream

// The whole prefix, or a wide window: a request's pages stream through shared
// memory.  A team is four warps that compute and one that copies: it reads a
// chunk's page ids, waits for a free slot of the ring (tiles of 64 keys) and
// starts one asynchronous bulk copy a page (64-row pages, whose block is a tile
// as it stands) or three (key codes, value codes, scales).
//
// Work: an item is up to rows_per query rows of one request (a decode step: one
// row), its columns rows x heads of one KV head; its keys are cut into chunks
// of chunk_tiles tiles at absolute places, so what is added to what depends on
// the call's shapes and the row's own length, not on other requests.  The tiles
// of all chunks, in order, are shared out evenly over one wave of teams, whole
// chunks at a time: each CTA adds up the items' tiles (from the lengths, in
// one block-wide scan), and each team takes its part and walks it, the copies
// running on across chunks and items.  The four warps take every fourth tile of a
// chunk and meet in shared memory at its end.  Chunks of a longer item go to the
// workspace, joined by a second kernel.
//
// One column tile: one CTA an SM with four teams, not a CTA a team.  A quarter of
// an SM's registers holds five warps of 96, and four CTAs of five warps fit only
// if each puts its fifth in another quarter; where they did not, three ran, and
// the fourth when all else was done (the batch below: 67 us with the join, and
// 55).  More columns: two CTAs of a team an SM, for their registers (a CTA of two
// teams may have 168 a thread: 64 requests of 4 to 8 rows, 32 columns, 75 us and 71).
//
// Bounded by its instructions, next to the memory: 128 requests of 1024 to 32768
// rows, 8 / 2 heads (167 MB) take 44 us, 3.8 TB/s (the tiles' instructions 28 us
// of it, the memory would take 25; the rest is the start, the chunks' ends and
// an uneven end), one of 400001 rows, 16 / 2 heads (58 MB) 20.
constexpr int kStreamWarps = 4, kSlots = 8;

// Row r of a 16-key tile is key r ^ (r >> 2 & 1): the rows that lanes of one
// shared-memory pass read then lie in different banks, for keys (rows g) and
// values (rows 2t, 2t + 1) alike.
__device__ __forceinline__ int key_of(int r) { return r ^ ((r >> 2) & 1); }

// 16 GB keys (from key k0 of a tile that starts at key j0, its data at T) added
// to the columns' sums.  MASKED: some column may not attend some key.
template <int NT, int GB, bool EXACT, bool MASKED, typename Q>
__device__ __forceinline__ void stream_keys(const Kv4Args& a, const StreamArgs& sa, const Item& it, const Q& q, Acc<NT>& acc,
                                            const uint8_t* T, int j0, int k0, int pages, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int lgr = min(a.lgS, 6);
  const uint8_t* const kt = T + 32 * (k0 + key_of(g)) + 8 * t;
  const uint8_t* const st = T + 64 * kTile + 8 * (k0 + key_of(g)) + t;
  // does column 8 nt + 2 t + e attend key k of the tile?
  auto attends = [&](int nt, int e, int k) {
    const int p = it.pfirst + ((8 * nt + 2 * t + e) >> a.lgG), j = j0 + k;
    return j <= p && j >= p - sa.W && (pages >> (k >> lgr) & 1);
  };
  float s[GB][NT][4];
#pragma unroll
  for (int i = 0; i < GB; ++i) {
    key_products<NT>(q, *reinterpret_cast<const uint2*>(kt + 512 * i), *reinterpret_cast<const uint2*>(kt + 512 * i + 256),
                 (uint32_t)st[128 * i], (uint32_t)st[128 * i + 64], s[i]);
    if (MASKED) {
      const int ka = k0 + 16 * i + key_of(g);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!attends(nt, e, ka)) s[i][nt][e] = -INFINITY;
          if (!attends(nt, e, ka + 8)) s[i][nt][2 + e] = -INFINITY;
        }
    }
  }
  // the statistics move only when a logit passes them by more than kLag
  float top[NT][2];
  bool passes = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
      for (int i = 1; i < GB; ++i) x = fmaxf(x, fmaxf(s[i][nt][e], s[i][nt][2 + e]));
      top[nt][e] = x * q.c[nt][e];
      passes |= top[nt][e] > __fadd_rd(acc.m[nt][e], kLag);
    }
  if (__any_sync(0xffffffffu, passes))
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = top[nt][e];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        if (x > acc.m[nt][e]) {
          const float corr = ex2(acc.m[nt][e] - x);  // 0 on the first keys
          acc.m[nt][e] = x;
          acc.l[nt][e] *= corr;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            acc.o[nt][mt][e] *= corr;
            acc.o[nt][mt][2 + e] *= corr;
          }
        }
      }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float off = acc.m[nt][e] == -INFINITY ? 0.0f : __fsub_rd(kPShift, acc.m[nt][e]);
#pragma unroll
      for (int i = 0; i < GB; ++i) {
        s[i][nt][e] = ex2(fmaf(s[i][nt][e], q.c[nt][e], off));
        s[i][nt][2 + e] = ex2(fmaf(s[i][nt][2 + e], q.c[nt][e], off));
        acc.l[nt][e] += s[i][nt][e] + s[i][nt][2 + e];
      }
    }
  // rows 2t and 2t + 1 of a 16-key tile are keys kv and kv ^ 1
  const int kv = key_of(2 * t), kw = kv ^ 1;
  const uint8_t* const va = T + 32 * kTile + 32 * (k0 + kv) + 4 * g;
  const uint8_t* const vb = T + 32 * kTile + 32 * (k0 + kw) + 4 * g;
  const uint8_t* const sv = T + 64 * kTile + 8 * (k0 + kv) + 4 + (g >> 1);
  const uint8_t* const sw = T + 64 * kTile + 8 * (k0 + kw) + 4 + (g >> 1);
#pragma unroll
  for (int i = 0; i < GB; ++i) {
    const uint32_t w[4] = {*reinterpret_cast<const uint32_t*>(va + 512 * i), *reinterpret_cast<const uint32_t*>(vb + 512 * i),
                           *reinterpret_cast<const uint32_t*>(va + 512 * i + 256), *reinterpret_cast<const uint32_t*>(vb + 512 * i + 256)};
    uint32_t vs[4] = {sv[128 * i], sw[128 * i], sv[128 * i + 64], sw[128 * i + 64]};
    if (MASKED) {
      bool nan = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // rows that are not stored hold anything, a NaN scale perhaps; 0 * NaN must not reach the sums
        const int k = k0 + 16 * i + (e & 1 ? kw : kv) + 8 * (e >> 1);
        if (j0 + k > it.plast() || !(pages >> (k >> lgr) & 1)) vs[e] = 0;
        nan |= (vs[e] & 127u) == 127u;
      }
      if (__any_sync(0xffffffffu, nan)) {
        // a stored NaN reaches the columns that attend it, and no others
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((vs[e] & 127u) == 127u) vs[e] = 0;
#pragma unroll 1
        for (int k = k0 + 16 * i; k < k0 + 16 * i + 16; ++k)
          if ((T[64 * kTile + 8 * k + 4 + (g >> 1)] & 127u) == 127u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (attends(nt, e, k))
#pragma unroll
                  for (int mt = 0; mt < 4; ++mt) acc.o[nt][mt][e] = acc.o[nt][mt][2 + e] = __int_as_float(0x7fffffff);
      }
    }
    value_products<NT, EXACT>(w, vs[0] | vs[1] << 8, vs[2] | vs[3] << 8, s[i], acc.o);
  }
}

// One tile.  With one column tile 32 keys' logits are held at once: 204 clocks
// an SM a tile with its data at hand (197 is what the memory takes to bring
// one); 64 at once take 183, but then 16 warps' registers do not hold the rest.
// Masked tiles, and wider ones, take 16 keys at a time.
template <int NT, bool EXACT, typename Q>
__device__ __forceinline__ void stream_tile(const Kv4Args& a, const StreamArgs& sa, const Item& it, const Q& q, Acc<NT>& acc,
                                            const uint8_t* T, int j0, int pages, int all_pages, int lane) {
  constexpr int GB = NT == 1 ? 2 : 1;  // 16-key groups whose logits are held at once
  const bool full = pages == all_pages && j0 + kTile - 1 <= it.pfirst && j0 >= it.plast() - sa.W;
  if (full) {
#pragma unroll 1
    for (int k = 0; k < kTile; k += 16 * GB) stream_keys<NT, GB, EXACT, false>(a, sa, it, q, acc, T, j0, k, pages, lane);
  } else {
#pragma unroll 1
    for (int k = 0; k < kTile; k += 16) stream_keys<NT, 1, EXACT, true>(a, sa, it, q, acc, T, j0, k, pages, lane);
  }
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// The variant with NT column tiles: teams a CTA, CTAs an SM, shared memory of a team.
template <int NT>
constexpr int kStreamTeams = NT == 1 ? 4 : 1;
template <int NT>
constexpr int kStreamCtas = NT == 1 ? 1 : 2;
template <int NT>
constexpr int kTeamSmem = (kSlots * kTileBytes + 2 * kStreamWarps * 8 * NT * (66 * 4 + 8) + (NT == 4 ? 4 * NT * 512 + 8 * NT * 4 : 0) +
                           8 * (2 * kSlots + 4) + 4 * kSlots + 127) / 128 * 128;

template <typename TIO, int NT>
__global__ void __launch_bounds__(32 * (kStreamWarps + 1) * kStreamTeams<NT>, kStreamCtas<NT>)
    kv4_stream_kernel(const Kv4Args a, const StreamArgs sa) {
  constexpr bool kExact = sizeof(TIO) == 4;
  constexpr int NC = 8 * NT, TEAMS = kStreamTeams<NT>, kThr = 32 * (kStreamWarps + 1) * TEAMS;
  extern __shared__ __align__(128) uint8_t smem_all[];
  __shared__ int sums[kThr / 32];
  __shared__ RunStart where[TEAMS];
  const int tid = threadIdx.x, lane = tid & 31, cta_warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // the teams' computing warps, then their copying ones
  const bool copies = cta_warp >= kStreamWarps * TEAMS;
  const int team = TEAMS == 1 ? 0 : copies ? cta_warp - kStreamWarps * TEAMS : cta_warp / kStreamWarps;
  const int warp = TEAMS == 1 ? cta_warp : cta_warp % kStreamWarps;
  uint8_t* const smem = smem_all + team * kTeamSmem<NT>;
  float* const po = reinterpret_cast<float*>(smem + kSlots * kTileBytes);         // [2][warp][NC][66]
  float2* const ml = reinterpret_cast<float2*>(po + 2 * kStreamWarps * NC * 66);  // [2][warp][NC]
  uint4* const qs = reinterpret_cast<uint4*>(ml + 2 * kStreamWarps * NC);          // NT = 4: [step][column tile][lane]
  float* const qc = reinterpret_cast<float*>(qs + 4 * NT * 32);                   //         [NC]
  // the slots' full and empty barriers, the buffers' (filled by four warps, joined by one)
  uint64_t* const bars = NT == 4 ? reinterpret_cast<uint64_t*>(qc + NC) : reinterpret_cast<uint64_t*>(ml + 2 * kStreamWarps * NC);
  int* const pages = reinterpret_cast<int*>(bars + 2 * kSlots + 4);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kSlots;
  pdl_launch_dependents();
  if (copies && lane == 0) {
    for (int i = 0; i < 2 * kSlots + 4; ++i) mbar_init(full + 8 * i, i == 2 * kSlots || i == 2 * kSlots + 1 ? kStreamWarps : 1);
    mbar_fence_init();
  }
  pdl_wait();

  Cursor cur;
  if (!find_run<kThr, TEAMS>(a, sa, sums, where, team, cur)) return;

  if (copies) {
    copy_run<kSlots>(a, sa, cur, smem_u32(smem), full, empty, pages, cur.at == 0 ? a.debug_skip : -1, lane);
    return;
  }
  const int G = 1 << a.lgG;
  const int all_pages = (1 << (kTile >> min(a.lgS, 6))) - 1;
  std::conditional_t<NT == 4, QShared<NT>, QFrag<NT>> q;
  Acc<NT> acc;
  int qx = -1, qh = -1, n0 = 0, nchunk = 0;  // n0, nchunk: tiles and chunks of the run before this one
  bool dead = false;                         // a wait ran out: no more waits, no more work
  auto wait = [&](uint32_t bar, int phase) {
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_bounded(bar, phase, a.wait_cycles));
  };
  do {
    const int ncol = cur.it.nrows << a.lgG;
    if (cur.x != qx || cur.h != qh) {
      const TIO* base = static_cast<const TIO*>(a.q) + (int64_t)cur.it.row0 * a.q_stride + cur.h * G * kD;
      auto at = [&](int col) { return col < ncol ? cur.it.pfirst + (col >> a.lgG) : -1; };
      if constexpr (NT == 4) {  // a column tile a warp
        static_assert(NT == kStreamWarps && TEAMS == 1, "a column tile a warp; one team at the barrier");
        uint32_t hi[8], lo[8];
        const float back = load_queries(base, a.q_stride, a.lgG, at(8 * warp + g), a.rope, a.qmul, a.qexp, warp, lane, hi, lo);
        bar_sync(1, 32 * kStreamWarps);  // the last item's queries have been used
        if (t == 0) qc[8 * warp + g] = back;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          qs[(ks * NT + warp) * 32 + lane] = make_uint4(hi[2 * ks], hi[2 * ks + 1], lo[2 * ks], lo[2 * ks + 1]);
        bar_sync(1, 32 * kStreamWarps);
        q.frag = smem_u32(qs + lane);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) q.c[nt][e] = qc[8 * nt + 2 * t + e];
      } else {
        q.load(base, a.q_stride, a.lgG, at, a.rope, a.qmul, a.qexp, lane);
      }
      qx = cur.x;
      qh = cur.h;
    }
    acc.clear();
    for (int k = warp; k < cur.te - cur.tb; k += kStreamWarps) {
      const int n = n0 + k, slot = n % kSlots;
      wait(full + 8 * slot, n / kSlots & 1);
      if (dead) break;
      stream_tile<NT, kExact>(a, sa, cur.it, q, acc, smem + slot * kTileBytes, (cur.tb + k) * kTile, pages[slot], all_pages, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * slot);
    }
    n0 += cur.te - cur.tb;
    // The four warps' sums meet in one of two buffers.  No warp waits for the others here: the
    // warps take turns at joining a chunk's sums, and a buffer is waited for when it is filled again.
    acc.close();
    const int buf = nchunk & 1, round = nchunk >> 1;
    const uint32_t in = full + 8 * (2 * kSlots + buf), out_ = in + 16;
    if (round > 0) wait(out_, (round - 1) & 1);
    float* const pb = po + buf * kStreamWarps * NC * 66;
    float2* const mb = ml + buf * kStreamWarps * NC;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * nt + 2 * t + e;
        if (col >= ncol) continue;
        if (g == 0) mb[warp * NC + col] = make_float2(acc.m[nt][e], acc.l[nt][e]);
        float* out = pb + (warp * NC + col) * 66 + 8 * g;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) *reinterpret_cast<float2*>(out + 2 * mt) = make_float2(acc.o[nt][mt][e], acc.o[nt][mt][2 + e]);
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(in);
    if (warp != (nchunk++ & 3)) continue;
    wait(in, round & 1);
    for (int i = lane; i < 8 * ncol; i += 32) {  // eight lanes a column
      const int col = i >> 3, d = i & 7;
      float M = -INFINITY, l = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kStreamWarps; ++w) M = fmaxf(M, mb[w * NC + col].x);
#pragma unroll
      for (int w = 0; w < kStreamWarps; ++w) {
        const float2 v = mb[w * NC + col];
        const float f = v.x == -INFINITY ? 0.0f : ex2(v.x - M);
        l = fmaf(v.y, f, l);
        const float* y = pb + (w * NC + col) * 66 + 8 * d;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 z = *reinterpret_cast<const float2*>(y + e);
          x[e] = fmaf(z.x, f, x[e]);
          x[e + 1] = fmaf(z.y, f, x[e + 1]);
        }
      }
      if (cur.it.nch == 1) {
        write_head<TIO>(a, cur.it.row0 + (col >> a.lgG), cur.h * G + (col & (G - 1)), d, x, M, l);
      } else {
        const int64_t at = (((int64_t)cur.x * a.Hkv + cur.h) * sa.max_chunks + cur.c - cur.it.c0) * (G << sa.lg_rows) + col;
        store8(sa.part_o + at * kD + 8 * d, x);
        if (d == 0) sa.part_ml[at] = make_float2(M, l);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(out_);
  } while (cur.next(a, sa));
  if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
}

// (m, l, 8 sums) of some keys of a column; what other keys gave is added.
struct Part {
  float m = -INFINITY, l = 0.0f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  __device__ __forceinline__ void add(float m2, float l2, const float* z) {
    const float top = fmaxf(m, m2);
    const float f = m2 == -INFINITY ? 0.0f : ex2(m2 - top), back = m == -INFINITY ? 0.0f : ex2(m - top);
    m = top;
    l = fmaf(l, back, l2 * f);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], back, z[e] * f);
  }
  // lanes `step`, 2 step, .. apart
  __device__ __forceinline__ void add_lanes(int step) {
    for (int o = step; o < 32; o <<= 1) {
      float z[8];
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = __shfl_xor_sync(0xffffffffu, y[e], o);
      add(m2, l2, z);
    }
  }
};

// The chunks of one (item, KV head) joined: `lanes` lanes a CTA, each 8 dims of a
// column (8 or all 32 of four columns, or 2 of one, where columns are few), the
// chunks dealt out over the groups of lanes (their partial sums are read once,
// 264 bytes each: what counts is how many are in flight).  Bounded by latency:
// with the end of the grid before it, 6.5 us of 27 for a row of 400001 keys (782
// parts a head), 4 of 49 for 128 requests of 1024 to 32768.
constexpr int kJoinThreads = 512;

template <typename TIO>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4Args a, const StreamArgs sa, int lanes) {
  __shared__ float red[kJoinThreads / 32][10][32];
  pdl_launch_dependents();
  pdl_wait();
  const int x = blockIdx.x / a.Hkv, h = blockIdx.x - x * a.Hkv;
  const Item it = item_at(a, sa, x);
  const int ncol = it.nrows << a.lgG, G = 1 << a.lgG, width = G << sa.lg_rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int i = threadIdx.x & (lanes - 1), at8 = blockIdx.y * lanes + i, d = at8 & 7;  // the lane among all columns' lanes
  if (it.nch <= 1 || blockIdx.y * lanes >= 8 * ncol) return;
  const int col = min(at8 >> 3, ncol - 1);
  const int64_t at = ((int64_t)blockIdx.x * sa.max_chunks) * width + col;
  Part p;
#pragma unroll 4
  for (int c = threadIdx.x / lanes; c < it.nch; c += blockDim.x / lanes) {
    const float2 v = sa.part_ml[at + (int64_t)c * width];
    float z[8];
    load8(sa.part_o + (at + (int64_t)c * width) * kD + 8 * d, z);
    p.add(v.x, v.y, z);
  }
  p.add_lanes(lanes);
  red[warp][8][lane] = p.m;
  red[warp][9][lane] = p.l;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[warp][e][lane] = p.y[e];
  __syncthreads();
  if (warp > 0) return;
  // 32 / lanes warps' sums at a time
  Part q;
  for (int w = lane / lanes; w < warps; w += 32 / lanes) {
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = red[w][e][i];
    q.add(red[w][8][i], red[w][9][i], z);
  }
  q.add_lanes(lanes);
  if (lane < lanes && at8 < 8 * ncol) write_head<TIO>(a, it.row0 + (col >> a.lgG), h * G + (col & (G - 1)), d, q.y, q.m, q.l);
}

// The stream kernel's shape for a call; items = 0: the gather kernel takes it.
struct StreamShape {
  StreamArgs s;
  int nt, teams;
  int64_t slots;  // chunks the workspace has room for
  size_t bytes;   // the workspace
};

static StreamShape stream_shape(const Kv4Args& a, const Plan& p, bool ragged) {
  StreamShape z = {};
  const int64_t cap = (int64_t)a.max_pages << a.lgS;
  // few keys, or a wave of rows with few, or of clusters with some: one launch and
  // no workspace win.  (A cluster's keys: 16 units of 3000, 9.7 us streamed and
  // 10.0; 76 units of 4000, 17.5 and 15.0; 2 units of 2000 and 4000, 8.4 and 8.5
  // streamed, 7.9 and 9.4.)
  const int64_t keys = std::min<int64_t>(cap, (int64_t)p.W + 1), units_n = (int64_t)a.N * a.Hkv;
  if (p.n > 0 || keys <= 64 || (keys <= 512 && units_n <= 4 * kSMs)) return z;
  if (keys <= (units_n >= 16 ? 4096 : 2048) && clustered(a, keys)) return z;
  const int G = 1 << a.lgG;
  // columns a warp holds: as many rows as a request brings on average, 32 at most
  const int avg = ragged ? (a.N + a.R - 1) / a.R : 1;
  z.nt = G * avg > 16 ? 4 : G * avg > 8 ? 2 : 1;
  z.nt = std::max(z.nt, G > 16 ? 4 : G > 8 ? 2 : 1);
  // more than 32 columns: the tensor memory kernel (nt = 32; 64 requests of up to 20000 rows, 8 / 2 heads,
  // 12 rows each: 113 us, and 150 us in items of 32 columns; 6 rows each: 113 and 85; both a quarter less since)
  if (ragged && G * avg > 32) z.nt = kPromptColumns / 8;
  z.s.lg_rows = ragged ? __builtin_ctz((unsigned)(8 * z.nt / std::min(G, 8 * z.nt))) : 0;
  z.s.items = ragged ? (a.N >> z.s.lg_rows) + a.R : a.R;
  z.s.W = p.W;
  z.s.limit = (int)(a.rope ? std::min<int64_t>(cap, a.rope_T) : cap);
  z.teams = kSMs * (z.nt == 1 ? kStreamTeams<1> * kStreamCtas<1> : kStreamTeams<4> * kStreamCtas<4>);
  const int64_t units = (int64_t)z.s.items * a.Hkv;
  if (z.nt == kPromptColumns / 8) {  // cuts its work otherwise
    z.s.chunk_tiles = 1 << 18;
    z.s.lg_chunk = 18;
    z.s.max_chunks = 1;
    z.bytes = prompt_workspace(units);
    return z;
  }
  // chunks: 512 keys (two tiles a warp), 256 where that would leave teams without
  // one; more where the whole block table's worth of them would pass 16 a team
  // (which bounds the workspace; the teams' shares differ by a chunk at most)
  int64_t ck = (cap + 511) / 512 * units <= z.teams ? 256 : 512;
  while (ck < cap && (cap + ck - 1) / ck * units > 16 * z.teams) ck *= 2;
  // up to 2048 keys one chunk, without workspace and join (128 requests of 300 to 1900, 8 / 4 heads: 25.0 and
  // 21.0 us, 80 of 8 / 2 heads 14.8 and 14.4); with more columns only if there is one for each team (32: 100
  // requests 27.6 and 30.1, 300 47.0 and 45.4)
  if (cap <= 2048 && (z.nt == 1 || units >= z.teams)) ck = 2048;
  z.s.chunk_tiles = (int)(ck / kTile);
  z.s.lg_chunk = __builtin_ctz((unsigned)z.s.chunk_tiles);
  z.s.max_chunks = (int)((cap + ck - 1) / ck);
  z.slots = z.s.max_chunks > 1 ? units * z.s.max_chunks : 0;
  z.bytes = (size_t)z.slots * ((size_t)66 * 4 << (a.lgG + z.s.lg_rows));
  return z;
}

template <typename TIO>
static cudaError_t join(const Kv4Args& a, const StreamShape& z, cudaStream_t s) {
  if (z.slots == 0) return cudaSuccess;
  const int width = 1 << (a.lgG + z.s.lg_rows);
  // enough columns to fill the card: up to four a CTA, eight groups (four beyond a wave of CTAs of eight);
  // else a quarter column a CTA (400001 keys of 16 columns: 10.5 us with whole ones, 16 CTAs, and 8), and
  // groups for two chunks each
  const int64_t columns = (int64_t)z.s.items * a.Hkv * width;
  const bool fills = columns >= 4 * kSMs;
  const int lanes = fills ? std::min(32, 8 * width) : 2;
  int groups = !fills ? 32 : 8 * columns / lanes > 4 * kSMs ? 4 : 8;
  while (!fills && groups < kJoinThreads / 2 && 2 * groups < z.s.max_chunks) groups *= 2;
  return launch_pdl(kv4_join_kernel<TIO>, dim3((unsigned)(z.s.items * a.Hkv), (unsigned)(8 * width / lanes)), dim3(lanes * groups), 0, s, a,
                    z.s, lanes);
}

template <typename TIO, int NT>
static cudaError_t stream(const Kv4Args& a, const StreamShape& z, cudaStream_t s) {
  constexpr int smem = kStreamTeams<NT> * kTeamSmem<NT>;
  static_assert((smem + 512 + 1024) * kStreamCtas<NT> <= 228 * 1024, "CTAs an SM");
  const cudaError_t e = cudaFuncSetAttribute(kv4_stream_kernel<TIO, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_stream_kernel<TIO, NT>, dim3(kSMs * kStreamCtas<NT>), dim3(32 * (kStreamWarps + 1) * kStreamTeams<NT>), (size_t)smem, s,
                    a, z.s);
}

template <typename TIO>
static cudaError_t stream_and_join(const Kv4Args& a, const StreamShape& z, cudaStream_t s) {
  const cudaError_t e = z.nt == 1 ? stream<TIO, 1>(a, z, s) : z.nt == 2 ? stream<TIO, 2>(a, z, s) : stream<TIO, 4>(a, z, s);
  return e == cudaSuccess ? join<TIO>(a, z, s) : e;
}

bool kv4_attend_fits(const Kv4Args& a, const Plan& p, bool ragged) {
  const StreamShape z = stream_shape(a, p, ragged);
  const int64_t tiles = ((int64_t)a.max_pages << a.lgS) / kTile + 1;
  return (int64_t)z.s.items * a.Hkv * (tiles + (z.s.max_chunks + 1LL) * kChunkCost) < (1LL << 31);
}

size_t kv4_attend_workspace(const Kv4Args& a, const Plan& p, bool ragged) {
  return stream_shape(a, p, ragged).bytes;
}

int launch_kv4_attend(const Kv4Args& a, const Plan& p, int dtype, void* ws, void* stream_) {
  cudaStream_t s = (cudaStream_t)stream_;
  LaunchTimer tm(SFA_KERNEL_KV4_ATTEND, stream_);
  cudaError_t e;
  StreamShape z = stream_shape(a, p, a.cu_q != nullptr);
  if (z.s.items > 0) {
    z.s.row_bytes = a.Hq * kD * (dtype == SFA_BF16 ? 2 : 4);
    z.s.part_o = static_cast<float*>(ws);
    z.s.part_ml = reinterpret_cast<float2*>(z.s.part_o + ((size_t)z.slots * kD << (a.lgG + z.s.lg_rows)));
    e = z.nt == kPromptColumns / 8 ? launch_kv4_prompt(a, z.s, dtype, ws, s)
        : dtype == SFA_BF16        ? stream_and_join<bf16>(a, z, s)
                                   : stream_and_join<float>(a, z, s);
    return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
  }
  e = dtype == SFA_BF16 ? gather_any<bf16>(a, p, s) : gather_any<float>(a, p, s);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
