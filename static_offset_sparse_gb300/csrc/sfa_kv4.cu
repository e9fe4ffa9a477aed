// The paged 4-bit cache's bookkeeping, its write and its read-back: block
// tables and slot maps from request lengths, rotate + quantise + store, and
// rows as numbers.
#include <math.h>

#include <algorithm>

#include "sfa_kv4.cuh"
#include "sfa_launch.cuh"

namespace sfa {

// ---------------------------------------------------------------- plan

// One serving step.  Per request: pages released (n_new = -1) and pages newly
// needed, prefix sums of both and of the new rows; released pages are pushed
// on the stack of free pages in (request, page) order, then new pages are
// popped in (request, page) order.  The work is a few hundred bytes a request
// and bounded by latency, so one CTA does all of it between barriers (no
// atomics: the same inputs give the same pages); the row maps of more than
// kPlanRows rows are left to a second kernel over the whole card (47458 rows:
// 8.7 us, and 15 in the one CTA; 4096 rows 5.1 and 5.9; 2048 in the one CTA 4.5;
// 256 requests of a row each, with pages to move, 5.0).
constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 2 * kPlanThreads;

struct PlanArgs {
  const int32_t* n_new;
  const int32_t* lens;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* cu;
  int32_t* slots;
  int32_t* pos;
  int32_t* lens_out;
  int32_t* n_free_out;
  int32_t R, N, max_pages, n_pages, lgS;
  int* status;
};

// First index whose inclusive prefix exceeds x.
__device__ __forceinline__ int upper(const int* inc, int n, int x) {
  int lo = 0, len = n;
  while (len > 0) {
    const int half = len >> 1;
    if (inc[lo + half] <= x) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo;
}

__device__ __forceinline__ void put_row(const PlanArgs& a, int row, int p, const int32_t* trow) {
  const int page = trow[p >> a.lgS];
  const bool fine = page >= 0 && page < a.n_pages;
  if (!fine) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
  a.slots[row] = fine ? (page << a.lgS) + (p & ((1 << a.lgS) - 1)) : -1;
  a.pos[row] = p;
}

// MANY: more than a request a thread, whose numbers go through shared memory, so
// that neighbouring threads read neighbouring requests (8192 requests 24 us, and
// 17 so; with one a thread the detour costs 0.2 of 5).
template <bool MANY>
__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const PlanArgs a, int rows_here) {
  extern __shared__ int sm[];
  int* const back = sm;            // inclusive prefix of released pages
  int* const need = sm + a.R;      // of new pages
  int* const rows = sm + 2 * a.R;  // of new rows
  int* const kept = sm + 3 * a.R;  // rows that a request keeps
  __shared__ long long wsum[3][32];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid == 0) bad = 0;
  pdl_wait();
  __syncthreads();
  const int S1 = (1 << a.lgS) - 1;
  const long long cap = (long long)a.max_pages << a.lgS;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const int nf = *a.n_free;
  long long s[3] = {0, 0, 0};
  for (int r = MANY ? tid : r0; r < (MANY ? a.R : r1); r += MANY ? kPlanThreads : 1) {
    const int nn = a.n_new[r], len = a.lens[r];
    if (nn < -1 || len < 0 || len > cap || len + (long long)max(nn, 0) > cap) bad = 1;
    const int held = (len + S1) >> a.lgS;
    const int b = nn < 0 ? held : 0;
    const int keep = nn < 0 ? 0 : len;
    const int add = max(nn, 0);
    const int nd = (int)(((long long)keep + add + S1) >> a.lgS) - (held - b);
    if (!MANY) {
      s[0] += b;
      s[1] += nd;
      s[2] += add;
    }
    kept[r] = keep;
    back[r] = b;
    need[r] = nd;
    rows[r] = add;
  }
  if (MANY) {
    __syncthreads();
    for (int r = r0; r < r1; ++r) {
      s[0] += back[r];
      s[1] += need[r];
      s[2] += rows[r];
    }
  }
  long long mine[3] = {s[0], s[1], s[2]};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long x = __shfl_up_sync(0xffffffffu, s[i], off);
      if (lane >= off) s[i] += x;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) wsum[i][warp] = s[i];
  __syncthreads();
  long long tot[3], ex[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long x = wsum[i][lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    tot[i] = __shfl_sync(0xffffffffu, x, 31);
    const long long before = __shfl_sync(0xffffffffu, x, max(0, warp - 1));
    ex[i] = (warp ? before : 0) + s[i] - mine[i];
  }
  // nothing is changed unless the whole step fits
  const bool fits = tot[1] <= nf + tot[0] && nf + tot[0] <= a.n_pages && tot[2] <= a.N && nf >= 0;
  if (bad || !fits) {
    if (tid == 0) record_status(a.status, bad || nf < 0 || nf + tot[0] > a.n_pages ? SFA_ERR_DEVICE_BOUNDS : SFA_ERR_CAPACITY);
    for (int r = tid; r <= a.R; r += kPlanThreads) a.cu[r] = 0;
    for (int r = tid; r < a.R; r += kPlanThreads) a.lens_out[r] = a.lens[r];
    if (tid == 0) *a.n_free_out = nf;
    if (rows_here)
      for (int i = tid; i < a.N; i += kPlanThreads) a.slots[i] = a.pos[i] = -1;
    return;
  }
  const int left = nf + (int)tot[0] - (int)tot[1];
  for (int r = r0; r < r1; ++r) {
    const int add = rows[r];
    ex[0] += back[r];
    ex[1] += need[r];
    ex[2] += add;
    back[r] = (int)ex[0];
    need[r] = (int)ex[1];
    rows[r] = (int)ex[2];
    if (!MANY) {
      a.cu[r + 1] = (int)ex[2];
      a.lens_out[r] = kept[r] + add;
    }
  }
  if (tid == 0) {
    a.cu[0] = 0;
    *a.n_free_out = left;
  }
  __syncthreads();
  if (MANY)
    for (int r = tid; r < a.R; r += kPlanThreads) {
      a.cu[r + 1] = rows[r];
      a.lens_out[r] = kept[r] + rows[r] - (r ? rows[r - 1] : 0);
    }
  // the page at place x of the stack: the old free pages, then the released ones
  auto stacked = [&](int x) {
    if (x < nf) return a.free_pages[x];
    const int k = x - nf, r = upper(back, a.R, k);
    return a.table[(int64_t)r * a.max_pages + k - (r ? back[r - 1] : 0)];
  };
  const int top = nf + (int)tot[0];
  for (int k = tid; k < (int)tot[1]; k += kPlanThreads) {
    const int r = upper(need, a.R, k);
    const int j = ((kept[r] + S1) >> a.lgS) + k - (r ? need[r - 1] : 0);
    a.table[(int64_t)r * a.max_pages + j] = stacked(top - 1 - k);
  }
  for (int x = nf + tid; x < left; x += kPlanThreads) a.free_pages[x] = stacked(x);
  if (!rows_here) return;
  __syncthreads();
  for (int i = tid; i < a.N; i += kPlanThreads) {
    if (i >= (int)tot[2]) {
      a.slots[i] = a.pos[i] = -1;
      continue;
    }
    const int r = upper(rows, a.R, i);
    put_row(a, i, kept[r] + i - (r ? rows[r - 1] : 0), a.table + (int64_t)r * a.max_pages);
  }
}

// The row maps of a large step, a warp 32 rows: the first one's request by a
// search of 32 boundaries at a time, the others' among the 32 after it, and the
// next, held by the lanes.
__global__ void __launch_bounds__(256) kv4_plan_rows_kernel(const PlanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, i0 = i - lane;
  if (i0 >= a.N) return;
  const int last = a.cu[a.R];
  if (i0 >= last) {
    if (i < a.N) a.slots[i] = a.pos[i] = -1;
    return;
  }
  // the first request whose end lies beyond i0
  int lo = 0, len = a.R;
  while (len > 1) {
    const int step = (len + 31) >> 5, at = lane * step;
    const bool le = at < len && a.cu[lo + at] <= i0;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;  // cu does not decrease: the first k + 1 of them
    lo += k * step;
    len = min(step, len - k * step);
  }
  int r = -1, end = 0;
  for (; __any_sync(0xffffffffu, r < 0 && i < last); lo += 32) {
    const int mine = lo + lane < a.R ? a.cu[lo + lane + 1] : 0x7fffffff;
    int k = 0;  // ends among the 32 that are not beyond i
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) k += __shfl_sync(0xffffffffu, mine, k + s - 1) <= i ? s : 0;
    const int e = __shfl_sync(0xffffffffu, mine, k);
    if (r < 0 && i < last && e > i) {
      r = lo + k;
      end = e;
    }
  }
  if (r >= 0)
    put_row(a, (int)i, a.lens_out[r] - (end - (int)i), a.table + (int64_t)r * a.max_pages);
  else if (i < a.N)
    a.slots[i] = a.pos[i] = -1;
}

// ---------------------------------------------------------------- append

struct AppendArgs {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;  // elements between rows
  uint8_t* cache;
  const int32_t* slots;
  const int32_t* pos;
  const float2* rope;
  int32_t N, Hkv, lgS, n_pages, rope_T;
  float kscale, vscale, inv_kscale, inv_vscale;
  int* status;
};

// The largest size of three numbers; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// a / b from r = 1 / b, both quotients rounded to nearest: Markstein's theorem
// ("Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): with r the rounded reciprocal, one correction of a r by its exact
// remainder rounds correctly while nothing leaves the range of normal numbers.
// 3 operations, on two numbers at once, where a division takes about ten.
__device__ __forceinline__ float2 divide(float2 a, float b, float r) {
  const float2 r2 = make_float2(r, r), q = fma2(a, r2, make_float2(-0.0f, -0.0f));
  return fma2(fma2(q, make_float2(-b, -b), a), r2, q);
}

// 16 numbers -> 8 bytes of codes and their scale.  The numbers are first divided
// by `by` (its rounded reciprocal inv); scale = e4m3(amax / 6) to nearest even,
// 448 at most; code = e2m1(x / scale) to nearest even.  All quotients are the
// correctly rounded ones, so the bytes are a function of the numbers alone.  A
// NaN among them gives a NaN scale; a zero scale has zero codes.
template <typename DIV>
__device__ __forceinline__ uint2 quantise16_by(float* x, float m, float by, float inv, uint32_t& scale, DIV div) {
  if (by != 1.0f) {
    m = __fdiv_rn(m, by);  // rounding is monotone: the largest stays the largest
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 y = div(make_float2(x[e], x[e + 1]), by, inv);
      x[e] = y.x;
      x[e + 1] = y.y;
    }
  }
  scale = __nv_cvt_float_to_fp8(__fdiv_rn(m, 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = unpack_f16(e4m3x2_f16x2(scale)).x;
  if (s == 0.0f) return make_uint2(0, 0);
  const float r = __fdiv_rn(1.0f, s);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = div(make_float2(x[8 * h + 2 * e], x[8 * h + 2 * e + 1]), s, r);
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(w[h])
        : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
  }
  return make_uint2(w[0], w[1]);
}

// The rare blocks (all but zero, huge, infinite, NaN) apart: their divisions
// would fill the instruction cache of the others.
__device__ __noinline__ uint2 quantise16_rare(const float* x, float m, float by, uint32_t* scale) {
  float y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = x[e];
  return quantise16_by(y, m, by, 0.0f, *scale, [](float2 a, float b, float) { return make_float2(__fdiv_rn(a.x, b), __fdiv_rn(a.y, b)); });
}

__device__ __forceinline__ uint2 quantise16(float* x, float by, float inv, uint32_t& scale) {
  float m = max_abs(x[0], x[1], x[1]);
#pragma unroll
  for (int e = 2; e < 16; e += 2) m = max_abs(m, x[e], x[e + 1]);
  // where remainders are exact (what lies 2^-60 below the largest has code 0 either way)
  if (m >= 0x1p-40f && m <= 0x1p60f && by >= 0x1p-40f && by <= 0x1p40f) return quantise16_by(x, m, by, inv, scale, divide);
  float y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = x[e];
  uint32_t s;
  const uint2 c = quantise16_rare(y, m, by, &s);
  scale = s;
  return c;
}

template <typename TIO>
__device__ __forceinline__ void load16(const TIO* p, float* x) {
  load8(p, x);
  load8(p + 8, x + 8);
}

// Four threads a (row, head): two on the key, each with 16 rotation pairs (dims
// 16u.. and 32 + 16u..: two whole scale blocks), two on the value, in another
// warp, which has no rotation to go through.
// 2 * 64 elements in, 72 bytes out, but bounded by instructions and the loads'
// latency: 32741 rows of 2 heads in bf16 (22 MB, and 8 of the RoPE table) take
// 7.5 us, 5.5 of them without rotation (8.0 with the rows asked for when the
// slot is there, 8.2 with one number divided at a time besides).
template <typename TIO>
__global__ void __launch_bounds__(256) kv4_append_kernel(const AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t unit = blockIdx.x * 64u + (threadIdx.x >> 6) * 16u + ((threadIdx.x & 31) >> 1);  // (N * Hkv <= 2^27)
  const int u = threadIdx.x & 1;
  const bool value = threadIdx.x & 32;
  const int n = (int)(unit / (uint32_t)a.Hkv), h = (int)unit - n * a.Hkv;
  int slot = -1, p = 0;
  float lo[16], hi[16];
  if (n < a.N) {
    slot = a.slots[n];
    p = a.pos[n];
    // on their way while the slot is
    const TIO* row = value ? static_cast<const TIO*>(a.v) + n * a.v_stride + h * kD
                           : static_cast<const TIO*>(a.k) + n * a.k_stride + h * kD;
    load16(row + 16 * u, lo);
    load16(row + 32 + 16 * u, hi);
    // (a row is written whole or not at all)
    if (slot >= 0 && ((slot >> a.lgS) >= a.n_pages || (a.rope && (p < 0 || p >= a.rope_T)))) {
      record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
      slot = -1;
    }
  }
  uint32_t s0 = 0, s1 = 0;
  uint8_t* block = nullptr;
  const int S = 1 << a.lgS, at = slot & (S - 1);
  if (slot >= 0) {
    block = a.cache + ((int64_t)(slot >> a.lgS) * a.Hkv + h) * (kKv4Row * S);
    if (!value && a.rope) {
#pragma unroll
      for (int c = 0; c < 16; c += 8) {
        float cs[8], sn[8];
        load_rope8(a.rope, p, 16 * u + c, cs, sn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // each product rounded by itself
          const float x = lo[c + e], y = hi[c + e];
          lo[c + e] = __fsub_rn(__fmul_rn(x, cs[e]), __fmul_rn(y, sn[e]));
          hi[c + e] = __fadd_rn(__fmul_rn(x, sn[e]), __fmul_rn(y, cs[e]));
        }
      }
    }
    const float sc = value ? a.vscale : a.kscale, inv = value ? a.inv_vscale : a.inv_kscale;
    const uint2 c0 = quantise16(lo, sc, inv, s0), c1 = quantise16(hi, sc, inv, s1);
    uint8_t* codes = block + (value ? 32 * S : 0) + 32 * at;
    *reinterpret_cast<uint2*>(codes + 8 * u) = c0;
    *reinterpret_cast<uint2*>(codes + 16 + 8 * u) = c1;
  }
  // the four scales leave in one store
  uint32_t w = (s0 << (8 * u)) | (s1 << (16 + 8 * u));
  w |= __shfl_xor_sync(0xffffffffu, w, 1);
  if (block && u == 0) *reinterpret_cast<uint32_t*>(block + 64 * S + 8 * at + (value ? 4 : 0)) = w;
}

// ---------------------------------------------------------------- read

struct ReadArgs {
  const uint8_t* cache;
  const int32_t* slots;
  void* k;
  void* v;
  int32_t N, Hkv, lgS, n_pages;
  float kscale, vscale;
  int* status;
};

template <typename TIO>
__device__ __forceinline__ void to_words(const float* x, uint32_t* w) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if constexpr (sizeof(TIO) == 4) w[e] = __float_as_uint(x[e]);
  if constexpr (sizeof(TIO) == 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
}

// Eight threads a (row, head), one for each scale block of its key and value.
// Bounded by memory once there is enough to do: 65536 rows of 2 heads in bf16
// (43 MB moved) take 8.9 us, 4.9 TB/s, 32741 in fp32 (38 MB) 7.4; a few hundred
// rows 2 us, latency alone.
template <typename TIO>
__global__ void __launch_bounds__(256) kv4_read_kernel(const ReadArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, unit = i >> 3;  // (N * Hkv <= 2^27)
  const int n = (int)(unit / (uint32_t)a.Hkv);
  const int part = (int)(i & 7), h = (int)unit - n * a.Hkv, S = 1 << a.lgS;
  const bool value = part >= 4;
  const int slot = n < a.N ? a.slots[n] : -1;
  float x[16];
  if (slot >= 0 && (slot >> a.lgS) < a.n_pages) {
    const int at = slot & (S - 1);
    const uint8_t* block = a.cache + ((int64_t)(slot >> a.lgS) * a.Hkv + h) * (kKv4Row * S);
    const uint2 c = *reinterpret_cast<const uint2*>(block + (value ? 32 * S : 0) + 32 * at + 8 * (part & 3));
    const float s = unpack_f16(e4m3x2_f16x2(block[64 * S + 8 * at + part])).x;
    const float sc = value ? a.vscale : a.kscale;
    uint32_t y[8];
    e2m1x8_f16(c.x, y);
    e2m1x8_f16(c.y, y + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack_f16(y[e]);
      x[2 * e] = (f.x * s) * sc;
      x[2 * e + 1] = (f.y * s) * sc;
    }
  } else {
    if (slot >= 0) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
  }
  // Two lanes write a sector of 32 bytes together, first the even one's, then the odd one's: each store
  // then fills its sectors (in halves the fp32 rows above took 10.5 us).
  constexpr int kSectors = sizeof(TIO) / 2;  // of a lane's 16 numbers
  uint32_t w[8 * kSectors];
  to_words<TIO>(x, w);
  TIO* const mine = static_cast<TIO*>(value ? a.v : a.k) + (int64_t)unit * kD + 16 * (part & 3);
  const bool odd = part & 1;
#pragma unroll
  for (int j = 0; j < kSectors; ++j) {
    uint32_t* const v = w + 8 * j;
    uint32_t got[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) got[e] = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[4 + e], 1);
    if (n >= a.N) continue;
    uint4* const even_sector = reinterpret_cast<uint4*>(mine - (odd ? 16 : 0)) + 2 * j + odd;
    uint4* const odd_sector = reinterpret_cast<uint4*>(mine + (odd ? 0 : 16)) + 2 * j + odd;
    *even_sector = odd ? make_uint4(got[0], got[1], got[2], got[3]) : make_uint4(v[0], v[1], v[2], v[3]);
    *odd_sector = odd ? make_uint4(v[4], v[5], v[6], v[7]) : make_uint4(got[0], got[1], got[2], got[3]);
  }
}

// ---------------------------------------------------------------- entry points

static bool at16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool at4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

static int check_pool(const sfa_kv4_desc* d) {
  if (!d || d->n_pages <= 0 || d->page <= 0 || d->N < 0) return SFA_ERR_INVALID_ARG;
  if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128) return SFA_ERR_UNSUPPORTED;
  if ((int64_t)d->n_pages * d->page >= (1LL << 31)) return SFA_ERR_UNSUPPORTED;
  return SFA_OK;
}

// Below 128 GiB: rows of 32 bytes are counted in 32 bits.
static bool cache_fits(const sfa_kv4_desc* d, int Hkv) {
  return (int64_t)d->n_pages * d->page <= ((1LL << 37) - 1) / kKv4Row / Hkv;
}

// What append, read and attend share.
static int check_rows(const sfa_kv4_desc* d) {
  const int rc = check_pool(d);
  if (rc != SFA_OK) return rc;
  if (d->Hkv <= 0 || (d->dtype != SFA_F32 && d->dtype != SFA_BF16)) return SFA_ERR_INVALID_ARG;
  if (!(d->kscale > 0.0f && d->kscale <= 3.4e38f && d->vscale > 0.0f && d->vscale <= 3.4e38f)) return SFA_ERR_INVALID_ARG;
  if (d->D != kD || (int64_t)d->N * d->Hkv > (1 << 27)) return SFA_ERR_UNSUPPORTED;
  if (!cache_fits(d, d->Hkv)) return SFA_ERR_UNSUPPORTED;
  if (d->rope && (d->rope_T <= 0 || !at16(d->rope))) return SFA_ERR_INVALID_ARG;
  return SFA_OK;
}

static bool stride_ok(int64_t stride, int heads, int dtype) {
  return stride >= (int64_t)heads * kD && (stride * (dtype == SFA_BF16 ? 2 : 4)) % 16 == 0;
}

static int check_attend(const sfa_kv4_desc* d, Plan* p, Kv4Args* a) {
  int rc = check_rows(d);
  if (rc != SFA_OK) return rc;
  if (d->R < 0 || (d->R == 0 && d->N > 0) || d->max_pages <= 0 || d->Hq <= 0) return SFA_ERR_INVALID_ARG;
  if ((int64_t)d->max_pages * d->page > (1 << 24) || d->Hq % d->Hkv) return SFA_ERR_UNSUPPORTED;
  if ((int64_t)d->N + d->R > INT32_MAX) return SFA_ERR_UNSUPPORTED;  // (their items are counted in 32 bits)
  const int G = d->Hq / d->Hkv;
  if (G > 32 || (G & (G - 1)) || (int64_t)d->N * d->Hq > (1LL << 31) - 1) return SFA_ERR_UNSUPPORTED;
  if (d->dist) {
    sfa_desc s = {};
    s.dist = d->dist;
    s.n_dist = d->n_dist;
    if ((rc = build_int_plan(&s, p)) != SFA_OK) return rc;
    if (p->n > 0 && p->c[0] < 0) return SFA_ERR_INVALID_ARG;  // a cache has no future keys
  } else {
    p->W = 1 << 24;  // the whole prefix: a window no position leaves
    p->n = 0;
    p->interp = 0;
  }
  *a = Kv4Args{};
  a->R = d->R;
  a->N = d->N;
  a->Hq = d->Hq;
  a->Hkv = d->Hkv;
  a->lgG = __builtin_ctz((unsigned)G);
  a->max_pages = d->max_pages;
  a->n_pages = d->n_pages;
  a->lgS = __builtin_ctz((unsigned)d->page);
  a->rope = reinterpret_cast<const float2*>(d->rope);
  a->rope_T = d->rope_T;
  a->qmul = (float)(2.0 * frexp(0.125 * M_LOG2E * d->kscale, &a->qexp));
  a->qexp -= 1;
  a->vscale = d->vscale;
  a->q_stride = d->q_stride;
  if (d->N == 0) return SFA_OK;
  return kv4_attend_fits(*a, *p, true) && (d->N != d->R || kv4_attend_fits(*a, *p, false)) ? SFA_OK : SFA_ERR_UNSUPPORTED;
}

}  // namespace sfa

using namespace sfa;

extern "C" {

int sfa_kv4_cache_bytes(int32_t n_pages, int32_t page, int32_t Hkv, size_t* bytes) {
  sfa_kv4_desc d = {};
  d.n_pages = n_pages;
  d.page = page;
  if (!bytes || Hkv <= 0) return SFA_ERR_INVALID_ARG;
  const int rc = check_pool(&d);
  if (rc != SFA_OK) return rc;
  if (!cache_fits(&d, Hkv)) return SFA_ERR_UNSUPPORTED;
  *bytes = (size_t)n_pages * Hkv * page * kKv4Row;
  return SFA_OK;
}

int sfa_kv4_plan(const sfa_kv4_desc* d, const int32_t* n_new, const int32_t* seq_lens,
                 int32_t* block_table, int32_t* free_pages, const int32_t* n_free, int32_t* cu_q,
                 int32_t* slots, int32_t* pos, int32_t* lens_out, int32_t* n_free_out, void* stream) {
  int rc = check_pool(d);
  if (rc != SFA_OK) return rc;
  if (d->R <= 0 || d->max_pages <= 0) return SFA_ERR_INVALID_ARG;
  if (d->R > 8192 || (int64_t)d->max_pages * d->page > (1 << 24)) return SFA_ERR_UNSUPPORTED;
  const void* ptrs[] = {n_new, seq_lens, block_table, free_pages, n_free, cu_q, lens_out, n_free_out};
  for (const void* x : ptrs)
    if (!x || !at4(x)) return SFA_ERR_INVALID_ARG;
  if (d->N > 0 && (!slots || !pos || !at4(slots) || !at4(pos))) return SFA_ERR_INVALID_ARG;
  PlanArgs a = {n_new, seq_lens, block_table, free_pages, n_free, cu_q, slots, pos, lens_out, n_free_out,
                d->R, d->N, d->max_pages, d->n_pages, __builtin_ctz((unsigned)d->page), nullptr};
  if ((rc = device_status(&a.status)) != SFA_OK) return rc;
  const size_t smem = (size_t)d->R * 16;
  auto kern = d->R > kPlanThreads ? kv4_plan_kernel<true> : kv4_plan_kernel<false>;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024) != cudaSuccess)
    return SFA_ERR_CUDA;
  const int here = d->N <= kPlanRows;
  LaunchTimer tm(SFA_KERNEL_KV4_PLAN, stream);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(kern, dim3(1), dim3(kPlanThreads), smem, s, a, here);
  if (e == cudaSuccess && !here) e = launch_pdl(kv4_plan_rows_kernel, dim3((unsigned)(((int64_t)d->N + 255) / 256)), dim3(256), 0, s, a);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int sfa_kv4_append(const sfa_kv4_desc* d, const void* k, const void* v, void* cache,
                   const int32_t* slots, const int32_t* pos, void* stream) {
  int rc = check_rows(d);
  if (rc != SFA_OK) return rc;
  if (d->N == 0) return SFA_OK;
  if (!k || !v || !cache || !slots || !pos) return SFA_ERR_INVALID_ARG;
  if (!at16(k) || !at16(v) || !at16(cache) || !at4(slots) || !at4(pos)) return SFA_ERR_INVALID_ARG;
  if (!stride_ok(d->k_stride, d->Hkv, d->dtype) || !stride_ok(d->v_stride, d->Hkv, d->dtype)) return SFA_ERR_INVALID_ARG;
  AppendArgs a = {k, v, d->k_stride, d->v_stride, static_cast<uint8_t*>(cache), slots, pos,
                  reinterpret_cast<const float2*>(d->rope), d->N, d->Hkv, __builtin_ctz((unsigned)d->page),
                  d->n_pages, d->rope_T, d->kscale, d->vscale, 1.0f / d->kscale, 1.0f / d->vscale, nullptr};
  if ((rc = device_status(&a.status)) != SFA_OK) return rc;
  const dim3 grid((unsigned)(((int64_t)d->N * d->Hkv * 4 + 255) / 256));
  LaunchTimer tm(SFA_KERNEL_KV4_APPEND, stream);
  const cudaError_t e = d->dtype == SFA_BF16 ? launch_pdl(kv4_append_kernel<bf16>, grid, dim3(256), 0, (cudaStream_t)stream, a)
                                             : launch_pdl(kv4_append_kernel<float>, grid, dim3(256), 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int sfa_kv4_read(const sfa_kv4_desc* d, const void* cache, const int32_t* slots, void* k, void* v,
                 void* stream) {
  int rc = check_rows(d);
  if (rc != SFA_OK) return rc;
  if (d->N == 0) return SFA_OK;
  if (!k || !v || !cache || !slots) return SFA_ERR_INVALID_ARG;
  if (!at16(k) || !at16(v) || !at16(cache) || !at4(slots)) return SFA_ERR_INVALID_ARG;
  ReadArgs a = {static_cast<const uint8_t*>(cache), slots, k, v, d->N, d->Hkv, __builtin_ctz((unsigned)d->page),
                d->n_pages, d->kscale, d->vscale, nullptr};
  if ((rc = device_status(&a.status)) != SFA_OK) return rc;
  const dim3 grid((unsigned)(((int64_t)d->N * d->Hkv * 8 + 255) / 256));
  LaunchTimer tm(SFA_KERNEL_KV4_READ, stream);
  const cudaError_t e = d->dtype == SFA_BF16 ? launch_pdl(kv4_read_kernel<bf16>, grid, dim3(256), 0, (cudaStream_t)stream, a)
                                             : launch_pdl(kv4_read_kernel<float>, grid, dim3(256), 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int sfa_kv4_workspace_size(const sfa_kv4_desc* d, size_t* bytes) {
  Plan p;
  Kv4Args a;
  if (!bytes) return SFA_ERR_INVALID_ARG;
  const int rc = check_attend(d, &p, &a);
  if (rc != SFA_OK) return rc;
  // without cu_q N = R; with N = R the call may be of either kind
  *bytes = 0;
  if (d->N == 0) return SFA_OK;
  *bytes = kv4_attend_workspace(a, p, true);
  if (d->N == d->R) *bytes = std::max(*bytes, kv4_attend_workspace(a, p, false));
  return SFA_OK;
}

int sfa_kv4_attend(const sfa_kv4_desc* d, const void* q, const void* cache,
                   const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* o,
                   float* lse, void* ws, size_t ws_bytes, void* stream) {
  Plan p;
  Kv4Args a;
  int rc = check_attend(d, &p, &a);
  if (rc != SFA_OK) return rc;
  if (!cu_q && d->N != d->R) return SFA_ERR_INVALID_ARG;
  if (d->N == 0) return SFA_OK;
  if (!q || !cache || !block_table || !seq_lens || !o) return SFA_ERR_INVALID_ARG;
  if (!at16(q) || !at16(cache) || !at16(o) || !at4(block_table) || !at4(seq_lens) || !at4(cu_q) || !at4(lse))
    return SFA_ERR_INVALID_ARG;
  if (!stride_ok(d->q_stride, d->Hq, d->dtype)) return SFA_ERR_INVALID_ARG;
  const size_t need = kv4_attend_workspace(a, p, cu_q != nullptr);
  if (need && (!ws || !at16(ws))) return SFA_ERR_INVALID_ARG;
  if (ws_bytes < need) return SFA_ERR_CAPACITY;
  a.q = q;
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q;
  a.o = o;
  a.lse = lse;
  wait_injection(&a.wait_cycles, &a.debug_skip);
  if ((rc = device_status(&a.status)) != SFA_OK) return rc;
  return launch_kv4_attend(a, p, d->dtype, ws, stream);
}

}  // extern "C"
