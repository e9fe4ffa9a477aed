// The paged 4-bit key/value cache: its layout, and the warp-level pieces that
// turn its rows into tensor-core operands.
//
// A cache is [n_pages][Hkv] blocks of 72 * S bytes (S rows a page):
//   key codes    S x 32 bytes   dim 2i in the low, 2i + 1 in the high half of byte i
//   value codes  S x 32 bytes
//   scales       S x 8 bytes    e4m3: keys' dims 0-15, 16-31, 32-47, 48-63, then the values'
// A code is e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign).  A code times its
// scale has at most 6 significant bits and lies in 2^-10 .. 2688, so it is a
// whole f16 number: dequantising into f16 operands loses nothing.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sfa_device.cuh"
#include "sfa_mma.cuh"
#include "sfa_tma.cuh"

namespace sfa {

constexpr int kKv4Row = 72;  // bytes of one (row, head)

// Eight e2m1 codes (a word, byte by byte, first in the low half) -> 4 x two
// f16.  Naming the bytes lets the conversion pick them from the word: 3.4
// clocks an SM for a word and its four scalings, against 6.1 with the bytes
// shifted out first (and 6.3 for the conversion by masks and shifts).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* o) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Two e4m3 numbers (16 bits: first in the low byte) -> two f16 (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
  return __half22float2(*reinterpret_cast<__half2*>(&u));
}
// Transpose of an 8x8 b16 matrix held one row per four lanes.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
// d += a * b (f16 inputs, fp32 accumulate); fragments as in sfa_mma.cuh.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two fp32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// What takes an accumulator (of a query whose largest number has exponent bits
// ex, scaled to 2^8 and times Kv4Args::qmul) to its logit in log2 units: a power
// of two, so that the product is exact and 2^(s c - m) cannot pass 1 by what
// rounding a large maximum m leaves out.  It is a normal number whatever kscale
// is: a masked logit is -inf times it, and for a factor raised to 2^-126 no logit
// reaches 2^-98.
__device__ __forceinline__ float logit_factor(int ex, int qexp) {
  return __uint_as_float((uint32_t)min(max(ex - 8 + qexp, 1), 254) << 23);
}

// Arguments of an attend call, passed by value.
struct Kv4Args {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;     // [R, max_pages]
  const int32_t* seq_lens;  // [R]
  const int32_t* cu_q;      // [R + 1] or nullptr (row r is request r's last token)
  void* o;
  float* lse;               // [N, Hq] or nullptr
  const float2* rope;       // [rope_T][32] or nullptr
  int64_t q_stride;         // elements between query rows
  int32_t R, N, Hq, Hkv, lgG, max_pages, n_pages, lgS, rope_T;
  float qmul, vscale;       // kscale log2(e) / 8 = qmul 2^qexp, qmul in [1, 2]
  int32_t qexp;
  int* status;
  long long wait_cycles;    // limit of every bounded wait
  int32_t debug_skip;       // test injection: tile whose copies the first warp of the first chunk's CTA never starts, or -1
};

// The request of packed row n, and the row's position; found by the whole
// warp, 32 boundaries at a time.  Returns false for a row behind the last one.
__device__ __forceinline__ bool kv4_row(const Kv4Args& a, int n, int lane, int& r, int& pos) {
  if (!a.cu_q) {
    r = n;
    pos = a.seq_lens[n] - 1;
    return true;
  }
  // largest r in [0, R) with cu_q[r] <= n, among requests with rows
  int lo = 0, len = a.R;  // the answer lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < len && a.cu_q[at] <= n;
    const uint32_t b = __ballot_sync(0xffffffffu, le);
    const int k = b ? 31 - __clz(b) : 0;  // cu_q is non-decreasing: the set bits are a prefix
    lo += k * step;
    len = min(step, len - k * step);
  }
  r = lo;
  const int end = a.cu_q[r + 1];
  pos = a.seq_lens[r] - (end - n);
  return n < end;
}

// sfa_kv4_attend.cu: whether the tiles of an attend call (ragged: with cu_q)
// can be counted in 31 bits, its scratch bytes, and the call.
bool kv4_attend_fits(const Kv4Args& a, const Plan& p, bool ragged);
size_t kv4_attend_workspace(const Kv4Args& a, const Plan& p, bool ragged);
int launch_kv4_attend(const Kv4Args& a, const Plan& p, int dtype, void* ws, void* stream);

}  // namespace sfa
