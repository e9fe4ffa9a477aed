// Shared by the kernels of attention to states of another length (sfa_cross_*)
// and of a decode step behind a shared prefix (sfa_prefix_decode).
//
// Rows of a (sequence, KV head): its G heads' queries, row r is head r mod G of
// query r / G, so that one pass over the keys serves the whole group and rows
// behind a sequence's last query come last.
//
// Where rows are few, the keys are split: a part holds the sums of some keys
// for each row, o = sum_j 2^(x_j - m) v_j, l = sum_j 2^(x_j - m), m = max x_j (x:
// logits times log2(e)), all fp32; join_parts puts them together, always in the
// same order.
#pragma once

#include <math.h>

#include "sfa_device.cuh"
#include "sfa_launch.cuh"
#include "sfa_mma.cuh"
#include "sfa_tma.cuh"

namespace sfa {

constexpr int kSMs = 152;
constexpr float kLogitScale = 0.125f * kLog2e;  // logits in log2 units: 1/sqrt(64) * log2(e)

struct Strides {
  int64_t b, h, t;  // elements between sequences, heads, rows
};

struct CrossArgs {
  const void *q, *k, *v;
  Strides qs, ks, vs;
  void* o;     // [rows][64]
  float* lse;  // [rows], or nullptr
  Strides rs;  // where a query's row is: the order of [B, Hq, Tq], or of [Tq, Hq] for a batch's queries of a shared prefix
  int64_t rows;  // B * Hq * Tq
  const int32_t *q_len, *kv_len;  // [B] or nullptr (all rows)
  int kv_add;  // added to kv_len (1 where it holds the position of the last key)
  int B, Tq, Tk, Hq, Hkv, G;
  int splits;       // parts that the keys of a row (dk, dv: the rows of a key) are split into
  bool parts;       // whether parts are written (always with more than one split), or o and lse
  float* part_o;    // [splits][rows][64]
  float2* part_ml;  // [splits][rows] (m, l); l < 0: no key, and no sum in part_o
  // backward
  const void *out, *dO;
  const float2* stat;  // [B * Hq * Tq]: lse * log2(e) (+inf for rows that count for nothing), delta
  void *dq, *dk, *dv;
  float *part_a, *part_b;  // [splits][dq's] or [splits][dk's], [splits][dv's]
  int* status;
  long long wait_cycles;

  // Valid queries and keys of sequence b; a length out of range counts as none
  // and is recorded.
  __device__ __forceinline__ int queries(int b) const { return length(q_len, 0, b, Tq); }
  __device__ __forceinline__ int keys(int b) const { return length(kv_len, kv_add, b, Tk); }
  __device__ __forceinline__ int length(const int32_t* lens, int add, int b, int most) const {
    if (!lens) return most;
    const int64_t n = (int64_t)lens[b] + add;
    if (n < add || n > most) {
      record_status(status, SFA_ERR_DEVICE_BOUNDS);
      return 0;
    }
    return (int)n;
  }
  // Where row r of (b, KV head) is in o, lse and the parts.
  __device__ __forceinline__ int64_t row(int b, int kvh, int r) const {
    const int t = r / G;
    return b * rs.b + ((int64_t)kvh * G + (r - t * G)) * rs.h + t * rs.t;
  }
};

// Keys of split s of n, in whole tiles of `tile`: begin and end.
__device__ __forceinline__ void split_keys(int n, int tile, int splits, int s, int& begin, int& end) {
  const int tiles = (n + tile - 1) / tile;
  const int lo = (int)((int64_t)tiles * s / splits), hi = (int)((int64_t)tiles * (s + 1) / splits);
  begin = lo * tile;
  end = min(n, hi * tile);
}

// Two fp32 numbers at once.
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// What 2^(x - m) is taken against: 0 for a maximum of -inf (no key, or logits
// that are all -inf), so that -inf - m stays -inf.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

// host side
int launch_cross_stream(const CrossArgs& a, bool q32, int dtype, void* stream);
int launch_cross_join(const CrossArgs& a, int dtype, const int32_t* pos, int pos_T, void* stream);
int launch_cross_fwd_simt(const CrossArgs& a, void* stream);
// Tiles of 128 rows of the tensor-core kernels: 2^lgR queries of 128 / 2^lgR
// heads of a KV head each, so that short sequences share tiles; tile i holds
// head group i mod groups of query block i / groups (queries behind a length come last).
struct RowTiles {
  int lgR, groups, blocks, tiles;
};
RowTiles row_tiles(int G, int Tq);
// A tensor map of bf16 rows: boxes of `heads` x `rows` rows, 128-byte swizzle (sfa_api.cu).
int make_rows4_map(CUtensorMap* m, const void* base, int T, int H, int B, int64_t s_t, int64_t s_h, int64_t s_b, int box_rows, int box_heads);
inline int make_view_map(CUtensorMap* m, const void* base, int T, int H, int B, const Strides& s, int rows, int heads) {
  return make_rows4_map(m, base, T, H, B, s.t, s.h, s.b, rows, heads);
}
// bf16; two: queries as two bf16 parts, the second a sequence's stride behind the first
int launch_cross_fwd_tc(const CrossArgs& a, bool two, void* stream);
int launch_cross_bwd_tc(const CrossArgs& a, bool dkv, void* stream);  // bf16
int launch_cross_dq_simt(const CrossArgs& a, void* stream);           // fp32
int launch_cross_dkv_simt(const CrossArgs& a, void* stream);
constexpr int kStreamRows = 8;  // rows that cross_stream_kernel takes at once
constexpr int kSimtTile = 64;   // rows and keys of the fp32 kernels' tiles

// Splits of `units` units of work a CTA where there are `ctas` CTAs and room for
// `slots`: one wave of them, `least` units each.
inline int wave_splits(int64_t ctas, int64_t slots, int64_t units, int64_t least) {
  const int64_t want = slots / ctas, most = units / least;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : (int)s;
}

}  // namespace sfa
