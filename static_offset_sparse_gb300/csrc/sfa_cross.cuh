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

// What 2^(x - m) is taken against: 0 for a maximum of -inf (no key, or logits
// that are all -inf), so that -inf - m stays -inf.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

// host side
int launch_cross_stream(const CrossArgs& a, bool q32, int dtype, void* stream);
int launch_cross_join(const CrossArgs& a, int dtype, const int32_t* pos, int pos_T, void* stream);
int launch_cross_fwd_simt(const CrossArgs& a, int dtype, void* stream);
int launch_cross_dq_simt(const CrossArgs& a, int dtype, void* stream);
int launch_cross_dkv_simt(const CrossArgs& a, int dtype, void* stream);
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
