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
#include "sfa_umma.cuh"

namespace sfa {

constexpr int kSMs = 152;
constexpr float kLogitScale = 0.125f * kLog2e;  // logits in log2 units: 1/sqrt(64) * log2(e)

// What 2^(x - m) is taken against: 0 for a maximum of -inf (no key, or logits
// that are all -inf), so that -inf - m stays -inf.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

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
  bool parts;       // whether parts are written, or o and lse
  bool cluster;     // few rows: a cluster's CTAs are a row's splits, which meet in shared memory
  float* part_o;    // [splits][rows][64]
  float2* part_ml;  // [splits][rows] (m, l); l < 0: no key, and no sum in part_o
  // backward
  const void *out, *dO;
  const float2* stat;  // [B * Hq * Tq]: lse * log2(e), delta, of rows that count
  void *dq, *dk, *dv;
  float *part_a, *part_b;  // fp32 kernels: [splits][dq's] or [splits][dk's], [splits][dv's]
  int* status;
  long long wait_cycles;
  int debug_skip;  // test injection: the copy that CTA 0 of a tensor-core kernel leaves out, or -1

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

// Tiles of 128 rows of the tensor-core kernels: 2^lgR queries of 128 / 2^lgR
// heads of a KV head each, so that short sequences share tiles; tile i holds
// head group i mod groups of query block i / groups (queries behind a length come last).
struct RowTiles {
  int lgR, groups, blocks, tiles;
  // tiles with one of a sequence's nq queries: the first of them
  __host__ __device__ __forceinline__ int used(int nq) const { return groups * ((nq + (1 << lgR) - 1) >> lgR); }
};
RowTiles row_tiles(int G, int Tq);

// Query and head (of its group) of row r of a row tile.
struct RowOf {
  int t, g;
  bool mine;
};
__device__ __forceinline__ RowOf row_of(const CrossArgs& a, const RowTiles& rt, int tile, int r) {
  const int tb = tile / rt.groups, hb = tile - tb * rt.groups;
  RowOf o;
  o.t = (tb << rt.lgR) + (r & ((1 << rt.lgR) - 1));
  o.g = (hb << (7 - rt.lgR)) + (r >> rt.lgR);
  o.mine = tile < rt.tiles && o.t < a.Tq && o.g < a.G;
  return o;
}

// How the tensor-core kernels share out their work: sequence b has units(b)
// units (tiles that stay on an SM) of steps(b) steps each; all steps of all units,
// in order, are dealt out evenly over the CTAs, to the step.  Lengths are known
// on the device only, and whole units are too uneven: with a unit a CTA in turn, 32
// ragged sequences of up to 1024 x 2048 gave one CTA 70 steps where the mean is 40.
// A unit that spans CTAs leaves a part from each.  A CTA's share has one unit at
// most that began before it and one that ends behind it, so two places for parts a
// CTA are enough: 2 c for a part that does not begin its unit, 2 c + 1 for one that
// does.  What a unit costs besides its steps counts as kUnitCost steps, with the CTA
// that begins it.  A CTA has `least` steps at least, or a unit.
constexpr int kUnitCost = 2;

struct Shares {
  int64_t share, rest;
  int ctas;
  __host__ __device__ __forceinline__ void set(int64_t total, int64_t units, int most, int least) {
    const int64_t n = units > total / least ? units : total / least;
    ctas = n < 1 ? 1 : n < most ? (int)n : most;
    share = total / ctas;
    rest = total - share * ctas;
  }
  __host__ __device__ __forceinline__ int64_t begin(int c) const { return share * c + (c < rest ? c : rest); }
  __host__ __device__ __forceinline__ int owner(int64_t w) const {
    const int64_t big = (share + 1) * rest;
    if (((w | share) >> 31) == 0 && (big >> 31) == 0) {  // (64-bit division is slow)
      const uint32_t x = (uint32_t)w, n = (uint32_t)share, b = (uint32_t)big;
      return (int)(x < b ? x / (n + 1) : (uint32_t)rest + (x - b) / n);
    }
    return (int)(w < big ? w / (share + 1) : rest + (w - big) / share);
  }
};

// Shares of `units` units of weight w among `most` CTAs.  Where all are alike and whole
// units take at most `extra` steps longer than a division to the step, they stay whole:
// parts are written, read and joined for less than that.
inline Shares deal(int64_t units, int64_t w, int most, int least, bool alike, int extra) {
  Shares s;
  s.set(units * w, units, most, least);
  const int64_t per = (units + most - 1) / most;
  if (alike && units % per == 0 && per * w <= s.share + extra) s.set(units * w, units, (int)(units / per), least);
  return s;
}

// The CTA's pieces of units, one after another.
struct Walk {
  int64_t begin, end;      // weight before the unit, where the share ends
  int b, u, units, steps;  // the unit: number u of sequence b's
  int s0, s1;              // the piece: its steps s0 .. s1 - 1
  __device__ __forceinline__ bool whole() const { return s0 == 0 && s1 == steps; }
  // from weight `off` of the unit on; false if no step of it lies in the share
  __device__ __forceinline__ bool set(int64_t off) {
    s0 = off > kUnitCost ? (int)off - kUnitCost : 0;
    const int64_t left = end - begin - kUnitCost;
    s1 = left < steps ? (int)left : steps;
    // the same in all lanes, and known to be
    s0 = __shfl_sync(0xffffffffu, s0, 0);
    s1 = __shfl_sync(0xffffffffu, s1, 0);
    return s0 < s1;
  }
  template <typename F>
  __device__ __forceinline__ bool next(int B, const F& counts) {
    begin += steps + kUnitCost;
    if (begin >= end) return false;
    if (++u == units) {
      u = 0;
      do {
        if (++b >= B) return false;
        counts(b, units, steps);
      } while (units == 0);
    }
    return set(0);  // (without a step it is the share's last unit)
  }
};

struct WalkShared {
  long long sums[32], units;
  Walk first;
  Shares shares;
  int any;
};

// The first piece of CTA c of ctas, by all its THREADS threads; false if it has none.
template <int THREADS, typename F>
__device__ __forceinline__ bool find_walk(int B, const F& counts, int c, int ctas, int least, WalkShared& sh, Walk& wk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (B + THREADS - 1) / THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  if (tid == 0) {
    sh.any = 0;
    sh.units = 0;
  }
  __syncthreads();
  int64_t mine = 0, n = 0;
  int units, steps;
  for (int b = b0; b < b1; ++b) {
    counts(b, units, steps);
    mine += (int64_t)units * (steps + kUnitCost);
    n += units;
  }
  if (n > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.units), (unsigned long long)n);
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 31) sh.sums[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i == warp) upto += total;
    total += sh.sums[i];
  }
  Shares s;
  s.set(total, sh.units, ctas, least);
  const int64_t from = s.begin(c), to = s.begin(c + 1);
  int64_t at = upto - mine;
  if (c < s.ctas && from < to && from >= at && from < upto)
    for (int b = b0; b < b1; ++b) {
      counts(b, units, steps);
      const int64_t w = steps + kUnitCost, here = (int64_t)units * w;
      if (from < at + here) {
        wk.u = (int)((from - at) / w);
        wk.begin = at + wk.u * w;
        wk.end = to;
        wk.b = b;
        wk.units = units;
        wk.steps = steps;
        sh.first = wk;
        sh.shares = s;
        sh.any = 1;
        break;
      }
      at += here;
    }
  __syncthreads();
  if (!sh.any) return false;
  wk = sh.first;
  return wk.set(from - wk.begin) || wk.next(B, counts);
}

// For each x = c, c + ctas, .. below n with empty(x), todo(x), by whole warps; a lane
// looks at an x, so that the lengths of 32 are asked for at once.
template <typename E, typename D>
__device__ __forceinline__ void each_empty(int64_t n, int c, int ctas, int lane, const E& empty, const D& todo) {
#pragma unroll 1
  for (int64_t from = c; from < n; from += 32 * (int64_t)ctas) {
    const int64_t x = from + (int64_t)lane * ctas;
#pragma unroll 1
    for (unsigned left = __ballot_sync(0xffffffffu, x < n && empty(x)); left; left &= left - 1)
      todo(from + (int64_t)(__ffs(left) - 1) * ctas);
  }
}

// Keys of split s of n, in whole tiles of `tile`: begin and end.
__device__ __forceinline__ void split_keys(int n, int tile, int splits, int s, int& begin, int& end) {
  const int tiles = (n + tile - 1) / tile;
  const int lo = (int)((int64_t)tiles * s / splits), hi = (int)((int64_t)tiles * (s + 1) / splits);
  begin = lo * tile;
  end = min(n, hi * tile);
}

// n parts of a row (ml(i): its maximum and sum, a sum below 0 for a part without
// a key, which has no o; o(i): its 64 sums) to o and lse, by a warp: a part's sums by
// eight lanes, four parts at a time, always in the same order.  No key at all: zeros,
// lse = -inf.  4 S parts' sums are asked for at once, before anything is known of their
// weights: S = 8 for many parts (1024 rows of 30: 10.5 us one after another, so 6.4), 2 for up
// to 8 (8000 rows of 3 took 5 us longer with the registers of S = 8).
constexpr int kFewParts = 8;
template <int S, typename TIO, typename ML, typename O>
__device__ __forceinline__ void join_row(const CrossArgs& a, int64_t row, int n, int lane, const ML& ml, const O& o) {
  float m = -INFINITY, l = 0.0f, y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  bool any = false;
  for (int i0 = 0; i0 < n; i0 += 4 * S) {
    const int k = min(4 * S, n - i0), mine = lane >> 3;
    float z[S][8];
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (4 * s < k) load8(o(i0 + min(4 * s + mine, k - 1)) + 8 * (lane & 7), z[s]);
    const float2 v = lane < k ? ml(i0 + lane) : make_float2(-INFINITY, -1.0f);
    const unsigned there = __ballot_sync(0xffffffffu, !(v.y < 0.0f));
    any |= there != 0;
    float top = v.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float to = fmaxf(m, top), corr = exp2f(m - shift_of(to));  // (0 on the first)
    m = to;
    l *= corr;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= corr;
    const float f = exp2f(v.x - shift_of(m));
    if (there >> lane & 1) l = fmaf(f, v.y, l);
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (4 * s < k) {
        const int i = 4 * s + mine;
        const float fi = __shfl_sync(0xffffffffu, f, i);
        if (there >> i & 1)  // (else it may be anything)
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = fmaf(fi, z[s][e], y[e]);
      }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] += __shfl_xor_sync(0xffffffffu, y[e], 8);
    y[e] += __shfl_xor_sync(0xffffffffu, y[e], 16);
    y[e] = any ? y[e] / l : 0.0f;
  }
  if (lane < 8) store8(static_cast<TIO*>(a.o) + row * kD + 8 * lane, y);
  if (a.lse && lane == 0) a.lse[row] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
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
// The largest of three (NaN counts as nothing).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
// This warpgroup's registers a thread, of those the block was launched with.
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
// 8 columns of this thread's lane, as tmem_ld16 and tmem_st16.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// 96 and 32 columns of this thread's lane, there when the call returns.  (One
// statement: a wait of its own that passes the values on costs a move for each.)
__device__ __forceinline__ void tmem_take96(uint32_t taddr, float* v) {
  asm volatile(
      "{\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%96];\n"
      " .reg .b32 t32;\n add.u32 t32, %96, 32;\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [t32];\n"
      " .reg .b32 t64;\n add.u32 t64, %96, 64;\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [t64];\n"
      " tcgen05.wait::ld.sync.aligned;\n}\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]),
        "=f"(v[64]), "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
        "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]),
        "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]),
        "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_take32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// One K = 16 step of a product, as umma_ss_lo and umma_ts_lo, with the choice
// between setting and adding known to the compiler: from a register it costs
// more to bring to the tensor core than the rest of the step's operands.
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(hi), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// host side
int launch_cross_stream(const CrossArgs& a, bool q32, int dtype, void* stream);
// Two in one launch, of fp32 queries; a's rows are as many as b's or more.
int launch_cross_stream_two(const CrossArgs& a, const CrossArgs& b, int dtype, void* stream);
int launch_cross_join(const CrossArgs& a, int dtype, const int32_t* pos, int pos_T, void* stream);
int launch_cross_fwd_f32(const CrossArgs& a, void* stream);
// A tensor map of bf16 rows: boxes of `heads` x `rows` rows, 128-byte swizzle (sfa_api.cu).
int make_rows4_map(CUtensorMap* m, const void* base, int T, int H, int B, int64_t s_t, int64_t s_h, int64_t s_b, int box_rows, int box_heads);
inline int make_view_map(CUtensorMap* m, const void* base, int T, int H, int B, const Strides& s, int rows, int heads) {
  return make_rows4_map(m, base, T, H, B, s.t, s.h, s.b, rows, heads);
}
// Forward pass, bf16; ws: cross_tc_bytes.
size_t cross_tc_bytes(int B, int Hkv, int G, int Tq, int Tk);
int launch_cross_fwd_tc(const CrossArgs& a, void* ws, void* stream);
// The same into parts, the batch as one sequence of queries, those as two bf16
// parts, a sequence's stride apart; and the join with the sequences' own rows'
// a.splits parts, which stand behind the prefix's in out.part_o and out.part_ml.
int launch_prefix_tc(const CrossArgs& a, void* ws, void* stream);
int launch_prefix_join(const CrossArgs& prefix, const CrossArgs& out, void* ws, const int32_t* pos, int T, void* stream);
// Backward pass, bf16; ws: cross_bwd_tc_bytes.
size_t cross_bwd_tc_bytes(int B, int Hkv, int G, int Tq, int Tk);
int launch_cross_bwd_tc(const CrossArgs& a, void* ws, void* stream);
// Backward pass, fp32: dq, and dk and dv.
int launch_cross_bwd_f32(const CrossArgs& q, const CrossArgs& kv, void* stream);
constexpr int kStreamRows = 8, kStreamRowsBf16 = 16;  // rows that a CTA of the kernels for few rows takes
constexpr int kClusterSplits = 8;  // splits whose CTAs may be a cluster
constexpr int kF32Tile = 64;  // rows and keys of the fp32 kernels' tiles
constexpr int kF32Keys = 32;  // keys the fp32 forward kernel takes at a time

// Splits of `units` units of work a CTA where there are `ctas` CTAs and room for
// `slots`: one wave of them, `least` units each.
inline int wave_splits(int64_t ctas, int64_t slots, int64_t units, int64_t least) {
  const int64_t want = slots / ctas, most = units / least;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : (int)s;
}

}  // namespace sfa
