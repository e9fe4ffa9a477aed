// What the streaming attention kernels over the paged 4-bit cache share: how
// the work is cut and shared out, the warp that copies, the outputs.
#pragma once

#include <math.h>

#include "sfa_kv4.cuh"

namespace sfa {

// Probabilities are kept times 2^kPShift, relative to a maximum that may lag
// the true one by 2^kLag (the statistics move only when a logit passes it by
// more): at most 2^15 in f16, whose smallest steps then lie 2^-35 below the
// largest probability of a column.  (Sums with a maximum are rounded downwards: to
// nearest, one of 2^26 would let 2^19 through.)
constexpr float kPShift = 11.0f, kLag = 4.0f;

// One head's output row (dims 8g .. 8g + 7 of lane (g, t)) and log-sum-exp, of
// sums of 2^(logit + (shift - m)), the difference rounded downwards as it was
// there.  l = 0: no keys, a zero row and -inf.
template <typename TIO>
__device__ __forceinline__ void write_head(const Kv4Args& a, int64_t n, int head, int g, const float* x, float m, float l,
                                           float shift = kPShift) {
  float y[8];
  const float inv = l == 0.0f ? 0.0f : a.vscale / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = l == 0.0f ? 0.0f : x[e] * inv;
  store8(static_cast<TIO*>(a.o) + (n * a.Hq + head) * kD + 8 * g, y);
  if (a.lse && g == 0) a.lse[n * a.Hq + head] = l == 0.0f ? -INFINITY : __fsub_ru(m, shift) * kLn2 + logf(l);
}

constexpr int kTile = 64, kTileBytes = kTile * kKv4Row;
constexpr int kSMs = 152;

struct StreamArgs {
  int32_t items, lg_rows, chunk_tiles, lg_chunk, max_chunks, W;
  int32_t limit, row_bytes;  // positions that the block table and the RoPE table have room for; bytes of a row of o
  float* part_o;   // [item][KV head][chunk][column][64]
  float2* part_ml; // [item][KV head][chunk][column] (m, l)
};

struct Item {
  int r, row0, nrows, pfirst, c0, nch;  // nch = 0: no rows
  __device__ __forceinline__ int plast() const { return pfirst + nrows - 1; }
};

// What is wrong with an item: rows behind the tables' end, which are not among
// the item's, or before the request's first position.
struct Bad {
  int row = 0, rows = 0;  // those behind the end
  bool any = false;
  // The status, and the rows behind the end written as rows without keys: by
  // thread i of n, where `write` says so.
  __device__ __forceinline__ void settle(const Kv4Args& a, const StreamArgs& s, bool write, int i, int n) const {
    if (!any) return;
    record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
    if (!write) return;
    uint4* const o = reinterpret_cast<uint4*>(static_cast<char*>(a.o) + (int64_t)row * s.row_bytes);
#pragma unroll 1
    for (int j = i; j < rows * (s.row_bytes / 16); j += n) o[j] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int j = i; a.lse && j < rows * a.Hq; j += n) a.lse[(int64_t)row * a.Hq + j] = -INFINITY;
  }
};

// Item x.  Requests start at item cu_q[r] / rows + r: room for each one's last,
// shorter item without a scan over the requests.  Rows whose positions leave the
// tables are zero rows, and the status says so: those before a request's first
// position attend nothing, and a request's items end before those behind the
// tables' end.  CHECK: what is wrong with it goes to bad, for who looks every item
// over (each CTA as it finds its share, the prompts' join).
template <bool CHECK>
__device__ __forceinline__ Item item_check(const Kv4Args& a, const StreamArgs& s, int x, Bad& bad) {
  Item it;
  if (!a.cu_q) {
    const int len = max(a.seq_lens[x], -1);
    it.r = it.row0 = x;
    it.nrows = 1;
    it.pfirst = len - 1;
    if (CHECK) bad.any = len < 0 || len > s.limit;
  } else {
    int lo = 0, n = a.R;  // largest r with cu_q[r] / rows + r <= x
    while (n > 1) {
      const int half = n >> 1;
      const bool le = (a.cu_q[lo + half] >> s.lg_rows) + lo + half <= x;
      lo += le ? half : 0;
      n = le ? n - half : half;
    }
    const int c = a.cu_q[lo], end = min(a.cu_q[lo + 1], a.N), len = max(a.seq_lens[lo], -1);
    const int past = end - max(len - s.limit, 0);  // the first row behind the tables' end
    it.r = lo;
    it.row0 = c + ((x - lo - (c >> s.lg_rows)) << s.lg_rows);
    it.nrows = min(1 << s.lg_rows, past - it.row0);
    it.pfirst = len - (end - it.row0);
    const bool none = c < 0 || it.row0 < c;
    if (CHECK && !none) {
      bad.row = max(it.row0, past);
      bad.rows = max(min(it.row0 + (1 << s.lg_rows), end) - bad.row, 0);
      bad.any = bad.rows > 0 || (it.nrows > 0 && it.pfirst < 0);
    }
    if (none || it.nrows <= 0) {
      it.nrows = it.nch = it.pfirst = it.c0 = 0;
      return it;
    }
  }
  if (it.plast() < 0 || it.pfirst >= s.limit) {  // no row has a position
    it.pfirst = -it.nrows;
    it.c0 = 0;
    it.nch = 1;
    return it;
  }
  const int lg = s.lg_chunk + 6;  // 64 keys a tile
  it.c0 = max(0, it.pfirst - s.W) >> lg;
  it.nch = (it.plast() >> lg) - it.c0 + 1;
  return it;
}
__device__ __forceinline__ Item item_at(const Kv4Args& a, const StreamArgs& s, int x) {
  Bad bad;
  return item_check<false>(a, s, x, bad);
}

// What a chunk counts for besides its tiles, in tiles, when the shares are made:
// its four warps' odd tiles, their meeting, and that shares end at whole chunks.
// Not one of these measured by itself: with 0 the teams with more and shorter
// chunks ended last, and any number from 8 to 48 evens the shares out about as
// well.  0, 8, 16, 24, 48: 128 requests of 1024 to 32768 rows 86.4, 86.1, 84.5,
// 84.5, 84.3 us; 300 of 100 to 6000 48.5, 46.1, 46.3, 46.1, 46.0; 700 of up to
// 3000 62.7, 57.6, 58.0, 57.7, 59.8; 64 of 4 to 8 rows over up to 20000 97.7,
// 94.8, 93.3, 93.2, 93.0; one of 400001 27.1, 26.7, 26.8, 26.7, 26.8.
constexpr int kChunkCost = 24;

// A place in a team's run of chunks: chunk c of (item x, KV head h), its tiles
// tb .. te - 1, and the run's weight (tiles and chunks' costs) up to here.
struct Cursor {
  Item it;
  int x, h, c, tb, te;
  int at, end;
  __device__ __forceinline__ void tiles(const StreamArgs& s) {
    tb = max(c * s.chunk_tiles, max(0, it.pfirst - s.W) / kTile);
    te = it.plast() < 0 ? tb : min((c + 1) * s.chunk_tiles, it.plast() / kTile + 1);
  }
  // the next chunk; false at the end of the run
  __device__ __forceinline__ bool next(const Kv4Args& a, const StreamArgs& s) {
    at += te - tb + kChunkCost;
    if (at >= end) return false;
    if (++c == it.c0 + it.nch) {
      if (++h == a.Hkv) {
        h = 0;
        do {
          if (x + 1 >= s.items) return false;
          it = item_at(a, s, ++x);
        } while (it.nch == 0);
      }
      c = it.c0;
    }
    tiles(s);
    return true;
  }
};

// Weight of one KV head of an item.
__device__ __forceinline__ int run_weight(const StreamArgs& s, const Item& it) {
  return it.nch * kChunkCost + (it.nch == 0 || it.plast() < 0 ? 0 : it.plast() / kTile + 1 - max(0, it.pfirst - s.W) / kTile);
}

// Sums of the warps' `mine` before a thread's own and over the CTA; one barrier.
template <int THREADS>
__device__ __forceinline__ void cta_sums(int mine, int* sums, int& before, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  static_assert(THREADS <= 1024, "a lane a warp");
  const int v = lane < THREADS / 32 ? sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, v);
  before = inc - mine + __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
}

// Where a team's run begins: the first item, its head and chunk, the weight there.
struct RunStart {
  Item it;
  int x, h, c, at;
};

// A team's run of chunks: those that begin in its share of the weight; false if
// there are none.  All THREADS threads of the CTA's TEAMS teams call it, with
// shared memory for THREADS / 32 sums and a RunStart a team (`where`).  Its one
// loop over the items runs twice, to count and to find: the code is cold when a
// kernel starts, and a second copy of item_at cost 2300 clocks.
template <int THREADS, int TEAMS>
__device__ __forceinline__ bool find_run(const Kv4Args& a, const StreamArgs& sa, int* sums, RunStart* where, int team, Cursor& cur) {
  const int tid = threadIdx.x;
  const int per = (sa.items + THREADS - 1) / THREADS;
  const int x0 = min(sa.items, tid * per), x1 = min(sa.items, x0 + per);
  if (tid < TEAMS) where[tid].x = -1;
  // the teams of an SM (CTAs kSMs apart come to lie on one) have neighbouring shares, whose roundings to
  // whole chunks cancel
  const int teams = gridDim.x * TEAMS, b0 = (blockIdx.x % kSMs * (gridDim.x / kSMs) + blockIdx.x / kSMs) * TEAMS;
  int share = 0, rest = 0, before = 0;
  auto begin = [&](int b) { return share * b + min(b, rest); };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int at = before;
#pragma unroll 1
    for (int x = x0; x < x1; ++x) {
      Bad bad;
      const Item it = item_check<true>(a, sa, x, bad);
      bad.settle(a, sa, blockIdx.x == 0, 0, 1);
      const int wt = run_weight(sa, it), end = at + wt * a.Hkv;
      if (pass > 0 && end > begin(b0) && at < begin(b0 + TEAMS)) {
#pragma unroll 1
        for (int i = 0; i < TEAMS; ++i) {
          const int first = begin(b0 + i);
          if (first == begin(b0 + i + 1) || first < at || first >= end) continue;
          // the first chunk that begins at `first` or later; its head's end is a chunk's beginning too
          const int h = (first - at) / wt, in = first - at - h * wt;
          // chunk j > 0 begins j (tiles + cost) - skip into the head
          const int skip = max(0, it.pfirst - sa.W) / kTile - it.c0 * sa.chunk_tiles, step = sa.chunk_tiles + kChunkCost;
          const int j = in == 0 ? 0 : min((in + skip + step - 1) / step, it.nch);
          where[i] = {it, x, h, it.c0 + j, at + h * wt + (j == 0 ? 0 : j < it.nch ? j * step - skip : wt)};
        }
      }
      at = end;
    }
    if (pass == 0) {
      int total;
      cta_sums<THREADS>(at, sums, before, total);
      share = total / teams;
      rest = total - share * teams;
    }
  }
  __syncthreads();
  const RunStart& w = where[team];
  if (w.x < 0) return false;
  cur.it = w.it;
  cur.x = w.x;
  cur.h = w.h;
  cur.c = w.c;
  cur.at = w.at;
  cur.end = begin(b0 + team + 1);
  if (cur.at >= cur.end) return false;
  if (cur.c >= cur.it.c0 + cur.it.nch) {  // the share begins inside a head's last chunk: step to the next head
    cur.c = cur.it.c0 + cur.it.nch - 1;
    cur.te = cur.tb = 0;
    cur.at -= kChunkCost;
    return cur.next(a, sa);
  }
  cur.tiles(sa);
  return true;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// The copying warp: every tile of the team's run, in order, into slot n mod
// SLOTS as soon as tile n - SLOTS has been read.
template <int SLOTS, typename CURSOR>
__device__ __forceinline__ void copy_run(const Kv4Args& a, const StreamArgs& sa, CURSOR cur, uint32_t ring, uint32_t full, uint32_t empty,
                                         volatile int* pages, int skip, int lane) {
  const int S = 1 << a.lgS, rows = min(S, kTile), np = kTile / rows, lgnp = __ffs(np) - 1, batch = 32 >> lgnp;
  const int64_t block = kKv4Row * S;
  int n = 0;
  bool dead = false;
  do {
    const int32_t* trow = a.table + (int64_t)cur.it.r * a.max_pages;
    const uint8_t* head = a.cache + cur.h * block;
    const int last = cur.it.plast();
    for (int t0 = cur.tb; t0 < cur.te && !dead; t0 += batch) {
      // lane: page `lane mod np` of tile t0 + lane / np
      const int j = (t0 + (lane >> lgnp)) * kTile + (lane & (np - 1)) * rows;
      const bool mine = t0 + (lane >> lgnp) < cur.te && j <= last;
      const int pid = mine ? trow[j >> a.lgS] : 0;
      const bool ok = mine && pid >= 0 && pid < a.n_pages;
      if (mine && !ok) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
      const uint32_t there = __ballot_sync(0xffffffffu, ok);
      const uint8_t* src = head + pid * (block * a.Hkv);
      const int k1 = min(batch, cur.te - t0);
      for (int k = 0; k < k1; ++k, ++n) {
        const int slot = n % SLOTS;
        if (n >= SLOTS && !mbar_wait_bounded(empty + 8 * slot, (n / SLOTS - 1) & 1, a.wait_cycles)) {
          record_status(a.status, SFA_ERR_TIMEOUT);
          dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        if (n == skip) continue;
        const uint32_t b = full + 8 * slot, d = ring + slot * kTileBytes;
        const uint32_t here = (there >> (k << lgnp)) & ((1u << np) - 1);
        if (lane == 0) {
          pages[slot] = (int)here;
          mbar_expect_tx(b, __popc(here) * rows * kKv4Row);
        }
        __syncwarp();
        if (ok && lane >> lgnp == k) {
          const int p = lane & (np - 1), row = j & (S - 1);
          if (S == kTile) {
            bulk_load(d, src, kTileBytes, b);
          } else {
            bulk_load(d + 32 * p * rows, src + 32 * row, 32 * rows, b);
            bulk_load(d + 32 * kTile + 32 * p * rows, src + 32 * S + 32 * row, 32 * rows, b);
            bulk_load(d + 64 * kTile + 8 * p * rows, src + 64 * S + 8 * row, 8 * rows, b);
          }
        }
      }
    }
  } while (!dead && cur.next(a, sa));
  // the copies end before the CTA does, whatever became of their readers
  for (int i = max(0, n - SLOTS); i < n; ++i)
    if (i != skip && !mbar_wait_bounded(full + 8 * (i % SLOTS), i / SLOTS & 1, a.wait_cycles)) record_status(a.status, SFA_ERR_TIMEOUT);
}

// sfa_kv4_prompt.cu: the stream of many rows a request, 256 columns an item,
// with its join; ws: prompt_workspace(units) bytes.
constexpr int kPromptColumns = 256;
size_t prompt_workspace(int64_t units);
cudaError_t launch_kv4_prompt(const Kv4Args& a, StreamArgs s, int dtype, void* ws, cudaStream_t stream);

}  // namespace sfa
