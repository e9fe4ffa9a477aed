// Prompts over the paged 4-bit cache: many query rows a request, on the
// fifth-generation tensor cores.
//
// An item is two tiles of 128 columns (256 / G rows x the G heads of a KV head)
// of one request, a step 128 keys.  Per step
//   four warps turn the raw codes and scales (as the copying warp brings them)
//     into f16 keys and values in shared memory, a thread a key: code * scale
//     is a whole f16 number;
//   one thread issues S = Q K^T for each tile, twice (the query's two f16
//     parts: logits good to fp32's last bits), 128 x 128 sums in tensor memory;
//   four warps a tile, a thread a column (a lane of tensor memory), take the
//     maximum, exponentiate, and put P in f16 back into tensor memory, where
//     the issuing thread takes it as the left operand of O += P V.
// One tile's exponentials run under the other's products, and both use the same
// keys and values.  fp32 outputs add a second product with what rounding P to
// f16 dropped (it takes the place of logits already read).  What bounds it is
// the chain from a step's logits over its softmax (1300 clocks of exponentials,
// scalings, sums and packings) to the next step's logits, about 3000 clocks a
// step, of them 1536 of products, and next to it shared memory, which the logits'
// products read at its full rate (8 KB in 64 clocks) for 1024 clocks and all else
// uses for some 700.  (P in shared memory in odd steps, so that exponentials need
// not wait for the last step's outputs, took 109 us where this takes 94.)  8
// prompts of 300 to 700 rows over 2048 to 16384, 8 / 2 heads: 94 us with the
// join, 39% of the tensor cores' cycles.
//
// The steps of all (item, KV head) units, in order, are shared out evenly over
// one CTA an SM, to the step (and what a unit costs besides): units are long and
// few, and whole chunks of them left a quarter of the SMs' time idle.  A unit
// that spans CTAs leaves a part from each in the workspace (two a CTA at most),
// joined by a second kernel; so the last bits of a split row depend on the batch
// it is in.
#include "sfa_kv4_stream.cuh"
#include "sfa_launch.cuh"
#include "sfa_umma.cuh"

namespace sfa {

constexpr int kPSlots = 8, kStep = 128;
// Probabilities times 2^8, relative to a maximum that lags the true one: the
// 128 of a step then sum up to 2^15 at most while the maximum stands, and a sum
// below 65000 says that none has left f16's range.  (fp32 outputs know the
// maximum in every step and keep kPShift.)
template <bool EXACT>
constexpr float kPromptShift = EXACT ? kPShift : 8.0f;
constexpr float kSumLimit = 65000.0f;
constexpr int kPWarps = 14, kPThreads = 32 * kPWarps;  // softmax 0-3 and 4-7, dequantise 8-11, copy 12, products 13
// tensor memory of a tile: logits, probabilities, outputs
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192, kColTile = 256, kPCols = 512;
// shared memory: Q [tile][part], K [2], V [2] (128 rows of 128 bytes each,
// 128-byte swizzle), the raw ring, then what is small
constexpr int kPTile = 128 * 128;
constexpr int kPromptSmem = 8 * kPTile + kPSlots * kTileBytes + 1024;

// Where a CTA's share begins: the unit, and how far into its weight.
struct PieceStart {
  Item it;
  int x, h, in;
};

struct PromptShared {
  uint64_t raw_full[kPSlots], raw_empty[kPSlots];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // by step parity
  uint64_t s_full[2], p_full[2], pv_done[2], q_full[2];   // by tile
  int pages[kPSlots];
  int step_pages[2];      // pages there of a step's two 64-key tiles: bits 0-3 and 4-7
  int step_nan[2][4];     // whether a warp's values of the step hold a NaN
  uint8_t nan[2][kStep];  // per key: the scale blocks of its value that are NaN
  int sums[kPWarps];
  PieceStart where;
  uint32_t tmem;
};

// Parts of split units: two a CTA, [column][64] and (m, l); which parts a unit has.
struct PromptParts {
  float* o;     // [2 kSMs][256][64]
  float2* ml;   // [2 kSMs][256]
  int2* units;  // [unit]: first part, their number
};

__device__ __forceinline__ int first_tile(const StreamArgs& s, const Item& it) { return max(0, it.pfirst - s.W) / kTile; }
// Steps of an (item, KV head): 1 for an empty one, 0 for none.
__device__ __forceinline__ int item_steps(const StreamArgs& s, const Item& it) {
  return it.nch == 0 ? 0 : it.plast() < 0 ? 1 : (it.plast() / kTile - first_tile(s, it)) / 2 + 1;
}

// What a piece costs besides its steps (its queries, its first logits, its
// outputs), in steps: the CTA where a unit begins has it in its share.  Without
// it the CTAs with more pieces ran a quarter longer than the average.  0, 3, 6,
// 10, 16: 8 prompts of 300 to 700 rows over 2048 to 16384 141, 125, 119, 123, 130
// us; 30 of 50 to 200 over up to 4000 89, 58, 57.5, 61, 62; 500 of 20 to 40 over
// up to 1500 201, 164, 161, 162, 171; 64 of 12 over up to 20000 139, 131, 128,
// 133, 139.
constexpr int kUnitCost = 6;
__device__ __forceinline__ int item_weight(const StreamArgs& s, const Item& it) {
  const int n = item_steps(s, it);
  return n == 0 ? 0 : n + kUnitCost;
}

// A CTA's piece of a unit: its steps s0 .. s1 - 1, tiles tb .. te - 1.
struct Piece {
  Item it;
  int x, h, s0, s1, steps, tb, te;
  int begin, end;  // the weight before this unit, and where the CTA's share ends
  // the unit from weight `off` of it on; false if no step of it lies in the share
  __device__ __forceinline__ bool set(const StreamArgs& s, int off) {
    steps = item_steps(s, it);
    s0 = max(0, off - kUnitCost);
    s1 = max(s0, min(steps, end - begin - kUnitCost));
    const int t0 = first_tile(s, it);
    tb = t0 + 2 * s0;
    te = it.plast() < 0 ? tb : min(t0 + 2 * s1, it.plast() / kTile + 1);
    return s0 < s1;
  }
  __device__ __forceinline__ bool next(const Kv4Args& a, const StreamArgs& s) {
    begin += steps + kUnitCost;
    if (begin >= end) return false;
    if (++h == a.Hkv) {
      h = 0;
      do {
        if (x + 1 >= s.items) return false;
        it = item_at(a, s, ++x);
        asm volatile("" ::: "memory");  // moves no code; without it the steps' loops came out slower (119 us, 122)
      } while (it.nch == 0);
    }
    return set(s, 0);  // (without a step it is the share's last unit)
  }
};

// The shares of the weight: CTA b's begins at share * b + min(b, rest).
struct Shares {
  int share, rest;
  __device__ __forceinline__ int begin(int b) const { return share * b + min(b, rest); }
  __device__ __forceinline__ int owner(int w) const {
    const int big = (share + 1) * rest;
    return w < big ? w / (share + 1) : rest + (w - big) / share;
  }
};

// This CTA's first piece; false if it has none.  Called by all threads.  (One
// loop run twice, as in find_run.)
__device__ __forceinline__ bool find_piece(const Kv4Args& a, const StreamArgs& sa, int* sums, PieceStart* where, Shares& sh, Piece& cur) {
  const int tid = threadIdx.x;
  const int per = (sa.items + kPThreads - 1) / kPThreads;
  const int x0 = min(sa.items, tid * per), x1 = min(sa.items, x0 + per);
  int before = 0, first = 0, last = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int at = before;
#pragma unroll 1
    for (int x = x0; x < x1; ++x) {
      const Item it = item_at(a, sa, x);
      const int n = item_weight(sa, it), end = at + n * a.Hkv;
      if (pass > 0 && first < last && first >= at && first < end) *where = {it, x, (first - at) / n, (first - at) % n};
      at = end;
    }
    if (pass == 0) {
      int total;
      cta_sums<kPThreads>(at, sums, before, total);
      sh.share = total / (int)gridDim.x;
      sh.rest = total - sh.share * (int)gridDim.x;
      first = sh.begin(blockIdx.x);
      last = sh.begin(blockIdx.x + 1);
    }
  }
  __syncthreads();
  if (first == last) return false;
  cur.it = where->it;
  cur.x = where->x;
  cur.h = where->h;
  cur.begin = first - where->in;
  cur.end = last;
  return cur.set(sa, where->in) || cur.next(a, sa);
}

// 64 codes and 4 scales -> a row of f16 at row r of a swizzled tile; zero: zeros.
__device__ __forceinline__ void dequantise_row(const uint8_t* codes, uint32_t scales, bool zero, uint8_t* tile, int r) {
  const uint4 c0 = reinterpret_cast<const uint4*>(codes)[0], c1 = reinterpret_cast<const uint4*>(codes)[1];
  const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t f = e4m3x2_f16x2(((scales >> (8 * b)) & 255u) * 0x101u);
    uint32_t x[8];
    e2m1x8_f16(c[2 * b], x);
    e2m1x8_f16(c[2 * b + 1], x + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = zero ? 0u : hmul2(x[e], f);
    *reinterpret_cast<uint4*>(tile + swz(r, 2 * b)) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(tile + swz(r, 2 * b + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The keys of a step that a column attends: lo .. hi, where their pages are there.
struct Keys {
  int lo, hi, pages, lgr;
  __device__ __forceinline__ bool attended(int k) const {
    return k >= lo && k <= hi && (pages >> ((k >> 6) * 4 + ((k & 63) >> lgr)) & 1);
  }
  // keys c .. c + 31 as bits
  __device__ __forceinline__ uint32_t bits(int c) const {
    const int a = max(lo - c, 0), b = min(hi - c, 31);
    if (a > b) return 0;
    uint32_t m = (0xffffffffu << a) & (0xffffffffu >> (31 - b));
    const int pg = pages >> ((c >> 6) * 4);
    if (lgr >= 5) return pg >> ((c & 63) >> lgr) & 1 ? m : 0;
    if (!(pg >> ((c & 63) >> 4) & 1)) m &= 0xffff0000u;
    if (!(pg >> (((c & 63) >> 4) + 1) & 1)) m &= 0x0000ffffu;
    return m;
  }
};

// Logits of 32 keys from c on, at v; the next 32 are asked for before they are used.
template <bool MASKED>
__device__ __forceinline__ void column_take(uint32_t s, int c, const Keys& keys, float* v, float* next, bool more) {
  tmem_wait_ld32(v);
  if (more) tmem_ld32(s + c + 32, next);
  if (MASKED) {
    const uint32_t m = keys.bits(c);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(m >> e & 1)) v[e] = -INFINITY;
  }
}

// The largest of a column's 128 logits (its own lane of tensor memory).  Both
// walks are loops over 64 keys: unrolled over 128, with the masked form beside
// it, the eight softmax warps waited for instructions longer than they ran.
template <bool MASKED>
__device__ __forceinline__ float column_top(uint32_t s, const Keys& keys) {
  float top = -INFINITY, v[2][32];
  tmem_ld32(s, v[0]);
#pragma unroll 1
  for (int c = 0; c < kStep; c += 64)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      column_take<MASKED>(s, c + 32 * h, keys, v[h], v[h ^ 1], h == 0 || c == 0);
#pragma unroll
      for (int e = 0; e < 32; e += 2) top = fmaxf(top, fmaxf(v[h][e], v[h][e + 1]));
    }
  return top;
}

// P = 2^(s cs + off) of a column, into tensor memory; returns their sum.
template <bool EXACT, bool MASKED>
__device__ __forceinline__ float column_exp(uint32_t tl, const Keys& keys, float cs, float off) {
  const float2 cs2 = make_float2(cs, cs), off2 = make_float2(off, off);
  float2 sum = make_float2(0.0f, 0.0f);
  float v[2][32];
  tmem_ld32(tl + kColS, v[0]);
#pragma unroll 1
  for (int c = 0; c < kStep; c += 64)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      column_take<MASKED>(tl + kColS, c + 32 * h, keys, v[h], v[h ^ 1], h == 0 || c == 0);
      float w[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 y = fma2(make_float2(v[h][e], v[h][e + 1]), cs2, off2);
        v[h][e] = ex2(y.x);
        v[h][e + 1] = ex2(y.y);
        sum = add2(sum, make_float2(v[h][e], v[h][e + 1]));
        w[e >> 1] = __uint_as_float(pack_f16(v[h][e], v[h][e + 1]));
      }
      tmem_st16(tl + kColP + c / 2 + 16 * h, w);
      if (EXACT) {  // the rest of P goes over logits that have been read (those asked for lie behind)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 r = unpack_f16(__float_as_uint(w[e]));
          w[e] = __uint_as_float(pack_f16(v[h][2 * e] - r.x, v[h][2 * e + 1] - r.y));
        }
        tmem_st16(tl + kColS + c / 2 + 16 * h, w);
      }
    }
  return sum.x + sum.y;
}

template <typename TIO>
__global__ void __launch_bounds__(kPThreads, 1) kv4_prompt_kernel(const Kv4Args a, const StreamArgs sa, const PromptParts parts) {
  constexpr bool kExact = sizeof(TIO) == 4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PromptShared sh;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const kt = smem + 4 * kPTile;
  uint8_t* const vt = smem + 6 * kPTile;
  uint8_t* const raw = smem + 8 * kPTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(smem_u32(&sh.raw_full[i]), 1);
      mbar_init(smem_u32(&sh.raw_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), 4);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), 4);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
      mbar_init(smem_u32(&sh.q_full[i]), 4);
    }
    mbar_fence_init();
  }
  if (warp == kPWarps - 1) {
    tmem_alloc(smem_u32(&sh.tmem), kPCols);
    tmem_relinquish();
  }
  pdl_wait();
  Piece cur;
  Shares shares;
  tc05_fence_before();
  const bool work = find_piece(a, sa, sh.sums, &sh.where, shares, cur);  // (two barriers of the CTA inside)
  tc05_fence_after();
  const uint32_t tm = sh.tmem;
  const int G = 1 << a.lgG;
  bool dead = false;  // a wait ran out: no more waits, no more work
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_u32(bar), phase & 1, a.wait_cycles));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
  };
  if (!work) {
  } else if (warp == 12) {
    copy_run<kPSlots>(a, sa, cur, smem_u32(raw), smem_u32(sh.raw_full), smem_u32(sh.raw_empty), sh.pages,
                      cur.begin == 0 && cur.s0 == 0 ? a.debug_skip : -1, lane);
  } else if (warp == 13) {
    // ---- the products
    constexpr uint32_t idS = idesc_f16(128, kStep, false, false), idO = idesc_f16(128, 64, false, true);
    // descriptors' low words of the bases; a row is 128 bytes, a tile kPTile: in 16-byte units
    constexpr uint32_t kHi = smem_desc_hi(1024), kTileU = kPTile / 16;
    const uint32_t q0 = smem_desc_lo(smem_u32(smem), 16), k0 = smem_desc_lo(smem_u32(kt), 16), v0 = smem_desc_lo(smem_u32(vt), 8192);
    int nq[2] = {0, 0}, ns[2] = {0, 0}, np[2] = {0, 0};  // query loads, logit and value products of each tile
    // S = Q K^T of tile T in step j; last: the step's last one
    auto logits = [&](int T, int j, bool fresh, bool last) {
      if (fresh) wait(&sh.q_full[T], nq[T]++);
      if (T == 0) wait(&sh.k_full[j & 1], j >> 1);  // (the first tile has columns in every step)
      if (kExact && ns[T] > 0) wait(&sh.pv_done[T], ns[T] - 1);  // the logits' columns hold the rest of P until then
      if (dead) return;
      if (elect_one()) {
        tc05_fence_after();
        const uint32_t d = tm + kColTile * T + kColS, q = q0 + 2 * T * kTileU, k = k0 + (j & 1) * kTileU;
#pragma unroll
        for (int i = 0; i < 8; ++i) umma_ss_lo(d, q + (i >> 2) * kTileU + 2 * (i & 3), k + 2 * (i & 3), kHi, idS, i > 0);
        umma_commit(smem_u32(&sh.s_full[T]));
        if (last) umma_commit(smem_u32(&sh.k_empty[j & 1]));
      }
      __syncwarp();
      ++ns[T];
    };
    // O (+)= P V
    auto outputs = [&](int T, int j, bool begin, bool last) {
      if (T == 0) wait(&sh.v_full[j & 1], j >> 1);
      if (dead) return;
      if (elect_one()) {
        tc05_fence_after();
        const uint32_t d = tm + kColTile * T, v = v0 + (j & 1) * kTileU;
#pragma unroll
        for (int i = 0; i < (kExact ? 16 : 8); ++i)  // 16 keys: two groups of 8 rows
          umma_ts_lo(d + kColO, d + (i >= 8 ? kColS : kColP) + 8 * (i & 7), v + 128 * (i & 7), kHi, idO, !begin || i > 0);
        umma_commit(smem_u32(&sh.pv_done[T]));
        if (last) umma_commit(smem_u32(&sh.v_empty[j & 1]));
      }
      __syncwarp();
      ++np[T];
    };
    bool more = true;
    while (more && cur.te == cur.tb) more = cur.next(a, sa);
    int t = cur.tb, j = 0;
    bool two = (cur.it.nrows << a.lgG) > 128;
    if (more) {
      logits(0, 0, true, !two);
      if (two) logits(1, 0, true, true);
    }
    while (more && !dead) {
      const bool begin = t == cur.tb, was_two = two;
      bool fresh = false;
      t += 2;
      if (t >= cur.te) {
        do more = cur.next(a, sa);
        while (more && cur.te == cur.tb);
        fresh = true;
        t = cur.tb;
        two = (cur.it.nrows << a.lgG) > 128;
      }
      // the next logits first, where the queries stay: their readers wait longest (fp32 outputs: the rest
      // of P lies there)
      for (int T = 0; T < (was_two ? 2 : 1); ++T) {
        const bool last = T == was_two;
        wait(&sh.p_full[T], np[T]);  // the logits have been read (with a piece's first step: the last piece's O too)
        if (more && !fresh && !kExact) logits(T, j + 1, false, last);
        outputs(T, j, begin, last);
        if (more && !fresh && kExact) logits(T, j + 1, false, last);
      }
      if (more && fresh) {
        logits(0, j + 1, true, !two);
        if (two) logits(1, j + 1, true, true);
      }
      ++j;
    }
    if (dead && lane == 0) {  // products still under way end before their memory goes
      record_status(a.status, SFA_ERR_TIMEOUT);
      for (int T = 0; T < 2; ++T) {
        if (ns[T] > 0) mbar_wait_bounded(smem_u32(&sh.s_full[T]), (ns[T] - 1) & 1, a.wait_cycles);
        if (np[T] > 0) mbar_wait_bounded(smem_u32(&sh.pv_done[T]), (np[T] - 1) & 1, a.wait_cycles);
      }
    }
  } else if (warp >= 8) {
    // ---- codes to f16, a thread a key of the step
    const int key = tid - 256, half = key >> 6, k64 = key & 63;
    const int lgr = min(a.lgS, 6);
    int j = 0, n = 0;  // steps and raw tiles before the current one
    do {
      for (int t = cur.tb; t < cur.te && !dead; t += 2, ++j) {
        const bool two = t + 1 < cur.te;
        const int s0 = n % kPSlots, s1 = (n + 1) % kPSlots, buf = j & 1;
        wait(&sh.raw_full[s0], n / kPSlots);
        if (two) wait(&sh.raw_full[s1], (n + 1) / kPSlots);
        const int pg0 = sh.pages[s0], pg1 = two ? sh.pages[s1] : 0;
        const uint8_t* T = raw + (half ? s1 : s0) * kTileBytes;
        const bool zero = (half && !two) || t * kTile + key > cur.it.plast() || !((half ? pg1 : pg0) >> (k64 >> lgr) & 1);
        const uint2 sc = zero ? make_uint2(0, 0) : *reinterpret_cast<const uint2*>(T + 64 * kTile + 8 * k64);
        if (j > 1) wait(&sh.k_empty[buf], (j >> 1) - 1);
        if (dead) break;
        dequantise_row(T + 32 * k64, sc.x, zero, kt + buf * kPTile, key);
        fence_async_smem();
        arrive(&sh.k_full[buf]);
        // a NaN value block is stored as zeros: the columns that attend its key are told (0 * NaN would reach all)
        uint32_t nan = 0, vs = sc.y;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if ((vs >> (8 * b) & 127u) == 127u) {
            nan |= 1u << b;
            vs &= ~(255u << (8 * b));
          }
        const bool any = __any_sync(0xffffffffu, nan != 0);
        if (j > 1) wait(&sh.v_empty[buf], (j >> 1) - 1);  // (both tiles have done with that step)
        if (dead) break;
        sh.nan[buf][key] = (uint8_t)nan;
        if (lane == 0) {
          sh.step_nan[buf][warp - 8] = any;
          if (warp == 8) sh.step_pages[buf] = pg0 | pg1 << 4;
        }
        dequantise_row(T + 32 * kTile + 32 * k64, vs, zero, vt + buf * kPTile, key);
        fence_async_smem();
        arrive(&sh.v_full[buf]);
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.raw_empty[s0]));
          if (two) mbar_arrive(smem_u32(&sh.raw_empty[s1]));
        }
        n += two ? 2 : 1;
      }
    } while (!dead && cur.next(a, sa));
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  } else {
    // ---- softmax, a thread a column
    const int T = warp >> 2, lane_row = tid & 127;
    const uint32_t tl = tm + kColTile * T + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes of tensor memory
    uint8_t* const qt = smem + 2 * T * kPTile;
    const int row = tid >> a.lgG, lgr = min(a.lgS, 6);
    const int all_pages = (1 << (kTile >> lgr)) - 1;
    const int full_pages = all_pages | all_pages << 4;
    // Steps before the current one, and those in which this tile had columns.  A barrier's phase is
    // known by its parity alone, and a tile may sit steps out: once its own logits are there, the
    // step's other barriers are at that step's phase.
    int j = 0, jt = 0;
    float cs = 0.0f;
    bool first = true;  // the CTA's first piece
    do {
      const int ncol = cur.it.nrows << a.lgG;
      if (tid == 0 && cur.s0 == 0) {  // the unit begins here: which parts it leaves
        const int b = blockIdx.x, count = shares.owner(cur.begin + kUnitCost + cur.steps - 1) - b + 1;
        parts.units[(int64_t)cur.x * a.Hkv + cur.h] = make_int2(2 * b + (first ? 0 : 1), count);
      }
      if (dead) {  // (the join reads every unit's parts, whatever is in them)
        first = false;
        continue;
      }
      const bool whole = cur.s0 == 0 && cur.s1 == cur.steps;
      if (ncol <= 128 * T) {  // no column of this tile
        j += (cur.te - cur.tb + 1) >> 1;
        first = false;
        continue;
      }
      const bool mine = tid < ncol;
      const int p = cur.it.pfirst + row, head = cur.h * G + (tid & (G - 1));
      const int64_t out_row = cur.it.row0 + row;
      if (cur.te > cur.tb) {
        // the column's query: rotated, scaled by a power of two to its own size, in two f16 parts.  The
        // products that read the last one have ended: this thread has seen their sums
        const TIO* src = static_cast<const TIO*>(a.q) + out_row * a.q_stride + head * kD;
        const bool there = mine && p >= 0;
        float big = 0.0f;
#pragma unroll 2
        for (int c = 0; c < 4; ++c) {
          float lo[8], hi[8];
          if (there) {
            load_pair_chunk(src, c, a.rope, p, lo, hi);
#pragma unroll
            for (int e = 0; e < 8; ++e) big = fmaxf(big, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
          }
        }
        const int ex = min(max((int)(__float_as_uint(big) >> 23), 9), 253);
        const float f = __uint_as_float((uint32_t)(254 - ex) << 23) * 256.0f * a.qmul;
        cs = logit_factor(ex, a.qexp);
#pragma unroll 2
        for (int c = 0; c < 4; ++c) {
          float x[2][8] = {{0, 0, 0, 0, 0, 0, 0, 0}, {0, 0, 0, 0, 0, 0, 0, 0}};
          if (there) load_pair_chunk(src, c, a.rope, p, x[0], x[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u = x[i][2 * e] * f, v = x[i][2 * e + 1] * f;
              h[e] = pack_f16(u, v);
              const float2 r = unpack_f16(h[e]);
              l[e] = pack_f16(u - r.x, v - r.y);
            }
            *reinterpret_cast<uint4*>(qt + swz(lane_row, c + 4 * i)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(qt + kPTile + swz(lane_row, c + 4 * i)) = make_uint4(l[0], l[1], l[2], l[3]);
          }
        }
        fence_async_smem();
        arrive(&sh.q_full[T]);
      }
      float m = -INFINITY, l = 0.0f;
      uint32_t nans = 0;  // scale blocks of the output that an attended NaN reaches
      for (int t = cur.tb; t < cur.te && !dead; t += 2, ++j, ++jt) {
        const int buf = j & 1, j0 = t * kTile;
        wait(&sh.s_full[T], jt);
        wait(&sh.v_full[buf], j >> 1);  // (what is said about the step's keys; in this order, see below)
        if (dead) break;
        tc05_fence_after();
        const int pg = sh.step_pages[buf];
        const bool full = pg == full_pages && j0 + kStep - 1 <= cur.it.pfirst && j0 >= cur.it.plast() - sa.W;
        const int k_lo = max(p - sa.W - j0, 0), k_hi = mine ? min(p - j0, kStep - 1) : -1;
        const Keys keys = {k_lo, k_hi, pg, lgr};
        if (sh.step_nan[buf][0] | sh.step_nan[buf][1] | sh.step_nan[buf][2] | sh.step_nan[buf][3])
          for (int k = 0; k < kStep; ++k)
            if (sh.nan[buf][k] && keys.attended(k)) nans |= sh.nan[buf][k];
        if (jt > 0) wait(&sh.pv_done[T], jt - 1);  // P's columns are free, O stands still
        if (dead) break;
        tc05_fence_after();
        // After a piece's first step P is taken with the maximum so far: only if a sum passes the limit, or
        // a column that had no key so far has some, are the logits looked at, the maximum moved and P taken
        // anew.  (fp32 outputs look first: their P takes the logits' place.)
        const bool look = kExact || t == cur.tb;
        float sum = 0.0f, off = m == -INFINITY ? 0.0f : __fsub_rd(kPromptShift<kExact>, m);
        if (!look) sum = full ? column_exp<kExact, false>(tl, keys, cs, off) : column_exp<kExact, true>(tl, keys, cs, off);
        const bool again = look || __any_sync(0xffffffffu, sum > kSumLimit || (m == -INFINITY && k_lo <= k_hi));
        if (again) {
          const float top = cs * (full ? column_top<false>(tl + kColS, keys) : column_top<true>(tl + kColS, keys));
          float corr = 1.0f;
          if (top > __fadd_rd(m, kLag)) {
            corr = ex2(m - top);  // 0 on the first keys
            m = top;
            l *= corr;
          }
          if (t > cur.tb)
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float o[16];
              tmem_ld16(tl + kColO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= corr;
              tmem_st16(tl + kColO + c, o);
            }
          off = m == -INFINITY ? 0.0f : __fsub_rd(kPromptShift<kExact>, m);
          sum = full ? column_exp<kExact, false>(tl, keys, cs, off) : column_exp<kExact, true>(tl, keys, cs, off);
        }
        l += sum;
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full[T]);
      }
      const bool any = cur.te > cur.tb;  // (an empty item has no step)
      if (any) {
        wait(&sh.pv_done[T], jt - 1);
        tc05_fence_after();
      }
      const int64_t at = (int64_t)(2 * blockIdx.x + (first ? 0 : 1)) * kPromptColumns + tid;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        float o[16];
        if (any && !dead) {
          tmem_ld16(tl + kColO + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.0f;
        }
        if (nans >> (c / 16) & 1)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __int_as_float(0x7fffffff);
        if (!mine) {
        } else if (whole) {
          write_head<TIO>(a, out_row, head, c / 8, o, m, l, kPromptShift<kExact>);
          write_head<TIO>(a, out_row, head, c / 8 + 1, o + 8, m, l, kPromptShift<kExact>);
        } else {
          store8(parts.o + at * kD + c, o);
          store8(parts.o + at * kD + c + 8, o + 8);
          if (c == 0) parts.ml[at] = make_float2(m, l);
        }
      }
      tc05_fence_before();
      first = false;
    } while (cur.next(a, sa));
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == kPWarps - 1) tmem_dealloc(tm, kPCols);
}

// The parts of one unit joined, in the order of their keys: 32 columns a CTA, 8
// lanes a column.  Items' bad rows are seen to here.
template <typename TIO>
__global__ void __launch_bounds__(256) kv4_prompt_join_kernel(const Kv4Args a, const StreamArgs sa, const PromptParts parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int x = blockIdx.x / a.Hkv, h = blockIdx.x - x * a.Hkv, G = 1 << a.lgG;
  Bad bad;
  const Item it = item_check<true>(a, sa, x, bad);
  bad.settle(a, sa, h == 0 && blockIdx.y == 0, threadIdx.x, blockDim.x);
  const int col = 32 * blockIdx.y + (threadIdx.x >> 3), d = threadIdx.x & 7;
  if (it.nch == 0 || col >= it.nrows << a.lgG) return;
  const int2 u = parts.units[blockIdx.x];
  if (u.y <= 1) return;
  // its first part is the last of CTA u.x / 2 or all of it; the others are their CTAs' first
  auto place = [&](int i) { return (int64_t)(i == 0 ? u.x : 2 * (u.x / 2 + i)) * kPromptColumns + col; };
  float M = -INFINITY, l = 0.0f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int i = 0; i < u.y; ++i) M = fmaxf(M, parts.ml[place(i)].x);
  for (int i = 0; i < u.y; ++i) {
    const float2 v = parts.ml[place(i)];
    const float f = v.x == -INFINITY ? 0.0f : ex2(v.x - M);
    float z[8];
    load8(parts.o + place(i) * kD + 8 * d, z);
    l = fmaf(v.y, f, l);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(z[e], f, y[e]);
  }
  write_head<TIO>(a, it.row0 + (col >> a.lgG), h * G + (col & (G - 1)), d, y, M, l, kPromptShift<sizeof(TIO) == 4>);
}

static constexpr size_t kPartBytes = (size_t)2 * kSMs * kPromptColumns * (kD + 2) * sizeof(float);

size_t prompt_workspace(int64_t units) { return kPartBytes + (size_t)units * sizeof(int2); }

cudaError_t launch_kv4_prompt(const Kv4Args& a, StreamArgs s, int dtype, void* ws, cudaStream_t stream) {
  static_assert(kPromptSmem + (int)sizeof(PromptShared) + 1024 <= 228 * 1024, "shared memory of an SM");
  PromptParts parts;
  parts.o = static_cast<float*>(ws);
  parts.ml = reinterpret_cast<float2*>(parts.o + (size_t)2 * kSMs * kPromptColumns * kD);
  parts.units = reinterpret_cast<int2*>(parts.ml + (size_t)2 * kSMs * kPromptColumns);
  auto kern = dtype == SFA_BF16 ? kv4_prompt_kernel<bf16> : kv4_prompt_kernel<float>;
  auto join = dtype == SFA_BF16 ? kv4_prompt_join_kernel<bf16> : kv4_prompt_join_kernel<float>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPromptSmem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(kSMs), dim3(kPThreads), kPromptSmem, stream, a, s, parts);
  if (e != cudaSuccess) return e;
  return launch_pdl(join, dim3((unsigned)(s.items * a.Hkv), kPromptColumns / 32), dim3(256), 0, stream, a, s, parts);
}

}  // namespace sfa
