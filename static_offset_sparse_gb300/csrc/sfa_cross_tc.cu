// Forward pass of attention to states of another length on the fifth-generation
// tensor cores (bf16).
//
// A unit is two tiles of 128 rows of one (sequence, KV head), a step 96 of their
// keys; both tiles use the same keys and values.  Per step and tile
//   one thread issues S = Q K^T (128 x 96 sums in tensor memory);
//   four warps, a thread a row (a lane of tensor memory), take 2^x of the row's 96
//     logits and their sum, and put P in bf16 over them;
//   the issuing thread takes P as the left operand of O += P V, O in tensor memory.
// 96 keys, because two such S for each of two tiles fit tensor memory beside O: the
// next S is there when a step's exponentials end.  (With 128, one S and P beside it,
// a step took the chain of both, 2300 to 3000 clocks where the tensor cores need
// 1024 and the exponentials as many.)
//
// The shift of 2^x is the maximum of a row's first 96 logits.  Later steps do not look
// for theirs: a row whose sum over a step passes kSumLimit (or is no number) takes the
// step again, with its maximum, and moves its sums; P, O and the sum are thus at most
// kSumLimit times too large, which fp32 and bf16 hold as well as 1.  Maxima cost a
// fifth of the instructions, and the step's first 200 clocks.  The sums are taken in
// fp32 from probabilities before their rounding to
// bf16.  A unit's first products start under the last unit's outputs: one warp walks
// the CTA's share of the steps and writes down each piece a little ahead, the
// others read it there (each for itself, they waited 1000 clocks a piece for lengths
// and divisions), coupled by mbarriers only.
#include <limits.h>

#include "sfa_cross.cuh"

namespace sfa {

constexpr int kTcThreads = 384;  // 2 x 4 warps of softmax, a copying warp, two that issue, one that plans and clears tails
// Registers: 168 a thread at launch, 3 x 128 x 168 = 2 x 128 x 216 + 128 x 72.
constexpr int kTcMoreRegs = 216, kTcFewerRegs = 72;
constexpr int kTcTile = 128 * 128;  // bytes of 128 rows of 64 bf16
constexpr int kKeys = 96, kKeyTile = kKeys * 128;  // keys of a step, bytes of that many rows
constexpr int kTcCols = 512, kTcTileCols = 256, kTcO = 2 * kKeys;  // tensor memory columns of a tile: S or P of even steps, of odd ones, O
// Steps a CTA has at least (8 / 2 heads, 17 queries over 1000: 12.4 us, with 6 14.9; 4 x 8 / 2,
// 128 over 2000: 17.7 and 20.8).
constexpr int kTcLeast = 3;
constexpr float kSumLimit = 16384.0f;
// Maxima beyond this are taken from x before the multiplication: a fused
// 2^(x c - m c) would keep what rounding m c dropped, a factor of 2^(2^-5) and more.
constexpr float kFar = 1048576.0f;

template <int PARTS>
struct TcShape {
  static constexpr int kSlots = 8;                   // key and value tiles in flight
  static constexpr int kQBufs = PARTS == 1 ? 2 : 1;  // units whose queries are there
  static constexpr int kQBytes = 2 * PARTS * kTcTile;
  static constexpr int kOut = 8 * 4096;              // outputs on their way: 32 rows of 128 bytes a warp
  static constexpr int kSmem = kQBufs * kQBytes + kSlots * kKeyTile + kOut + 1024;
};

constexpr int kPlans = 4;  // pieces written down ahead

// A piece as the roles need it.
struct TcPiece {
  int steps;                // none: there are no more pieces
  int b, kvh, tile, k0, k1;  // the first of its tiles, its keys
  int two;                  // whether the second tile has queries
  int place;                // of its rows in place_o: -1 for a whole unit
};

struct TcShared {
  uint64_t full[8], empty[8], q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // by tile and step's parity
  uint64_t v_ready[4];  // by value slot: what stands behind the last key is zeros
  uint64_t plan_full[kPlans], plan_empty[kPlans];
  TcPiece plan[kPlans];
  int rows[kPlans][256];  // where a row is in o and lse: ~ of it for one without keys or behind the last query, INT_MIN for none
  WalkShared walk;
  uint32_t tmem;
};

struct TcWork {
  RowTiles rt;
  float* place_o;    // [2 CTAs][256][64]: parts of units that span CTAs
  float2* place_ml;  // [2 CTAs][256]
  int4* split;       // [CTAs]: the unit that a CTA begins and does not end: sequence, KV head, pair of tiles, parts (0: none)
};

// A row's logits of a step, -inf from the `left`th on.
__device__ __forceinline__ void row_logits(uint32_t s, int left, float* x) {
  tmem_take96(s, x);
  if (left < kKeys) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e)
      if (e >= left) x[e] = -INFINITY;
  }
}

__device__ __forceinline__ float row_top(const float* v) {
  float tops[4] = {fmaxf(v[0], v[1]), fmaxf(v[2], v[3]), fmaxf(v[4], v[5]), fmaxf(v[6], v[7])};
#pragma unroll
  for (int e = 8; e < kKeys; e += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], v[e + 2 * i], v[e + 2 * i + 1]);
  return max3(tops[0], tops[1], fmaxf(tops[2], tops[3]));
}

// x to P = 2^(x c - m c) in bf16, two a word; returns their sum.
__device__ __forceinline__ float row_exp(float* x, float mc) {
  const float2 c2 = make_float2(kLogitScale, kLogitScale), off2 = make_float2(-mc, -mc);
  float2 sum[4] = {};
#pragma unroll
  for (int e = 0; e < kKeys; e += 2) {
    const float2 y = pair_fma(make_float2(x[e], x[e + 1]), c2, off2);
    const float2 p = make_float2(ex2(y.x), ex2(y.y));
    sum[(e >> 1) & 3] = pair_add(sum[(e >> 1) & 3], p);
    x[e >> 1] = __uint_as_float(pack_bf16(p.x, p.y));
  }
  const float2 both = pair_add(pair_add(sum[0], sum[1]), pair_add(sum[2], sum[3]));
  return both.x + both.y;
}

// The same for any m, in a loop, P over the logits that have been read.
__device__ __forceinline__ float row_exp_any(uint32_t s, int left, float m) {
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < kKeys; c += 16) {
    float v[16];
    tmem_ld8(s + c, v);
    tmem_ld8(s + c + 8, v + 8);
    tmem_wait_ld8(v);
    tmem_wait_ld8(v + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      v[e] = c + e < left ? ex2((v[e] - m) * kLogitScale) : 0.0f;
      sum += v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(pack_bf16(v[2 * e], v[2 * e + 1]));
    tmem_st8(s + c / 2, v);
  }
  return sum;
}

__device__ __forceinline__ void st_stage(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)),
               "r"(__float_as_uint(d))
               : "memory");
}

template <int PARTS>
__global__ void __launch_bounds__(kTcThreads, 1)
    cross_fwd_tc_kernel(const CrossArgs a, const TcWork w, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                        const __grid_constant__ CUtensorMap vm) {
  using Shape = TcShape<PARTS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcShared sh;
  const uint32_t smem = smem_u32(smem_raw) + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem + Shape::kQBufs * Shape::kQBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, and known to be)
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < Shape::kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 1);
      mbar_init(smem_u32(&sh.q_empty[i]), 2);
      for (int j = 0; j < 2; ++j) {
        mbar_init(smem_u32(&sh.s_full[i][j]), 1);
        mbar_init(smem_u32(&sh.p_full[i][j]), 4);
        mbar_init(smem_u32(&sh.pv_done[i][j]), 1);
      }
    }
    for (int i = 0; i < Shape::kSlots / 2; ++i) mbar_init(smem_u32(&sh.v_ready[i]), 1);
    for (int i = 0; i < kPlans; ++i) {
      mbar_init(smem_u32(&sh.plan_full[i]), 1);
      mbar_init(smem_u32(&sh.plan_empty[i]), 11);  // every other warp
    }
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.tmem), kTcCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane < 3) prefetch_map(lane == 0 ? &qm : lane == 1 ? &km : &vm);
  pdl_wait();
  auto counts = [&](int b, int& units, int& steps) {
    const int nk = a.keys(b);
    steps = (nk + kKeys - 1) / kKeys;
    units = nk > 0 ? a.Hkv * ((w.rt.used(a.queries(b)) + 1) >> 1) : 0;
  };
  Walk wk;
  tc05_fence_before();
  const bool some = find_walk<kTcThreads>(a.B, counts, blockIdx.x, gridDim.x, kTcLeast, sh.walk, wk);  // (with barriers of the CTA)
  tc05_fence_after();
  const uint32_t tm = sh.tmem;
  bool dead = false;  // a wait ran out: no more waits, no more work
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_u32(bar), phase & 1, a.wait_cycles));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(bar));
  };

  int pieces = 0;  // taken so far
  // The next piece; false if there is none.
  auto take = [&](TcPiece& p) {
    const int i = pieces % kPlans;
    wait(&sh.plan_full[i], pieces / kPlans);
    if (dead) return false;
    p = sh.plan[i];
    p.steps = __shfl_sync(0xffffffffu, p.steps, 0);  // (known to be the same in all lanes)
    p.two = __shfl_sync(0xffffffffu, p.two, 0);
    return p.steps > 0;
  };
  auto give_back = [&]() { arrive(&sh.plan_empty[pieces++ % kPlans]); };

  if (warp < 8) {
    // ---- softmax: a thread a row of tile T
    more_registers<kTcMoreRegs>();
    const int T = warp >> 2, r = tid & 127;
    const uint32_t tl = tm + kTcTileCols * T + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    // rows of tiles without work: zeros (parts have no such rows)
    if (!a.parts && (a.q_len || a.kv_len))
      each_empty(
          (int64_t)a.B * a.Hkv * w.rt.tiles, blockIdx.x, gridDim.x, lane,
          [&](int64_t x) {
            const int bh = (int)(x / w.rt.tiles), b = bh / a.Hkv;
            return x - (int64_t)bh * w.rt.tiles >= (a.keys(b) > 0 ? (w.rt.used(a.queries(b)) + 1) & ~1 : 0);
          },
          [&](int64_t x) {
            const int bh = (int)(x / w.rt.tiles), b = bh / a.Hkv;
            const RowOf ro = row_of(a, w.rt, (int)(x - (int64_t)bh * w.rt.tiles), r);
            if (!ro.mine) return;
            const int64_t row = a.row(b, bh - b * a.Hkv, ro.t * a.G + ro.g);
#pragma unroll
            for (int c = 32 * T; c < 32 * T + 32; c += 8) *reinterpret_cast<uint4*>(static_cast<bf16*>(a.o) + row * kD + c) = make_uint4(0, 0, 0, 0);
            if (a.lse && T == 0) a.lse[row] = -INFINITY;
          });
    int np = 0;  // steps of this tile
    for (;;) {
      int steps, keys;
      bool none;  // the row counts for nothing: whatever its sums become, no step is taken again for it
      {
        TcPiece p;
        if (!take(p)) break;
        steps = T == 0 || p.two ? p.steps : 0;
        keys = p.k1 - p.k0;
        none = sh.rows[pieces % kPlans][tid] < 0;
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < steps; ++j, ++np) {
        wait(&sh.s_full[T][np & 1], np >> 1);
        if (dead) break;
        tc05_fence_after();
        const uint32_t ts = tl + kKeys * (np & 1);
        const int left = keys - kKeys * j;
        float sum = 0.0f;
        bool again = true;  // of all lanes or none
        {
          float v[kKeys];
          row_logits(ts, left, v);
          if (j == 0) m = row_top(v);
          if (__all_sync(0xffffffffu, none || fabsf(m) <= kFar)) {
            sum = row_exp(v, m * kLogitScale);
            again = !__all_sync(0xffffffffu, none || sum <= kSumLimit);
            if (!again)
#pragma unroll
              for (int c = 0; c < kKeys / 2; c += 16) tmem_st16(ts + c, v + c);
          }
        }
        if (again) {
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 8) {
            float v[8];
            tmem_ld8(ts + c, v);
            tmem_wait_ld8(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, c + e < left ? v[e] : -INFINITY);
          }
          const float to = fmaxf(m, top), corr = ex2((m - shift_of(to)) * kLogitScale);  // 0 on the first keys
          m = to;
          l *= corr;
          if (j > 0 && __any_sync(0xffffffffu, corr != 1.0f)) {
            wait(&sh.pv_done[T][(np - 1) & 1], (np - 1) >> 1);
            tc05_fence_after();
#pragma unroll 1
            for (int c = 0; c < 64; c += 8) {
              float o[8];
              tmem_ld8(tl + kTcO + c, o);
              tmem_wait_ld8(o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= corr;
              tmem_st8(tl + kTcO + c, o);
            }
          }
          sum = row_exp_any(ts, left, shift_of(m));
        }
        l += sum;
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full[T][np & 1]);
      }
      if (steps > 0) {
        wait(&sh.pv_done[T][(np - 1) & 1], (np - 1) >> 1);
        tc05_fence_after();
      }
      const float mc = shift_of(m) * kLogitScale;
      if (dead) break;
      const int plan = pieces % kPlans, code = sh.rows[plan][tid], place = sh.plan[plan].place;
      const bool mine = code != INT_MIN, whole = place < 0;
      const int row = none ? ~code : code;
      // parts: (o, m, l) as they are; else o / l.  Through shared memory, so that eight
      // lanes write a row's 128 bytes together.  (Loops: this code runs once a piece, and
      // fetching it costs more than running it.)
      const uint32_t stage = ring + Shape::kSlots * kKeyTile + warp * 4096;
      const bool part = a.parts || !whole;
      char* const to = part ? reinterpret_cast<char*>(whole ? a.part_o : w.place_o) : static_cast<char*>(a.o);
      const int at = part && !whole ? place + tid : row;
      const float f = part ? 1.0f : 1.0f / l;
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        float o[16];
        if (steps > 0) {
          tmem_ld8(tl + kTcO + c, o);
          tmem_ld8(tl + kTcO + c + 8, o + 8);
          tmem_wait_ld8(o);
          tmem_wait_ld8(o + 8);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * f;
        if (part) {  // 32 dims of fp32 at a time
#pragma unroll
          for (int k = 0; k < 4; ++k) st_stage(stage + swz(lane, ((c >> 2) & 4) + k), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (!(c & 16)) continue;
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            st_stage(stage + swz(lane, (c >> 3) + k), __uint_as_float(pack_bf16(o[8 * k], o[8 * k + 1])),
                     __uint_as_float(pack_bf16(o[8 * k + 2], o[8 * k + 3])), __uint_as_float(pack_bf16(o[8 * k + 4], o[8 * k + 5])),
                     __uint_as_float(pack_bf16(o[8 * k + 6], o[8 * k + 7])));
          if (c < 48) continue;
        }
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 32; i += 8)
#pragma unroll
          for (int h = 0; h < 8; h += 4) {
            const int rr = i + h + (lane >> 3), k = lane & 7;
            const int there = __shfl_sync(0xffffffffu, mine ? at : -1, rr);
            uint4 x;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(stage + swz(rr, k)) : "memory");
            if (there >= 0) *reinterpret_cast<uint4*>(to + (int64_t)there * (part ? 256 : 128) + (part ? 4 * (c & 32) : 0) + 16 * k) = x;
          }
        __syncwarp();
      }
      tc05_fence_before();
      if (mine) {
        if (part)
          (whole ? a.part_ml[row] : w.place_ml[at]) = none ? make_float2(-INFINITY, -1.0f) : make_float2(mc, l);
        else if (a.lse)
          a.lse[row] = none ? -INFINITY : (mc + log2f(l)) * kLn2;
      }
      give_back();
    }
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  } else {
    fewer_registers<kTcFewerRegs>();
    if (warp == 8) {
      // ---- copies
      int n = 0, nq = 0;  // key and value tiles, pieces so far
      TcPiece p;
      for (; take(p); give_back()) {
        const int buf = nq % Shape::kQBufs;
        if (nq >= Shape::kQBufs) wait(&sh.q_empty[buf], nq / Shape::kQBufs - 1);
        if (dead) break;
        if (elect_one()) {
          const uint32_t bar = smem_u32(&sh.q_full[buf]);
          mbar_expect_tx(bar, (p.two ? 2 : 1) * PARTS * kTcTile);
          for (int T = 0; T < (p.two ? 2 : 1); ++T) {
            const int tb = (p.tile + T) / w.rt.groups, hb = p.tile + T - tb * w.rt.groups;
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
              tma_load_4d(smem + buf * Shape::kQBytes + (T * PARTS + i) * kTcTile, &qm, 0, tb << w.rt.lgR,
                          p.kvh * a.G + (hb << (7 - w.rt.lgR)), p.b + i, bar);
          }
        }
        __syncwarp();
        ++nq;
        for (int j = p.k0; j < p.k1 && !dead; j += kKeys)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = n % Shape::kSlots;
            if (n >= Shape::kSlots) wait(&sh.empty[slot], n / Shape::kSlots - 1);
            if (dead) break;
            if (elect_one() && (n != a.debug_skip || blockIdx.x > 0)) {
              const uint32_t bar = smem_u32(&sh.full[slot]);
              mbar_expect_tx(bar, kKeyTile);
              tma_load_4d(ring + slot * kKeyTile, kv ? &vm : &km, 0, j, p.kvh, p.b, bar);
            }
            __syncwarp();
            ++n;
          }
      }
      if (dead) {  // copies under way end before their memory goes (whatever the limit of the others)
        if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
        for (int i = max(0, n - Shape::kSlots); i < n; ++i)
          mbar_wait_bounded(smem_u32(&sh.full[i % Shape::kSlots]), (i / Shape::kSlots) & 1, kDefaultWaitCycles);
        for (int i = max(0, nq - Shape::kQBufs); i < nq; ++i)
          mbar_wait_bounded(smem_u32(&sh.q_full[i % Shape::kQBufs]), (i / Shape::kQBufs) & 1, kDefaultWaitCycles);
      }
    } else if (warp < 11) {
      // ---- products of tile T: a step's logits are issued before the last step's
      // outputs.  A warp a tile: one for both took 2800 clocks a step to issue what the
      // tensor cores do in 1024, two take half each, side by side.
      constexpr uint32_t idS = idesc_bf16(128, kKeys, false, false), idO = idesc_bf16(128, 64, false, true);
      constexpr uint32_t kHi = smem_desc_hi(1024), kTileU = kTcTile / 16, kKeyU = kKeyTile / 16;
      const int T = warp - 9;
      const bool lead = elect_one();
      const uint32_t q0 = smem_desc_lo(smem, 16) + T * PARTS * kTileU, k0 = smem_desc_lo(ring, 16), v0 = smem_desc_lo(ring, 8192);
      const uint32_t d = tm + kTcTileCols * T;
      int n = 0, nq = 0, ns = 0;       // steps of the CTA, pieces, steps of this tile
      bool had = false, begin = false;  // whether the last step was this tile's, a piece's first
      auto outputs = [&]() {  // O (+)= P V of step n - 1
        const int slot = (2 * n - 1) % Shape::kSlots;
        wait(&sh.v_ready[slot >> 1], (n - 1) / (Shape::kSlots / 2));
        if (had) wait(&sh.p_full[T][(ns - 1) & 1], (ns - 1) >> 1);
        if (dead) return;
        if (lead) {
          if (had) {
            tc05_fence_after();
            const uint32_t v = v0 + slot * kKeyU, p = d + kKeys * ((ns - 1) & 1);
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)  // 16 keys: two groups of 8 rows, 8 columns of P
              if (i > 0)
                mma_ts<true>(d + kTcO, p + 8 * i, v + 128 * i, kHi, idO);
              else if (begin)
                mma_ts<false>(d + kTcO, p, v, kHi, idO);
              else
                mma_ts<true>(d + kTcO, p, v, kHi, idO);
            umma_commit(smem_u32(&sh.pv_done[T][(ns - 1) & 1]));
          }
          umma_commit(smem_u32(&sh.empty[slot]));
        }
        __syncwarp();
      };
      TcPiece p;
      for (; take(p); give_back()) {
        const int buf = nq % Shape::kQBufs, steps = p.steps;
        const bool mine = T == 0 || p.two;
        wait(&sh.q_full[buf], nq / Shape::kQBufs);
        ++nq;
        for (int j = 0; j < steps && !dead; ++j) {
          const int at = 2 * n, slot = at % Shape::kSlots;
          wait(&sh.full[slot], at / Shape::kSlots);  // (not only its own: what it frees is there by then)
          if (mine && ns > 1) wait(&sh.pv_done[T][ns & 1], (ns - 2) >> 1);  // P of the step before the last lies where S goes
          if (dead) break;
          if (lead) {
            if (mine) {
              tc05_fence_after();
              const uint32_t q = q0 + buf * 2 * PARTS * kTileU, k = k0 + slot * kKeyU, to = d + kKeys * (ns & 1);
#pragma unroll
              for (int i = 0; i < 4 * PARTS; ++i)
                if (i > 0)
                  mma_ss<true>(to, q + (i >> 2) * kTileU + 2 * (i & 3), k + 2 * (i & 3), kHi, idS);
                else
                  mma_ss<false>(to, q, k, kHi, idS);
              umma_commit(smem_u32(&sh.s_full[T][ns & 1]));
            }
            umma_commit(smem_u32(&sh.empty[slot]));
            if (j == steps - 1) umma_commit(smem_u32(&sh.q_empty[buf]));
          }
          __syncwarp();
          if (n > 0) outputs();
          if (dead) break;
          had = mine;
          begin = j == 0;
          ++n;
          ns += mine;
        }
      }
      if (n > 0 && !dead) outputs();
      if (dead) {  // products under way end before their memory goes
        if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
        for (int i = max(0, ns - 1); i <= ns; ++i) {
          mbar_wait_bounded(smem_u32(&sh.s_full[T][i & 1]), (i >> 1) & 1, kDefaultWaitCycles);
          if (i > 0) mbar_wait_bounded(smem_u32(&sh.pv_done[T][(i - 1) & 1]), ((i - 1) >> 1) & 1, kDefaultWaitCycles);
        }
      }
    } else {
      // ---- the pieces; and values behind a sequence's last key are made zeros (they may be
      // anything, and 0 * NaN would reach every row)
      int4 split = make_int4(0, 0, 0, 0);
      bool more = some, ended = false;
      int n = 0, planned = 0;
      auto plan = [&]() {  // one more piece, or that there is none
        const int i = planned % kPlans;
        if (planned >= kPlans) wait(&sh.plan_empty[i], planned / kPlans - 1);
        if (dead) return;
        if (!more) {
          if (lane == 0) sh.plan[i].steps = 0;
          ended = true;
        } else {
          const int pairs = wk.units / a.Hkv, kvh = wk.u / pairs, tile = 2 * (wk.u - kvh * pairs);
          const int nq = a.queries(wk.b), nk = a.keys(wk.b);
          const bool two = tile + 1 < w.rt.used(nq);
          if (lane == 0) {
            TcPiece p;
            p.steps = wk.s1 - wk.s0;
            p.b = wk.b;
            p.kvh = kvh;
            p.tile = tile;
            p.k0 = kKeys * wk.s0;
            p.k1 = min(kKeys * wk.s1, nk);
            p.two = two;
            p.place = wk.whole() ? -1 : (2 * blockIdx.x + (wk.s0 == 0)) * 256;
            sh.plan[i] = p;
          }
          if (!wk.whole() && wk.s0 == 0) split = make_int4(wk.b, kvh, tile, sh.walk.shares.owner(wk.begin + wk.steps + kUnitCost - 1) - blockIdx.x + 1);
#pragma unroll 1
          for (int r = lane; r < 256; r += 32) {
            const RowOf ro = row_of(a, w.rt, tile + (r >> 7), r & 127);
            const int row = (int)(wk.b * a.rs.b + (kvh * a.G + ro.g) * a.rs.h + ro.t * a.rs.t);
            sh.rows[i][r] = !ro.mine ? INT_MIN : ro.t >= nq || (r >= 128 && !two) ? ~row : row;
          }
          more = wk.next(a.B, counts);
        }
        ++planned;
        arrive(&sh.plan_full[i]);
      };
      plan();
      for (int x = 0; !dead; ++x) {
        while (planned < x + 3 && !ended && !dead) plan();
        if (x == planned - 1 && ended) break;
        const int k0 = sh.plan[x % kPlans].k0, k1 = sh.plan[x % kPlans].k1;
        for (int j = k0; j < k1 && !dead; j += kKeys, ++n) {
          const int at = 2 * n + 1, slot = at % Shape::kSlots;
          wait(&sh.full[slot], at / Shape::kSlots);
          if (dead) break;
          if (k1 - j < kKeys) {
#pragma unroll 1
            for (int r = k1 - j + lane; r < kKeys; r += 32)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_stage(ring + slot * kKeyTile + r * 128 + 16 * c, 0.0f, 0.0f, 0.0f, 0.0f);
            fence_async_smem();
          }
          arrive(&sh.v_ready[slot >> 1]);
        }
      }
      if (lane == 0) w.split[blockIdx.x] = split;
      if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 9) tmem_dealloc(tm, kTcCols);
}

// Units that span CTAs: their parts to o and lse.
// FEW units have many parts each: CTA (u, y) has 8 rows of unit u, a warp a row.
// Many have two, and most have none: CTA (c, y) has 64 rows of the unit that CTA c
// began, eight lanes a row.  (A row a warp, and 32 CTAs for each that began one,
// took 20 us for 32 sequences of up to 1024 x 2048.)
template <bool FEW>
__global__ void __launch_bounds__(256) cross_join_places_kernel(const CrossArgs a, const TcWork w, int ctas) {
  __shared__ int4 found;
  __shared__ int from;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  int4 s;
  int c;
  if (FEW) {
    const int pairs = (w.rt.tiles + 1) >> 1, bh = blockIdx.x / pairs, tile = 2 * (blockIdx.x - bh * pairs);
    if (threadIdx.x == 0) found.w = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < ctas; i += 256) {
      const int4 x = w.split[i];
      if (x.w > 1 && x.x * a.Hkv + x.y == bh && x.z == tile) {
        found = x;
        from = i;
      }
    }
    __syncthreads();
    s = found;
    c = from;
  } else {
    c = blockIdx.x;
    s = w.split[c];
  }
  if (s.w <= 1) return;
  auto place = [&](int x, int i) { return (int64_t)(x == 0 ? 2 * c + 1 : 2 * (c + x)) * 256 + i; };
  if (FEW) {
    const int i = blockIdx.y * 8 + (threadIdx.x >> 5);
    const RowOf ro = row_of(a, w.rt, s.z + (i >> 7), i & 127);
    if (ro.mine)
      join_row<8, bf16>(a, s.x * a.rs.b + (s.y * a.G + ro.g) * a.rs.h + ro.t * a.rs.t, s.w, lane, [&](int x) { return w.place_ml[place(x, i)]; },
                     [&](int x) { return w.place_o + place(x, i) * kD; });
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = blockIdx.y * 64 + 32 * h + (threadIdx.x >> 3), d8 = (threadIdx.x & 7) * 8;
    const RowOf ro = row_of(a, w.rt, s.z + (i >> 7), i & 127);
    if (!ro.mine) continue;
    const int64_t row = s.x * a.rs.b + (s.y * a.G + ro.g) * a.rs.h + ro.t * a.rs.t;
    float m = -INFINITY, l = 0.0f, y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, z[8];
    bool any = false;
    for (int x = 0; x < s.w; ++x) m = fmaxf(m, w.place_ml[place(x, i)].x);
    const float sh = shift_of(m);
    for (int x = 0; x < s.w; ++x) {
      const float2 v = w.place_ml[place(x, i)];
      load8(w.place_o + place(x, i) * kD + d8, z);
      const bool none = v.y < 0.0f;  // (the part's sums are zeros then)
      const float f = none ? 0.0f : exp2f(v.x - sh);
      any |= !none;
      l = fmaf(f, none ? 0.0f : v.y, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(f, z[e], y[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = any ? y[e] / l : 0.0f;
    store8(static_cast<bf16*>(a.o) + row * kD + d8, y);
    if (a.lse && d8 == 0) a.lse[row] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

// A decode step behind a prefix: the prefix's parts, whole units' in the rows' own
// places, and those of the sequences' own rows behind them (a.part_o + rows * 64 on).
template <int S>
__global__ void __launch_bounds__(256) prefix_join_kernel(const CrossArgs a, const TcWork w, const Shares shares, int steps, const int32_t* pos, int T) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // [B][Hq]
  if (row >= a.rows) return;
  const int b = (int)(row / a.Hq), h = (int)(row - (int64_t)b * a.Hq), kvh = h / a.G, g = h - kvh * a.G;
  const int t = pos[b];
  const bool there = t >= 0 && t < T;
  const int tile = (b >> w.rt.lgR) * w.rt.groups + (g >> (7 - w.rt.lgR));
  const int i = (tile & 1) * 128 + ((g & ((1 << (7 - w.rt.lgR)) - 1)) << w.rt.lgR) + (b & ((1 << w.rt.lgR) - 1));
  const int64_t begin = ((int64_t)kvh * ((w.rt.tiles + 1) >> 1) + (tile >> 1)) * (steps + kUnitCost);
  const int c0 = shares.owner(begin + kUnitCost), c1 = shares.owner(begin + kUnitCost + steps - 1), n = c1 - c0 + 1;
  auto place = [&](int x) { return (int64_t)(x == 0 ? 2 * c0 + 1 : 2 * (c0 + x)) * 256 + i; };
  join_row<S, bf16>(a, row, there ? n + a.splits : 0, lane,
                 [&](int x) { return x >= n ? a.part_ml[(1 + x - n) * a.rows + row] : n == 1 ? a.part_ml[row] : w.place_ml[place(x)]; },
                 [&](int x) {
                   return x >= n ? a.part_o + ((1 + x - n) * a.rows + row) * kD : n == 1 ? a.part_o + row * kD : w.place_o + place(x) * kD;
                 });
}

RowTiles row_tiles(int G, int Tq) {
  RowTiles best = {};
  for (int lg = 7; lg >= 2; --lg) {  // fewest tiles, then most queries a tile (32 heads at most)
    RowTiles t;
    t.lgR = lg;
    t.groups = (G + (1 << (7 - lg)) - 1) >> (7 - lg);
    t.blocks = (Tq + (1 << lg) - 1) >> lg;
    t.tiles = t.groups * t.blocks;
    if (lg == 7 || t.tiles < best.tiles) best = t;
  }
  return best;
}

// Shares, of the most that the lengths may come to.  (A unit in parts costs a launch and
// their writing: 8 x 8 / 2 heads, 512 x 512 22.3 us in 152 shares of 6.7 steps, 14.0 in 128
// whole units of 8; 2 x 16 / 2, 2048 x 300 27.1 and 18.2; with 12 steps for 8, 17 x 1000 took
// 14.1 us for 12.3.  A prefix's are written and joined with the own rows' anyway.)
static Shares tc_shares(int B, int Hkv, const RowTiles& rt, int Tk, bool alike, int extra) {
  return deal((int64_t)B * Hkv * ((rt.tiles + 1) / 2), (Tk + kKeys - 1) / kKeys + kUnitCost, kSMs, kTcLeast, alike, extra);
}
static Shares call_shares(const CrossArgs& a, const RowTiles& rt) {
  return tc_shares(a.B, a.Hkv, rt, a.Tk, !a.q_len && !a.kv_len, a.parts ? 0 : 8);
}

static size_t places_o(int ctas) { return (size_t)2 * ctas * 256 * kD * sizeof(float); }

size_t cross_tc_bytes(int B, int Hkv, int G, int Tq, int Tk) {
  const int ctas = tc_shares(B, Hkv, row_tiles(G, Tq), Tk, false, 0).ctas;  // (lengths may differ)
  return align256(places_o(ctas) + (size_t)2 * ctas * 256 * sizeof(float2) + ctas * sizeof(int4));
}

static TcWork tc_work(const CrossArgs& a, void* ws, int* ctas) {
  TcWork w;
  w.rt = row_tiles(a.G, a.Tq);
  *ctas = call_shares(a, w.rt).ctas;
  w.place_o = static_cast<float*>(ws);
  w.place_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + places_o(*ctas));
  w.split = reinterpret_cast<int4*>(w.place_ml + (size_t)2 * *ctas * 256);
  return w;
}

template <int PARTS>
static int fwd_tc(const CrossArgs& a, const TcWork& w, int ctas, cudaStream_t st) {
  CUtensorMap qm, km, vm;
  int rc = make_view_map(&qm, a.q, a.Tq, a.Hq, PARTS == 2 ? 2 : a.B, a.qs, 1 << w.rt.lgR, 128 >> w.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&km, a.k, a.Tk, a.Hkv, a.B, a.ks, kKeys, 1);
  if (rc == SFA_OK) rc = make_view_map(&vm, a.v, a.Tk, a.Hkv, a.B, a.vs, kKeys, 1);
  if (rc != SFA_OK) return rc;
  auto* f = cross_fwd_tc_kernel<PARTS>;
  static_assert(TcShape<PARTS>::kSmem + sizeof(TcShared) + 1024 <= 228 * 1024, "shared memory of an SM");
  LaunchTimer tm(SFA_KERNEL_CROSS_FWD, st);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<PARTS>::kSmem);
  if (e == cudaSuccess) e = launch_pdl(f, dim3((unsigned)ctas), dim3(kTcThreads), TcShape<PARTS>::kSmem, st, a, w, qm, km, vm);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int launch_cross_fwd_tc(const CrossArgs& a, void* ws, void* stream) {
  int ctas;
  const TcWork w = tc_work(a, ws, &ctas);
  const int rc = fwd_tc<1>(a, w, ctas, (cudaStream_t)stream);
  // where all lengths are alike and each CTA has whole units, there is nothing to join
  const Shares s = call_shares(a, w.rt);
  if (rc != SFA_OK || ctas == 1 || (!a.q_len && !a.kv_len && s.rest == 0 && s.share % ((a.Tk + kKeys - 1) / kKeys + kUnitCost) == 0)) return rc;
  LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
  const int64_t units = (int64_t)a.B * a.Hkv * ((w.rt.tiles + 1) / 2);
  const bool few = 4 * units <= ctas;
  const dim3 grid = few ? dim3((unsigned)units, 32) : dim3((unsigned)ctas, 4);
  const cudaError_t e = launch_pdl(few ? cross_join_places_kernel<true> : cross_join_places_kernel<false>, grid, dim3(256), 0,
                                   (cudaStream_t)stream, a, w, ctas);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int launch_prefix_tc(const CrossArgs& a, void* ws, void* stream) {
  int ctas;
  const TcWork w = tc_work(a, ws, &ctas);
  return fwd_tc<2>(a, w, ctas, (cudaStream_t)stream);
}

int launch_prefix_join(const CrossArgs& prefix, const CrossArgs& out, void* ws, const int32_t* pos, int T, void* stream) {
  int ctas;
  const TcWork w = tc_work(prefix, ws, &ctas);
  const Shares s = call_shares(prefix, w.rt);
  const int steps = (prefix.Tk + kKeys - 1) / kKeys;
  const bool few = steps / s.share + 2 + out.splits <= kFewParts;
  LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
  const cudaError_t e = launch_pdl(few ? prefix_join_kernel<kFewParts / 4> : prefix_join_kernel<8>, dim3((unsigned)((out.rows + 7) / 8)), dim3(256), 0,
                                   (cudaStream_t)stream, out, w, s, steps, pos, T);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
