// Backward pass of attention to states of another length on the
// fifth-generation tensor cores (bf16): dq, and dk and dv, which are the same walk
// with the roles of queries and keys exchanged.
//
//   dq     a tile of 128 rows stays, their keys and values pass by:
//            S = Q K^T, dP = dO V^T, dS = P (dP - delta), dQ += dS K
//   dk,dv  a tile of 128 keys stays, the rows that attend it (all heads of the
//          group) pass by:
//            S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//
// Each sum has one owner, or a fixed order of parts, so nothing is added atomically
// and equal inputs give equal bits; the price is S and dP twice (7 products instead
// of 5).  In both the probabilities come out of tensor memory the way they go back in
// as a left operand: a lane per row of the tile that stays, so P and dS never pass
// shared memory.  Per step one warp issues the next S and dP as soon as 16 warps
// hold this step's in registers (32 columns of both a thread), another the
// accumulations when P and dS are back.  P and dS are rounded to bf16 for their
// products; everything else is fp32.  The steps of all tiles are dealt out evenly
// over the SMs, and planned ahead by one warp, as in the forward pass.
#include <limits.h>

#include <algorithm>

#include "sfa_cross.cuh"

namespace sfa {

// 16 warps of softmax, a copying warp, two that issue, one that clears rows, one that
// plans (three more make a warpgroup).
constexpr int kBtSoftmax = 16, kBtThreads = 32 * (kBtSoftmax + 8);
// Registers: 80 a thread at launch, 768 x 80 = 512 x 96 + 256 x 48.
constexpr int kBtMoreRegs = 96, kBtFewerRegs = 48;
constexpr int kBtTile = 128 * 128;  // bytes of 128 rows of 64 bf16
constexpr int kBtStages = 4;
constexpr int kBtStat = 1024;  // bytes of a row tile's numbers: 128 of -lse log2(e), 128 of -delta
constexpr int kBtStays = 0, kBtRing = kBtStays + 2 * 2 * kBtTile, kBtOut = kBtRing + kBtStages * 2 * kBtTile,
              kBtStatRing = kBtOut + kBtSoftmax * 1024, kBtStatStays = kBtStatRing + kBtStages * kBtStat, kBtSmem = kBtStatStays + 2 * kBtStat + 1024;
constexpr int kBtPlans = 4;
constexpr int kBtLeast = 6;  // steps a CTA has at least (with 3, 4 x 8 / 2 heads, 64 x 64 took 15.7 us, so 14.1)
// tensor memory: S, dP, P, dS, sums of dq or dk, of dv
constexpr int kBtDp = 128, kBtP = 256, kBtDs = 320, kBtSum = 384, kBtSum2 = 448;

// A piece as the roles need it.
struct BtPiece {
  int steps;                  // none: there are no more pieces
  int b, kvh, tile, t0;       // the tile that stays, the first that passes by
  int nq, nk, place;          // place: of its sums, -1 for a whole unit
};

struct BtShared {
  uint64_t full[kBtStages], empty[kBtStages], ready[kBtStages];  // ready: rows that count for nothing are zeros
  uint64_t a_full[2], a_empty[2], s_full, s_free, p_full, done;
  uint64_t plan_full[kBtPlans], plan_empty[kBtPlans];
  BtPiece plan[kBtPlans];
  int rows[kBtPlans][128];  // dq: where a row is; ~ of it for one behind the last query, INT_MIN for none
  WalkShared walk;
  uint32_t tmem;
};

struct BtWork {
  RowTiles rt;
  int key_tiles;
  const float* stat;  // [B][Hkv][row tiles][2][128]
  float* places;      // [2 CTAs][128][64], dk and dv: twice that, dv's behind dk's
  int ctas;
  int4* split;        // [CTAs]: the unit that a CTA begins and does not end: sequence, KV head, tile, parts (0: none)
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_out(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// CTA cta of ctas.
template <bool DKV>
__device__ __forceinline__ void cross_bwd_tc(const CrossArgs& a, const BtWork& w, const CUtensorMap& qm, const CUtensorMap& gm, const CUtensorMap& km,
                                             const CUtensorMap& vm, uint8_t* smem_raw, BtShared& sh, int cta, int ctas) {
  const uint32_t smem = smem_u32(smem_raw) + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, and known to be)
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kBtStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
      mbar_init(smem_u32(&sh.ready[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.a_full[i]), 1);
      mbar_init(smem_u32(&sh.a_empty[i]), DKV ? 1 : kBtSoftmax + 1);  // (dq: the softmax warps read the staying rows' numbers)
    }
    for (int i = 0; i < kBtPlans; ++i) {
      mbar_init(smem_u32(&sh.plan_full[i]), 1);
      mbar_init(smem_u32(&sh.plan_empty[i]), kBtSoftmax + 3);  // all others that take pieces
    }
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.s_free), kBtSoftmax);
    mbar_init(smem_u32(&sh.p_full), kBtSoftmax);
    mbar_init(smem_u32(&sh.done), 1);
    mbar_fence_init();
  }
  if (warp == kBtSoftmax + 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  if (warp == kBtSoftmax && lane < 4) prefetch_map(lane == 0 ? &qm : lane == 1 ? &gm : lane == 2 ? &km : &vm);
  pdl_wait();
  auto counts = [&](int b, int& units, int& steps) {
    const int nk = a.keys(b), nq = a.queries(b), keys = (nk + 127) >> 7, rows = w.rt.used(nq);
    units = nk > 0 && nq > 0 ? a.Hkv * (DKV ? keys : rows) : 0;
    steps = DKV ? rows : keys;
  };
  Walk wk;
  tc05_fence_before();
  const bool some = find_walk<kBtThreads>(a.B, counts, cta, ctas, kBtLeast, sh.walk, wk);  // (with barriers of the CTA)
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
  auto take = [&](BtPiece& p) {
    const int i = pieces % kBtPlans;
    wait(&sh.plan_full[i], pieces / kBtPlans);
    if (dead) return false;
    p = sh.plan[i];
    p.steps = __shfl_sync(0xffffffffu, p.steps, 0);  // (known to be the same in all lanes)
    return p.steps > 0;
  };
  auto give_back = [&]() { arrive(&sh.plan_empty[pieces++ % kBtPlans]); };

  if (warp < kBtSoftmax) {
    // ---- P and dS: a thread a row of the tile that stays, 32 of the 128 that pass by
    more_registers<kBtMoreRegs>();
    const int quarter = warp >> 2, r = tid & 127;
    const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    // tiles without work: zeros
    if (a.q_len || a.kv_len) {
      const int own = DKV ? w.key_tiles : w.rt.tiles;
      each_empty(
          (int64_t)a.B * a.Hkv * own, cta, ctas, lane,
          [&](int64_t x) {
            const int bh = (int)(x / own);
            int units, steps;
            counts(bh / a.Hkv, units, steps);
            return x - (int64_t)bh * own >= units / a.Hkv;
          },
          [&](int64_t x) {
            const int bh = (int)(x / own), tile = (int)(x - (int64_t)bh * own), b = bh / a.Hkv;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            if (DKV) {
              const int j = tile * 128 + r;
              if (j >= a.Tk) return;
              uint4* const out = reinterpret_cast<uint4*>(static_cast<bf16*>(quarter >> 1 ? a.dv : a.dk) + ((int64_t)bh * a.Tk + j) * kD + 32 * (quarter & 1));
#pragma unroll
              for (int c = 0; c < 4; ++c) out[c] = zero;
            } else {
              const RowOf ro = row_of(a, w.rt, tile, r);
              if (!ro.mine) return;
              uint4* const out = reinterpret_cast<uint4*>(static_cast<bf16*>(a.dq) + a.row(b, bh - b * a.Hkv, ro.t * a.G + ro.g) * kD + 16 * quarter);
              out[0] = zero;
              out[1] = zero;
            }
          });
    }
    int n = 0;
    for (;;) {
      int steps, nk, t0;
      unsigned counted;  // dk, dv: which of this warp's keys count
      {
        BtPiece p;
        if (!take(p)) break;
        steps = p.steps;
        nk = p.nk;
        t0 = p.t0;
        counted = DKV ? __ballot_sync(0xffffffffu, r < p.nk - 128 * p.tile) : 0;
      }
      float2 own = make_float2(-INFINITY, 0.0f);
      if (!DKV) {
        const int buf = pieces & 1;
        wait(&sh.a_full[buf], pieces >> 1);
        const uint32_t at = smem + kBtStatStays + buf * kBtStat + 4 * r;
        asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(own.x) : "r"(at) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(own.y) : "r"(at + 512) : "memory");
      }
      for (int j = 0; j < steps; ++j, ++n) {
        const int st = n % kBtStages;
        if (DKV) wait(&sh.full[st], n / kBtStages);  // (the rows' numbers)
        wait(&sh.s_full, n);
        if (dead) break;
        tc05_fence_after();
        float s[32], d[32];
        tmem_take32(tl + 32 * quarter, s);
        tmem_take32(tl + kBtDp + 32 * quarter, d);
        tc05_fence_before();
        arrive(&sh.s_free);
        const float2 c2 = make_float2(kLogitScale, kLogitScale);
        const uint32_t stat = smem + kBtStatRing + st * kBtStat + 128 * quarter;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4 nl, nd;
          if (DKV) {
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(nl.x), "=f"(nl.y), "=f"(nl.z), "=f"(nl.w) : "r"(stat + 4 * e));
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(nd.x), "=f"(nd.y), "=f"(nd.z), "=f"(nd.w) : "r"(stat + 512 + 4 * e));
          } else {
            nl = make_float4(own.x, own.x, own.x, own.x);
            nd = make_float4(own.y, own.y, own.y, own.y);
          }
          const float2 y0 = pair_fma(make_float2(s[e], s[e + 1]), c2, make_float2(nl.x, nl.y));
          const float2 y1 = pair_fma(make_float2(s[e + 2], s[e + 3]), c2, make_float2(nl.z, nl.w));
          const float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
          const float2 g0 = pair_mul(p0, pair_add(make_float2(d[e], d[e + 1]), make_float2(nd.x, nd.y)));
          const float2 g1 = pair_mul(p1, pair_add(make_float2(d[e + 2], d[e + 3]), make_float2(nd.z, nd.w)));
          if (DKV) {
            s[e >> 1] = __uint_as_float(pack_bf16(p0.x, p0.y));
            s[(e >> 1) + 1] = __uint_as_float(pack_bf16(p1.x, p1.y));
          }
          d[e >> 1] = __uint_as_float(pack_bf16(g0.x, g0.y));
          d[(e >> 1) + 1] = __uint_as_float(pack_bf16(g1.x, g1.y));
        }
        // Rows that count for nothing are zeros, whose products with a key or value that is not finite
        // are NaN: their P and dS are made zeros too.  If one of the 32 counts for nothing, the last
        // does, so its dS says whether to look, of keys that count (32 x 8 / 2 heads, 1024 x 2048 ragged
        // rows: 238 us, and 248 with zeros made in each tile that has such rows, whatever their products).
        if (DKV && (__ballot_sync(0xffffffffu, (__float_as_uint(d[15]) & 0x7fffffffu) > 0x7f80ffffu) & counted) != 0) {
          const RowOf ro = row_of(a, w.rt, t0 + j, 32 * quarter + lane);
          const unsigned in = __ballot_sync(0xffffffffu, ro.mine && ro.t < sh.plan[pieces % kBtPlans].nq);
#pragma unroll
          for (int e = 0; e < 32; ++e)  // (two a register)
            if (!(in >> e & 1)) {
              const uint32_t keep = e & 1 ? 0x0000ffffu : 0xffff0000u;
              s[e >> 1] = __uint_as_float(__float_as_uint(s[e >> 1]) & keep);
              d[e >> 1] = __uint_as_float(__float_as_uint(d[e >> 1]) & keep);
            }
        }
        const int left = DKV ? 128 : nk - 128 * (t0 + j) - 32 * quarter;  // keys of this quarter that are there
        if (left < 32) {
#pragma unroll
          for (int e = 0; e < 32; ++e)  // (two a register)
            if (e >= left) d[e >> 1] = __uint_as_float(__float_as_uint(d[e >> 1]) & (e & 1 ? 0x0000ffffu : 0u));
        }
        if (n > 0) wait(&sh.done, n - 1);  // the last step's P and dS have been read
        if (dead) break;
        tc05_fence_after();
        if (DKV) tmem_st16(tl + kBtP + 16 * quarter, s);
        tmem_st16(tl + kBtDs + 16 * quarter, d);
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full);
      }
      // (Not before the last use: given back right after the reads above, the buffer was now
      // and then filled with the piece after next's numbers before `own` had been read.)
      if (!DKV) arrive(&sh.a_empty[pieces & 1]);
      if (!dead) {
        wait(&sh.done, n - 1);
        tc05_fence_after();
      }
      if (dead) break;
      // The first eight warps have dk, the others dv, half the dims each; dq: a quarter of
      // the dims each.  16 dims at a time through shared memory, so that lanes write rows
      // together.
      const int plan = pieces % kBtPlans, dv = DKV ? quarter >> 1 : 0;
      const BtPiece p = sh.plan[plan];
      const bool whole = p.place < 0;
      int row;  // of this thread, where it is written; INT_MIN: nowhere, ~: as zeros
      if (DKV) {
        const int key = p.tile * 128 + r;
        row = whole ? (p.b * a.Hkv + p.kvh) * a.Tk + key : (p.place + (dv ? ctas * 2 : 0)) * 128 + r;
        row = key >= a.Tk ? INT_MIN : key >= p.nk ? ~row : row;
      } else {
        row = sh.rows[plan][r];
        if (!whole && row != INT_MIN) row = row < 0 ? ~(p.place * 128 + r) : p.place * 128 + r;
      }
      const bool none = row < 0;
      const int at = row == INT_MIN ? -1 : none ? ~row : row;
      const float f = none ? 0.0f : dv ? 1.0f : 0.125f;
      char* const to = whole ? static_cast<char*>(DKV ? (dv ? a.dv : a.dk) : a.dq) : reinterpret_cast<char*>(w.places);
      const uint32_t stage = smem + kBtOut + warp * 1024;
      const int lgc = whole ? 1 : 2;  // 16-byte pieces of 16 dims: 2 of bf16, 4 of fp32
#pragma unroll 1
      for (int c = 0; c < (DKV ? 32 : 16); c += 16) {
        const int dim = DKV ? 32 * (quarter & 1) + c : 16 * quarter;
        float o[16];
        const uint32_t src = tl + (dv ? kBtSum2 : kBtSum) + dim;
        tmem_ld8(src, o);
        tmem_ld8(src + 8, o + 8);
        tmem_wait_ld8(o);
        tmem_wait_ld8(o + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * f;
        auto spot = [&](int rr, int k) { return stage + (rr & 15) * 64 + ((k ^ ((rr >> 1) & 3)) << 4); };
#pragma unroll 1
        for (int h = 0; h < 32; h += 16) {  // 16 rows
          if ((lane & 16) == h) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                st_out(spot(lane, k), pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]), pack_bf16(o[8 * k + 4], o[8 * k + 5]),
                       pack_bf16(o[8 * k + 6], o[8 * k + 7]));
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                st_out(spot(lane, k), __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                       __float_as_uint(o[4 * k + 3]));
            }
          }
          __syncwarp();
          for (int i = h; i < h + 16; i += 32 >> lgc) {
            const int rr = i + (lane >> lgc), k = lane & ((1 << lgc) - 1);
            const int there = __shfl_sync(0xffffffffu, at, rr);
            uint4 x;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(spot(rr, k)) : "memory");
            if (there >= 0) *reinterpret_cast<uint4*>(to + (int64_t)there * (whole ? 128 : 256) + dim * (whole ? 2 : 4) + 16 * k) = x;
          }
          __syncwarp();
        }
      }
      tc05_fence_before();
      give_back();
    }
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  } else {
    fewer_registers<kBtFewerRegs>();
    if (warp == kBtSoftmax) {
      // ---- copies
      int n = 0;  // steps so far
      const bool lead = elect_one();
      const int heads = 1 << (7 - w.rt.lgR);
      BtPiece p;
      for (; take(p); give_back()) {
        const int buf = pieces & 1;
        if (pieces >= 2) wait(&sh.a_empty[buf], (pieces >> 1) - 1);
        if (dead) break;
        const int row_tile = DKV ? p.t0 : p.tile;
        int tb = row_tile / w.rt.groups, hb = row_tile - tb * w.rt.groups;
        const float* stat = w.stat + (((int64_t)p.b * a.Hkv + p.kvh) * w.rt.tiles + row_tile) * 256;
        if (lead) {
          const uint32_t bar = smem_u32(&sh.a_full[buf]), dst = smem + kBtStays + buf * 2 * kBtTile;
          mbar_expect_tx(bar, 2 * kBtTile + (DKV ? 0 : kBtStat));
          if (DKV) {
            tma_load_4d(dst, &km, 0, p.tile * 128, p.kvh, p.b, bar);
            tma_load_4d(dst + kBtTile, &vm, 0, p.tile * 128, p.kvh, p.b, bar);
          } else {
            tma_load_4d(dst, &qm, 0, tb << w.rt.lgR, p.kvh * a.G + hb * heads, p.b, bar);
            tma_load_4d(dst + kBtTile, &gm, 0, tb << w.rt.lgR, p.kvh * a.G + hb * heads, p.b, bar);
            bulk_copy(smem + kBtStatStays + buf * kBtStat, stat, kBtStat, bar);
          }
        }
        __syncwarp();
        for (int t = p.t0; t < p.t0 + p.steps && !dead; ++t, ++n) {
          const int st = n % kBtStages;
          if (n >= kBtStages) wait(&sh.empty[st], n / kBtStages - 1);
          if (dead) break;
          if (lead && (n != a.debug_skip || cta > 0)) {
            const uint32_t bar = smem_u32(&sh.full[st]), dst = smem + kBtRing + st * 2 * kBtTile;
            mbar_expect_tx(bar, 2 * kBtTile + (DKV ? kBtStat : 0));
            if (DKV) {
              tma_load_4d(dst, &qm, 0, tb << w.rt.lgR, p.kvh * a.G + hb * heads, p.b, bar);
              tma_load_4d(dst + kBtTile, &gm, 0, tb << w.rt.lgR, p.kvh * a.G + hb * heads, p.b, bar);
              bulk_copy(smem + kBtStatRing + st * kBtStat, stat, kBtStat, bar);
            } else {
              tma_load_4d(dst, &km, 0, t * 128, p.kvh, p.b, bar);
              tma_load_4d(dst + kBtTile, &vm, 0, t * 128, p.kvh, p.b, bar);
            }
          }
          __syncwarp();
          if (DKV) {
            stat += 256;
            if (++hb == w.rt.groups) {
              hb = 0;
              ++tb;
            }
          }
        }
        if (dead) break;
      }
      if (dead) {  // copies under way end before their memory goes
        if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
        for (int i = max(0, n - kBtStages); i < n; ++i) mbar_wait_bounded(smem_u32(&sh.full[i % kBtStages]), (i / kBtStages) & 1, kDefaultWaitCycles);
        for (int i = max(0, pieces - 1); i <= pieces; ++i) mbar_wait_bounded(smem_u32(&sh.a_full[i & 1]), (i / 2) & 1, kDefaultWaitCycles);
      }
    } else if (warp == kBtSoftmax + 1) {
      // ---- S and dP
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false), kHi = smem_desc_hi(1024), kTileU = kBtTile / 16;
      const uint32_t a0 = smem_desc_lo(smem + kBtStays, 16), b0 = smem_desc_lo(smem + kBtRing, 16);
      const bool lead = elect_one();
      int n = 0;
      BtPiece p;
      for (; take(p); give_back()) {
        const int buf = pieces & 1;
        wait(&sh.a_full[buf], pieces >> 1);
        for (int j = 0; j < p.steps && !dead; ++j, ++n) {
          const int st = n % kBtStages;
          wait(&sh.ready[st], n / kBtStages);
          if (n > 0) wait(&sh.s_free, n - 1);
          if (dead) break;
          if (lead) {
            tc05_fence_after();
            const uint32_t aa = a0 + 2 * buf * kTileU, b = b0 + 2 * st * kTileU;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i > 0)
                mma_ss<true>(tm, aa + 2 * i, b + 2 * i, kHi, idS);
              else
                mma_ss<false>(tm, aa, b, kHi, idS);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i > 0)
                mma_ss<true>(tm + kBtDp, aa + kTileU + 2 * i, b + kTileU + 2 * i, kHi, idS);
              else
                mma_ss<false>(tm + kBtDp, aa + kTileU, b + kTileU, kHi, idS);
            umma_commit(smem_u32(&sh.s_full));
            if (j == p.steps - 1) umma_commit(smem_u32(&sh.a_empty[buf]));
          }
          __syncwarp();
        }
        if (dead) break;
      }
      if (dead) {  // products under way end before their memory goes
        if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
        for (int i = max(0, n - 1); i <= n; ++i) mbar_wait_bounded(smem_u32(&sh.s_full), i & 1, kDefaultWaitCycles);
      }
    } else if (warp == kBtSoftmax + 2) {
      // ---- the sums
      constexpr uint32_t idO = idesc_bf16(128, 64, false, true), kHi = smem_desc_hi(1024), kTileU = kBtTile / 16;
      const uint32_t b0 = smem_desc_lo(smem + kBtRing, 8192);
      const bool lead = elect_one();
      int n = 0;
      for (int x = 0; !dead; ++x) {
        // (the plan stays until the softmax warps, which need this, give it back)
        const int i = x % kBtPlans;
        wait(&sh.plan_full[i], x / kBtPlans);
        if (dead) break;
        const int steps = __shfl_sync(0xffffffffu, sh.plan[i].steps, 0);
        if (steps == 0) break;
        for (int j = 0; j < steps && !dead; ++j, ++n) {
          const int st = n % kBtStages;
          wait(&sh.p_full, n);
          if (dead) break;
          if (lead) {
            tc05_fence_after();
            const uint32_t b = b0 + 2 * st * kTileU;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i > 0)
                mma_ts<true>(tm + kBtSum, tm + kBtDs + 8 * i, b + 128 * i, kHi, idO);
              else if (j == 0)
                mma_ts<false>(tm + kBtSum, tm + kBtDs, b, kHi, idO);
              else
                mma_ts<true>(tm + kBtSum, tm + kBtDs, b, kHi, idO);
            if (DKV)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i > 0)
                  mma_ts<true>(tm + kBtSum2, tm + kBtP + 8 * i, b + kTileU + 128 * i, kHi, idO);
                else if (j == 0)
                  mma_ts<false>(tm + kBtSum2, tm + kBtP, b + kTileU, kHi, idO);
                else
                  mma_ts<true>(tm + kBtSum2, tm + kBtP, b + kTileU, kHi, idO);
            umma_commit(smem_u32(&sh.done));
            umma_commit(smem_u32(&sh.empty[st]));
          }
          __syncwarp();
        }
      }
      if (dead) {  // products under way end before their memory goes
        if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
        for (int i = max(0, n - 1); i <= n; ++i) mbar_wait_bounded(smem_u32(&sh.done), i & 1, kDefaultWaitCycles);
      }
    } else if (warp == kBtSoftmax + 3) {
      // ---- rows that pass by and count for nothing are made zeros (they may hold
      // anything, and 0 * NaN would reach every sum)
      int n = 0;
      BtPiece p;
      for (; take(p); give_back()) {
        int tb = DKV ? p.t0 / w.rt.groups : 0, hb = DKV ? p.t0 - tb * w.rt.groups : 0;
        for (int t = p.t0; t < p.t0 + p.steps && !dead; ++t, ++n) {
          const int st = n % kBtStages;
          const bool clean = DKV ? (tb + 1) << w.rt.lgR <= p.nq && (hb + 1) << (7 - w.rt.lgR) <= a.G : (t + 1) * 128 <= p.nk;
          wait(&sh.full[st], n / kBtStages);
          if (dead) break;
          if (!clean) {
#pragma unroll 1
            for (int r = lane; r < 128; r += 32) {
              bool in;
              if (DKV) {
                const RowOf ro = row_of(a, w.rt, t, r);
                in = ro.g < a.G && ro.t < p.nq;
              } else {
                in = t * 128 + r < p.nk;
              }
              if (!in)
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  st_out(smem + kBtRing + st * 2 * kBtTile + (c >> 3) * kBtTile + r * 128 + 16 * (c & 7), 0, 0, 0, 0);
            }
            fence_async_smem();
          }
          arrive(&sh.ready[st]);
          if (DKV && ++hb == w.rt.groups) {
            hb = 0;
            ++tb;
          }
        }
        if (dead) break;
      }
      if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
    } else if (warp == kBtSoftmax + 4) {
      // ---- the pieces (a warp of its own: lengths and divisions take 3000 clocks a piece)
      int4 split = make_int4(0, 0, 0, 0);
      bool more = some;
      for (int planned = 0; !dead; ++planned) {
        const int i = planned % kBtPlans;
        if (planned >= kBtPlans) wait(&sh.plan_empty[i], planned / kBtPlans - 1);
        if (dead) break;
        if (!more) {
          if (lane == 0) sh.plan[i].steps = 0;
          arrive(&sh.plan_full[i]);
          break;
        }
        const int own = wk.units / a.Hkv, kvh = wk.u / own, tile = wk.u - kvh * own;
        const int nq = a.queries(wk.b), nk = a.keys(wk.b);
        if (lane == 0) {
          BtPiece p;
          p.steps = wk.s1 - wk.s0;
          p.b = wk.b;
          p.kvh = kvh;
          p.tile = tile;
          p.t0 = wk.s0;
          p.nq = nq;
          p.nk = nk;
          p.place = wk.whole() ? -1 : 2 * cta + (wk.s0 == 0);
          sh.plan[i] = p;
        }
        if (!wk.whole() && wk.s0 == 0) split = make_int4(wk.b, kvh, tile, sh.walk.shares.owner(wk.begin + wk.steps + kUnitCost - 1) - cta + 1);
        if (!DKV)
#pragma unroll 1
          for (int r = lane; r < 128; r += 32) {
            const RowOf ro = row_of(a, w.rt, tile, r);
            const int row = (int)a.row(wk.b, kvh, ro.t * a.G + ro.g);
            sh.rows[i][r] = !ro.mine ? INT_MIN : ro.t >= nq ? ~row : row;
          }
        more = wk.next(a.B, counts);
        arrive(&sh.plan_full[i]);
      }
      if (lane == 0) w.split[cta] = split;
      if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == kBtSoftmax + 1) tmem_dealloc(tm, 512);
}

// dq's CTAs, dk's and dv's, or both in one launch, kv's first (BtPlan says which).  Each
// in a kernel of its own, because with both in one the registers of a thread do not reach
// (32 x 8 / 2 heads, 1024 x 2048 ragged rows through it in two launches: 251 us, so 238).
enum BtPart { kBtDq, kBtDkv, kBtBoth };
template <BtPart PART>
__global__ void __launch_bounds__(kBtThreads, 1)
    cross_bwd_tc_kernel(const CrossArgs a, const BtWork q, const BtWork kv, const __grid_constant__ CUtensorMap qm,
                        const __grid_constant__ CUtensorMap gm, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ BtShared sh;
  const int first = PART == kBtBoth ? kv.ctas : 0, cta = blockIdx.x;  // dq's first
  if (PART == kBtDkv || (PART == kBtBoth && cta < first))
    cross_bwd_tc<true>(a, kv, qm, gm, km, vm, smem_raw, sh, cta, PART == kBtDkv ? gridDim.x : kv.ctas);
  else
    cross_bwd_tc<false>(a, q, qm, gm, km, vm, smem_raw, sh, cta - first, PART == kBtDq ? gridDim.x : q.ctas);
}

// What the kernels need of each row, tile by tile: -lse log2(e) and -delta, eight
// lanes a row, a CTA a tile; rows that count for nothing get -inf, which makes their
// probabilities 0.  A thread asks for its four rows at once (memory bounds this: with a
// row a thread, gradients of 4 x 8 heads, 4096 x 77 took 57.9 us, so 56.8).
__global__ void __launch_bounds__(256) cross_stat_tc_kernel(const CrossArgs a, const RowTiles rt, float* stat) {
  pdl_launch_dependents();
  pdl_wait();
  const int d8 = (threadIdx.x & 7) * 8;
  const int bh = (int)(blockIdx.x / rt.tiles), tile = (int)(blockIdx.x - (int64_t)bh * rt.tiles), b = bh / a.Hkv;
  const int nq = a.keys(b) > 0 ? a.queries(b) : 0;
  uint4 o[4], g[4];
  float lse[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const RowOf ro = row_of(a, rt, tile, 32 * i + (threadIdx.x >> 3));
    o[i] = g[i] = make_uint4(0, 0, 0, 0);
    lse[i] = INFINITY;
    if (ro.mine && ro.t < nq) {
      const int64_t row = a.row(b, bh - b * a.Hkv, ro.t * a.G + ro.g);
      o[i] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.out) + row * kD + d8);
      g[i] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.dO) + row * kD + d8);
      lse[i] = a.lse[row] * kLog2e;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t ow[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpack_bf16(ow[e]), y = unpack_bf16(gw[e]);
      sum = fmaf(x.x, y.x, sum);
      sum = fmaf(x.y, y.y, sum);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (d8 == 0) {
      float* const at = stat + (int64_t)blockIdx.x * 256 + 32 * i + (threadIdx.x >> 3);
      at[0] = -lse[i];
      at[128] = -sum;
    }
  }
}

// Units that span CTAs: the sums of their parts, in order.  CTA (c, y) has 32 rows of
// the unit that CTA c of the dq kernel (c < q_ctas) or of the dk, dv kernel began, eight
// lanes a row.
__global__ void __launch_bounds__(256) cross_sum_places_kernel(const CrossArgs a, const BtWork q, const BtWork kv) {
  pdl_launch_dependents();
  pdl_wait();
  const bool dkv = (int)blockIdx.x >= q.ctas;
  const int c = dkv ? blockIdx.x - q.ctas : blockIdx.x, lane = threadIdx.x & 31, d8 = (lane & 7) * 8;
  const int4 s = dkv ? kv.split[c] : q.split[c];
  if (s.w <= 1) return;
  // many parts: four at a time, 8 rows of the CTA's 32 at once; few: a row's one after
  // another, all rows at once
  const bool many = s.w >= 8;
  const int ways = many ? 4 : 1, first = many ? lane >> 3 : 0;
#pragma unroll 2
  for (int i = 0; i < (many ? 4 : 1) * (dkv ? 2 : 1); ++i) {
    const int dv = dkv ? i & 1 : 0, k = dkv ? i >> 1 : i;
    const int r = blockIdx.y * 32 + (many ? 8 * k + (threadIdx.x >> 5) : threadIdx.x >> 3);
    int64_t row = -1;
    if (dkv) {
      const int key = s.z * 128 + r;
      if (key < a.Tk) row = ((int64_t)s.x * a.Hkv + s.y) * a.Tk + key;
    } else {
      const RowOf ro = row_of(a, q.rt, s.z, r);
      if (ro.mine) row = a.row(s.x, s.y, ro.t * a.G + ro.g);
    }
    const float* const from = (dkv ? kv.places : q.places) + (dv ? (int64_t)kv.ctas * 2 * 128 * kD : 0) + r * kD + d8;
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, z[8];
    if (row >= 0)
#pragma unroll 2
      for (int x = first; x < s.w; x += ways) {
        load8(from + (int64_t)(x == 0 ? 2 * c + 1 : 2 * (c + x)) * 128 * kD, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += z[e];
      }
    if (many)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] += __shfl_xor_sync(0xffffffffu, y[e], 8);
        y[e] += __shfl_xor_sync(0xffffffffu, y[e], 16);
      }
    if (row >= 0 && first == 0) store8(static_cast<bf16*>(dkv ? (dv ? a.dv : a.dk) : a.dq) + row * kD + d8, y);
  }
}

struct BtPlan {
  RowTiles rt;
  bool one;  // whether dq, and dk and dv, are one launch
  int key_tiles, q_ctas, kv_ctas;
  size_t stat, q_places, kv_places, bytes;
};

// Steps that whole units may take longer (8 x 8 / 2 heads, 512 x 512: 34.7 us in parts, so 30.9).
constexpr int kBtExtra = 4;
static BtPlan bt_plan(int B, int Hkv, int G, int Tq, int Tk, bool alike) {
  BtPlan p;
  p.rt = row_tiles(G, Tq);
  p.key_tiles = (Tk + 127) / 128;
  const int64_t u = (int64_t)B * Hkv, qu = u * p.rt.tiles, ku = u * p.key_tiles;
  // Both in one launch, the SMs shared out by weights (and 15 : 14, a step of dk and dv
  // against one of dq): a start and an uneven end less (4 x 8 / 2 heads, 64 x 64: 22.8 us in
  // two, so 14.3; 4 x 8 / 8, 4096 x 77: 56.7 and 50.2).  From 128 steps an SM on what the
  // weights do not know costs more than that (32 x 8 / 2 heads, 1024 x 2048: 425 us in two
  // launches, 436 in one; 200 x 8 / 2, 33 x 1500: 267 and 290).
  const int64_t qw = qu * (p.key_tiles + kUnitCost), kw = ku * (p.rt.tiles + kUnitCost);
  p.one = qw + kw <= 128 * kSMs;
  Shares q = deal(qu, p.key_tiles + kUnitCost, kSMs, kBtLeast, alike, kBtExtra), kv = deal(ku, p.rt.tiles + kUnitCost, kSMs, kBtLeast, alike, kBtExtra);
  if (p.one && q.ctas + kv.ctas > kSMs) {
    const int n = (int)((kSMs * 15 * kw + (15 * kw + 14 * qw) / 2) / (15 * kw + 14 * qw));
    kv = deal(ku, p.rt.tiles + kUnitCost, n < 1 ? 1 : n < kSMs ? n : kSMs - 1, kBtLeast, alike, kBtExtra);
    q = deal(qu, p.key_tiles + kUnitCost, kSMs - kv.ctas, kBtLeast, alike, kBtExtra);
  }
  p.q_ctas = q.ctas;
  p.kv_ctas = kv.ctas;
  p.stat = align256((size_t)qu * kBtStat);
  p.q_places = (size_t)p.q_ctas * 2 * 128 * kD * sizeof(float);
  p.kv_places = (size_t)p.kv_ctas * 4 * 128 * kD * sizeof(float);
  p.bytes = p.stat + p.q_places + p.kv_places + align256((size_t)(p.q_ctas + p.kv_ctas) * sizeof(int4));
  return p;
}

size_t cross_bwd_tc_bytes(int B, int Hkv, int G, int Tq, int Tk) {
  return std::max(bt_plan(B, Hkv, G, Tq, Tk, false).bytes, bt_plan(B, Hkv, G, Tq, Tk, true).bytes);
}

int launch_cross_bwd_tc(const CrossArgs& a, void* ws, void* stream) {
  static_assert(kBtSmem + sizeof(BtShared) + 1024 <= 228 * 1024, "shared memory of an SM");
  const BtPlan p = bt_plan(a.B, a.Hkv, a.G, a.Tq, a.Tk, !a.q_len && !a.kv_len);
  char* const at = static_cast<char*>(ws);
  float* const stat = static_cast<float*>(ws);
  BtWork q = {p.rt, p.key_tiles, stat, reinterpret_cast<float*>(at + p.stat), p.q_ctas, reinterpret_cast<int4*>(at + p.stat + p.q_places + p.kv_places)};
  BtWork kv = {p.rt, p.key_tiles, stat, reinterpret_cast<float*>(at + p.stat + p.q_places), p.kv_ctas, q.split + p.q_ctas};
  CUtensorMap qm, gm, km, vm;
  const Strides dense = {(int64_t)a.Hq * a.Tq * kD, (int64_t)a.Tq * kD, kD};
  int rc = make_view_map(&qm, a.q, a.Tq, a.Hq, a.B, a.qs, 1 << p.rt.lgR, 128 >> p.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&gm, a.dO, a.Tq, a.Hq, a.B, dense, 1 << p.rt.lgR, 128 >> p.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&km, a.k, a.Tk, a.Hkv, a.B, a.ks, 128, 1);
  if (rc == SFA_OK) rc = make_view_map(&vm, a.v, a.Tk, a.Hkv, a.B, a.vs, 128, 1);
  if (rc != SFA_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  {
    LaunchTimer tm(SFA_KERNEL_CROSS_STAT, stream);
    e = launch_pdl(cross_stat_tc_kernel, dim3((unsigned)((int64_t)a.B * a.Hkv * p.rt.tiles)), dim3(256), 0, st, a, p.rt, stat);
  }
  auto launch = [&](int kind, auto* f, int ctas) {
    LaunchTimer tm(kind, stream);
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kBtSmem);
    return e != cudaSuccess ? e : launch_pdl(f, dim3((unsigned)ctas), dim3(kBtThreads), kBtSmem, st, a, q, kv, qm, gm, km, vm);
  };
  if (p.one) {
    if (e == cudaSuccess) e = launch(SFA_KERNEL_CROSS_BWD_KV, cross_bwd_tc_kernel<kBtBoth>, p.q_ctas + p.kv_ctas);
  } else {
    if (e == cudaSuccess) e = launch(SFA_KERNEL_CROSS_BWD_Q, cross_bwd_tc_kernel<kBtDq>, p.q_ctas);
    if (e == cudaSuccess) e = launch(SFA_KERNEL_CROSS_BWD_KV, cross_bwd_tc_kernel<kBtDkv>, p.kv_ctas);
  }
  if (e == cudaSuccess) {
    LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
    e = launch_pdl(cross_sum_places_kernel, dim3((unsigned)(p.q_ctas + p.kv_ctas), 4), dim3(256), 0, st, a, q, kv);
  }
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
