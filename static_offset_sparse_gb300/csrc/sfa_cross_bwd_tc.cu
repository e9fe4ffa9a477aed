// Backward pass of attention to states of another length on the
// fifth-generation tensor cores (bf16): one kernel for dq, one for dk and dv,
// which are the same walk with the roles of queries and keys exchanged.
//
//   dq     a tile of 128 rows stays, their keys and values pass by:
//            S = Q K^T, dP = dO V^T, dS = P (dP - delta), dQ += dS K
//   dk,dv  a tile of 128 keys stays, the rows that attend it (all heads of the
//          group) pass by:
//            S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//
// Each sum has one owner, so nothing is added atomically and equal inputs give
// equal bits; the price is S and dP twice (7 products instead of 5).  In both
// the probabilities come out of tensor memory the way they go back in as a left
// operand: a lane per row of the tile that stays, so P and dS never pass shared
// memory.  Per step one thread issues the next S and dP as soon as eight warps
// hold this step's in registers (64 columns of both a thread), and the
// accumulations when P and dS are back.  P and dS are rounded to bf16 for
// their products; everything else is fp32.
#include "sfa_cross.cuh"

namespace sfa {

constexpr int kBtThreads = 384;  // 8 warps of softmax, a copying, an issuing and a preparing warp
constexpr int kBtTile = 128 * 128;  // bytes of 128 rows of 64 bf16
constexpr int kBtStages = 4;
constexpr int kBtSmem = 2 * 2 * kBtTile + kBtStages * 2 * kBtTile + 1024;
// tensor memory: S, dP, P, dS, sums of dq or dk, of dv
constexpr int kBtDp = 128, kBtP = 256, kBtDs = 320, kBtSum = 384, kBtSum2 = 448;

struct BtShared {
  uint64_t full[kBtStages], empty[kBtStages], ready[kBtStages];  // ready: rows that count for nothing are zeros, their numbers are there
  uint64_t a_full[2], a_empty[2], s_full, s_free, p_full, done;
  float nlse[kBtStages][128], ndelta[kBtStages][128];  // of the rows that pass by: -lse log2(e), -delta
  uint32_t tmem;
};

struct BtWork {
  RowTiles rt;
  int key_tiles, items;
};

// An item: a tile that stays, and tiles t0 .. t1 - 1 that pass by.
struct BtItem {
  int b, kvh, s, tile, t0, t1, nq, nk;
};

template <bool DKV>
__device__ __forceinline__ BtItem bt_item(const CrossArgs& a, const BtWork& w, int x) {
  BtItem it;
  it.s = x % a.splits;
  x /= a.splits;
  const int own = DKV ? w.key_tiles : w.rt.tiles;
  it.tile = x % own;
  x /= own;
  it.kvh = x % a.Hkv;
  it.b = x / a.Hkv;
  it.nq = a.queries(it.b);
  it.nk = a.keys(it.b);
  const int rows = it.nk > 0 ? w.rt.groups * ((it.nq + (1 << w.rt.lgR) - 1) >> w.rt.lgR) : 0;
  const int keys = it.nq > 0 ? (it.nk + 127) >> 7 : 0;
  const bool some = DKV ? it.tile < keys : it.tile < rows;
  const int n = !some ? 0 : DKV ? rows : keys;
  it.t0 = (int)((int64_t)n * it.s / a.splits);
  it.t1 = (int)((int64_t)n * (it.s + 1) / a.splits);
  return it;
}

template <bool DKV>
__global__ void __launch_bounds__(kBtThreads, 1)
    cross_bwd_tc_kernel(const CrossArgs a, const BtWork w, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap gm,
                        const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ BtShared sh;
  const uint32_t smem = smem_u32(smem_raw) + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem + 2 * 2 * kBtTile;
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
      mbar_init(smem_u32(&sh.a_empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.s_free), 8);
    mbar_init(smem_u32(&sh.p_full), 8);
    mbar_init(smem_u32(&sh.done), 1);
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tm = sh.tmem;
  pdl_wait();
  bool dead = false;  // a wait ran out: no more waits, no more work
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_u32(bar), phase & 1, a.wait_cycles));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(bar));
  };

  if (warp == 8) {
    // ---- copies
    int n = 0, na = 0;  // steps, items so far
    auto rows = [&](uint32_t dst, const CUtensorMap* m, const BtItem& it, int tile, uint32_t bar) {
      const int tb = tile / w.rt.groups, hb = tile - tb * w.rt.groups;
      tma_load_4d(dst, m, 0, tb << w.rt.lgR, it.kvh * a.G + (hb << (7 - w.rt.lgR)), it.b, bar);
    };
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const BtItem it = bt_item<DKV>(a, w, x);
      if (it.t1 <= it.t0) continue;
      const int buf = na & 1;
      if (na >= 2) wait(&sh.a_empty[buf], na / 2 - 1);
      if (dead) break;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&sh.a_full[buf]), dst = smem + buf * 2 * kBtTile;
        mbar_expect_tx(bar, 2 * kBtTile);
        if (DKV) {
          tma_load_4d(dst, &km, 0, it.tile * 128, it.kvh, it.b, bar);
          tma_load_4d(dst + kBtTile, &vm, 0, it.tile * 128, it.kvh, it.b, bar);
        } else {
          rows(dst, &qm, it, it.tile, bar);
          rows(dst + kBtTile, &gm, it, it.tile, bar);
        }
      }
      __syncwarp();
      ++na;
      for (int t = it.t0; t < it.t1 && !dead; ++t, ++n) {
        const int st = n % kBtStages;
        if (n >= kBtStages) wait(&sh.empty[st], n / kBtStages - 1);
        if (dead) break;
        if (elect_one()) {
          const uint32_t bar = smem_u32(&sh.full[st]), dst = ring + st * 2 * kBtTile;
          mbar_expect_tx(bar, 2 * kBtTile);
          if (DKV) {
            rows(dst, &qm, it, t, bar);
            rows(dst + kBtTile, &gm, it, t, bar);
          } else {
            tma_load_4d(dst, &km, 0, t * 128, it.kvh, it.b, bar);
            tma_load_4d(dst + kBtTile, &vm, 0, t * 128, it.kvh, it.b, bar);
          }
        }
        __syncwarp();
      }
    }
    if (dead) {  // copies under way end before their memory goes
      if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
      for (int i = max(0, n - kBtStages); i < n; ++i) mbar_wait_bounded(smem_u32(&sh.full[i % kBtStages]), (i / kBtStages) & 1, a.wait_cycles);
      for (int i = max(0, na - 2); i < na; ++i) mbar_wait_bounded(smem_u32(&sh.a_full[i & 1]), (i / 2) & 1, a.wait_cycles);
    }
  } else if (warp == 9) {
    // ---- products
    constexpr uint32_t idS = idesc_bf16(128, 128, false, false), idO = idesc_bf16(128, 64, false, true);
    constexpr uint32_t kHi = smem_desc_hi(1024), kTileU = kBtTile / 16;
    const uint32_t a0 = smem_desc_lo(smem, 16), b0 = smem_desc_lo(ring, 16), bt0 = smem_desc_lo(ring, 8192);
    int n = 0, na = 0, np = 0;  // steps, items, accumulations so far
    auto sums = [&](bool begin) {  // of step np
      wait(&sh.p_full, np);
      if (dead) return;
      const int st = np % kBtStages;
      if (elect_one()) {
        tc05_fence_after();
        const uint32_t b = bt0 + 2 * st * kTileU;
#pragma unroll
        for (int i = 0; i < 8; ++i) umma_ts_lo(tm + kBtSum, tm + kBtDs + 8 * i, b + 128 * i, kHi, idO, !begin || i > 0);
        if (DKV)
#pragma unroll
          for (int i = 0; i < 8; ++i) umma_ts_lo(tm + kBtSum2, tm + kBtP + 8 * i, b + kTileU + 128 * i, kHi, idO, !begin || i > 0);
        umma_commit(smem_u32(&sh.done));
        umma_commit(smem_u32(&sh.empty[st]));
      }
      __syncwarp();
      ++np;
    };
    bool had_begin = false;
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const BtItem it = bt_item<DKV>(a, w, x);
      if (it.t1 <= it.t0) continue;
      const int buf = na & 1;
      wait(&sh.a_full[buf], na / 2);
      ++na;
      for (int t = it.t0; t < it.t1 && !dead; ++t) {
        const int st = n % kBtStages;
        wait(&sh.full[st], n / kBtStages);
        wait(&sh.ready[st], n / kBtStages);
        if (n > 0) wait(&sh.s_free, n - 1);
        if (dead) break;
        if (elect_one()) {
          tc05_fence_after();
          const uint32_t aa = a0 + 2 * buf * kTileU, b = b0 + 2 * st * kTileU;
#pragma unroll
          for (int i = 0; i < 4; ++i) umma_ss_lo(tm, aa + 2 * i, b + 2 * i, kHi, idS, i > 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) umma_ss_lo(tm + kBtDp, aa + kTileU + 2 * i, b + kTileU + 2 * i, kHi, idS, i > 0);
          umma_commit(smem_u32(&sh.s_full));
          if (t == it.t1 - 1) umma_commit(smem_u32(&sh.a_empty[buf]));
        }
        __syncwarp();
        if (n > 0) sums(had_begin);
        had_begin = t == it.t0;
        ++n;
      }
    }
    if (n > 0 && !dead) sums(had_begin);
    if (dead) {  // products under way end before their memory goes
      if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
      if (n > 0) mbar_wait_bounded(smem_u32(&sh.s_full), (n - 1) & 1, a.wait_cycles);
      if (np > 0) mbar_wait_bounded(smem_u32(&sh.done), (np - 1) & 1, a.wait_cycles);
    }
  } else if (warp == 10) {
    // ---- what the products need besides the copies: rows that count for nothing
    // are made zeros (they may hold anything, and 0 * NaN would reach every sum),
    // and the passing rows' numbers are brought
    int n = 0;
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const BtItem it = bt_item<DKV>(a, w, x);
      for (int t = it.t0; t < it.t1 && !dead; ++t, ++n) {
        const int st = n % kBtStages;
        if (n >= kBtStages) wait(&sh.empty[st], n / kBtStages - 1);
        if (dead) break;
        uint32_t bad = 0;  // of rows lane + 32 i
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          if (DKV) {
            const RowOf ro = row_of(a, w.rt, t, r);
            const bool in = ro.mine && ro.t < it.nq;
            const float2 v = in ? a.stat[a.row(it.b, it.kvh, ro.t * a.G + ro.g)] : make_float2(INFINITY, 0.0f);
            sh.nlse[st][r] = -v.x;
            sh.ndelta[st][r] = -v.y;
            bad |= (in ? 0u : 1u) << i;
          } else {
            bad |= (t * 128 + r < it.nk ? 0u : 1u) << i;
          }
        }
        if (__any_sync(0xffffffffu, bad != 0)) {
          wait(&sh.full[st], n / kBtStages);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (bad >> i & 1)
#pragma unroll
              for (int c = 0; c < 16; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(ring + st * 2 * kBtTile + (c >> 3) * kBtTile +
                                                                               (lane + 32 * i) * 128 + 16 * (c & 7)),
                             "r"(0)
                             : "memory");
          fence_async_smem();
        }
        arrive(&sh.ready[st]);
      }
    }
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  } else if (warp < 8) {
    // ---- P and dS: a thread a row of the tile that stays, 64 of the 128 that pass by
    const int half = warp >> 2, r = tid & 127;
    const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    int n = 0;
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const BtItem it = bt_item<DKV>(a, w, x);
      const RowOf ro = DKV ? RowOf{} : row_of(a, w.rt, it.tile, r);
      float2 own = make_float2(-INFINITY, 0.0f);
      if (!DKV && ro.mine) {
        const float2 v = a.stat[a.row(it.b, it.kvh, ro.t * a.G + ro.g)];
        own = make_float2(-v.x, -v.y);
      }
      for (int t = it.t0; t < it.t1 && !dead; ++t, ++n) {
        const int st = n % kBtStages;
        if (DKV) wait(&sh.ready[st], n / kBtStages);
        wait(&sh.s_full, n);
        if (dead) break;
        tc05_fence_after();
        float s[64], d[64];
        tmem_ld32(tl + 64 * half, s);
        tmem_ld32(tl + 64 * half + 32, s + 32);
        tmem_ld32(tl + kBtDp + 64 * half, d);
        tmem_ld32(tl + kBtDp + 64 * half + 32, d + 32);
        tmem_wait_ld32(s);
        tmem_wait_ld32(s + 32);
        tmem_wait_ld32(d);
        tmem_wait_ld32(d + 32);
        tc05_fence_before();
        arrive(&sh.s_free);
        const float2 c2 = make_float2(kLogitScale, kLogitScale);
        const int left = DKV ? 128 : it.nk - 128 * t - 64 * half;  // keys of this half that are there
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          float4 nl, nd;
          if (DKV) {
            nl = *reinterpret_cast<const float4*>(&sh.nlse[st][64 * half + e]);
            nd = *reinterpret_cast<const float4*>(&sh.ndelta[st][64 * half + e]);
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
        if (left < 64) {
#pragma unroll
          for (int e = 0; e < 64; ++e)  // (two a register)
            if (e >= left) d[e >> 1] = __uint_as_float(__float_as_uint(d[e >> 1]) & (e & 1 ? 0x0000ffffu : 0u));
        }
        if (n > 0) wait(&sh.done, n - 1);  // the last step's P and dS have been read
        if (dead) break;
        tc05_fence_after();
        if (DKV) {
          tmem_st16(tl + kBtP + 32 * half, s);
          tmem_st16(tl + kBtP + 32 * half + 16, s + 16);
        }
        tmem_st16(tl + kBtDs + 32 * half, d);
        tmem_st16(tl + kBtDs + 32 * half + 16, d + 16);
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full);
      }
      const bool any = it.t1 > it.t0;
      if (any && !dead) {
        wait(&sh.done, n - 1);
        tc05_fence_after();
      }
      if (DKV) {  // the first four warps have dk, the others dv
        const int j = it.tile * 128 + r;
        const int64_t row = ((int64_t)it.b * a.Hkv + it.kvh) * a.Tk + j;
        const float f = half ? 1.0f : 0.125f;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          float o[16];
          if (any && !dead) {
            tmem_ld16(tl + (half ? kBtSum2 : kBtSum) + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = any && j < it.nk ? o[e] * f : 0.0f;
          if (j >= a.Tk) continue;
          if (a.parts) {
            float* const out = (half ? a.part_b : a.part_a) + ((int64_t)it.s * a.B * a.Hkv * a.Tk + row) * kD + c;
            store8(out, o);
            store8(out + 8, o + 8);
          } else {
            bf16* const out = static_cast<bf16*>(half ? a.dv : a.dk) + row * kD + c;
            store8(out, o);
            store8(out + 8, o + 8);
          }
        }
      } else {  // half the dims each
        const int64_t row = ro.mine ? a.row(it.b, it.kvh, ro.t * a.G + ro.g) : 0;
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
          float o[16];
          if (any && !dead) {
            tmem_ld16(tl + kBtSum + 32 * half + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = any && ro.t < it.nq ? o[e] * 0.125f : 0.0f;
          if (!ro.mine) continue;
          if (a.parts) {
            float* const out = a.part_a + (it.s * a.rows + row) * kD + 32 * half + c;
            store8(out, o);
            store8(out + 8, o + 8);
          } else {
            bf16* const out = static_cast<bf16*>(a.dq) + row * kD + 32 * half + c;
            store8(out, o);
            store8(out + 8, o + 8);
          }
        }
      }
      tc05_fence_before();
    }
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 9) tmem_dealloc(tm, 512);
}

int launch_cross_bwd_tc(const CrossArgs& a, bool dkv, void* stream) {
  static_assert(kBtSmem + sizeof(BtShared) + 1024 <= 228 * 1024, "shared memory of an SM");
  BtWork w;
  w.rt = row_tiles(a.G, a.Tq);
  w.key_tiles = (a.Tk + 127) / 128;
  w.items = (int)((int64_t)a.B * a.Hkv * (dkv ? w.key_tiles : w.rt.tiles) * a.splits);
  CUtensorMap qm, gm, km, vm;
  const Strides dense = {(int64_t)a.Hq * a.Tq * kD, (int64_t)a.Tq * kD, kD};
  int rc = make_view_map(&qm, a.q, a.Tq, a.Hq, a.B, a.qs, 1 << w.rt.lgR, 128 >> w.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&gm, a.dO, a.Tq, a.Hq, a.B, dense, 1 << w.rt.lgR, 128 >> w.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&km, a.k, a.Tk, a.Hkv, a.B, a.ks, 128, 1);
  if (rc == SFA_OK) rc = make_view_map(&vm, a.v, a.Tk, a.Hkv, a.B, a.vs, 128, 1);
  if (rc != SFA_OK) return rc;
  LaunchTimer tm(dkv ? SFA_KERNEL_CROSS_BWD_KV : SFA_KERNEL_CROSS_BWD_Q, stream);
  auto* f = dkv ? cross_bwd_tc_kernel<true> : cross_bwd_tc_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kBtSmem);
  if (e == cudaSuccess)
    e = launch_pdl(f, dim3((unsigned)(w.items < kSMs ? w.items : kSMs)), dim3(kBtThreads), kBtSmem, (cudaStream_t)stream, a, w, qm, gm, km, vm);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
