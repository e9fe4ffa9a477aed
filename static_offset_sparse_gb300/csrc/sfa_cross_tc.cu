// Forward pass of attention to states of another length on the fifth-generation
// tensor cores (bf16).
//
// A CTA an SM works through items: two tiles of 128 rows of one (sequence, KV
// head) and a split of its keys, 128 keys a step.  Both tiles use the same keys
// and values.  Per step and tile
//   one thread issues S = Q K^T (128 x 128 sums in tensor memory);
//   four warps, a thread a row, take the row's 128 logits into registers at
//     once, which frees S for the next step's product while they work;
//     the maximum, 2^x, the sum, and P in bf16 back into tensor memory;
//   the issuing thread takes P as the left operand of O += P V, O in tensor
//     memory.
// The sum of a row is moved to a new maximum only where that grew by more than
// 2^8 (P and O are then at most 2^8 times too large, which fp32 and bf16 hold as
// well as 1).  The sums are taken in fp32 from probabilities before their
// rounding to bf16.  An item's first products start under the last item's
// outputs: each role walks the items by itself, the only coupling is through
// mbarriers.
#include "sfa_cross.cuh"
#include "sfa_umma.cuh"

namespace sfa {

constexpr int kTcThreads = 320;  // 2 x 4 warps of softmax, a copying warp, an issuing warp
constexpr int kTcTile = 128 * 128;  // bytes of 128 rows of 64 bf16
constexpr int kTcCols = 512, kTcTileCols = 256, kTcP = 128, kTcO = 192;  // tensor memory columns of a tile: S, P, O
constexpr float kGrow = 8.0f;  // log2 of how far P and O may be too large
// Beyond this, x - m is taken before its multiplication: a fused 2^(x c - m c)
// would keep what rounding m c dropped, a factor of 2^(2^-4) and more.
constexpr float kFar = 1048576.0f;

template <int PARTS>
struct TcShape {
  static constexpr int kSlots = 8;                  // key and value tiles in flight
  static constexpr int kQBufs = PARTS == 1 ? 2 : 1;  // items whose queries are there
  static constexpr int kQBytes = 2 * PARTS * kTcTile;
  static constexpr int kSmem = kQBufs * kQBytes + kSlots * kTcTile + 1024;
};

struct TcShared {
  uint64_t full[8], empty[8], q_full[2], q_empty[2];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];  // by tile
  uint32_t tmem;
};

// An item: what every role needs of it.
struct TcItem {
  int b, kvh, s, tile, k0, k1, nq;
  bool two;  // whether its second tile has queries
  __device__ __forceinline__ int steps() const { return (k1 - k0 + 127) >> 7; }
};

struct TcWork {
  RowTiles rt;
  int pairs, items;
};

__device__ __forceinline__ TcItem tc_item(const CrossArgs& a, const TcWork& w, int x) {
  TcItem it;
  it.s = x % a.splits;
  x /= a.splits;
  it.tile = 2 * (x % w.pairs);
  x /= w.pairs;
  it.kvh = x % a.Hkv;
  it.b = x / a.Hkv;
  it.nq = a.queries(it.b);
  const int nk = a.keys(it.b);
  split_keys(nk, 128, a.splits, it.s, it.k0, it.k1);
  if ((it.tile / w.rt.groups) << w.rt.lgR >= it.nq) it.k1 = it.k0;
  it.two = it.tile + 1 < w.rt.tiles && ((it.tile + 1) / w.rt.groups) << w.rt.lgR < it.nq;
  return it;
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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < Shape::kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 1);
      mbar_init(smem_u32(&sh.q_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_free[i]), 4);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
    }
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.tmem), kTcCols);
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
    int n = 0, nq = 0;  // key and value tiles, items so far
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const TcItem it = tc_item(a, w, x);
      if (it.k1 <= it.k0) continue;
      const int buf = nq % Shape::kQBufs;
      if (nq >= Shape::kQBufs) wait(&sh.q_empty[buf], nq / Shape::kQBufs - 1);
      if (dead) break;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&sh.q_full[buf]);
        mbar_expect_tx(bar, (it.two ? 2 : 1) * PARTS * kTcTile);
        for (int T = 0; T < (it.two ? 2 : 1); ++T) {
          const int tb = (it.tile + T) / w.rt.groups, hb = it.tile + T - tb * w.rt.groups;
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
            tma_load_4d(smem + buf * Shape::kQBytes + (T * PARTS + p) * kTcTile, &qm, 0, tb << w.rt.lgR,
                        it.kvh * a.G + (hb << (7 - w.rt.lgR)), it.b + p, bar);
        }
      }
      __syncwarp();
      ++nq;
      for (int j = it.k0; j < it.k1 && !dead; j += 128)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int slot = n % Shape::kSlots;
          if (n >= Shape::kSlots) wait(&sh.empty[slot], n / Shape::kSlots - 1);
          if (dead) break;
          if (elect_one()) {
            const uint32_t bar = smem_u32(&sh.full[slot]);
            mbar_expect_tx(bar, kTcTile);
            tma_load_4d(ring + slot * kTcTile, kv ? &vm : &km, 0, j, it.kvh, it.b, bar);
          }
          __syncwarp();
          ++n;
        }
    }
    if (dead) {  // copies under way end before their memory goes
      if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
      for (int i = max(0, n - Shape::kSlots); i < n; ++i)
        mbar_wait_bounded(smem_u32(&sh.full[i % Shape::kSlots]), (i / Shape::kSlots) & 1, a.wait_cycles);
      for (int i = max(0, nq - Shape::kQBufs); i < nq; ++i)
        mbar_wait_bounded(smem_u32(&sh.q_full[i % Shape::kQBufs]), (i / Shape::kQBufs) & 1, a.wait_cycles);
    }
  } else if (warp == 9) {
    // ---- products: a step's logits are issued before the last step's outputs
    constexpr uint32_t idS = idesc_bf16(128, 128, false, false), idO = idesc_bf16(128, 64, false, true);
    constexpr uint32_t kHi = smem_desc_hi(1024), kTileU = kTcTile / 16;
    const uint32_t q0 = smem_desc_lo(smem, 16), k0 = smem_desc_lo(ring, 16), v0 = smem_desc_lo(ring, 8192);
    int n = 0, nq = 0, ns[2] = {0, 0}, np[2] = {0, 0};  // steps, items, products of each tile so far
    auto outputs = [&](int step, bool two, bool begin) {  // O (+)= P V of a step
      const int slot = (2 * step + 1) % Shape::kSlots;
      wait(&sh.full[slot], (2 * step + 1) / Shape::kSlots);
      for (int T = 0; T < (two ? 2 : 1); ++T) {
        wait(&sh.p_full[T], np[T]++);
        if (dead) return;
        if (elect_one()) {
          tc05_fence_after();
          const uint32_t d = tm + kTcTileCols * T, v = v0 + slot * kTileU;
#pragma unroll
          for (int i = 0; i < 8; ++i)  // 16 keys: two groups of 8 rows, 8 columns of P
            umma_ts_lo(d + kTcO, d + kTcP + 8 * i, v + 128 * i, kHi, idO, !begin || i > 0);
          umma_commit(smem_u32(&sh.pv_done[T]));
          if (T == (int)two) umma_commit(smem_u32(&sh.empty[slot]));
        }
        __syncwarp();
      }
    };
    bool had = false, had_two = false, had_begin = false;
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const TcItem it = tc_item(a, w, x);
      if (it.k1 <= it.k0) continue;
      const int buf = nq % Shape::kQBufs, steps = it.steps();
      wait(&sh.q_full[buf], nq / Shape::kQBufs);
      ++nq;
      for (int j = 0; j < steps && !dead; ++j, ++n) {
        const int slot = (2 * n) % Shape::kSlots;
        wait(&sh.full[slot], 2 * n / Shape::kSlots);
        for (int T = 0; T < (it.two ? 2 : 1); ++T) {
          if (ns[T] > 0) wait(&sh.s_free[T], ns[T] - 1);
          ++ns[T];
          if (dead) break;
          if (elect_one()) {
            tc05_fence_after();
            const uint32_t q = q0 + (buf * 2 + T) * PARTS * kTileU, k = k0 + slot * kTileU;
#pragma unroll
            for (int i = 0; i < 4 * PARTS; ++i)
              umma_ss_lo(tm + kTcTileCols * T, q + (i >> 2) * kTileU + 2 * (i & 3), k + 2 * (i & 3), kHi, idS, i > 0);
            umma_commit(smem_u32(&sh.s_full[T]));
            if (T == (int)it.two) {
              umma_commit(smem_u32(&sh.empty[slot]));
              if (j == steps - 1) umma_commit(smem_u32(&sh.q_empty[buf]));
            }
          }
          __syncwarp();
        }
        if (had && !dead) outputs(n - 1, had_two, had_begin);
        had = true;
        had_two = it.two;
        had_begin = j == 0;
      }
    }
    if (had && !dead) outputs(n - 1, had_two, had_begin);
    if (dead) {  // products under way end before their memory goes
      if (lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
      for (int T = 0; T < 2; ++T) {
        if (ns[T] > 0) mbar_wait_bounded(smem_u32(&sh.s_full[T]), (ns[T] - 1) & 1, a.wait_cycles);
        if (np[T] > 0) mbar_wait_bounded(smem_u32(&sh.pv_done[T]), (np[T] - 1) & 1, a.wait_cycles);
      }
    }
  } else {
    // ---- softmax: a thread a row of tile T
    const int T = warp >> 2, r = tid & 127;
    const uint32_t tl = tm + kTcTileCols * T + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    int n = 0, np = 0;  // steps of the CTA, of this tile
    for (int x = blockIdx.x; x < w.items && !dead; x += gridDim.x) {
      const TcItem it = tc_item(a, w, x);
      const int tile = it.tile + T, tb = tile / w.rt.groups, hb = tile - tb * w.rt.groups;
      const int t = (tb << w.rt.lgR) + (r & ((1 << w.rt.lgR) - 1)), g = (hb << (7 - w.rt.lgR)) + (r >> w.rt.lgR);
      const bool mine = tile < w.rt.tiles && t < a.Tq && g < a.G;
      const int steps = T == 0 || it.two ? it.steps() : 0;
      float m = -INFINITY, mc = 0.0f, l = 0.0f;  // what the shift of 2^x was set by, the shift
      for (int j = 0; j < steps && !dead; ++j, ++np) {
        wait(&sh.s_full[T], np);
        if (dead) break;
        tc05_fence_after();
        float v[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(tl + c, v + c);
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_wait_ld32(v + c);
        tc05_fence_before();
        arrive(&sh.s_free[T]);
        const int left = it.k1 - it.k0 - 128 * j;
        if (left < 128) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= left) v[e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 128; e += 2) top = fmaxf(top, fmaxf(v[e], v[e + 1]));
        const bool grown = j == 0 || top > m + kGrow / kLogitScale;
        if (__any_sync(0xffffffffu, grown)) {
          float corr = 1.0f;
          if (grown) {
            const float to = fmaxf(m, top);
            corr = ex2((m - shift_of(to)) * kLogitScale);  // 0 on the first keys
            m = to;
            mc = shift_of(m) * kLogitScale;
            l *= corr;
          }
          if (j > 0) {
            wait(&sh.pv_done[T], np - 1);
            tc05_fence_after();
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float o[16];
              tmem_ld16(tl + kTcO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= corr;
              tmem_st16(tl + kTcO + c, o);
            }
          }
        }
        float off = -mc;
        if (__any_sync(0xffffffffu, !(fabsf(mc) <= kFar))) {
          off = 0.0f;
#pragma unroll
          for (int e = 0; e < 128; ++e) v[e] -= shift_of(m);
        }
        const float2 c2 = make_float2(kLogitScale, kLogitScale), off2 = make_float2(off, off);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int e = 0; e < 128; e += 2) {
          const float2 y = pair_fma(make_float2(v[e], v[e + 1]), c2, off2);
          v[e] = ex2(y.x);
          v[e + 1] = ex2(y.y);
          sum[(e >> 1) & 1] = pair_add(sum[(e >> 1) & 1], make_float2(v[e], v[e + 1]));
          v[e >> 1] = __uint_as_float(pack_bf16(v[e], v[e + 1]));
        }
        const float2 both = pair_add(sum[0], sum[1]);
        l += both.x + both.y;
        if (j > 0) wait(&sh.pv_done[T], np - 1);  // the last step's P has been read
        if (dead) break;
        tc05_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 16) tmem_st16(tl + kTcP + c, v + c);
        if (left < 128 && T == 0 && left <= r) {
          // values behind the last key may be anything, and 0 * NaN would reach every row
          const int at = 2 * (n + j) + 1, slot = at % Shape::kSlots;
          if (!mbar_wait_bounded(smem_u32(&sh.full[slot]), (at / Shape::kSlots) & 1, a.wait_cycles)) record_status(a.status, SFA_ERR_TIMEOUT);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(ring + slot * kTcTile + r * 128 + 16 * c), "r"(0) : "memory");
          fence_async_smem();
        }
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full[T]);
      }
      n += it.steps();
      if (steps > 0 && !dead) {
        wait(&sh.pv_done[T], np - 1);
        tc05_fence_after();
      }
      const bool none = steps == 0 || t >= it.nq;
      const int64_t row = mine ? a.row(it.b, it.kvh, t * a.G + g) : 0;
      const int64_t at = it.s * a.rows + row;
      const float inv = 1.0f / l;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        float o[16];
        if (steps > 0 && !dead) {
          tmem_ld16(tl + kTcO + c, o);
          tmem_wait_ld();
        }
        if (!mine) {
        } else if (a.parts) {
          if (!none) {
            store8(a.part_o + at * kD + c, o);
            store8(a.part_o + at * kD + c + 8, o + 8);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * inv;
          bf16* const out = static_cast<bf16*>(a.o) + row * kD + c;
          store8(out, o);
          store8(out + 8, o + 8);
        }
      }
      tc05_fence_before();
      if (mine) {
        if (a.parts)
          a.part_ml[at] = none ? make_float2(-INFINITY, -1.0f) : make_float2(mc, l);
        else if (a.lse)
          a.lse[row] = none ? -INFINITY : (mc + log2f(l)) * kLn2;
      }
    }
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 9) tmem_dealloc(tm, kTcCols);
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

template <int PARTS>
static cudaError_t fwd_tc(const CrossArgs& a, const TcWork& w, const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                          cudaStream_t st) {
  auto* f = cross_fwd_tc_kernel<PARTS>;
  static_assert(TcShape<PARTS>::kSmem + sizeof(TcShared) + 1024 <= 228 * 1024, "shared memory of an SM");
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<PARTS>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(f, dim3((unsigned)(w.items < kSMs ? w.items : kSMs)), dim3(kTcThreads), TcShape<PARTS>::kSmem, st, a, w, qm, km, vm);
}

int launch_cross_fwd_tc(const CrossArgs& a, bool two, void* stream) {
  TcWork w;
  w.rt = row_tiles(a.G, a.Tq);
  w.pairs = (w.rt.tiles + 1) / 2;
  w.items = (int)((int64_t)a.B * a.Hkv * w.pairs * a.splits);
  CUtensorMap qm, km, vm;
  int rc = make_view_map(&qm, a.q, a.Tq, a.Hq, two ? 2 : a.B, a.qs, 1 << w.rt.lgR, 128 >> w.rt.lgR);
  if (rc == SFA_OK) rc = make_view_map(&km, a.k, a.Tk, a.Hkv, a.B, a.ks, 128, 1);
  if (rc == SFA_OK) rc = make_view_map(&vm, a.v, a.Tk, a.Hkv, a.B, a.vs, 128, 1);
  if (rc != SFA_OK) return rc;
  LaunchTimer tm(SFA_KERNEL_CROSS_FWD, stream);
  const cudaError_t e = two ? fwd_tc<2>(a, w, qm, km, vm, (cudaStream_t)stream) : fwd_tc<1>(a, w, qm, km, vm, (cudaStream_t)stream);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
