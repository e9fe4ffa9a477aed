// Prompts over the paged 4-bit cache: many query rows a request, on the
// fifth-generation tensor cores.
//
// An item is 128 columns (128 / G rows x the G heads of a KV head) of one
// request, a step 128 keys.  Per step
//   four warps turn the raw codes and scales (as the copying warp brings them)
//     into f16 keys and values in shared memory, a thread a key: code * scale
//     is a whole f16 number;
//   one thread issues S = Q K^T, twice (the query's two f16 parts: logits good
//     to fp32's last bits), 128 x 128 sums in tensor memory;
//   four warps, a thread a column of the item (a lane of tensor memory), take
//     the maximum, exponentiate, and put P in f16 back into tensor memory, where
//     the same issuing thread takes it as the left operand of O += P V.
// fp32 outputs add a second product with what rounding P to f16 dropped (it
// takes the place of the logits already read).
// Two CTAs an SM: one's exponentials run under the other's products.  What
// bounds it is the softmax: 128 x 128 exponentials, scalings and packings a
// step against 384 clocks of products.
//
// Work is cut and shared out as for single rows (sfa_kv4_stream.cuh), chunks
// joined by the same kernel.
#include "sfa_kv4_stream.cuh"
#include "sfa_launch.cuh"
#include "sfa_umma.cuh"

namespace sfa {

constexpr int kPSlots = 6, kStep = 128;
constexpr int kPWarps = 10, kPThreads = 32 * kPWarps;  // softmax 0-3, dequantise 4-7, copy 8, products 9
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192, kPCols = 256;
// shared memory: Q hi, Q lo, K, V (128 rows of 128 bytes each, 128-byte
// swizzle), the raw ring, then what is small
constexpr int kPTile = 128 * 128;
constexpr int kPromptSmem = 4 * kPTile + kPSlots * kTileBytes + 1024;

struct PromptShared {
  uint64_t raw_full[kPSlots], raw_empty[kPSlots];
  uint64_t k_full, v_full, s_full, p_full, pv_done, q_full;
  int pages[kPSlots];
  int step_pages[2];    // pages there of a step's two tiles: bits 0-3 and 4-7
  int step_nan[2][4];   // whether a warp's values of the step hold a NaN
  uint8_t nan[2][kStep];  // per key: the scale blocks of its value that are NaN
  int sums[kPWarps], where[4];
  uint32_t tmem;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
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

template <typename TIO>
__global__ void __launch_bounds__(kPThreads, kPromptCtas) kv4_prompt_kernel(const Kv4Args a, const StreamArgs sa) {
  constexpr bool kExact = sizeof(TIO) == 4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PromptShared sh;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const kt = smem + 2 * kPTile;
  uint8_t* const vt = smem + 3 * kPTile;
  uint8_t* const raw = smem + 4 * kPTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(smem_u32(&sh.raw_full[i]), 1);
      mbar_init(smem_u32(&sh.raw_empty[i]), 4);
    }
    mbar_init(smem_u32(&sh.k_full), 4);
    mbar_init(smem_u32(&sh.v_full), 4);
    mbar_init(smem_u32(&sh.s_full), 2);  // the products' end, and the issuing thread: what it has seen of the step, its readers see
    mbar_init(smem_u32(&sh.p_full), 4);
    mbar_init(smem_u32(&sh.pv_done), 1);
    mbar_init(smem_u32(&sh.q_full), 4);
    mbar_fence_init();
  }
  if (warp == kPWarps - 1) {
    tmem_alloc(smem_u32(&sh.tmem), kPCols);
    tmem_relinquish();
  }
  pdl_wait();
  Cursor cur;
  tc05_fence_before();
  const bool work = find_run<kPThreads>(a, sa, sh.sums, sh.where, cur);  // (two barriers of the CTA inside)
  tc05_fence_after();
  const uint32_t tm = sh.tmem;
  const int G = 1 << a.lgG;
  bool dead = false;
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_u32(bar), phase, a.wait_cycles));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
  };
  int j = 0, n = 0, nq = 0;  // steps, raw tiles and query loads before the current one
  int qx = -1, qh = -1;
  if (!work) {
  } else if (warp == 8) {
    copy_run<kPSlots>(a, sa, cur, smem_u32(raw), smem_u32(sh.raw_full), smem_u32(sh.raw_empty), sh.pages,
                      cur.at == 0 ? a.debug_skip : -1, lane);
  } else if (warp == 9) {
    // ---- the products
    constexpr uint32_t idS = idesc_f16(128, kStep, false, false), idO = idesc_f16(128, 64, false, true);
    const uint32_t q0 = smem_u32(smem), k0 = smem_u32(kt), v0 = smem_u32(vt);
    int last = 0;  // steps whose S product was issued
    do {
      if (cur.te > cur.tb && (cur.x != qx || cur.h != qh)) {
        qx = cur.x;
        qh = cur.h;
        wait(&sh.q_full, nq++ & 1);
      }
      for (int t = cur.tb; t < cur.te && !dead; t += 2, ++j) {
        wait(&sh.k_full, j & 1);
        if (dead) break;
        if (lane == 0) {
          tc05_fence_after();
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(tm + kColS, smem_desc_sw128(q0 + part * kPTile + 32 * k, 16, 1024), smem_desc_sw128(k0 + 32 * k, 16, 1024), idS,
                        part + k > 0);
          umma_commit(smem_u32(&sh.s_full));
          mbar_arrive(smem_u32(&sh.s_full));
        }
        last = j + 1;
        wait(&sh.v_full, j & 1);
        wait(&sh.p_full, j & 1);  // (with a chunk's first step: the last chunk's O has been read)
        if (dead) break;
        if (lane == 0) {
          tc05_fence_after();
#pragma unroll
          for (int part = 0; part < (kExact ? 2 : 1); ++part)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_ts(tm + kColO, tm + (part ? kColS : kColP) + 8 * k, smem_desc_sw128(v0 + 2048 * k, 8192, 1024), idO,
                      t > cur.tb || part + k > 0);
          umma_commit(smem_u32(&sh.pv_done));
        }
        if (kExact) wait(&sh.pv_done, j & 1);  // the logits' columns hold the rest of P until then
      }
    } while (!dead && cur.next(a, sa));
    if (dead) {  // products still under way end before their memory goes
      if (lane == 0) {
        record_status(a.status, SFA_ERR_TIMEOUT);
        if (last > 0) mbar_wait_bounded(smem_u32(&sh.s_full), (last - 1) & 1, a.wait_cycles);
        if (last > 1) mbar_wait_bounded(smem_u32(&sh.pv_done), (last - 2) & 1, a.wait_cycles);
      }
    }
  } else if (warp >= 4) {
    // ---- codes to f16, a thread a key of the step
    const int key = tid - 128, half = key >> 6, k64 = key & 63;
    const int lgr = min(a.lgS, 6);
    do {
      for (int t = cur.tb; t < cur.te && !dead; t += 2, ++j) {
        const bool two = t + 1 < cur.te;
        const int s0 = n % kPSlots, s1 = (n + 1) % kPSlots;
        wait(&sh.raw_full[s0], n / kPSlots & 1);
        if (two) wait(&sh.raw_full[s1], (n + 1) / kPSlots & 1);
        const int slot = half ? s1 : s0;
        const int pg0 = sh.pages[s0], pg1 = two ? sh.pages[s1] : 0;
        const uint8_t* T = raw + slot * kTileBytes;
        const bool zero = (half && !two) || t * kTile + key > cur.it.plast() || !((half ? pg1 : pg0) >> (k64 >> lgr) & 1);
        const uint2 sc = zero ? make_uint2(0, 0) : *reinterpret_cast<const uint2*>(T + 64 * kTile + 8 * k64);
        if (j > 0) wait(&sh.s_full, (j - 1) & 1);  // the last step's keys have been read
        if (dead) break;
        dequantise_row(T + 32 * k64, sc.x, zero, kt, key);
        // a NaN value block is stored as zeros: the columns that attend its key are told (0 * NaN would reach all)
        uint32_t nan = 0, vs = sc.y;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if ((vs >> (8 * b) & 127u) == 127u) {
            nan |= 1u << b;
            vs &= ~(255u << (8 * b));
          }
        const int buf = j & 1;
        sh.nan[buf][key] = (uint8_t)nan;
        const bool any = __any_sync(0xffffffffu, nan != 0);
        if (lane == 0) {
          sh.step_nan[buf][warp - 4] = any;
          if (warp == 4) sh.step_pages[buf] = pg0 | pg1 << 4;
        }
        fence_async_smem();
        arrive(&sh.k_full);
        if (j > 0) wait(&sh.pv_done, (j - 1) & 1);  // and its values
        if (dead) break;
        dequantise_row(T + 32 * kTile + 32 * k64, vs, zero, vt, key);
        fence_async_smem();
        arrive(&sh.v_full);
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
    const uint32_t tl = tm + ((uint32_t)(32 * warp) << 16);  // this warp's lanes of tensor memory
    const int row = tid >> a.lgG, lgr = min(a.lgS, 6);
    const int all_pages = (1 << (kTile >> lgr)) - 1;
    const int full_pages = all_pages | all_pages << 4;
    float cs = 0.0f;
    do {
      const int ncol = cur.it.nrows << a.lgG;
      const bool mine = tid < ncol;
      const int p = cur.it.pfirst + row, head = cur.h * G + (tid & (G - 1));
      const int64_t out_row = cur.it.row0 + row;
      if (cur.te > cur.tb && (cur.x != qx || cur.h != qh)) {
        qx = cur.x;
        qh = cur.h;
        // the column's query: rotated, scaled by a power of two to its own size, in two f16 parts.  The
        // products that read the last one have ended: this thread has seen their sums
        const TIO* src = static_cast<const TIO*>(a.q) + out_row * a.q_stride + head * kD;
        const bool there = mine && p >= 0;
        float big = 0.0f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float lo[8], hi[8];
          if (there) {
            load_pair_chunk(src, c, a.rope, p, lo, hi);
#pragma unroll
            for (int e = 0; e < 8; ++e) big = fmaxf(big, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
          }
        }
        const int ex = min(max((int)(__float_as_uint(big) >> 23), 9), 253);
        const float f = __uint_as_float((uint32_t)(254 - ex) << 23) * 256.0f;
        cs = __uint_as_float((uint32_t)ex << 23) * (0.125f * kLog2e * a.kscale * 0.00390625f);
#pragma unroll 1
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
            *reinterpret_cast<uint4*>(smem + swz(tid, c + 4 * i)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(smem + kPTile + swz(tid, c + 4 * i)) = make_uint4(l[0], l[1], l[2], l[3]);
          }
        }
        fence_async_smem();
        arrive(&sh.q_full);
      }
      float m = -INFINITY, l = 0.0f;
      uint32_t nans = 0;  // scale blocks of the output that an attended NaN reaches
      for (int t = cur.tb; t < cur.te && !dead; t += 2, ++j) {
        const int buf = j & 1, j0 = t * kTile;
        wait(&sh.s_full, j & 1);
        if (dead) break;
        tc05_fence_after();
        const int pg = sh.step_pages[buf];
        const bool full = pg == full_pages && j0 + kStep - 1 <= cur.it.pfirst && j0 >= cur.it.plast() - sa.W;
        const int k_lo = max(p - sa.W - j0, 0), k_hi = mine ? min(p - j0, kStep - 1) : -1;
        auto attends = [&](int k) { return k >= k_lo && k <= k_hi && (pg >> ((k >> 6) * 4 + ((k & 63) >> lgr)) & 1); };
        if (sh.step_nan[buf][0] | sh.step_nan[buf][1] | sh.step_nan[buf][2] | sh.step_nan[buf][3])
          for (int k = 0; k < kStep; ++k)
            if (sh.nan[buf][k] && attends(k)) nans |= sh.nan[buf][k];
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kStep; c += 32) {
          float s[32];
          tmem_ld32(tl + kColS + c, s);
          tmem_wait_ld();
          if (!full)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!attends(c + e)) s[e] = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e) top = fmaxf(top, s[e]);
        }
        top *= cs;
        // the maximum moves only when a logit passes it by more than kLag
        const bool move = top > m + kLag;
        float corr = 1.0f;
        if (move) {
          corr = ex2(m - top);  // 0 on the first keys
          m = top;
          l *= corr;
        }
        if (j > 0) wait(&sh.pv_done, (j - 1) & 1);  // P's columns are free, O stands still
        if (dead) break;
        tc05_fence_after();
        if (t > cur.tb && __any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float o[16];
            tmem_ld16(tl + kColO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= corr;
            tmem_st16(tl + kColO + c, o);
          }
        }
        const float off = m == -INFINITY ? 0.0f : kPShift - m;
        float part[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kStep; c += 32) {
          float s[32], w[16];
          tmem_ld32(tl + kColS + c, s);
          tmem_wait_ld();
          if (!full)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!attends(c + e)) s[e] = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            s[e] = ex2(fmaf(s[e], cs, off));
            part[e & 1] += s[e];
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __uint_as_float(pack_f16(s[2 * e], s[2 * e + 1]));
          tmem_st16(tl + kColP + c / 2, w);
          if (kExact) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 r = unpack_f16(__float_as_uint(w[e]));
              w[e] = __uint_as_float(pack_f16(s[2 * e] - r.x, s[2 * e + 1] - r.y));
            }
            tmem_st16(tl + kColS + c / 2, w);  // over logits that have been read
          }
        }
        l += part[0] + part[1];
        tmem_wait_st();
        tc05_fence_before();
        arrive(&sh.p_full);
      }
      const bool any = cur.te > cur.tb;  // (an empty item has no step)
      if (any) {
        wait(&sh.pv_done, (j - 1) & 1);
        tc05_fence_after();
      }
      const int64_t at = (((int64_t)cur.x * a.Hkv + cur.h) * sa.max_chunks + cur.c - cur.it.c0) * kPromptColumns + tid;
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
        } else if (cur.it.nch == 1) {
          write_head<TIO>(a, out_row, head, c / 8, o, m, l);
          write_head<TIO>(a, out_row, head, c / 8 + 1, o + 8, m, l);
        } else {
          store8(sa.part_o + at * kD + c, o);
          store8(sa.part_o + at * kD + c + 8, o + 8);
          if (c == 0) sa.part_ml[at] = make_float2(m, l);
        }
      }
      tc05_fence_before();
    } while (!dead && cur.next(a, sa));
    if (dead && lane == 0) record_status(a.status, SFA_ERR_TIMEOUT);
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == kPWarps - 1) tmem_dealloc(tm, kPCols);
}

cudaError_t launch_kv4_prompt(const Kv4Args& a, const StreamArgs& s, int dtype, cudaStream_t stream) {
  static_assert((kPromptSmem + (int)sizeof(PromptShared) + 1024) * kPromptCtas <= 228 * 1024, "CTAs an SM");
  auto kern = dtype == SFA_BF16 ? kv4_prompt_kernel<bf16> : kv4_prompt_kernel<float>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPromptSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(kSMs * kPromptCtas), dim3(kPThreads), kPromptSmem, stream, a, s);
}

}  // namespace sfa
