// Few rows over many keys: the step of a decoder over an encoder's states, and
// the own rows of the sequences behind a shared prefix.
//
// Every key and value is read once for the (up to 8) rows of its KV head and
// used for a few multiplications a row: memory bounds it.  Eight lanes hold a
// key, 8 dims each, so a warp reads four whole rows at a time straight into
// registers; a row's products are summed over the eight lanes by halving
// exchanges that leave row r's logit in lane r (7 shuffles for 8 rows, not 24).
// fp32 throughout.
#include "sfa_cross.cuh"

namespace sfa {

constexpr int kStreamWarps = 4;

// Sums of acc[0 .. NR) over the eight lanes of a key; lane l gets row l mod NR's.
template <int NR>
__device__ __forceinline__ float sum_rows(float* acc, int lane) {
#pragma unroll
  for (int bit = 4, n = NR; bit > 0; bit >>= 1) {
    if (n > bit) {  // rows' halves are exchanged: n -> n / 2 (bit is n / 2 then)
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i)
        if (i < n / 2) {
          const float mine = up ? acc[i + n / 2] : acc[i], other = up ? acc[i] : acc[i + n / 2];
          acc[i] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
        }
      n /= 2;
    } else {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (i < n) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], bit);
    }
  }
  return acc[0];
}

template <typename TQ, typename TIO, int NR>
__global__ void __launch_bounds__(32 * kStreamWarps) cross_stream_kernel(const CrossArgs a) {
  constexpr int U = sizeof(TIO) == 2 ? 4 : 2;  // keys a lane takes at a time
  constexpr int kStep = 4 * U;                  // keys a warp takes at a time
  __shared__ float so[kStreamWarps][NR][kD];
  __shared__ float2 sml[kStreamWarps][NR];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kg = lane >> 3, d8 = (lane & 7) * 8;
  const int rows = a.G * a.Tq, groups = (rows + NR - 1) / NR;
  int64_t x = blockIdx.x;
  const int s = (int)(x % a.splits);
  x /= a.splits;
  const int r0 = (int)(x % groups) * NR;
  x /= groups;
  const int kvh = (int)(x % a.Hkv), b = (int)(x / a.Hkv);
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kStep, a.splits, s, k0, k1);

  float q[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int t = (r0 + r) / a.G, h = kvh * a.G + (r0 + r - t * a.G);
    if (r0 + r < rows && t < nq) {
      load8(static_cast<const TQ*>(a.q) + b * a.qs.b + h * a.qs.h + t * a.qs.t + d8, q[r]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[r][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q[r][e] *= kLogitScale;
  }
  const TIO* kp = static_cast<const TIO*>(a.k) + b * a.ks.b + kvh * a.ks.h + d8;
  const TIO* vp = static_cast<const TIO*>(a.v) + b * a.vs.b + kvh * a.vs.h + d8;
  float m = -INFINITY, l = 0.0f;  // of row lane mod NR
  float o[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) o[r][e] = 0.0f;

  for (int base = k0 + warp * kStep; base < k1; base += kStep * kStreamWarps) {
    float kf[U][8], vf[U][8], p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + 4 * u + kg;
      const int64_t at = j < k1 ? j : k0;  // (a row that is there)
      load8(kp + at * a.ks.t, kf[u]);
      load8(vp + at * a.vs.t, vf[u]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y = fmaf(q[r][e], kf[u][e], y);
        acc[r] = y;
      }
      p[u] = sum_rows<NR>(acc, lane);
      if (base + 4 * u + kg >= k1) p[u] = -INFINITY;
      top = fmaxf(top, p[u]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (__any_sync(0xffffffffu, top > m)) {
      const float mn = fmaxf(m, top), corr = exp2f(m - shift_of(mn));
      l *= corr;
      m = mn;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float c = __shfl_sync(0xffffffffu, corr, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] *= c;
      }
    }
    const float sh = shift_of(m);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = base + 4 * u + kg < k1;
      p[u] = exp2f(p[u] - sh);
      l += p[u];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float pr = __shfl_sync(0xffffffffu, p[u], (lane & 24) | r);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] = there ? fmaf(pr, vf[u][e], o[r][e]) : o[r][e];
      }
    }
  }
  // the warp's four keys, then the warps
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (lane < NR) sml[warp][lane] = make_float2(m, l);
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 8);
      o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 16);
    }
  if (kg == 0)
#pragma unroll
    for (int r = 0; r < NR; ++r) st_smem8(&so[warp][r][d8], o[r]);
  __syncthreads();
  for (int i = threadIdx.x; i < NR * 32; i += 32 * kStreamWarps) {
    const int r = i >> 5, d = (i & 31) * 2;
    if (r0 + r >= rows) break;
    const int t = (r0 + r) / a.G;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) mm = fmaxf(mm, sml[w][r].x);
    const float sh = shift_of(mm);
    float ll = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) {
      const float f = exp2f(sml[w][r].x - sh);
      ll = fmaf(f, sml[w][r].y, ll);
      y0 = fmaf(f, so[w][r][d], y0);
      y1 = fmaf(f, so[w][r][d + 1], y1);
    }
    const int64_t row = a.row(b, kvh, r0 + r);
    const bool none = t >= nq || k1 <= k0;
    if (a.parts) {
      const int64_t at = s * a.rows + row;
      if (!none) store2(a.part_o + at * kD + d, y0, y1);
      if (d == 0) a.part_ml[at] = none ? make_float2(-INFINITY, -1.0f) : make_float2(mm, ll);
    } else {
      const float inv = none ? 0.0f : 1.0f / ll;
      store2(static_cast<TIO*>(a.o) + row * kD + d, none ? 0.0f : y0 * inv, none ? 0.0f : y1 * inv);
      if (a.lse && d == 0) a.lse[row] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  }
}

// Parts of each row to o and lse, a warp a row.  pos (of sequences whose rows
// are queries' heads, Tq = 1): a position outside [0, T) leaves a zero row.
template <typename TIO>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossArgs a, const int32_t* pos, int T) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.rows, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  int n = a.splits;
  if (pos) {
    const int p = pos[row / a.Hq];
    if (p < 0 || p >= T) n = 0;
  }
  join_row<TIO>(a, row, n, lane, [&](int i) { return a.part_ml[i * rows + row]; }, [&](int i) { return a.part_o + (i * rows + row) * kD; });
}

int launch_cross_join(const CrossArgs& a, int dtype, const int32_t* pos, int pos_T, void* stream) {
  const int64_t rows = a.rows;
  const dim3 grid((unsigned)((rows + 7) / 8));
  cudaStream_t st = (cudaStream_t)stream;
  LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
  const cudaError_t e = dtype == SFA_BF16 ? launch_pdl(cross_join_kernel<bf16>, grid, dim3(256), 0, st, a, pos, pos_T)
                                          : launch_pdl(cross_join_kernel<float>, grid, dim3(256), 0, st, a, pos, pos_T);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

template <typename TQ, typename TIO>
static cudaError_t stream_rows(const CrossArgs& a, cudaStream_t st) {
  const int rows = a.G * a.Tq, nr = rows == 1 ? 1 : rows == 2 ? 2 : rows <= 4 ? 4 : 8;
  const int64_t grid = (int64_t)a.B * a.Hkv * ((rows + nr - 1) / nr) * a.splits;
  auto* f = nr == 1 ? cross_stream_kernel<TQ, TIO, 1> : nr == 2 ? cross_stream_kernel<TQ, TIO, 2>
          : nr == 4 ? cross_stream_kernel<TQ, TIO, 4> : cross_stream_kernel<TQ, TIO, 8>;
  return launch_pdl(f, dim3((unsigned)grid), dim3(32 * kStreamWarps), 0, st, a);
}

int launch_cross_stream(const CrossArgs& a, bool q32, int dtype, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  LaunchTimer tm(SFA_KERNEL_CROSS_FWD, stream);
  const cudaError_t e = dtype == SFA_F32 ? stream_rows<float, float>(a, st)
                        : q32            ? stream_rows<float, bf16>(a, st)
                                         : stream_rows<bf16, bf16>(a, st);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace sfa
