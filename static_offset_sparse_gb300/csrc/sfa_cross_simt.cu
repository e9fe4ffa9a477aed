// Attention to states of another length in fp32, forward and backward: tiles of
// 64 rows x 64 keys in shared memory, products on the fp32 units.
//
// The fp32 units bound it: what a tile's product reads from shared memory (two
// or three 16-byte reads for 16 or 32 multiplications a thread) takes half as
// long.  Both operands of a product are held with the summed index outermost,
// so that a thread reads 4 neighbouring rows and 4 neighbouring columns at once.
#include "sfa_cross.cuh"

namespace sfa {

constexpr int kTileN = kSimtTile;
constexpr int kPitch = 68;  // floats a line: 16-byte reads, lines on other banks
constexpr int kLine = kTileN * kPitch;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// acc[i][j] += sum_x A[x][i0 + i] B[x][j0 + j]; A and B [64][kPitch].
template <int MR>
__device__ __forceinline__ void tile_product(float (*acc)[4], const float* A, const float* B, int i0, int j0) {
#pragma unroll 8
  for (int x = 0; x < kTileN; ++x) {
    float ar[MR];
#pragma unroll
    for (int i = 0; i < MR; i += 4) {
      const float4 v = ld4(A + x * kPitch + i0 + i);
      ar[i] = v.x; ar[i + 1] = v.y; ar[i + 2] = v.z; ar[i + 3] = v.w;
    }
    const float4 b = ld4(B + x * kPitch + j0);
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      acc[i][0] = fmaf(ar[i], b.x, acc[i][0]);
      acc[i][1] = fmaf(ar[i], b.y, acc[i][1]);
      acc[i][2] = fmaf(ar[i], b.z, acc[i][2]);
      acc[i][3] = fmaf(ar[i], b.w, acc[i][3]);
    }
  }
}

// n8 chunks of 8 dims of one row (nullptr: zeros) from chunk c0 on: transposed
// into line c of tr, and as they are into row r of pl (either may be nullptr).
__device__ __forceinline__ void load_row(const float* row, int r, int c0, int n8, float mul, float* tr, float* pl) {
#pragma unroll
  for (int c = c0; c < c0 + n8; ++c) {
    float x[8];
    if (row) {
      load8(row + 8 * c, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= mul;
    if (tr)
#pragma unroll
      for (int e = 0; e < 8; ++e) tr[(8 * c + e) * kPitch + r] = x[e];
    if (pl) st_smem8(pl + r * kPitch + 8 * c, x);
  }
}

// ---- forward: a CTA has 64 rows of a (sequence, KV head) and a split of its keys
constexpr int kFwdThreads = 128;
constexpr size_t kFwdSmemBytes = 4 * kLine * sizeof(float);

__global__ void __launch_bounds__(kFwdThreads) cross_fwd_kernel(const CrossArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *const Qt = sm, *const Kt = sm + kLine, *const Vs = sm + 2 * kLine, *const Pt = sm + 3 * kLine;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int rows = a.G * a.Tq, tiles = (rows + kTileN - 1) / kTileN;
  int64_t x = blockIdx.x;
  const int s = (int)(x % a.splits);
  x /= a.splits;
  const int r0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = (int)(x % a.Hkv), b = (int)(x / a.Hkv);
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kTileN, a.splits, s, k0, k1);
  if (r0 >= (int64_t)nq * a.G) k1 = k0;  // no query in the tile
  {
    const int r = r0 + (tid & 63), t = r / a.G, h = kvh * a.G + (r - t * a.G);
    const float* row = r < rows && t < nq ? static_cast<const float*>(a.q) + b * a.qs.b + h * a.qs.h + t * a.qs.t : nullptr;
    load_row(row, tid & 63, 4 * (tid >> 6), 4, kLogitScale, Qt, (float*)nullptr);
  }
  float o[8][4], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  }
  for (int j0 = k0; j0 < k1; j0 += kTileN) {
    {
      const int j = j0 + (tid & 63);
      const bool in = j < k1;
      load_row(in ? static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h + j * a.ks.t : nullptr, tid & 63, 4 * (tid >> 6), 4, 1.0f, Kt, (float*)nullptr);
      load_row(in ? static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h + j * a.vs.t : nullptr, tid & 63, 4 * (tid >> 6), 4, 1.0f, (float*)nullptr, Vs);
    }
    __syncthreads();
    float p[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j] = 0.0f;
    tile_product<8>(p, Qt, Kt, 8 * ty, 4 * tx);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j0 + 4 * tx + j >= k1) p[i][j] = -INFINITY;
        top = fmaxf(top, p[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float mn = fmaxf(m[i], top), sh = shift_of(mn), corr = exp2f(m[i] - sh);
      m[i] = mn;
      l[i] *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[i][j] *= corr;
        p[i][j] = exp2f(p[i][j] - sh);
        l[i] += p[i][j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(Pt + (4 * tx + j) * kPitch + 8 * ty + i) = make_float4(p[i][j], p[i + 1][j], p[i + 2][j], p[i + 3][j]);
    __syncthreads();
    tile_product<8>(o, Pt, Vs, 8 * ty, 4 * tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    const int r = r0 + 8 * ty + i;
    if (r >= rows) continue;
    const bool none = k1 <= k0 || r / a.G >= nq;
    const int64_t row = a.row(b, kvh, r);
    if (a.parts) {
      const int64_t at = s * a.rows + row;
      if (!none) *reinterpret_cast<float4*>(a.part_o + at * kD + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
      if (tx == 0) a.part_ml[at] = none ? make_float2(-INFINITY, -1.0f) : make_float2(m[i], l[i]);
    } else {
      const float inv = 1.0f / l[i];
      float* out = static_cast<float*>(a.o) + row * kD + 4 * tx;
      store2(out, none ? 0.0f : o[i][0] * inv, none ? 0.0f : o[i][1] * inv);
      store2(out + 2, none ? 0.0f : o[i][2] * inv, none ? 0.0f : o[i][3] * inv);
      if (a.lse && tx == 0) a.lse[row] = none ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
  }
}

// ---- backward
constexpr int kBwdThreads = 256;  // 16 x 16 threads, 4 x 4 sums each
constexpr size_t kDqSmemBytes = 6 * kLine * sizeof(float), kDkvSmemBytes = 8 * kLine * sizeof(float);

// dq: a CTA has 64 rows and a split of their keys.
//   ds = p (dO v - delta), dq = sum ds k / 8
__global__ void __launch_bounds__(kBwdThreads) cross_dq_kernel(const CrossArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *const Qt = sm, *const Dt = sm + kLine, *const Kt = sm + 2 * kLine, *const Vt = sm + 3 * kLine, *const Ks = sm + 4 * kLine,
               *const St = sm + 5 * kLine;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lr = tid & 63, lc = 2 * (tid >> 6);
  const int rows = a.G * a.Tq, tiles = (rows + kTileN - 1) / kTileN;
  int64_t x = blockIdx.x;
  const int s = (int)(x % a.splits);
  x /= a.splits;
  const int r0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = (int)(x % a.Hkv), b = (int)(x / a.Hkv);
  const int nq = a.queries(b), nk = a.keys(b);
  int k0, k1;
  split_keys(nk, kTileN, a.splits, s, k0, k1);
  if (r0 >= (int64_t)nq * a.G) k1 = k0;
  {
    const int r = r0 + lr, t = r / a.G, h = kvh * a.G + (r - t * a.G);
    const bool in = r < rows && t < nq;
    load_row(in ? static_cast<const float*>(a.q) + b * a.qs.b + h * a.qs.h + t * a.qs.t : nullptr, lr, lc, 2, kLogitScale, Qt, (float*)nullptr);
    load_row(in ? static_cast<const float*>(a.dO) + a.row(b, kvh, r) * kD : nullptr, lr, lc, 2, 1.0f, Dt, (float*)nullptr);
  }
  float2 st[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    st[i] = r < rows ? a.stat[a.row(b, kvh, r)] : make_float2(INFINITY, 0.0f);
  }
  float dq[4][4] = {};
  for (int j0 = k0; j0 < k1; j0 += kTileN) {
    const int j = j0 + lr;
    const bool in = j < k1;
    load_row(in ? static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h + j * a.ks.t : nullptr, lr, lc, 2, 1.0f, Kt, Ks);
    load_row(in ? static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h + j * a.vs.t : nullptr, lr, lc, 2, 1.0f, Vt, (float*)nullptr);
    __syncthreads();
    float p[4][4] = {}, dp[4][4] = {};
    tile_product<4>(p, Qt, Kt, 4 * ty, 4 * tx);
    tile_product<4>(dp, Dt, Vt, 4 * ty, 4 * tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const bool there = j0 + 4 * tx + jj < k1 && st[i].x != INFINITY;
        p[i][jj] = there ? exp2f(p[i][jj] - st[i].x) * (dp[i][jj] - st[i].y) : 0.0f;
      }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
      *reinterpret_cast<float4*>(St + (4 * tx + jj) * kPitch + 4 * ty) = make_float4(p[0][jj], p[1][jj], p[2][jj], p[3][jj]);
    __syncthreads();
    tile_product<4>(dq, St, Ks, 4 * ty, 4 * tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    if (r >= rows) continue;
    const int64_t row = a.row(b, kvh, r);
    if (a.parts) {
      float* out = a.part_a + (s * a.rows + row) * kD + 4 * tx;
      *reinterpret_cast<float4*>(out) = make_float4(0.125f * dq[i][0], 0.125f * dq[i][1], 0.125f * dq[i][2], 0.125f * dq[i][3]);
    } else {
      float* out = static_cast<float*>(a.dq) + row * kD + 4 * tx;
      store2(out, 0.125f * dq[i][0], 0.125f * dq[i][1]);
      store2(out + 2, 0.125f * dq[i][2], 0.125f * dq[i][3]);
    }
  }
}

// dk, dv: a CTA has 64 keys and a split of the rows that attend them.
//   dv = sum p dO, dk = sum ds q / 8
__global__ void __launch_bounds__(kBwdThreads) cross_dkv_kernel(const CrossArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *const Kt = sm, *const Vt = sm + kLine, *const Qt = sm + 2 * kLine, *const Dt = sm + 3 * kLine, *const Qs = sm + 4 * kLine,
               *const Ds = sm + 5 * kLine, *const Pt = sm + 6 * kLine, *const St = sm + 7 * kLine;
  __shared__ float2 stat[kTileN];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lr = tid & 63, lc = 2 * (tid >> 6);
  const int tiles = (a.Tk + kTileN - 1) / kTileN;
  int64_t x = blockIdx.x;
  const int s = (int)(x % a.splits);
  x /= a.splits;
  const int j0 = (int)(x % tiles) * kTileN;
  x /= tiles;
  const int kvh = (int)(x % a.Hkv), b = (int)(x / a.Hkv);
  const int nq = a.queries(b), nk = a.keys(b), rows = a.G * nq;
  int b0, b1;
  split_keys(j0 < nk ? rows : 0, kTileN, a.splits, s, b0, b1);
  {
    const int j = j0 + lr;
    load_row(j < nk ? static_cast<const float*>(a.k) + b * a.ks.b + kvh * a.ks.h + j * a.ks.t : nullptr, lr, lc, 2, 1.0f, Kt, (float*)nullptr);
    load_row(j < nk ? static_cast<const float*>(a.v) + b * a.vs.b + kvh * a.vs.h + j * a.vs.t : nullptr, lr, lc, 2, 1.0f, Vt, (float*)nullptr);
  }
  float dk[4][4] = {}, dv[4][4] = {};
  for (int r0 = b0; r0 < b1; r0 += kTileN) {
    const int r = r0 + lr, t = r / a.G, h = kvh * a.G + (r - t * a.G);
    const bool in = r < b1;
    load_row(in ? static_cast<const float*>(a.q) + b * a.qs.b + h * a.qs.h + t * a.qs.t : nullptr, lr, lc, 2, 1.0f, Qt, Qs);
    load_row(in ? static_cast<const float*>(a.dO) + a.row(b, kvh, r) * kD : nullptr, lr, lc, 2, 1.0f, Dt, Ds);
    if (tid < kTileN) stat[tid] = in ? a.stat[a.row(b, kvh, r)] : make_float2(INFINITY, 0.0f);
    __syncthreads();
    float p[4][4] = {}, dp[4][4] = {};  // [key][row]
    tile_product<4>(p, Kt, Qt, 4 * ty, 4 * tx);
    tile_product<4>(dp, Vt, Dt, 4 * ty, 4 * tx);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const float2 st = stat[4 * tx + jj];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = j0 + 4 * ty + i < nk && st.x != INFINITY;
        p[i][jj] = there ? exp2f(fmaf(p[i][jj], kLogitScale, -st.x)) : 0.0f;
        dp[i][jj] = there ? p[i][jj] * (dp[i][jj] - st.y) : 0.0f;
      }
      *reinterpret_cast<float4*>(Pt + (4 * tx + jj) * kPitch + 4 * ty) = make_float4(p[0][jj], p[1][jj], p[2][jj], p[3][jj]);
      *reinterpret_cast<float4*>(St + (4 * tx + jj) * kPitch + 4 * ty) = make_float4(dp[0][jj], dp[1][jj], dp[2][jj], dp[3][jj]);
    }
    __syncthreads();
    tile_product<4>(dv, Pt, Ds, 4 * ty, 4 * tx);
    tile_product<4>(dk, St, Qs, 4 * ty, 4 * tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 4 * ty + i;
    if (j >= a.Tk) continue;
    const int64_t row = ((int64_t)b * a.Hkv + kvh) * a.Tk + j;
    if (a.parts) {
      const int64_t at = ((int64_t)s * a.B * a.Hkv * a.Tk + row) * kD + 4 * tx;
      *reinterpret_cast<float4*>(a.part_a + at) = make_float4(0.125f * dk[i][0], 0.125f * dk[i][1], 0.125f * dk[i][2], 0.125f * dk[i][3]);
      *reinterpret_cast<float4*>(a.part_b + at) = make_float4(dv[i][0], dv[i][1], dv[i][2], dv[i][3]);
    } else {
      float *ok = static_cast<float*>(a.dk) + row * kD + 4 * tx, *ov = static_cast<float*>(a.dv) + row * kD + 4 * tx;
      store2(ok, 0.125f * dk[i][0], 0.125f * dk[i][1]);
      store2(ok + 2, 0.125f * dk[i][2], 0.125f * dk[i][3]);
      store2(ov, dv[i][0], dv[i][1]);
      store2(ov + 2, dv[i][2], dv[i][3]);
    }
  }
}

static int launch_tiles(int kind, void (*f)(const CrossArgs), const CrossArgs& a, int tiles, int threads, size_t smem, void* stream) {
  const int64_t grid = (int64_t)a.B * a.Hkv * tiles * a.splits;
  LaunchTimer tm(kind, stream);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(f, dim3((unsigned)grid), dim3(threads), smem, (cudaStream_t)stream, a);
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

static int tiles_of(int rows) { return (rows + kTileN - 1) / kTileN; }

int launch_cross_fwd_simt(const CrossArgs& a, void* stream) {
  return launch_tiles(SFA_KERNEL_CROSS_FWD, cross_fwd_kernel, a, tiles_of(a.G * a.Tq), kFwdThreads, kFwdSmemBytes, stream);
}
int launch_cross_dq_simt(const CrossArgs& a, void* stream) {
  return launch_tiles(SFA_KERNEL_CROSS_BWD_Q, cross_dq_kernel, a, tiles_of(a.G * a.Tq), kBwdThreads, kDqSmemBytes, stream);
}
int launch_cross_dkv_simt(const CrossArgs& a, void* stream) {
  return launch_tiles(SFA_KERNEL_CROSS_BWD_KV, cross_dkv_kernel, a, tiles_of(a.Tk), kBwdThreads, kDkvSmemBytes, stream);
}

}  // namespace sfa
