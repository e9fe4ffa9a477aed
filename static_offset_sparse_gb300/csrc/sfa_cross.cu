// Attention to states of another length (sfa_cross_forward, sfa_cross_backward)
// and a decode step of a batch that shares a prefix (sfa_prefix_decode): checks
// of arguments, which kernels a call runs, its workspace, and the small kernels
// around them.
#include "sfa_cross.cuh"

namespace sfa {

static bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// ---- small kernels

// lse * log2(e) and delta = sum(o * dO) of each row, eight lanes a row (of rows that
// count for nothing: zeros, which nothing reads).
__global__ void __launch_bounds__(256) cross_stat_kernel(const CrossArgs a, float2* stat) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  const int d8 = (threadIdx.x & 7) * 8;
  float sum = 0.0f;
  bool valid = false;
  if (row < a.rows) {
    const int64_t bh = row / a.Tq;
    const int b = (int)(bh / a.Hq);
    valid = row - bh * a.Tq < a.queries(b) && a.keys(b) > 0;
  }
  if (valid) {
    float o[8], g[8];
    load8(static_cast<const float*>(a.out) + row * kD + d8, o);
    load8(static_cast<const float*>(a.dO) + row * kD + d8, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(o[e], g[e], sum);
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (row < a.rows && d8 == 0) stat[row] = valid ? make_float2(a.lse[row] * kLog2e, sum) : make_float2(0.0f, 0.0f);
}

// blockIdx.y-th: out = the sum of n-number parts, in order (n = 0: nothing).
struct SumArgs {
  const float* parts[3];
  float* out[3];
  int64_t n[3];
  int splits[3];
};
__global__ void __launch_bounds__(256) cross_sum_kernel(const __grid_constant__ SumArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = a.n[blockIdx.y];
  if (i >= n) return;
  const float* const parts = a.parts[blockIdx.y] + i;
  const int splits = a.splits[blockIdx.y];
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(parts + s * n);
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  *reinterpret_cast<float4*>(a.out[blockIdx.y] + i) = x;
}

struct PrefixArgs {
  const void *q, *k_new, *v_new;
  int64_t q_stride, k_stride, v_stride;
  void *k_cache, *v_cache;
  const int32_t* pos;
  const float2* rope;
  float* q32;  // [B, Hq, 64] rotated queries
  bf16* q16;   // or nullptr: the same as two bf16 parts, [2][B, Hq, 64]
  int B, P, T, Hq, Hkv;
  int* status;
};

// Rotates a step's queries, and its key rows into the caches next to the
// values: a warp a head's row, a pair (j, j + 32) a lane.
template <typename TIO>
__global__ void __launch_bounds__(128) prefix_prep_kernel(const PrefixArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, heads = a.Hq + (a.k_new ? 2 * a.Hkv : 0);
  const int64_t x = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (x >= (int64_t)a.B * heads) return;
  const int b = (int)(x / heads), h = (int)(x - (int64_t)b * heads);
  const int t = a.pos[b];
  const bool there = t >= 0 && t < a.T;
  if (!there && lane == 0) record_status(a.status, SFA_ERR_DEVICE_BOUNDS);
  float lo = 0.0f, hi = 0.0f;
  if (there) {
    const TIO* in = h < a.Hq ? static_cast<const TIO*>(a.q) + b * a.q_stride + h * kD
                  : h < a.Hq + a.Hkv ? static_cast<const TIO*>(a.k_new) + b * a.k_stride + (h - a.Hq) * kD
                                     : static_cast<const TIO*>(a.v_new) + b * a.v_stride + (h - a.Hq - a.Hkv) * kD;
    lo = (float)in[lane];
    hi = (float)in[lane + 32];
    if (a.rope && h < a.Hq + a.Hkv) {
      const float2 cs = __ldg(a.rope + ((int64_t)a.P + t) * 32 + lane);
      const float x0 = lo, x1 = hi;
      lo = x0 * cs.x - x1 * cs.y;
      hi = x0 * cs.y + x1 * cs.x;
    }
  }
  if (h < a.Hq) {
    float* out = a.q32 + ((int64_t)b * a.Hq + h) * kD;
    out[lane] = lo;
    out[lane + 32] = hi;
    if (a.q16) {
      bf16* const first = a.q16 + ((int64_t)b * a.Hq + h) * kD;
      bf16* const second = first + (int64_t)a.B * a.Hq * kD;
      first[lane] = (bf16)lo;
      first[lane + 32] = (bf16)hi;
      second[lane] = (bf16)(lo - (float)(bf16)lo);
      second[lane + 32] = (bf16)(hi - (float)(bf16)hi);
    }
  } else if (there) {
    const bool key = h < a.Hq + a.Hkv;
    TIO* out = static_cast<TIO*>(key ? a.k_cache : a.v_cache) + (((int64_t)b * a.Hkv + (h - a.Hq) % a.Hkv) * a.T + t) * kD;
    out[lane] = (TIO)lo;
    out[lane + 32] = (TIO)hi;
  }
}

// ---- which kernels a call runs

// Few rows go to the kernels that stream keys.  bf16: as many as one CTA of them takes (16).
// fp32: up to four CTAs' of 8, each of which reads the keys (from L2), because the other kernel
// has tiles of 64 rows, however few there are (8 x 8 / 2 heads, 8 queries over 2000: 30.4 us in
// a tile, 24.8 so; with 64 rows both take the same).
enum Kind { kFewRows, kTensor, kFp32 };
static int stream_rows(int dtype) { return dtype == SFA_BF16 ? kStreamRowsBf16 : kStreamRows; }
static Kind forward_kind(int rows, int dtype) {
  if (dtype == SFA_BF16) return rows <= kStreamRowsBf16 ? kFewRows : kTensor;
  return rows <= 4 * kStreamRows ? kFewRows : kFp32;
}

// Whether a row's splits are a cluster, without workspace and join (32 x 8 / 2 heads over
// 1500 10.0 -> 8.3 us): where all CTAs are on the card at once (64 x 8 / 2 heads, 4 queries
// over 2000, bf16, 7 splits: 18.5 us with a join, 26.3 in clusters), three an SM in bf16, two
// in fp32, four of up to 4 rows.
static bool clustered(int rows, int64_t units, int splits, int dtype) {
  const int64_t ctas = units * ((rows + stream_rows(dtype) - 1) / stream_rows(dtype)) * splits;
  return splits > 1 && splits <= kClusterSplits && ctas <= (dtype == SFA_BF16 ? 3 : rows > 4 ? 2 : 4) * kSMs;
}

// Parts of a call over `units` (sequence, KV head) pairs of Tq queries of G heads (not the
// tensor cores').  Few rows, bf16: two waves of the three CTAs that fit an SM (128 x 8 / 2
// heads over 2048: 31.1 us, one wave of four 37.2), 256 keys a part at least (with 128,
// 32 x 8 / 2 heads over 1500 took 11.4 us, so 9.9), 128 where all parts are an SM's each
// and there is a join anyway (4 heads over 1000: 5.8 us for 7.1).  fp32: a part's keys take
// longer and its join as long, so fewer, and sqrt(Tk / 12) parts at most (8 / 2 heads over
// 1000: 9.1 us for 13.5; over 10000 16.8 us, and 31 without the limit).  A call whose parts
// are joined by themselves takes kClusterSplits for up to two more, if they can be a cluster
// then (8 / 2 heads over 1300 7.8 us in 10 parts, 7.3 so; over 2200 8.6 in 13, 8.9 in 8).  A
// prefix's and the own rows' parts are joined together, never in a cluster (`joined`: 4
// sequences behind 1300, 8 / 2 heads, 12.1 us in 10 parts, 12.7 in 8).
static int forward_splits(int64_t units, int G, int Tq, int Tk, Kind kind, int dtype, bool joined) {
  if (kind == kFewRows) {
    const int64_t ctas = units * ((G * Tq + stream_rows(dtype) - 1) / stream_rows(dtype));
    if (dtype == SFA_BF16) return wave_splits(ctas, 6 * kSMs, Tk, Tk >= 512 && ctas * (Tk / 128) <= kSMs ? 128 : 256);
    int s = wave_splits(ctas, 4 * kSMs, Tk, 64);
    while (s > 1 && 12 * s * s > Tk) --s;
    return !joined && s > kClusterSplits && s <= kClusterSplits + 2 && clustered(G * Tq, units, kClusterSplits, dtype) ? kClusterSplits : s;
  }
  return wave_splits(units * ((G * Tq + kF32Tile - 1) / kF32Tile), 3 * kSMs, (Tk + kF32Keys - 1) / kF32Keys, 1);
}

static size_t part_bytes(int splits, int64_t rows) {
  return align256((size_t)splits * rows * kD * sizeof(float)) + align256((size_t)splits * rows * sizeof(float2));
}

static void set_parts(CrossArgs* a, char* ws, int splits, int64_t rows, int first) {
  a->part_o = reinterpret_cast<float*>(ws) + first * rows * kD;
  a->part_ml = reinterpret_cast<float2*>(ws + align256((size_t)splits * rows * kD * sizeof(float))) + first * rows;
}

// ---- attention to states of another length

// Strides of a [B, H, T, 64] tensor: 16-byte steps that do not overlap, where
// there is more than one.
static bool strides_ok(const int64_t* s, int B, int H, int T, int dtype) {
  const int n[3] = {B, H, T};
  const int64_t step = dtype == SFA_BF16 ? 8 : 4;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < kD || s[i] % step || s[i] >= ((int64_t)1 << 38))) return false;
  return true;
}

static int check_cross(const sfa_cross_desc* d) {
  if (!d) return SFA_ERR_INVALID_ARG;
  if (d->B <= 0 || d->Tq <= 0 || d->Tk <= 0 || d->Hq <= 0 || d->Hkv <= 0) return SFA_ERR_INVALID_ARG;
  if (d->dtype != SFA_F32 && d->dtype != SFA_BF16) return SFA_ERR_INVALID_ARG;
  if (d->D != kD || d->Hq % d->Hkv) return SFA_ERR_UNSUPPORTED;
  if (d->Hq / d->Hkv > 32) return SFA_ERR_UNSUPPORTED;
  if (d->Tq > (1 << 24) || d->Tk > (1 << 24)) return SFA_ERR_UNSUPPORTED;
  if ((__int128)d->B * d->Hq * d->Tq >= ((__int128)1 << 30) || (__int128)d->B * d->Hkv * d->Tk >= ((__int128)1 << 30))
    return SFA_ERR_UNSUPPORTED;
  if (!strides_ok(d->q_stride, d->B, d->Hq, d->Tq, d->dtype) || !strides_ok(d->k_stride, d->B, d->Hkv, d->Tk, d->dtype) ||
      !strides_ok(d->v_stride, d->B, d->Hkv, d->Tk, d->dtype) || !aligned(d->q_len, 4) || !aligned(d->kv_len, 4))
    return SFA_ERR_INVALID_ARG;
  return SFA_OK;
}

static int cross_args(const sfa_cross_desc* d, CrossArgs* a) {
  *a = CrossArgs{};
  a->qs = {d->q_stride[0], d->q_stride[1], d->q_stride[2]};
  a->ks = {d->k_stride[0], d->k_stride[1], d->k_stride[2]};
  a->vs = {d->v_stride[0], d->v_stride[1], d->v_stride[2]};
  a->rs = {(int64_t)d->Hq * d->Tq, d->Tq, 1};
  a->rows = (int64_t)d->B * d->Hq * d->Tq;
  a->q_len = d->q_len;
  a->kv_len = d->kv_len;
  a->B = d->B;
  a->Tq = d->Tq;
  a->Tk = d->Tk;
  a->Hq = d->Hq;
  a->Hkv = d->Hkv;
  a->G = d->Hq / d->Hkv;
  wait_injection(&a->wait_cycles, &a->debug_skip);
  return device_status(&a->status);
}

struct ForwardPlan {
  Kind kind;
  int splits;
  bool cluster;
  size_t bytes;
};

static ForwardPlan forward_plan(const sfa_cross_desc* d) {
  const int G = d->Hq / d->Hkv;
  ForwardPlan p = {forward_kind(G * d->Tq, d->dtype), 1, false, 0};
  if (p.kind == kTensor) {
    p.bytes = cross_tc_bytes(d->B, d->Hkv, G, d->Tq, d->Tk);
  } else {
    p.splits = forward_splits((int64_t)d->B * d->Hkv, G, d->Tq, d->Tk, p.kind, d->dtype, false);
    p.cluster = p.kind == kFewRows && clustered(G * d->Tq, (int64_t)d->B * d->Hkv, p.splits, d->dtype);
    if (p.splits > 1 && !p.cluster) p.bytes = part_bytes(p.splits, (int64_t)d->B * d->Hq * d->Tq);
  }
  return p;
}

struct BackwardPlan {  // (what is not bytes is the fp32 kernels')
  int dq_splits, dkv_splits;
  int64_t rows, keys;
  size_t stat, bytes;   // bytes of the rows' numbers, of the workspace
  size_t dq_parts;      // numbers of dq's parts, before those of dk and dv
};

static BackwardPlan backward_plan(const sfa_cross_desc* d) {
  BackwardPlan p = {};
  const int64_t units = (int64_t)d->B * d->Hkv;
  const int G = d->Hq / d->Hkv;
  if (d->dtype == SFA_BF16) {
    p.bytes = cross_bwd_tc_bytes(d->B, d->Hkv, G, d->Tq, d->Tk);
    return p;
  }
  const int rt = (G * d->Tq + kF32Tile - 1) / kF32Tile, kt = (d->Tk + kF32Tile - 1) / kF32Tile;
  // (three CTAs fit an SM: two waves of dq's, fewer of the heavier others; with 8 and 8,
  // 2 x 8 / 2 heads, 333 x 1000 ragged rows took 94 us, so 78)
  p.dq_splits = wave_splits(units * rt, 6 * kSMs, kt, 1);
  p.dkv_splits = wave_splits(units * kt, 4 * kSMs, rt, 1);
  p.rows = (int64_t)d->B * d->Hq * d->Tq;
  p.keys = units * d->Tk;
  p.stat = align256((size_t)p.rows * sizeof(float2));
  p.dq_parts = p.dq_splits > 1 ? (size_t)p.dq_splits * p.rows * kD : 0;
  p.bytes = p.stat + (p.dq_parts + (p.dkv_splits > 1 ? 2 * (size_t)p.dkv_splits * p.keys * kD : 0)) * sizeof(float);
  return p;
}

// ---- a decode step behind a shared prefix

static int check_prefix(const sfa_prefix_desc* d) {
  if (!d) return SFA_ERR_INVALID_ARG;
  if (d->B <= 0 || d->P < 0 || d->T <= 0 || d->Hq <= 0 || d->Hkv <= 0) return SFA_ERR_INVALID_ARG;
  if (d->dtype != SFA_F32 && d->dtype != SFA_BF16) return SFA_ERR_INVALID_ARG;
  if (d->D != kD || d->Hq % d->Hkv) return SFA_ERR_UNSUPPORTED;
  if (d->Hq / d->Hkv > 32) return SFA_ERR_UNSUPPORTED;
  if (d->P > (1 << 24) || d->T > (1 << 24) || (__int128)d->B * d->Hq >= (1 << 24) || (__int128)d->Hkv * d->P >= ((__int128)1 << 30) ||
      (__int128)d->B * d->Hkv * d->T >= ((__int128)1 << 30))
    return SFA_ERR_UNSUPPORTED;
  const int64_t step = d->dtype == SFA_BF16 ? 8 : 4;
  const int64_t s[5] = {d->q_stride, d->k_stride, d->v_stride, d->prefix_k_stride, d->prefix_v_stride};
  const int64_t least[5] = {(int64_t)d->Hq * kD, (int64_t)d->Hkv * kD, (int64_t)d->Hkv * kD, (int64_t)d->P * kD, (int64_t)d->P * kD};
  for (int i = 0; i < 5; ++i)
    if ((i < 3 ? d->B : d->P ? d->Hkv : 1) > 1 && (s[i] < least[i] || s[i] % step || s[i] >= ((int64_t)1 << 38))) return SFA_ERR_INVALID_ARG;
  if (d->rope && (!aligned(d->rope, 16) || (int64_t)d->rope_T < (int64_t)d->P + d->T)) return SFA_ERR_INVALID_ARG;
  return SFA_OK;
}

struct PrefixPlan {
  Kind kind;        // of the prefix's part
  int shared, own;  // parts of the prefix and of the sequences' own rows
  int64_t rows;
  bool two;   // on the tensor cores: the queries are wanted as two bf16 parts
  bool both;  // few rows: the prefix's and the sequences' own rows in one launch
  size_t q32, q16, parts, bytes;
};

static PrefixPlan prefix_plan(const sfa_prefix_desc* d) {
  PrefixPlan p;
  const int G = d->Hq / d->Hkv;
  p.rows = (int64_t)d->B * d->Hq;
  p.kind = forward_kind(G * d->B, d->dtype);
  p.two = d->P && p.kind == kTensor;
  // In fp32 one kernel for both has the prefix's rows a CTA, 8 of more than 4, which costs more
  // than a launch over many own rows of fewer heads.  In one launch and apart: 8 x 16 / 4 heads
  // behind 1000, own rows of 100 12.4 and 18.7 us, of 1000 17.6 and 20.1, of 4000 30.3 and 24.3;
  // 8 x 8 / 2, 4000 20.3 and 23.1, 16000 52.4 and 41.0; 32 x 8 / 8, 100 18.1 and 19.5, 1000 53.7
  // and 42.9; up to 4 rows (4 x 8 / 8), 4000 20.1 and 21.8, 16000 59.7 and 60.0; more than 4 heads
  // (4 x 64 / 8), 16000 85.7 and 88.8.
  p.both = d->P && p.kind == kFewRows &&
           (d->dtype == SFA_BF16 || G > 4 || G * d->B <= 4 || (int64_t)d->B * d->Hkv * d->T <= 1 << 16);
  p.shared = !d->P ? 0 : p.two ? 1 : forward_splits(d->Hkv, G, d->B, d->P, p.kind, d->dtype, true);
  p.own = forward_splits((int64_t)d->B * d->Hkv, G, 1, d->T, kFewRows, d->dtype, true);
  p.q32 = align256((size_t)p.rows * kD * sizeof(float));
  p.q16 = p.two ? align256((size_t)p.rows * kD * 2 * sizeof(bf16)) : 0;
  p.parts = part_bytes(p.shared + p.own, p.rows);
  p.bytes = p.q32 + p.q16 + p.parts + (p.two ? cross_tc_bytes(1, d->Hkv, G, d->B, d->P) : 0);
  return p;
}

}  // namespace sfa

using namespace sfa;

extern "C" {

int sfa_cross_workspace_size(const sfa_cross_desc* d, int backward, size_t* bytes) {
  if (!bytes) return SFA_ERR_INVALID_ARG;
  const int rc = check_cross(d);
  if (rc != SFA_OK) return rc;
  if (backward) {
    *bytes = backward_plan(d).bytes;
  } else {
    *bytes = forward_plan(d).bytes;
  }
  return SFA_OK;
}

int sfa_cross_forward(const sfa_cross_desc* d, const void* q, const void* k, const void* v, void* o, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
  int rc = check_cross(d);
  if (rc != SFA_OK) return rc;
  if (!q || !k || !v || !o || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return SFA_ERR_INVALID_ARG;
  const ForwardPlan p = forward_plan(d);
  if (p.bytes && (!ws || !aligned(ws, 16))) return SFA_ERR_INVALID_ARG;
  if (ws_bytes < p.bytes) return SFA_ERR_CAPACITY;
  CrossArgs a;
  if ((rc = cross_args(d, &a)) != SFA_OK) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  if (p.kind == kTensor) return launch_cross_fwd_tc(a, ws, stream);
  a.splits = p.splits;
  a.cluster = p.cluster;
  a.parts = a.splits > 1 && !a.cluster;
  if (a.parts) set_parts(&a, static_cast<char*>(ws), a.splits, a.rows, 0);
  rc = p.kind == kFewRows ? launch_cross_stream(a, false, d->dtype, stream) : launch_cross_fwd_f32(a, stream);
  return rc != SFA_OK || !a.parts ? rc : launch_cross_join(a, d->dtype, nullptr, 0, stream);
}

int sfa_cross_backward(const sfa_cross_desc* d, const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                       void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_cross(d);
  if (rc != SFA_OK) return rc;
  const void* ptrs[] = {q, k, v, o, dO, dq, dk, dv, ws};
  for (const void* x : ptrs)
    if (!x || !aligned(x, 16)) return SFA_ERR_INVALID_ARG;
  if (!lse || !aligned(lse, 4)) return SFA_ERR_INVALID_ARG;
  const BackwardPlan p = backward_plan(d);
  if (ws_bytes < p.bytes) return SFA_ERR_CAPACITY;
  CrossArgs a;
  if ((rc = cross_args(d, &a)) != SFA_OK) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = o;
  a.lse = const_cast<float*>(lse);  // read only
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  if (d->dtype == SFA_BF16) return launch_cross_bwd_tc(a, ws, stream);
  float2* const stat = static_cast<float2*>(ws);
  float* const parts = reinterpret_cast<float*>(static_cast<char*>(ws) + p.stat);
  {
    LaunchTimer tm(SFA_KERNEL_CROSS_STAT, stream);
    if (launch_pdl(cross_stat_kernel, dim3((unsigned)((p.rows + 31) / 32)), dim3(256), 0, (cudaStream_t)stream, a, stat) != cudaSuccess)
      return SFA_ERR_CUDA;
  }
  a.stat = stat;
  CrossArgs kv = a;
  a.splits = p.dq_splits;
  a.parts = a.splits > 1;
  a.part_a = parts;
  kv.splits = p.dkv_splits;
  kv.parts = kv.splits > 1;
  kv.part_a = parts + p.dq_parts;
  kv.part_b = kv.part_a + (size_t)kv.splits * p.keys * kD;
  if ((rc = launch_cross_bwd_f32(a, kv, stream)) != SFA_OK || (!a.parts && !kv.parts)) return rc;
  const int64_t n = a.parts ? p.rows * kD : 0, m = kv.parts ? p.keys * kD : 0;
  const SumArgs sums = {{a.part_a, kv.part_a, kv.part_b},
                        {static_cast<float*>(dq), static_cast<float*>(dk), static_cast<float*>(dv)},
                        {n, m, m},
                        {a.splits, kv.splits, kv.splits}};
  LaunchTimer tm(SFA_KERNEL_CROSS_JOIN, stream);
  const dim3 grid((unsigned)(((n > m ? n : m) / 4 + 255) / 256), 3);
  return launch_pdl(cross_sum_kernel, grid, dim3(256), 0, (cudaStream_t)stream, sums) == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

int sfa_prefix_workspace_size(const sfa_prefix_desc* d, size_t* bytes) {
  if (!bytes) return SFA_ERR_INVALID_ARG;
  const int rc = check_prefix(d);
  if (rc != SFA_OK) return rc;
  *bytes = prefix_plan(d).bytes;
  return SFA_OK;
}

int sfa_prefix_decode(const sfa_prefix_desc* d, const void* q, const void* k_new, const void* v_new, const void* prefix_k,
                      const void* prefix_v, void* k_cache, void* v_cache, const int32_t* pos, void* o, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
  int rc = check_prefix(d);
  if (rc != SFA_OK) return rc;
  if (!q || !k_cache || !v_cache || !pos || !o || !ws || !k_new != !v_new || (d->P && (!prefix_k || !prefix_v))) return SFA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k_new, v_new, prefix_k, prefix_v, k_cache, v_cache, o, ws};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return SFA_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(lse, 4)) return SFA_ERR_INVALID_ARG;
  const PrefixPlan p = prefix_plan(d);
  if (ws_bytes < p.bytes) return SFA_ERR_CAPACITY;
  CrossArgs a = {};
  wait_injection(&a.wait_cycles, &a.debug_skip);
  if ((rc = device_status(&a.status)) != SFA_OK) return rc;
  char* const w = static_cast<char*>(ws);
  char* const parts = w + p.q32 + p.q16;
  PrefixArgs x = {q, k_new, v_new, d->q_stride, d->k_stride, d->v_stride, k_cache, v_cache, pos, reinterpret_cast<const float2*>(d->rope),
                  reinterpret_cast<float*>(w), p.two ? reinterpret_cast<bf16*>(w + p.q32) : nullptr, d->B, d->P, d->T, d->Hq, d->Hkv, a.status};
  {
    LaunchTimer tm(SFA_KERNEL_CROSS_STAT, stream);
    const int64_t heads = (int64_t)d->B * (d->Hq + (k_new ? 2 * d->Hkv : 0));
    const dim3 grid((unsigned)((heads + 3) / 4));
    const cudaError_t e = d->dtype == SFA_BF16 ? launch_pdl(prefix_prep_kernel<bf16>, grid, dim3(128), 0, (cudaStream_t)stream, x)
                                               : launch_pdl(prefix_prep_kernel<float>, grid, dim3(128), 0, (cudaStream_t)stream, x);
    if (e != cudaSuccess) return SFA_ERR_CUDA;
  }
  a.rows = p.rows;
  a.q = x.q32;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.G = d->Hq / d->Hkv;
  a.parts = true;
  if (d->P) {  // the batch as one sequence of B queries
    a.B = 1;
    a.Tq = d->B;
    a.Tk = d->P;
    a.qs = {p.rows * kD, kD, (int64_t)d->Hq * kD};
    if (p.two) a.q = x.q16;
    a.ks = {0, d->prefix_k_stride, kD};
    a.vs = {0, d->prefix_v_stride, kD};
    a.rs = {0, 1, d->Hq};
    a.k = prefix_k;
    a.v = prefix_v;
    a.splits = p.shared;
    set_parts(&a, parts, p.shared + p.own, p.rows, 0);
    if (p.two)
      rc = launch_prefix_tc(a, parts + p.parts, stream);
    else if (p.kind == kFp32)
      rc = launch_cross_fwd_f32(a, stream);
    else if (!p.both)
      rc = launch_cross_stream(a, true, d->dtype, stream);
    if (rc != SFA_OK) return rc;
  }
  const CrossArgs prefix = a;
  a.q = x.q32;
  a.B = d->B;
  a.Tq = 1;
  a.Tk = d->T;
  a.qs = {(int64_t)d->Hq * kD, kD, kD};
  a.ks = a.vs = {(int64_t)d->Hkv * d->T * kD, (int64_t)d->T * kD, kD};
  a.rs = {d->Hq, 1, 1};
  a.k = k_cache;
  a.v = v_cache;
  a.kv_len = pos;
  a.kv_add = 1;
  a.splits = p.own;
  set_parts(&a, parts, p.shared + p.own, p.rows, p.shared);
  rc = p.both ? launch_cross_stream_two(prefix, a, d->dtype, stream) : launch_cross_stream(a, true, d->dtype, stream);
  if (rc != SFA_OK) return rc;
  a.o = o;
  a.lse = lse;
  set_parts(&a, parts, p.shared + p.own, p.rows, 0);
  if (p.two) return launch_prefix_join(prefix, a, parts + p.parts, pos, d->T, stream);
  a.splits = p.shared + p.own;
  return launch_cross_join(a, d->dtype, pos, d->T, stream);
}

}  // extern "C"
