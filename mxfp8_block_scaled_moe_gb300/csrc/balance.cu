// The router's load-balance loss, the per-expert counts and the gradient of
// the logits.
//
//   p_te = softmax of logits[t, :]                      fp32
//   n    = tokens with mask[t] != 0 (all of them without a mask)
//   c_e  = assignments of those tokens to expert e (or the caller's counts,
//          e.g. summed over micro-batches);  f_e = c_e / sum_e c_e
//   loss = coef * E * sum_e f_e * (1/n) sum_t p_te
//   dlogits[t, e] = coef * E / n * p_te * (f_e - sum_j p_tj f_j), 0 if masked
//
// f is a constant of the gradient (the counts are not differentiable).  Both
// results need the same per-token dot product s_t = sum_j p_tj f_j (the loss
// is coef * E / n * sum_t s_t), so one pass over the logits serves both:
// every logit is read once and every gradient written once.
//
//   1. balance_count_kernel: histograms in shared memory, one per CTA, added
//      over a cluster's CTAs through distributed shared memory; one partial
//      histogram per cluster (at most 18) goes to the workspace.
//   2. balance_rows_kernel: every CTA adds the partial histograms into f (CTA 0
//      writes the counts), then a warp per token; each CTA leaves the sum of
//      its tokens' s_t, and the last CTA to finish adds those in CTA order, so
//      the loss does not depend on the order in which the CTAs run.
// Up to 1024 tokens one cluster does both (balance_small_kernel): one launch,
// no workspace.
//
// A logit of -inf has p = 0; a row of -inf only has p = 0 throughout.  NaN
// (or +inf) in a row that is not masked reaches the loss and that row.
//
// Roofline: HBM-bound for many tokens (4 E bytes read, 4 E written per token).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "topk.cuh"

namespace mxmoe {
namespace balance {

constexpr int kErrDeviceCheck = 8;  // MXMOE_ERR_DEVICE_CHECK
constexpr int kMaxE = 1024;
constexpr int kCluster = 8;
constexpr int kCountThreads = 512;
constexpr int kRowThreads = 256;
constexpr int kSmallThreads = 512;
constexpr int64_t kSmallTokens = 1024;

// Workspace, in 4-byte words: the CTA ticket, pad, then for each cluster of
// the count kernel its token count and histogram [E], then (8-byte aligned)
// the row CTAs' sums.
constexpr int kOffPart = 2;
__host__ __device__ inline int off_sums(int E, int clusters) {
  return (kOffPart + clusters * (E + 1) + 1) / 2 * 2;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_cluster_s32(const int* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), ra;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
  return v;
}

__device__ __forceinline__ double ld_cluster_f64(const double* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), ra;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(ra) : "memory");
  return v;
}

// Histogram of the ids of tokens [t0, t1) into hist (shared memory, zeroed) and
// their number into *n: a thread per token.  v4: four ids per load.
__device__ __forceinline__ void count_tokens(const int32_t* __restrict__ ids,
                                             const uint8_t* __restrict__ mask, int64_t t0,
                                             int64_t t1, int E, int k, bool v4, int* hist, int* n,
                                             int* status) {
  int live = 0;
  bool bad = false;
  auto one = [&](int e) {
    if (e < 0 || e >= E) bad = true;
    else atomicAdd(&hist[e], 1);
  };
  for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    if (mask && mask[t] == 0) continue;
    ++live;
    const int32_t* row = ids + t * k;
    if (v4) {
      for (int j = 0; j < k; j += 4) {
        const int4 e = __ldg(reinterpret_cast<const int4*>(row + j));
        one(e.x);
        one(e.y);
        one(e.z);
        one(e.w);
      }
    } else {
      for (int j = 0; j < k; ++j) one(__ldg(row + j));
    }
  }
  if (live) atomicAdd(n, live);
  if (bad) report_error(status, kErrDeviceCheck);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         int64_t T, int E, int k, bool v4, uint32_t* __restrict__ ws,
                         int* status) {
  __shared__ int s_hist[kMaxE + 1];  // [E]: the token count
  const uint32_t rank = cluster_rank();
  for (int e = threadIdx.x; e <= E; e += kCountThreads) s_hist[e] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const int64_t per = (T + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = min(T, blockIdx.x * per), t1 = min(T, t0 + per);
  count_tokens(ids, mask, t0, t1, E, k, v4, s_hist, &s_hist[E], status);
  __syncthreads();
  cluster_sync();
  // this CTA's share of the bins, added over the cluster (integers: any order)
  int* part = reinterpret_cast<int*>(ws) + kOffPart + (blockIdx.x / kCluster) * (E + 1);
  for (int e = rank + kCluster * threadIdx.x; e <= E; e += kCluster * kCountThreads) {
    int c = 0;
    for (int r = 0; r < kCluster; ++r) c += ld_cluster_s32(&s_hist[e], r);
    part[e] = c;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) ws[0] = 0;
  cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// Where a lane keeps expert i of its EPL: lane + 32 i, or with kGroup (E a
// multiple of 4) groups of four, 4 lane + i % 4 + 128 (i / 4).  The place
// depends on E alone and v4 (16-byte rows) only on how it is read, so the sums
// and their bits do not depend on a tensor's alignment.
template <bool kGroup>
__device__ __forceinline__ int expert_at(int lane, int i) {
  return kGroup ? 4 * lane + (i & 3) + 128 * (i >> 2) : lane + 32 * i;
}
template <int EPL, bool kGroup>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, bool v4,
                                         float (&v)[EPL]) {
  if (kGroup && v4) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      float4 u = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (expert_at<true>(lane, i) < E)
        u = __ldcs(reinterpret_cast<const float4*>(row + expert_at<true>(lane, i)));
      v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      v[i] = expert_at<kGroup>(lane, i) < E ? __ldcs(row + expert_at<kGroup>(lane, i)) : -INFINITY;
  }
}

// The warp's walk over tokens t, t + step, ... < T.  c: the counts (f times their
// sum) of the lane's experts.
// The next token's logits are loaded before this one's arithmetic, the first
// ones by start().  sum() is the tokens' sum of s_t (times the counts' sum), the same on every lane: two
// fp32 words, the second the first one's rounding errors.
template <int EPL, bool kGroup>
struct RowWalk {
  static constexpr bool kAhead = EPL <= 16;  // (two rows of 32 would not fit in the registers)
  const float* logits;
  int64_t ldl;
  const uint8_t* mask;
  int64_t t, step, T;
  int E, lane;
  bool v4;
  float v[EPL];
  bool live;
  float sum_hi, sum_lo;

  __device__ __forceinline__ void load(int64_t at, float (&x)[EPL], bool& l) {
    l = !mask || mask[at] != 0;
    if (l) load_row<EPL, kGroup>(logits + at * ldl, E, lane, v4, x);
  }
  __device__ __forceinline__ void start() {
    live = false;
    sum_hi = sum_lo = 0.f;
    if (kAhead && t < T) load(t, v, live);
  }
  __device__ __forceinline__ void walk(const float (&c)[EPL], float scale, float* dlogits) {
    float w[EPL];
    bool live_next = false;
    for (; t < T; t += step) {  // warp-uniform
      if (!kAhead) load(t, v, live);
      else if (t + step < T) load(t + step, w, live_next);
      if (live) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (m == -INFINITY) m = 0.f;  // an empty row: every exp below is 0 (NaN stays NaN)
        float z = 0.f, s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          v[i] = __expf(v[i] - m);
          z += v[i];
          s = fmaf(v[i], c[i], s);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          z += __shfl_xor_sync(0xffffffffu, z, off);
          s += __shfl_xor_sync(0xffffffffu, s, off);
        }
        const float iz = z == 0.f ? 0.f : 1.f / z;
        s *= iz;
        const float h = __fadd_rn(sum_hi, s);
        sum_lo = __fadd_rn(sum_lo, two_sum_err(sum_hi, s, h));
        sum_hi = h;
        const float g = scale * iz;
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = g * v[i] * (c[i] - s);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = 0.f;
      }
      if (dlogits) {
        float* out = dlogits + t * E;
        if (kGroup && v4) {
#pragma unroll
          for (int i = 0; i < EPL; i += 4)
            if (expert_at<true>(lane, i) < E)
              __stcs(reinterpret_cast<float4*>(out + expert_at<true>(lane, i)),
                     make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (expert_at<kGroup>(lane, i) < E) __stcs(out + expert_at<kGroup>(lane, i), v[i]);
        }
      }
      if (kAhead) {
        live = live_next;
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = w[i];
      }
    }
  }
  __device__ __forceinline__ double sum() const { return (double)sum_hi + (double)sum_lo; }
};

// The counts the loss uses, c of the lane's experts in fp32 (given: loaded by
// load_given before the own counts are known), and coef * E / (n sum c).  The
// rows work on c instead of f = c / sum c; this factor brings the sum back, so
// no CTA divides E times and none waits for another's total.
template <int EPL, bool kGroup>
__device__ __forceinline__ void load_given(const int64_t* __restrict__ counts_in, int E, int lane,
                                           float (&c)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_at<kGroup>(lane, i);
    c[i] = counts_in && e < E ? (float)__ldg(counts_in + e) : 0.f;
  }
}
template <int EPL, bool kGroup>
__device__ __forceinline__ float loss_scale(const int* s_cnt, bool given, int E, int lane,
                                            float coef, float (&c)[EPL]) {
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_at<kGroup>(lane, i);
    if (!given && e < E) c[i] = (float)s_cnt[e];
    total += c[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  const float n = (float)s_cnt[E];
  return n > 0.f && total > 0.f ? coef * (float)E / n / total : 0.f;
}

template <int EPL, bool kGroup>
__global__ void __launch_bounds__(kRowThreads)
    balance_rows_kernel(const float* __restrict__ logits, int64_t ldl,
                        const uint8_t* __restrict__ mask, const int64_t* __restrict__ counts_in,
                        int64_t T, int E, float coef, float* __restrict__ loss,
                        int64_t* __restrict__ counts, float* __restrict__ dlogits,
                        uint32_t* __restrict__ ws, int clusters, bool row4) {
  __shared__ double s_sum[kRowThreads / 32];
  __shared__ int s_cnt[kMaxE + 1];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  RowWalk<EPL, kGroup> rows = {logits, ldl, mask, (int64_t)blockIdx.x * (kRowThreads / 32) + warp,
                               (int64_t)gridDim.x * (kRowThreads / 32), T, E, lane, row4};
  rows.start();
  float c[EPL];
  load_given<EPL, kGroup>(counts_in, E, lane, c);
  const int* part = reinterpret_cast<const int*>(ws) + kOffPart;
  for (int e = threadIdx.x; e <= E; e += kRowThreads) {
    int sum = 0;
#pragma unroll 6
    for (int j = 0; j < clusters; ++j) sum += __ldcg(part + j * (E + 1) + e);
    s_cnt[e] = sum;
    if (blockIdx.x == 0 && e < E) counts[e] = sum;
  }
  __syncthreads();
  const float scale = loss_scale<EPL, kGroup>(s_cnt, counts_in != nullptr, E, lane, coef, c);
  rows.walk(c, scale, dlogits);
  if (lane == 0) s_sum[warp] = rows.sum();
  __syncthreads();
  double* sums = reinterpret_cast<double*>(ws + off_sums(E, clusters));
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kRowThreads / 32; ++w) a += s_sum[w];
    sums[blockIdx.x] = a;
    __threadfence();
    s_last = atomicAdd(&ws[0], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (warp == 0) {
    double a = 0.0;
    for (int b = lane; b < (int)gridDim.x; b += 32) a += __ldcg(&sums[b]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    if (lane == 0) *loss = scale == 0.f ? 0.f : (float)((double)scale * a);
  }
}

// Few tokens: one cluster counts, then walks the rows; the CTAs' histograms and
// sums meet through distributed shared memory.
template <int EPL, bool kGroup>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSmallThreads)
    balance_small_kernel(const float* __restrict__ logits, int64_t ldl,
                         const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         const int64_t* __restrict__ counts_in, int64_t T, int E, int k, bool v4,
                         float coef, float* __restrict__ loss, int64_t* __restrict__ counts,
                         float* __restrict__ dlogits, bool row4, int* status) {
  constexpr int kWarps = kSmallThreads / 32;
  __shared__ double s_sum[kWarps];
  __shared__ double s_cta;
  __shared__ int s_hist[kMaxE + 1], s_cnt[kMaxE + 1];
  const uint32_t rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= E; e += kSmallThreads) s_hist[e] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const int64_t per = (T + kCluster - 1) / kCluster;
  const int64_t t0 = min(T, rank * per), t1 = min(T, t0 + per);
  RowWalk<EPL, kGroup> rows = {logits, ldl, mask, t0 + warp, kWarps, t1, E, lane, row4};
  rows.start();
  float c[EPL];
  load_given<EPL, kGroup>(counts_in, E, lane, c);
  count_tokens(ids, mask, t0, t1, E, k, v4, s_hist, &s_hist[E], status);
  __syncthreads();
  cluster_sync();
  for (int e = threadIdx.x; e <= E; e += kSmallThreads) {
    int sum = 0;
    for (int r = 0; r < kCluster; ++r) sum += ld_cluster_s32(&s_hist[e], r);
    s_cnt[e] = sum;
    if (rank == 0 && e < E) counts[e] = sum;
  }
  __syncthreads();
  const float scale = loss_scale<EPL, kGroup>(s_cnt, counts_in != nullptr, E, lane, coef, c);
  rows.walk(c, scale, dlogits);
  if (lane == 0) s_sum[warp] = rows.sum();
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kWarps; ++w) a += s_sum[w];
    s_cta = a;
  }
  __syncthreads();
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    double a = 0.0;
    for (int r = 0; r < kCluster; ++r) a += ld_cluster_f64(&s_cta, r);
    *loss = scale == 0.f ? 0.f : (float)((double)scale * a);
  }
  cluster_sync();
}

static int row_blocks(int64_t T) {
  return (int)std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(T, kRowThreads / 32), 4 * (int64_t)num_sms()));
}
// Clusters of the count kernel: 512 tokens per CTA, at most one CTA per SM.
static int count_clusters(int64_t T) {
  const int64_t most = std::max(1, num_sms() / kCluster - 1);
  return (int)std::max<int64_t>(1, std::min(most, ceil_div(T, kCluster * kCountThreads)));
}

struct Args {
  const float* logits;
  int64_t ldl;
  const int32_t* ids;
  const uint8_t* mask;
  const int64_t* counts_in;
  int64_t T;
  int E, k;
  bool v4, row4;  // 16-byte aligned rows of ids, of logits and dlogits
  float coef;
  float* loss;
  int64_t* counts;
  float* dlogits;
  uint32_t* ws;
};

template <int EPL, bool kGroup>
static cudaError_t launch(const Args& a, cudaStream_t stream) {
  int* st = device_status_ptr();
  if (a.T <= kSmallTokens)
    return launch_pdl(balance_small_kernel<EPL, kGroup>, dim3(kCluster), dim3(kSmallThreads), 0,
                      stream, a.logits, a.ldl, a.ids, a.mask, a.counts_in, a.T, a.E, a.k, a.v4,
                      a.coef, a.loss, a.counts, a.dlogits, a.row4, st);
  const int clusters = count_clusters(a.T);
  const cudaError_t err =
      launch_pdl(balance_count_kernel, dim3(clusters * kCluster), dim3(kCountThreads), 0, stream,
                 a.ids, a.mask, a.T, a.E, a.k, a.v4, a.ws, st);
  if (err != cudaSuccess) return err;
  return launch_pdl(balance_rows_kernel<EPL, kGroup>, dim3(row_blocks(a.T)), dim3(kRowThreads), 0,
                    stream, a.logits, a.ldl, a.mask, a.counts_in, a.T, a.E, a.coef, a.loss,
                    a.counts, a.dlogits, a.ws, clusters, a.row4);
}

}  // namespace balance

size_t balance_workspace_bytes(int64_t T, int E) {
  using namespace balance;
  if (T <= kSmallTokens) return 0;
  return (size_t)off_sums(E, count_clusters(T)) * 4 + (size_t)row_blocks(T) * sizeof(double);
}

cudaError_t launch_balance_loss(const float* logits, int64_t ldl, const int32_t* ids,
                                const uint8_t* mask, const int64_t* counts_in, int64_t T, int E,
                                int k, float coef, float* loss, int64_t* counts, float* dlogits,
                                uint32_t* ws, cudaStream_t stream) {
  using namespace balance;
  const bool v4 = k % 4 == 0 && ((uintptr_t)ids & 15u) == 0;
  const bool row4 = E % 4 == 0 && ldl % 4 == 0 &&
                    (((uintptr_t)logits | (uintptr_t)dlogits) & 15u) == 0;
  const Args a = {logits, ldl,  ids,  mask, counts_in, T,       E, k,
                  v4,     row4, coef, loss, counts,    dlogits, ws};
  const int epl = (E + 31) / 32;
  if (E % 4 == 0 && E > 64) {
    if (epl <= 4) return launch<4, true>(a, stream);
    if (epl <= 8) return launch<8, true>(a, stream);
    if (epl <= 16) return launch<16, true>(a, stream);
    return launch<32, true>(a, stream);
  }
  if (epl <= 1) return launch<1, false>(a, stream);
  if (epl <= 2) return launch<2, false>(a, stream);
  if (epl <= 4) return launch<4, false>(a, stream);
  if (epl <= 8) return launch<8, false>(a, stream);
  if (epl <= 16) return launch<16, false>(a, stream);
  return launch<32, false>(a, stream);
}

}  // namespace mxmoe
