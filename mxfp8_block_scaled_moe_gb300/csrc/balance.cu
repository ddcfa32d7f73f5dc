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
//      writes the counts), then a warp takes 1 to 32
//      tokens at a time (8 experts a lane); each CTA leaves the sum of its
//      tokens' s_t, and the last CTA to finish adds those in CTA order, so the
//      loss does not depend on the order in which the CTAs run.
// For few tokens one cluster does both (balance_small_kernel): one launch,
// no workspace.
//
// A logit of -inf has p = 0; a row of -inf only has p = 0 throughout.  NaN
// (or +inf) in a row that is not masked reaches the loss and that row.
//
// Bound by HBM for many tokens (4 E bytes read, 4 E written per token): 65536 x
// 256, k = 8, takes 33.0 us, 4.1 TB/s, of which the count kernel, the second launch, the
// partial histograms and the last CTA's sum are 14 us whatever T (with nothing in the row
// loop); 16384 x 128 takes 13.3 us, 64 x 8 (one launch) 4.5 us.
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
constexpr int kRowThreads = 512;
constexpr int kSmallThreads = 512;

// One cluster, one launch: while its 128 warps have few tokens and experts to walk.
// (us, one cluster against two launches: 1024 x 128 9.2 / 8.9, 768 x 256 10.0 / 9.7, 256 x
// 1024 15.4 / 15.5; 1024 x 1024 25.9 / 15.5.)
static bool is_small(int64_t T, int E) { return T <= 1024 && T * E <= 196608; }

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

// A token takes G lanes of a warp (32 / G tokens side by side), EPL experts each: E
// <= G EPL.  Where lane l of them keeps expert i: l + G i, or with kQuad (E a multiple
// of 4) groups of four, 4 l + i % 4 + 4 G (i / 4).  The place depends on E alone and
// v4 (16-byte rows) only on how it is read, so the sums and their bits do not depend
// on a tensor's alignment.
template <int G, bool kQuad>
__device__ __forceinline__ int expert_at(int l, int i) {
  return kQuad ? 4 * l + (i & 3) + 4 * G * (i >> 2) : l + G * i;
}
template <int G, int EPL, bool kQuad>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, bool v4,
                                         float (&v)[EPL]) {
  if (kQuad && v4) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const int e = expert_at<G, true>(l, i);
      float4 u = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) u = __ldcs(reinterpret_cast<const float4*>(row + e));
      v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = expert_at<G, kQuad>(l, i);
      v[i] = e < E ? __ldcs(row + e) : -INFINITY;
    }
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A warp's walk over tokens: those of t, t + step, ... < T (t: the lane's own, the
// first of them the same distance from the warp's first).  c: the counts (f times
// their sum) of the lane's experts.  The next tokens' logits are loaded before these
// ones' arithmetic, the first ones by start().  A masked token, and one past T, is a
// row of -inf: p = 0 throughout.  sum_to() gives the sum of s_t (times the counts' sum) over
// the warp's tokens, kept in two fp32 words, the second the first one's rounding
// errors.
template <int G, int EPL, bool kQuad>
struct RowWalk {
  static constexpr bool kAhead = EPL <= 16;  // (two rows of 32 would not fit in the registers)
  const float* logits;
  int64_t ldl;
  const uint8_t* mask;
  int64_t t, step, T;
  int E;
  bool v4;
  int sub, l;  // the lane's token of the warp's, and its lane of the token's
  float v[EPL];
  float sum_hi, sum_lo;

  __device__ __forceinline__ void load(int64_t at, float (&x)[EPL]) {
    if (at < T && (!mask || mask[at] != 0)) {
      load_row<G, EPL, kQuad>(logits + at * ldl, E, l, v4, x);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = -INFINITY;
    }
  }
  // first: the warp's first token
  __device__ __forceinline__ void start(int64_t first) {
    const int lane = threadIdx.x & 31;
    sub = lane / G;
    l = lane % G;
    t = first;
    sum_hi = sum_lo = 0.f;
    if (kAhead) load(t + sub, v);
  }
  __device__ __forceinline__ void walk(const float (&c)[EPL], float scale, float* dlogits) {
    float w[EPL];
    for (; t < T; t += step) {  // warp-uniform
      if (!kAhead) load(t + sub, v);
      else load(t + step + sub, w);
      float m = v[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
#pragma unroll
      for (int off = G / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (m == -INFINITY) m = 0.f;  // an empty row: every exp below is 0 (NaN stays NaN)
      float z = 0.f, s = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        v[i] = __expf(v[i] - m);
        z += v[i];
        s = fmaf(v[i], c[i], s);
      }
      z = group_sum<G>(z);
      s = group_sum<G>(s);
      const float iz = z == 0.f ? 0.f : 1.f / z;
      s *= iz;
      const float h = __fadd_rn(sum_hi, s);
      sum_lo = __fadd_rn(sum_lo, two_sum_err(sum_hi, s, h));
      sum_hi = h;
      const float g = scale * iz;
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = g * v[i] * (c[i] - s);
      if (dlogits && t + sub < T) {
        float* out = dlogits + (t + sub) * E;
        if (kQuad && v4) {
#pragma unroll
          for (int i = 0; i < EPL; i += 4) {
            const int e = expert_at<G, true>(l, i);
            if (e < E)
              __stcs(reinterpret_cast<float4*>(out + e),
                     make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const int e = expert_at<G, kQuad>(l, i);
            if (e < E) __stcs(out + e, v[i]);
          }
        }
      }
      if (kAhead) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = w[i];
      }
    }
  }
  // (fp64 adds are slow here: one per warp, on lane 0)
  __device__ __forceinline__ void sum_to(double* out) {
#pragma unroll
    for (int off = G; off < 32; off <<= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, sum_hi, off);
      const float lo = __shfl_xor_sync(0xffffffffu, sum_lo, off);
      const float h = __fadd_rn(sum_hi, hi);
      sum_lo = __fadd_rn(__fadd_rn(sum_lo, lo), two_sum_err(sum_hi, hi, h));
      sum_hi = h;
    }
    if ((threadIdx.x & 31) == 0) *out = (double)sum_hi + (double)sum_lo;
  }
};

// The counts the loss uses, c of the lane's experts in fp32 (given: loaded by
// load_given before the own counts are known), and coef * E / (n sum c).  The
// rows work on c instead of f = c / sum c; this factor brings the sum back, so
// no CTA divides E times and none waits for another's total.
template <int G, int EPL, bool kQuad>
__device__ __forceinline__ void load_given(const int64_t* __restrict__ counts_in, int E,
                                           float (&c)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_at<G, kQuad>((int)(threadIdx.x % G), i);
    c[i] = counts_in && e < E ? (float)__ldg(counts_in + e) : 0.f;
  }
}
template <int G, int EPL, bool kQuad>
__device__ __forceinline__ float loss_scale(const int* s_cnt, bool given, int E, float coef,
                                            float (&c)[EPL]) {
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_at<G, kQuad>((int)(threadIdx.x % G), i);
    if (!given && e < E) c[i] = (float)s_cnt[e];
    total += c[i];
  }
  total = group_sum<G>(total);
  const float n = (float)s_cnt[E];
  return n > 0.f && total > 0.f ? coef * (float)E / n / total : 0.f;
}

template <int G, int EPL, bool kQuad>
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
  constexpr int64_t kTokens = 32 / G;  // of a warp at a time
  const int64_t first = ((int64_t)blockIdx.x * (kRowThreads / 32) + warp) * kTokens;
  RowWalk<G, EPL, kQuad> rows = {
      logits, ldl, mask, first, (int64_t)gridDim.x * (kRowThreads / 32) * kTokens, T, E, row4};
  rows.start(first);
  float c[EPL];
  load_given<G, EPL, kQuad>(counts_in, E, c);
  const int* part = reinterpret_cast<const int*>(ws) + kOffPart;
  for (int e = threadIdx.x; e <= E; e += kRowThreads) {
    int sum = 0;
#pragma unroll 6
    for (int j = 0; j < clusters; ++j) sum += __ldcg(part + j * (E + 1) + e);
    s_cnt[e] = sum;
    if (blockIdx.x == 0 && e < E) counts[e] = sum;
  }
  __syncthreads();
  const float scale = loss_scale<G, EPL, kQuad>(s_cnt, counts_in != nullptr, E, coef, c);
  rows.walk(c, scale, dlogits);
  rows.sum_to(&s_sum[warp]);
  __syncthreads();
  double* sums = reinterpret_cast<double*>(ws + off_sums(E, clusters));
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kRowThreads / 32; ++w) a += s_sum[w];
    sums[blockIdx.x] = a;
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(&ws[0])
                 : "memory");
    s_last = before == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
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
template <int G, int EPL, bool kQuad>
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
  const int64_t first = t0 + warp * (32 / G);
  RowWalk<G, EPL, kQuad> rows = {logits, ldl, mask, first, kWarps * (32 / G), t1, E, row4};
  rows.start(first);
  float c[EPL];
  load_given<G, EPL, kQuad>(counts_in, E, c);
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
  const float scale = loss_scale<G, EPL, kQuad>(s_cnt, counts_in != nullptr, E, coef, c);
  rows.walk(c, scale, dlogits);
  rows.sum_to(&s_sum[warp]);
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

// Lanes of a token: 8 experts each up to E = 256, all 32 lanes from there on.  (A warp
// per token: 65536 x 16, 60 and 16384 x 128 took 24.5, 26.7 and 13.3 us, against 12.0, 15.3 and
// 13.6.)
static int lanes_of(int E) {
  int g = 1;
  while (g < 32 && 8 * g < E) g *= 2;
  return g;
}
// Two CTAs of 512 threads per SM: half the tickets of four CTAs of 256 (the tickets and
// the last CTA's sum take 4 us with those: 15.2 us at 16384 x 128, 13.3 with these).
// Above 256 experts a thread's registers leave room for one.
static int row_blocks(int64_t T, int E) {
  return (int)std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(T * lanes_of(E), kRowThreads),
                               (E > 256 ? 1 : 2) * (int64_t)num_sms()));
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

template <int EPL, bool kQuad>
static cudaError_t launch_small(const Args& a, cudaStream_t stream) {
  return launch_pdl(balance_small_kernel<32, EPL, kQuad>, dim3(kCluster), dim3(kSmallThreads), 0,
                    stream, a.logits, a.ldl, a.ids, a.mask, a.counts_in, a.T, a.E, a.k, a.v4,
                    a.coef, a.loss, a.counts, a.dlogits, a.row4, device_status_ptr());
}
template <int G, int EPL, bool kQuad>
static cudaError_t launch_large(const Args& a, cudaStream_t stream) {
  const int clusters = count_clusters(a.T);
  const cudaError_t err =
      launch_pdl(balance_count_kernel, dim3(clusters * kCluster), dim3(kCountThreads), 0, stream,
                 a.ids, a.mask, a.T, a.E, a.k, a.v4, a.ws, device_status_ptr());
  if (err != cudaSuccess) return err;
  return launch_pdl(balance_rows_kernel<G, EPL, kQuad>, dim3(row_blocks(a.T, a.E)),
                    dim3(kRowThreads), 0, stream, a.logits, a.ldl, a.mask, a.counts_in, a.T, a.E,
                    a.coef, a.loss, a.counts, a.dlogits, a.ws, clusters, a.row4);
}

}  // namespace balance

size_t balance_workspace_bytes(int64_t T, int E) {
  using namespace balance;
  if (is_small(T, E)) return 0;
  return (size_t)off_sums(E, count_clusters(T)) * 4 + (size_t)row_blocks(T, E) * sizeof(double);
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
  const bool quad = E % 4 == 0;
  if (is_small(T, E)) {
    // one token per warp and as few experts per lane as there are: few rows wait for
    // one row's instructions (64 x 8: 4.5 us, and 5.7 with a lane per token)
    if (E <= 32) return launch_small<1, false>(a, stream);
    if (E <= 64) return launch_small<2, false>(a, stream);
    if (E <= 128) return quad ? launch_small<4, true>(a, stream) : launch_small<4, false>(a, stream);
    if (E <= 256) return quad ? launch_small<8, true>(a, stream) : launch_small<8, false>(a, stream);
    if (E <= 512)
      return quad ? launch_small<16, true>(a, stream) : launch_small<16, false>(a, stream);
    return quad ? launch_small<32, true>(a, stream) : launch_small<32, false>(a, stream);
  }
  if (E > 512)
    return quad ? launch_large<32, 32, true>(a, stream) : launch_large<32, 32, false>(a, stream);
  if (E > 256)
    return quad ? launch_large<32, 16, true>(a, stream) : launch_large<32, 16, false>(a, stream);
  switch (quad ? lanes_of(E) : -lanes_of(E)) {
    case 1: return launch_large<1, 8, true>(a, stream);
    case 2: return launch_large<2, 8, true>(a, stream);
    case 4: return launch_large<4, 8, true>(a, stream);
    case 8: return launch_large<8, 8, true>(a, stream);
    case 16: return launch_large<16, 8, true>(a, stream);
    case 32: return launch_large<32, 8, true>(a, stream);
    case -1: return launch_large<1, 8, false>(a, stream);
    case -2: return launch_large<2, 8, false>(a, stream);
    case -4: return launch_large<4, 8, false>(a, stream);
    case -8: return launch_large<8, 8, false>(a, stream);
    case -16: return launch_large<16, 8, false>(a, stream);
    default: return launch_large<32, 8, false>(a, stream);
  }
}

}  // namespace mxmoe
