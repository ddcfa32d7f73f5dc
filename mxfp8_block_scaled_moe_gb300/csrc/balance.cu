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
//   1. balance_count_kernel (one cluster): counts, n, f.
//   2. balance_rows_kernel: a warp per token; each CTA leaves the sum of its
//      tokens' s_t, and the last CTA to finish adds those in CTA order, so
//      the loss does not depend on the order in which the CTAs run.
//
// A logit of -inf has p = 0; a row of -inf only has p = 0 throughout.  NaN
// (or +inf) in a row that is not masked reaches the loss and that row.
//
// Roofline: HBM-bound for many tokens (4 E bytes read, 4 E written per token).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mxmoe {
namespace balance {

constexpr int kErrDeviceCheck = 8;  // MXMOE_ERR_DEVICE_CHECK
constexpr int kMaxE = 1024;
constexpr int kCluster = 8;
constexpr int kCountThreads = 1024;
constexpr int kRowThreads = 256;

// Workspace: n (int32), the CTA ticket (uint32), f [E], the CTAs' sums.
constexpr int kOffF = 4;  // in 4-byte words
__host__ __device__ inline int off_sums(int E) { return kOffF + (E + 3) / 4 * 4; }

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

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         const int64_t* __restrict__ counts_in, int64_t T, int E, int k,
                         int64_t* __restrict__ counts, uint32_t* __restrict__ ws, int* status) {
  __shared__ int s_hist[kMaxE];
  __shared__ int s_n;
  __shared__ unsigned long long s_total;
  const uint32_t rank = cluster_rank();
  for (int e = threadIdx.x; e < E; e += kCountThreads) s_hist[e] = 0;
  if (threadIdx.x == 0) { s_n = 0; s_total = 0; }
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const int64_t per = (T + kCluster - 1) / kCluster;
  const int64_t t0 = rank * per, t1 = min(T, t0 + per);
  int n = 0;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kCountThreads) n += !mask || mask[t] != 0;
  if (n) atomicAdd(&s_n, n);
  bool bad = false;
  for (int64_t i = t0 * k + threadIdx.x; i < t1 * k; i += kCountThreads) {
    if (mask && mask[i / k] == 0) continue;
    const int e = ids[i];
    if (e < 0 || e >= E) bad = true;
    else atomicAdd(&s_hist[e], 1);
  }
  if (bad) report_error(status, kErrDeviceCheck);
  __syncthreads();
  cluster_sync();
  if (rank == 0) {
    // every CTA's counts; the totals are integers, so the order is immaterial
    long long c[kMaxE / kCountThreads];
    long long mine = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / kCountThreads; ++i) {
      const int e = threadIdx.x + i * kCountThreads;
      c[i] = 0;
      if (e < E) {
        for (int r = 0; r < kCluster; ++r) c[i] += ld_cluster_s32(&s_hist[e], r);
        counts[e] = c[i];
        if (counts_in) c[i] = counts_in[e];
        mine += c[i];
      }
    }
    if (mine) atomicAdd(&s_total, (unsigned long long)mine);
    if (threadIdx.x == 0) {
      int all = 0;
      for (int r = 0; r < kCluster; ++r) all += ld_cluster_s32(&s_n, r);
      ws[0] = (uint32_t)all;
      ws[1] = 0;
    }
    __syncthreads();
    const long long total = (long long)s_total;
    float* f = reinterpret_cast<float*>(ws) + kOffF;
#pragma unroll
    for (int i = 0; i < kMaxE / kCountThreads; ++i) {
      const int e = threadIdx.x + i * kCountThreads;
      if (e < E) f[e] = total > 0 ? (float)((double)c[i] / (double)total) : 0.f;
    }
  }
  cluster_sync();  // no CTA leaves while rank 0 may still read its shared memory
}

// EPL experts per lane: lane + 32 i.
template <int EPL>
__global__ void __launch_bounds__(kRowThreads)
    balance_rows_kernel(const float* __restrict__ logits, int64_t ldl,
                        const uint8_t* __restrict__ mask, int64_t T, int E, float coef,
                        float* __restrict__ loss, float* __restrict__ dlogits,
                        uint32_t* __restrict__ ws) {
  __shared__ double s_sum[kRowThreads / 32];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const float* fs = reinterpret_cast<const float*>(ws) + kOffF;
  float f[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) f[i] = lane + 32 * i < E ? fs[lane + 32 * i] : 0.f;
  const int n = (int)ws[0];
  const float scale = n > 0 ? coef * (float)E / (float)n : 0.f;
  double sum = 0.0;
  for (int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32) + warp; t < T;
       t += (int64_t)gridDim.x * (kRowThreads / 32)) {
    float* out = dlogits ? dlogits + t * E : nullptr;
    if (mask && mask[t] == 0) {  // warp-uniform
      if (out)
        for (int e = lane; e < E; e += 32) out[e] = 0.f;
      continue;
    }
    const float* row = logits + t * ldl;
    float v[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = lane + 32 * i < E ? row[lane + 32 * i] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (m == -INFINITY) m = 0.f;  // an empty row: every exp below is 0 (NaN stays NaN)
    float z = 0.f, s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = __expf(v[i] - m);
      z += v[i];
      s = fmaf(v[i], f[i], s);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, off);
      s += __shfl_xor_sync(0xffffffffu, s, off);
    }
    const float iz = z == 0.f ? 0.f : 1.f / z;
    s *= iz;
    sum += s;
    if (out) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) out[lane + 32 * i] = scale * (v[i] * iz) * (f[i] - s);
    }
  }
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  double* sums = reinterpret_cast<double*>(ws + off_sums(E));
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kRowThreads / 32; ++w) a += s_sum[w];
    sums[blockIdx.x] = a;
    __threadfence();
    s_last = atomicAdd(&ws[1], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (warp == 0) {
    double a = 0.0;
    for (int b = lane; b < (int)gridDim.x; b += 32) a += __ldcg(&sums[b]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    if (lane == 0) *loss = n > 0 ? (float)((double)coef * E * a / n) : 0.f;
  }
}

static int row_blocks(int64_t T) {
  return (int)std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(T, kRowThreads / 32), 4 * (int64_t)num_sms()));
}

}  // namespace balance

size_t balance_workspace_bytes(int64_t T, int E) {
  return (size_t)balance::off_sums(E) * 4 + (size_t)balance::row_blocks(T) * sizeof(double);
}

cudaError_t launch_balance_loss(const float* logits, int64_t ldl, const int32_t* ids,
                                const uint8_t* mask, const int64_t* counts_in, int64_t T, int E,
                                int k, float coef, float* loss, int64_t* counts, float* dlogits,
                                uint32_t* ws, cudaStream_t stream) {
  using namespace balance;
  balance_count_kernel<<<kCluster, kCountThreads, 0, stream>>>(ids, mask, counts_in, T, E, k,
                                                               counts, ws, device_status_ptr());
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const int epl = (E + 31) / 32;
  auto kern = epl <= 1   ? balance_rows_kernel<1>
              : epl <= 2 ? balance_rows_kernel<2>
              : epl <= 4 ? balance_rows_kernel<4>
              : epl <= 8 ? balance_rows_kernel<8>
              : epl <= 16 ? balance_rows_kernel<16>
                          : balance_rows_kernel<32>;
  return launch_pdl(kern, dim3(row_blocks(T)), dim3(kRowThreads), 0, stream, logits, ldl, mask, T,
                    E, coef, loss, dlogits, ws);
}

}  // namespace mxmoe
