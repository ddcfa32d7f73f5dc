// Shared by the two kernels of the fused MXFP8 product (linear.cu,
// linear_pair.cu): parameters and the activations.
#pragma once

#include "gemm_common.cuh"

namespace mxmoe {
namespace linear {

using namespace gemm;

struct LinParams {
  const uint8_t* sfw;      // weight scales, MMA layout [ceil(N/128)][KT] chunks
  const uint8_t* sfx;      // activation scales, MMA layout
  const void* bias;        // [N] or null
  const uint16_t* res;     // [M, N] bf16 or null
  uint16_t* out;           // [M, N] bf16 (bf16 output)
  uint8_t* oq;             // [M, N] e4m3 (MXFP8 output)
  uint8_t* os;             // MMA layout, KT_out = ceil(N/128)
  int64_t M;
  int N, K, act;
  bool bias32;
  int NT, stages, nsplit;  // split kernel: token tile, pipeline stages, K ranges
  int tiles_n, tiles;      // pair kernel: n-tiles, tiles
  bool v32;                // pair kernel: out / residual rows are 32-byte aligned
  int* status;
  long long wait_limit;
};

// act(z).  silu(z) = z / (1 + e^-z); (1 + tanh u) / 2 = 1 / (1 + e^-2u), so
// the tanh form of gelu is z / (1 + e^-2u) with the same two hardware
// functions; erfcf (CUDA's) keeps gelu's relative accuracy where 1 + erf
// cancels.
constexpr float kGeluTanh = -2.f * 0.7978845608f * 1.4426950409f;  // -2 sqrt(2 / pi) log2 e

// One switch for a thread's N values (act is uniform).
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&v)[N]) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // NaN stays
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678f);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = v[i] * rcp_approx(1.f + ex2_approx(kGeluTanh * (v[i] + 0.044715f * v[i] * v[i] * v[i])));
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = swiglu(v[i], 1.f);
      break;
    default: break;
  }
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Whether the phase is over, without waiting for it.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// CTA pairs (linear_pair.cu).  cudaErrorNotSupported: the device cannot
// co-schedule pairs.
cudaError_t launch_pair(const uint8_t* xq, const uint8_t* wq, const LinParams& p, int bn,
                        cudaStream_t stream);
// Estimated SM cycles of the pair kernel on this product, and the tile width
// it would take.
double pair_cycles(int64_t M, int N, int K, int* bn);

}  // namespace linear
}  // namespace mxmoe
