// Shared by the two kernels of the fused MXFP8 product (linear.cu,
// linear_pair.cu): parameters and the activations.
#pragma once

#include "gemm_common.cuh"

namespace mxmoe {
namespace linear {

using namespace gemm;

struct LinParams {
  const uint16_t* x;       // [M, K] bf16 (split kernel that quantizes in place)
  const uint8_t* sfw;      // weight scales, MMA layout [ceil(N/128)][KT] chunks
  const uint8_t* sfx;      // activation scales, MMA layout
  const void* bias;        // [N] or null
  const uint16_t* res;     // [M, N] bf16 or null
  uint16_t* out;           // [M, N] bf16 (bf16 output)
  uint8_t* oq;             // [M, N] e4m3 (MXFP8 output), rows ldo bytes apart
  int64_t ldo, ldx, ldw;   // payload rows apart: output, activations, weights
  uint8_t* os;             // MMA layout, KT_out = ceil(N/128)
  int64_t M;
  int N, K, act;
  bool bias32;
  int NT, stages, nsplit;  // split kernel: token tile, pipeline stages, K ranges
  int tiles_n, tiles;      // pair kernel: n-tiles, tiles
  bool v32;                // pair kernel: rows of out and residual, or of oq, are 32-byte aligned
  int* status;
  long long wait_limit;
};

// Activations.  silu(z) = z * s(z) with s(z) = 1 / (1 + e^-z), and since
// (1 + tanh u) / 2 = s(2u), the tanh form of gelu is z * s(2u), u = sqrt(2 / pi) *
// (z + 0.044715 z^3).  erfcf (CUDA's) keeps gelu's relative accuracy where
// 1 + erf cancels.
//
// The hardware exp2 and reciprocal run at a quarter of a warp's instruction rate
// each, so two elements share one reciprocal: with d = 1 + 2^x, 1 / d0 =
// d1 / (d0 d1).  x is cut at 63 to keep d0 d1 finite: s below 2^-63 reads as
// 2^-63, which no sum with anything of z's size can tell from zero.
constexpr float kLog2e = 1.4426950409f;
constexpr float kGelu1 = -2.f * 0.7978845608f * kLog2e;  // -2u log2 e = z (kGelu1 + kGelu3 z^2)
constexpr float kGelu3 = 0.044715f * kGelu1;

// Two fp32 in one register pair, for the packed add / multiply / fma that do
// both in one instruction (each half as the scalar instruction, round to nearest).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// bf16 pair of a word as two fp32
__device__ __forceinline__ F2 bf16x2_f2(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// z * 1 / (1 + 2^x)
__device__ __forceinline__ F2 gate(F2 z, F2 x) {
  float x0, x1, d0, d1;
  unpack(x, x0, x1);
  const F2 d = add2(f2(ex2_approx(fminf(x0, 63.f)), ex2_approx(fminf(x1, 63.f))), f2(1.f, 1.f));
  unpack(d, d0, d1);
  const float r = rcp_approx(d0 * d1);
  return mul2(z, mul2(f2(r, r), f2(d1, d0)));
}

// One switch for a thread's 2 N values (act is uniform).
template <int N>
__device__ __forceinline__ void activate_all(int act, F2 (&v)[N]) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float a, b;
        unpack(v[i], a, b);
        v[i] = f2(a < 0.f ? 0.f : a, b < 0.f ? 0.f : b);  // NaN stays
      }
      break;
    case ACT_GELU:
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        float a, b;
        unpack(v[0], a, b);
        const F2 g = f2(0.5f * a * erfcf(a * -0.70710678f), 0.5f * b * erfcf(b * -0.70710678f));
#pragma unroll
        for (int j = 0; j + 1 < N; ++j) v[j] = v[j + 1];  // the values rotate: one copy of the code
        v[N - 1] = g;
      }
      break;
    case ACT_GELU_TANH: {
      const F2 k1 = f2(kGelu1, kGelu1), k3 = f2(kGelu3, kGelu3);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gate(v[i], mul2(v[i], fma2(k3, mul2(v[i], v[i]), k1)));
      break;
    }
    case ACT_SILU: {
      const F2 k = f2(-kLog2e, -kLog2e);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gate(v[i], mul2(v[i], k));
      break;
    }
    default: break;
  }
}

// MX scale of values whose largest magnitude is m, and their payload.
__device__ __forceinline__ float absmax3(float m, float a, float b) {
  return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 32-byte load the kernel may have written over (a residual updated in place:
// each element is read, then written, by one thread).
__device__ __forceinline__ void ld_v8(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
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

// e4m3 [outer, inner], rows ld bytes apart (a multiple of 16), 128-byte swizzled box.
inline bool make_map_ld(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                        uint64_t ld, uint32_t box_outer) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs (linear_pair.cu).  cudaErrorNotSupported: the device cannot
// co-schedule pairs.
cudaError_t launch_pair(const uint8_t* xq, const uint8_t* wq, const LinParams& p, int bn,
                        cudaStream_t stream);

}  // namespace linear
}  // namespace mxmoe
