// Dense MXFP8 product with bias, activation and residual in its epilogue.
//
//   z[t, n] = sum_k deq(xq)[t, k] * deq(wq)[n, k] + bias[n]      fp32
//   v       = act(z)                      none, relu, gelu, gelu_tanh, silu
//   out     = bf16(v + residual)          one rounding, or
//   (oq, os) = MX-quant(v) along n        payload and MMA-layout scales, what
//                                         the next product reads
//
// linear_split_kernel: the weights are the MMA's M side (128 rows of wq per
// CTA), NT tokens its N side (32, 64, 128 or 256), so few tokens cost a short
// instruction and a small operand tile.  K is split over the S <= 8 CTAs of a
// cluster: each accumulates its K range in TMEM, leaves the fp32 partial tile
// in its shared memory, and the CTAs then take tokens in turn, adding the S
// partials of a token in split order through distributed shared memory.  One
// launch, no partial sums in device memory, the same bits in every run.
//
// Roles (320 threads): warp 0 producer (TMA of both operand tiles, bulk
// copies of their scale chunks), warp 1 MMA issuer, warps 2-5 scale-factor
// writers (shared memory -> TMEM), warps 2-9 accumulator -> shared memory,
// all warps the epilogue (a warp per token, 4 columns of n per lane).
//
// Every mbarrier wait is bounded as in gemm.cu.
#include "linear.cuh"

namespace mxmoe {
namespace linear {

constexpr int WM = 128;              // weight rows per CTA
constexpr int W_BYTES = WM * BK;     // 16 KB per k-slice
constexpr int WARPS = 10;
constexpr int L_THREADS = 32 * WARPS;
constexpr int DRAIN_WARPS = 8;       // accumulator -> shared memory
constexpr int MAX_STAGES = 6;
constexpr int MAX_SPLIT = 8;

// Shared-memory layout (runtime NT and stage count).
struct Smem {
  int x, sfw, sfx, bar, misc, total;
};
__host__ __device__ inline Smem smem_layout(int NT, int stages) {
  Smem s;
  const int nx = NT > 128 ? 2 : 1;  // 128-row scale blocks of the token tile
  s.x = stages * W_BYTES;
  s.sfw = s.x + stages * NT * BK;
  s.sfx = s.sfw + stages * 512;
  s.bar = s.sfx + stages * nx * 512;
  s.misc = s.bar + (3 * MAX_STAGES + 1) * 8;
  s.total = s.misc + 16;
  return s;
}

__device__ __forceinline__ void tmem_st_1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_st_2(uint32_t taddr, uint32_t v0, uint32_t v1) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(v0), "r"(v1)
               : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A token's 4 columns n .. n + 3 (n + 3 < N) of this lane: bias, activation,
// residual, store.  bias: the lane's 4 values.  Called by a whole warp on one
// token t; lane l holds columns n0 + 4 l.
__device__ __forceinline__ void finish_token(const LinParams& p, int64_t t, int n0, int lane,
                                             float4 v, const float4& bias, uint2 res) {
  const int n = n0 + 4 * lane;
  const bool in = n < p.N;
  F2 a2[2] = {add2(f2(v.x, v.y), f2(bias.x, bias.y)), add2(f2(v.z, v.w), f2(bias.z, bias.w))};
  activate_all(p.act, a2);
  float a[4];
  unpack(a2[0], a[0], a[1]);
  unpack(a2[1], a[2], a[3]);
  if (p.out) {
    if (!in) return;
    a[0] += bf16_bits_to_float(res.x & 0xFFFFu);
    a[1] += bf16_bits_to_float(res.x >> 16);
    a[2] += bf16_bits_to_float(res.y & 0xFFFFu);
    a[3] += bf16_bits_to_float(res.y >> 16);
    uint2 o = make_uint2(cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]));
    *reinterpret_cast<uint2*>(p.out + t * p.N + n) = o;
    return;
  }
  // MXFP8: eight lanes hold a block of 32
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!in) a[i] = 0.f;
    m = umax(m, __float_as_uint(a[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) m = umax(m, __shfl_xor_sync(0xffffffffu, m, off));
  const uint32_t sb = e8m0_from_amax_bits(m);
  const float inv = inv_scale_from_e8m0(sb);
  if (in)
    *reinterpret_cast<uint32_t*>(p.oq + t * p.N + n) =
        cvt_e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
  // the 128 columns' four scale bytes are one word of the MMA layout; slots
  // past the row's last block hold 127
  const uint32_t byte = (n & ~31) < p.N ? sb : 127u;
  uint32_t word = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, byte, 8 * b) << (8 * b);
  if (lane == 0)
    *reinterpret_cast<uint32_t*>(p.os + tiled_scale_offset(t, n0 >> 5, (p.N + 127) / 128)) = word;
}

__global__ void __launch_bounds__(L_THREADS, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmX, const LinParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NT = p.NT, STAGES = p.stages;
  const Smem L = smem_layout(NT, STAGES);
  const int nx = NT > 128 ? 2 : 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L.misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L.misc + 4);
  auto bar_full = [&](int s) { return sbase + L.bar + 8u * s; };
  auto bar_empty = [&](int s) { return sbase + L.bar + 8u * (MAX_STAGES + s); };
  auto bar_sf = [&](int s) { return sbase + L.bar + 8u * (2 * MAX_STAGES + s); };
  const uint32_t bar_acc = sbase + L.bar + 8u * (3 * MAX_STAGES);
  // TMEM: NT accumulator columns, then 16 scale columns per stage
  const uint32_t tmem_cols = NT <= 64 ? 128u : NT <= 128 ? 256u : 512u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
      mbar_init(bar_sf(s), SF_WARPS);
    }
    mbar_init(bar_acc, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_tmem)),
                 "r"(tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const int rank = p.nsplit > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = blockIdx.x * WM;
  const int64_t t0 = (int64_t)blockIdx.y * NT;
  const int KT = (p.K + BK - 1) / BK;
  const int kper = (KT + p.nsplit - 1) / p.nsplit;
  const int k0 = rank * kper, k1 = min(KT, k0 + kper);  // non-empty for every rank
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 0) {
    // ================= producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      const uint32_t bytes = (uint32_t)(W_BYTES + NT * BK + 512 + 512 * nx);
      // the token tile's scale blocks; a block past the last token's is not read
      const int64_t rb = t0 >> 7, last_rb = (p.M - 1) >> 7;
      for (int kt = k0; kt < k1; ++kt) {
        if (!wait_bar(bar_empty(stage), phase ^ 1, p.wait_limit, p.status, s_abort)) break;
        mbar_arrive_expect_tx(bar_full(stage), bytes);
        tma_load_2d(sbase + stage * W_BYTES, &tmW, kt * BK, n0, bar_full(stage));
        tma_load_2d(sbase + L.x + stage * NT * BK, &tmX, kt * BK, (int)t0, bar_full(stage));
        bulk_copy_g2s(sbase + L.sfw + stage * 512, p.sfw + ((int64_t)blockIdx.x * KT + kt) * 512,
                      512, bar_full(stage));
        for (int b = 0; b < nx; ++b)
          bulk_copy_g2s(sbase + L.sfx + (stage * nx + b) * 512,
                        p.sfx + (min(rb + b, last_rb) * KT + kt) * 512, 512, bar_full(stage));
        armed |= 1u << stage;
        if (phase) armed_parity |= 1u << stage; else armed_parity &= ~(1u << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      // every copy this thread issued has landed before shared memory is reused
      for (int s = 0; s < STAGES; ++s)
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          wait_bar(bar_full(s), (armed_parity >> s) & 1u, 1ll << 32, nullptr, &no_abort);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================= MMA issuer
    if (lane == 0) {
      const uint32_t IDESC = make_idesc(WM, NT);
      int stage = 0;
      uint32_t phase = 0;
      bool issued = false;
      for (int kt = k0; kt < k1; ++kt) {
        if (!wait_bar(bar_sf(stage), phase, p.wait_limit, p.status, s_abort) ||
            !wait_bar(bar_full(stage), phase, p.wait_limit, p.status, s_abort))
          break;
        tc_fence_after();
        const uint64_t adesc = make_sdesc(sbase + stage * W_BYTES, 16, 1024, 2);
        const uint64_t bdesc = make_sdesc(sbase + L.x + stage * NT * BK, 16, 1024, 2);
        const uint32_t t_sf = tmem + NT + 16 * stage;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          tc_mma_mxf8(tmem, adesc + 2 * kk, bdesc + 2 * kk,
                      IDESC | ((uint32_t)kk << 29) | ((uint32_t)kk << 4), t_sf, t_sf + 4,
                      ((kt - k0) | kk) != 0 ? 1u : 0u);
        issued = true;
        tc_commit(bar_empty(stage));
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      // this thread waits too, so no MMA is in flight when shared memory is reused
      if (issued) {
        tc_commit(bar_acc);
        volatile int no_abort = 0;
        wait_bar(bar_acc, 0, 1ll << 32, nullptr, &no_abort);
      } else {
        mbar_arrive(bar_acc);
      }
    }
    __syncwarp();
  } else {
    if (warp < 2 + SF_WARPS) {
      // ================= scale-factor writers: 4 columns of weight scales, NT / 32
      // columns of token scales per stage (32-row groups g0 .. of their 128-row block)
      const uint32_t t_q = tmem + ((uint32_t)((warp & 3) * 32) << 16) + NT;
      const int g0 = (int)(t0 & 127) >> 5;
      int stage = 0;
      uint32_t phase = 0;
      for (int kt = k0; kt < k1; ++kt) {
        const bool got = wait_bar(bar_full(stage), phase, p.wait_limit, p.status, s_abort);
        if (!__all_sync(0xffffffffu, got)) break;
        const uint32_t col = t_q + 16 * stage;
        tmem_st_4(col, *reinterpret_cast<const uint4*>(smem + L.sfw + stage * 512 + lane * 16));
        const uint8_t* sx = smem + L.sfx + stage * nx * 512 + lane * 16;
        if (NT == 32) {
          tmem_st_1(col + 4, *reinterpret_cast<const uint32_t*>(sx + 4 * g0));
        } else if (NT == 64) {
          const uint2 w = *reinterpret_cast<const uint2*>(sx + 4 * g0);
          tmem_st_2(col + 4, w.x, w.y);
        } else {
          tmem_st_4(col + 4, *reinterpret_cast<const uint4*>(sx));
          if (NT == 256) tmem_st_4(col + 8, *reinterpret_cast<const uint4*>(sx + 512));
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf(stage));
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    // ================= accumulator -> shared memory [token][128], over the stages
    // (idle: every copy has landed and every MMA is done once bar_acc completes)
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool got = wait_bar(bar_acc, 0, p.wait_limit, p.status, s_abort);
    if (__all_sync(0xffffffffu, got)) {
      tc_fence_after();
      float* buf = reinterpret_cast<float*>(smem);
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16);
      const int cols = NT / 2, last = (int)min((int64_t)NT, p.M - t0);
      for (int c = half * cols; c < (half + 1) * cols && c < last; c += 16) {
        uint32_t v[16];
        tmem_ld_16(t_row + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) buf[(c + i) * WM + q * 32 + lane] = __uint_as_float(v[i]);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (p.nsplit > 1) cluster_sync();

  // ================= epilogue: a warp per token of this CTA's share
  {
    const int n = n0 + 4 * lane;
    const bool in = n < p.N;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.bias && in) {
      if (p.bias32) {
        bias = *reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + n);
      } else {
        const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.bias) + n);
        bias = make_float4(bf16_bits_to_float(b.x & 0xFFFFu), bf16_bits_to_float(b.x >> 16),
                           bf16_bits_to_float(b.y & 0xFFFFu), bf16_bits_to_float(b.y >> 16));
      }
    }
    const int last = (int)min((int64_t)NT, p.M - t0);
    for (int i = warp * p.nsplit + rank; i < last; i += WARPS * p.nsplit) {
      uint2 res = make_uint2(0, 0);
      if (p.res && in) res = *reinterpret_cast<const uint2*>(p.res + (t0 + i) * p.N + n);
      const uint32_t at = sbase + (uint32_t)(i * WM + 4 * lane) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.nsplit == 1) {
        v = *reinterpret_cast<const float4*>(smem + (i * WM + 4 * lane) * 4);
      } else {
        for (int r = 0; r < p.nsplit; ++r) {  // split order, whichever CTA adds
          const float4 u = ld_cluster_f4(mapa_cluster(at, r));
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
      }
      finish_token(p, t0 + i, n0, lane, v, bias, res);
    }
  }

  // ---- teardown
  __syncwarp();
  if (p.nsplit > 1) cluster_sync();  // the other CTAs still read this one's tile
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols)
                 : "memory");
  }
}

// Tile and split choice: the token tile covers the batch up to 256 tokens;
// K is split until the CTAs fill the GPU (two fit on an SM up to 64 tokens).
struct Plan {
  int NT, stages, nsplit;
};
static Plan make_plan(int64_t M, int N, int K) {
  Plan pl;
  pl.NT = M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  pl.stages = pl.NT <= 32 ? 5 : pl.NT <= 64 ? 4 : pl.NT <= 128 ? 6 : 4;
  const int64_t slots = (int64_t)num_sms() * (pl.NT <= 64 ? 2 : 1);
  const int64_t tiles = ceil_div(N, WM) * ceil_div(M, pl.NT);
  const int KT = (int)ceil_div(K, BK);
  int s = (int)std::min<int64_t>({slots / tiles, (int64_t)KT, (int64_t)MAX_SPLIT});
  if (s < 1) s = 1;
  const int kper = (int)ceil_div(KT, s);
  pl.nsplit = (int)ceil_div(KT, kper);  // no empty range
  return pl;
}

}  // namespace linear

cudaError_t launch_linear_fused(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                const uint8_t* ws, int64_t M, int N, int K, const void* bias,
                                bool bias32, int act, const uint16_t* residual, uint16_t* out,
                                uint8_t* oq, uint8_t* os, cudaStream_t stream) {
  using namespace linear;
  if (M == 0) return cudaSuccess;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static uint64_t configured[64] = {0};  // context id the attribute was set in
  const uint64_t ctx = context_id();
  if (ctx == 0 || configured[dev] != ctx) {
    const cudaError_t err = cudaFuncSetAttribute(
        linear_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (err != cudaSuccess) return err;
    configured[dev] = context_id();
  }
  LinParams p = {};
  p.sfw = ws;
  p.sfx = xs;
  p.bias = bias;
  p.res = residual;
  p.out = out;
  p.oq = oq;
  p.os = os;
  p.M = M;
  p.N = N;
  p.K = K;
  p.act = act;
  p.bias32 = bias32;
  p.status = device_status_ptr();
  p.wait_limit = wait_limit_cycles();
  if (M > 256) {
    int bn = 0;
    pair_cycles(M, N, K, &bn);
    const cudaError_t err = launch_pair(xq, wq, p, bn, stream);
    if (err != cudaErrorNotSupported) return err;
  }
  const Plan pl = make_plan(M, N, K);
  CUtensorMap tmW, tmX;
  if (!make_map(&tmW, wq, (uint64_t)K, (uint64_t)N, BK, WM) ||
      !make_map(&tmX, xq, (uint64_t)K, (uint64_t)M, BK, (uint32_t)pl.NT))
    return cudaErrorInvalidValue;
  p.NT = pl.NT;
  p.stages = pl.stages;
  p.nsplit = pl.nsplit;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = (unsigned)pl.nsplit;
  cfg.attrs = attr;
  cfg.numAttrs = pl.nsplit > 1 ? 2 : 1;
  cfg.gridDim = dim3((unsigned)ceil_div(N, WM), (unsigned)ceil_div(M, pl.NT), (unsigned)pl.nsplit);
  cfg.blockDim = dim3(L_THREADS);
  cfg.dynamicSmemBytes = (size_t)smem_layout(pl.NT, pl.stages).total + 1024;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel, tmW, tmX, p);
}

}  // namespace mxmoe
