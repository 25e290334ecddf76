// hicache_decode.cuh -- device code shared by the decode attention kernels
// (hicache_decode.cu, hicache_decode_latent.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hicache_serving.h"

namespace hicache {
namespace {

constexpr float kLn2 = 0.693147180559945309f;

// Scores are taken relative to a reference per head that follows the running maximum:
// it is put kAbove (log2) below the maximum whenever some score lies more than kRaise
// above it.  The exponentials, 2^kAbove for the maximum then and 2^kRaise at most, are
// rounded to the products' type.  fp16 has places from 2^-24 to 2^16: with the maximum
// at 2^6, what lies below half its smallest number, and is lost to the product though
// not to the sum of the exponentials, is under 2^-31 of the maximum: 2^-11 of the
// weight for a million such tokens, as much as fp16's own rounding (at 2^0 it
// was 2^-25, 3%).  bf16 has the exponents of the sums themselves, and exponentials
// above 1 would only take room from V: 2^40, which its places allow, times elements of
// 2^90 left 32 bits.  They stay under 1, so that the sum over a piece fits wherever that
// of V itself does; with the maximum at 2^-14, nothing is lost at the lower end.
template <bool FP16>
constexpr float kRaise = FP16 ? 15.f : 0.f;
template <bool FP16>
constexpr float kAbove = FP16 ? 6.f : -14.f;

// The tokens [start, len) that sequence b attends to.
__device__ __forceinline__ void seq_range(const DecodeParams &p, int b, int *start, int *len) {
  const int64_t cap = int64_t(p.max_pages) * p.P;
  const int n = max(0, __ldg(p.lens + b));
  *len = int(min(int64_t(n), cap));
  *start = p.window > 0 ? max(0, *len - p.window) : 0;
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

// 16 bytes, of which the first `bytes` (0 or 16) are read and the rest is zero
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x to two units of the last place; results under 2^-126 are zero
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

__device__ __forceinline__ void store_out(const DecodeParams &p, int b, int h, int col, float v) {
  if (col >= p.Dv) return;
  const int64_t at = int64_t(b) * p.o_sb + int64_t(h) * p.o_sh + col;
  if (p.bf16)
    static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half *>(p.out)[at] = __float2half_rn(v);
}
// four elements from a multiple of 4 on, times f
__device__ __forceinline__ void store_out4(const DecodeParams &p, int b, int h, int col, float4 v, float f) {
  if (col >= p.Dv) return;
  char *at = static_cast<char *>(p.out) + 2 * (int64_t(b) * p.o_sb + int64_t(h) * p.o_sh + col);
  *reinterpret_cast<uint2 *>(at) = p.bf16
                                       ? make_uint2(pack2<true>(v.x * f, v.y * f), pack2<true>(v.z * f, v.w * f))
                                       : make_uint2(pack2<false>(v.x * f, v.y * f), pack2<false>(v.z * f, v.w * f));
}
// l == 0: nothing attended to
__device__ __forceinline__ void store_lse(const DecodeParams &p, int b, int h, float m, float l) {
  const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
  if (p.lse) p.lse[int64_t(b) * p.lse_sb + h] = lse2 * kLn2;
  if (p.weights) p.lse2[int64_t(b) * p.Hq + h] = lse2;
}

// Exclusive prefix sums over the CTA's threads (WARPS of them) of `mine`; the
// total in *total.  Ends with every thread past its reads of `scratch`.
template <int WARPS, class T>
__device__ __forceinline__ T block_prefix(T mine, T *scratch, T *total) {
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  T inc = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  T before = 0, all = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scratch[w];
    all += scratch[w];
  }
  *total = all;
  return before + inc - mine;
}

// Launches a kernel that may start while the work before it on the stream ends:
// it waits (griddepcontrol.wait) before it touches memory.
inline int launch_dependent(void (*kernel)(const DecodeParams), dim3 grid, unsigned threads, cudaStream_t st,
                            const DecodeParams &p, size_t smem = 0) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, p);
  return int(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace
}  // namespace hicache
