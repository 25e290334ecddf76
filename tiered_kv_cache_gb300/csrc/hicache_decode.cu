// hicache_decode.cu -- attention of one new token per sequence over its pages.
//
// One CTA per sequence and query head; its warps take the tokens in turn, each
// with a running maximum and sum of its own, and are joined in shared memory.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "hicache_serving.h"

namespace hicache {
namespace {

constexpr int kSimpleWarps = 8;
constexpr int kSimpleElems = 18;   // elements of a row per lane: rows of up to 576
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float load_elem(const void *base, int64_t i, bool bf16, bool e4m3) {
  if (e4m3) {
    __nv_fp8_e4m3 x;
    x.__x = static_cast<const uint8_t *>(base)[i];
    return float(x);
  }
  if (bf16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[i]);
  return __half2float(static_cast<const __half *>(base)[i]);
}

__global__ void __launch_bounds__(kSimpleWarps * 32) decode_simple_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ float sm_m[kSimpleWarps], sm_l[kSimpleWarps];
  __shared__ float sm_o[kSimpleWarps][kSimpleElems * 32];
  const int h = blockIdx.x, b = blockIdx.y;
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int kvh = h / p.G;
  const int64_t cap = int64_t(p.max_pages) * p.P;
  const int len = int(min(int64_t(max(0, p.lens[b])), cap));
  const int start = p.window > 0 ? max(0, len - p.window) : 0;
  float q[kSimpleElems], o[kSimpleElems];
#pragma unroll
  for (int j = 0; j < kSimpleElems; ++j) {
    const int i = lane + 32 * j;
    q[j] = i < p.D ? load_elem(p.q, b * p.q_sb + h * p.q_sh + i, p.bf16, false) : 0.f;
    o[j] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = start + warp; t < len; t += kSimpleWarps) {
    const int pg = int(fast_div(uint32_t(t), p.fd_page));
    const int page = p.table[b * p.t_sb + pg];
    float s = -INFINITY;
    if (page >= 0 && page < p.num_pages) {
      const int64_t row = (int64_t(page) * p.P + (t - pg * p.P)) * p.row + int64_t(kvh) * p.D;
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < kSimpleElems; ++j) {
        const int i = lane + 32 * j;
        if (i < p.D) a = fmaf(q[j], load_elem(p.k, row + i, p.bf16, p.e4m3), a);
      }
      for (int x = 16; x > 0; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
      s = a * p.scale2;
      const float m2 = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - m2), e = exp2f(s - m2);
      m = m2;
      l = l * f + e;
#pragma unroll
      for (int j = 0; j < kSimpleElems; ++j) {
        const int i = lane + 32 * j;
        if (i < p.Dv) o[j] = o[j] * f + e * load_elem(p.v, row + i, p.bf16, p.e4m3);
      }
    }
    if (p.weights && lane == 0) p.scores[(int64_t(b) * p.Hq + h) * p.score_row + t] = s;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < kSimpleElems; ++j) sm_o[warp][lane + 32 * j] = o[j];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, sm_m[w]);
  float f[kSimpleWarps];
  for (int w = 0; w < kSimpleWarps; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - top);
    sum += f[w] * sm_l[w];
  }
  const float inv = sum > 0.f ? p.v_scale / sum : 0.f;
  for (int i = int(threadIdx.x); i < p.Dv; i += kSimpleWarps * 32) {
    float a = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) a += f[w] * sm_o[w][i];
    a *= inv;
    const int64_t at = b * p.o_sb + h * p.o_sh + i;
    if (p.bf16)
      static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(a);
    else
      static_cast<__half *>(p.out)[at] = __float2half_rn(a);
  }
  if (threadIdx.x == 0) {
    const float lse2 = top + log2f(sum);
    if (p.lse) p.lse[b * p.lse_sb + h] = lse2 * kLn2;
    if (p.weights) p.lse2[int64_t(b) * p.Hq + h] = lse2;
  }
}

// weights[b, p] <- decay * weights[b, p] + sum over heads and tokens of
// 2^(score - lse2).  A block takes as many whole pages as 256 tokens hold (one
// page if it is longer); each thread sums a token over the heads, then each
// page is summed in token order, so the result does not depend on timing.
constexpr int kWeightThreads = 256;

__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ float val[kWeightThreads];
  const int b = blockIdx.y, tid = int(threadIdx.x);
  const int64_t cap = int64_t(p.max_pages) * p.P;
  const int len = int(min(int64_t(max(0, p.lens[b])), cap));
  const int start = p.window > 0 ? max(0, len - p.window) : 0;
  const int per = max(1, kWeightThreads / p.P);            // pages of a block
  const int first = int(blockIdx.x) * per;
  const int pages = int(len > 0 ? fast_div(uint32_t(len - 1), p.fd_page) + 1 : 0);
  if (first >= pages) return;
  const int t0 = first * p.P, t1 = min(len, int(min(int64_t(len), (int64_t(first) + per) * p.P)));
  const float *lse2 = p.lse2 + int64_t(b) * p.Hq;
  const float *sc = p.scores + int64_t(b) * p.Hq * p.score_row;
  float sum = 0.f;
  for (int t = t0 + tid; t < t1; t += kWeightThreads) {
    if (t < start) continue;
    for (int h = 0; h < p.Hq; ++h) {
      const float s = sc[h * p.score_row + t];
      if (s != -INFINITY) sum += exp2f(s - __ldg(lse2 + h));
    }
  }
  val[tid] = sum;
  __syncthreads();
  if (p.P > kWeightThreads) {
    for (int o = kWeightThreads / 2; o > 0; o >>= 1) {
      if (tid < o) val[tid] += val[tid + o];
      __syncthreads();
    }
    if (tid == 0) p.weights[b * p.w_sb + first] = p.decay * p.weights[b * p.w_sb + first] + val[0];
  } else if (tid < per && first + tid < pages) {
    float s = 0.f;
    for (int i = 0; i < p.P; ++i) s += val[tid * p.P + i];
    float *w = p.weights + b * p.w_sb + first + tid;
    *w = p.decay * *w + s;
  }
}

}  // namespace

DecodeSpace decode_space(int64_t batch, int64_t q_heads, int64_t max_pages, int64_t page, bool weights) {
  DecodeSpace s{};
  s.score_row = (max_pages * page + 3) / 4 * 4;
  s.scores = (batch * q_heads * 4 + 255) / 256 * 256;
  s.bytes = weights ? s.scores + batch * q_heads * s.score_row * 4 : 256;
  return s;
}

int launch_decode(const DecodeParams &p, void *stream, int *launches) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  decode_simple_kernel<<<dim3(unsigned(p.Hq), unsigned(p.B)), kSimpleWarps * 32, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return int(e);
  ++*launches;
  if (p.weights) {
    const int per = p.P < kWeightThreads ? kWeightThreads / p.P : 1;
    weights_kernel<<<dim3(unsigned((p.max_pages + per - 1) / per), unsigned(p.B)), kWeightThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return int(e);
    ++*launches;
  }
  return 0;
}

}  // namespace hicache
