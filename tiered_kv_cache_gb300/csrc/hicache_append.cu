// hicache_append.cu -- norms of the query and key heads, the position rotation
// and the store of K and V into the paged cache, in one pass.
//
// Nothing is used twice, so memory binds: a head is read, normed, rotated and
// written once.  A unit of work is one head of one token (of q, k or v), taken
// by a group of lanes that each hold 16-byte vectors of it; the sum of squares
// is reduced by shuffles, and the rotation's partner elements are exchanged
// through shared memory, so that any rotation span and either pairing works on
// whole vectors.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "hicache_serving.h"

namespace hicache {
namespace {

constexpr int kAppendThreads = 256;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (BF16)
      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
    else
      f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x / scale in e4m3, saturated; a true division, so that the value rounded is
// the one a quotient in 32 bits gives.
__device__ __forceinline__ uint2 pack8_e4m3(const float *x, float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
    const float2 b = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
    w[i] = uint32_t(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
           (uint32_t(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16);
  }
  return make_uint2(w[0], w[1]);
}

// ITERS: 16-byte vectors of a head per lane of its group (lanes = 1 << lg).
template <int ITERS, bool BF16>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendParams p, int lg, FastDiv fd_units) {
  __shared__ float stage[kAppendThreads * 8 * ITERS];
  const int lanes = 1 << lg, group = int(threadIdx.x) >> lg, lane = int(threadIdx.x) & (lanes - 1);
  const uint32_t unit = blockIdx.x * uint32_t(kAppendThreads >> lg) + uint32_t(group);
  const uint32_t n = fast_div(unit, fd_units);
  const int u = int(unit - n * fd_units.d);
  const int kind = u < p.q_heads ? 0 : u < p.q_heads + p.kv_heads ? 1 : 2;   // q, k, v
  const int head = kind == 0 ? u : kind == 1 ? u - p.q_heads : u - p.q_heads - p.kv_heads;
  bool live = int64_t(n) < p.num_tokens;
  int64_t pos = 0, slot = 0;
  if (live && p.rot > 0) {
    pos = p.positions[n];
    live = pos >= 0 && pos < p.cos_sin_rows;
  }
  if (live && kind != 0) {
    slot = p.slots[n];
    live = slot >= 0 && slot < p.num_slots;
  }
  const int chunks = p.D >> 3;
  float x[ITERS][8];
  const char *src = static_cast<const char *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v);
  const int64_t off = kind == 0   ? int64_t(n) * p.q_st + int64_t(head) * p.q_sh
                      : kind == 1 ? int64_t(n) * p.k_st + int64_t(head) * p.k_sh
                                  : int64_t(n) * p.v_st + int64_t(head) * p.v_sh;
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int c = lane + it * lanes;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live && c < chunks) w = __ldcs(reinterpret_cast<const uint4 *>(src + 2 * off) + c);
    unpack8<BF16>(w, x[it]);
  }
  const int m = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : 0;
  float sum = 0.f;
#pragma unroll
  for (int it = 0; it < ITERS; ++it)
    if ((lane + it * lanes) * 8 < m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[it][i], x[it][i], sum);
    }
  for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (m > 0) {
    const float r = rsqrtf(sum / float(m) + p.eps);
    const uint4 *wt = static_cast<const uint4 *>(kind == 0 ? p.q_weight : p.k_weight);
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int c = lane + it * lanes;
      if (c * 8 < m) {
        float w[8];
        unpack8<BF16>(__ldg(wt + c), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[it][i] = x[it][i] * r * w[i];
      }
    }
  }
  if (p.rot > 0) {
    float *mine = stage + group * lanes * 8 * ITERS;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      float4 *d = reinterpret_cast<float4 *>(mine + (lane + it * lanes) * 8);
      d[0] = make_float4(x[it][0], x[it][1], x[it][2], x[it][3]);
      d[1] = make_float4(x[it][4], x[it][5], x[it][6], x[it][7]);
    }
    __syncwarp();
    if (live && kind != 2) {
      const int half = p.rot >> 1;
      const float *cs = p.cos_sin + pos * p.rot;
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int c = lane + it * lanes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = c * 8 + i - p.rot_off;
          if (c < chunks && e >= 0 && e < p.rot) {
            const bool second = p.interleaved ? (e & 1) : e >= half;
            const int j = p.interleaved ? e >> 1 : second ? e - half : e;
            const int mate = p.interleaved ? e ^ 1 : second ? e - half : e + half;
            const float y = mine[mate + p.rot_off], co = __ldg(cs + j), si = __ldg(cs + half + j);
            x[it][i] = second ? fmaf(x[it][i], co, y * si) : fmaf(x[it][i], co, -y * si);
          }
        }
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int c = lane + it * lanes;
    if (c >= chunks) continue;
    if (kind == 0) {
      char *dst = static_cast<char *>(p.q_out) + 2 * (int64_t(n) * p.o_st + int64_t(head) * p.o_sh);
      reinterpret_cast<uint4 *>(dst)[c] = pack8<BF16>(x[it]);
    } else {
      const int64_t at = slot * p.row + int64_t(head) * p.D;
      char *buf = static_cast<char *>(kind == 1 ? p.k_cache : p.v_cache);
      if (p.e4m3)
        reinterpret_cast<uint2 *>(buf + at)[c] = pack8_e4m3(x[it], kind == 1 ? p.k_scale : p.v_scale);
      else
        reinterpret_cast<uint4 *>(buf + 2 * at)[c] = pack8<BF16>(x[it]);
    }
  }
}

}  // namespace

int launch_append(const AppendParams &p, void *stream) {
  const int units = p.q_heads + p.kv_heads * (p.has_v ? 2 : 1);
  const int chunks = p.D / 8;
  int lg = 0;
  while (lg < 5 && (1 << lg) < chunks) ++lg;
  const int per_block = kAppendThreads >> lg;
  const int64_t total = p.num_tokens * units;
  const unsigned grid = unsigned((total + per_block - 1) / per_block);
  const FastDiv fd = make_fastdiv(uint32_t(units));
  auto *k = chunks <= 32 ? (p.bf16 ? append_kernel<1, true> : append_kernel<1, false>)
                         : (p.bf16 ? append_kernel<3, true> : append_kernel<3, false>);
  k<<<grid, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, lg, fd);
  return int(cudaGetLastError());
}

}  // namespace hicache
