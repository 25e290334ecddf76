// hicache_merge.cu -- results of attention over parts of the tokens, joined by their
// log-sums: lse = log sum_i exp(lse_i), out = sum_i exp(lse_i - lse) out_i.
//
// Bound by HBM: 2 bytes read per part and element, 2 written.  A thread takes 8 elements
// of a row, with the parts' loads on their way together; the log-sums of a row come from
// L1 for all its threads but one.  A part whose log-sum is -infinity is not read.  As many warps as
// an SM holds (8 blocks: 54 -> 48 us for 8,191 tokens of 32 heads of 128 from 4 parts of which a
// quarter is empty; two or four rows a thread instead took 62 and 113), and loads and stores
// that leave L2 to others (48 -> 45.4; 2 parts 37 -> 32.5): nothing is read twice.  4 parts without
// an empty one: 50.8 us, 8 parts 91, 97% and more of a plain copy's rate, 2 parts 92%.

#include "hicache_decode.cuh"

namespace hicache {
namespace {

constexpr int kMergeThreads = 256;

template <int PARTS, bool BF16>
__global__ void __launch_bounds__(kMergeThreads, PARTS <= 4 ? 8 : 5) merge_kernel(const __grid_constant__ MergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t at = int64_t(blockIdx.x) * kMergeThreads + threadIdx.x;
  if (at >= p.rows * p.fd_vecs.d) return;
  const uint32_t row = fast_div(uint32_t(at), p.fd_vecs), col = (uint32_t(at) - row * p.fd_vecs.d) * 8;
  const uint32_t token = fast_div(row, p.fd_heads), head = row - token * p.fd_heads.d;
  float z[PARTS];
  uint4 v[PARTS];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) z[i] = i < p.parts ? __ldg(p.lses[i] + token * p.l_st[i] + head) : -INFINITY;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    top = fmaxf(top, z[i]);
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (z[i] != -INFINITY)
      v[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(p.outs[i]) +
                                              2 * (token * p.o_st[i] + head * p.o_sh[i] + col)));
  }
  const float base = top == -INFINITY ? 0.f : top;
  // weights in eighths (exactly): the sum of as many parts near the largest bf16 would leave 32 bits,
  // though their mean does not
  float acc[8] = {}, sum = 0.f;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const float w = 0.125f * exp2_fast((z[i] - base) * 1.4426950408889634f);   // 0 for a part that is not there
    sum += w;
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]))
                            : __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
      acc[2 * j] += w * f.x;
      acc[2 * j + 1] += w * f.y;
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  static_assert(kMergeParts == 8, "eighths");
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = pack2<BF16>(acc[2 * j] * f, acc[2 * j + 1] * f);
  __stcs(reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + 2 * (token * p.out_st + head * p.out_sh + col)),
         make_uint4(r[0], r[1], r[2], r[3]));
  if (p.lse && col == 0) p.lse[token * p.lse_st + head] = sum == 0.f ? -INFINITY : base + log2f(8.f * sum) * kLn2;
}

template <int PARTS>
int launch_merge_as(const MergeParams &p, cudaStream_t st) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(unsigned((p.rows * p.fd_vecs.d + kMergeThreads - 1) / kMergeThreads));
  c.blockDim = dim3(kMergeThreads);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, p.bf16 ? merge_kernel<PARTS, true> : merge_kernel<PARTS, false>, p);
  return int(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

int launch_merge(const MergeParams &p, void *stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p.parts <= 2 ? launch_merge_as<2>(p, st) : p.parts <= 4 ? launch_merge_as<4>(p, st) : launch_merge_as<8>(p, st);
}

}  // namespace hicache
