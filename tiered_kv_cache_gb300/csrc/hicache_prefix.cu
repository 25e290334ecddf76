// hicache_prefix.cu -- the kernels of hicache_query.cuh for groups of sequences over shared
// prefixes, and the join with what the sequences have of their own.

#include "hicache_query.cuh"

namespace hicache {
namespace {

template <int TYPE>
int launch_prefix_type(const QueryParams &p, int device, cudaStream_t st, int *launches) {
  if (p.D <= 64) return launch_query_as<QueryConfig<64, TYPE, true>>(p, device, st, launches);
  if (p.D <= 128) return launch_query_as<QueryConfig<128, TYPE, true>>(p, device, st, launches);
  return launch_query_as<QueryConfig<256, TYPE, true>>(p, device, st, launches);
}

}  // namespace

int launch_prefix(const QueryParams &p, int device, void *stream, int *launches) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int e = p.e4m3 ? launch_prefix_type<kQE4m3>(p, device, st, launches)
          : p.bf16 ? launch_prefix_type<kQBf16>(p, device, st, launches)
                   : launch_prefix_type<kQFp16>(p, device, st, launches);
  if (e) return e;
  const int64_t blocks = (int64_t(p.N) * p.Hq * (p.D / 4) + kEndThreads - 1) / kEndThreads;
  e = query_launch(p.bf16 ? prefix_end_kernel<true> : prefix_end_kernel<false>, dim3(unsigned(blocks)), kEndThreads,
                   st, 0, p);
  *launches += e == 0;
  return e;
}

}  // namespace hicache
