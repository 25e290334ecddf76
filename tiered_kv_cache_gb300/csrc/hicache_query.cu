// hicache_query.cu -- the kernels of hicache_query.cuh, by type and head_dim.

#include "hicache_query.cuh"

namespace hicache {
namespace {

template <int TYPE>
int launch_query_type(const QueryParams &p, int device, cudaStream_t st, int *launches) {
  if (p.D <= 64) return launch_query_as<QueryConfig<64, TYPE>>(p, device, st, launches);
  if (p.D <= 128) return launch_query_as<QueryConfig<128, TYPE>>(p, device, st, launches);
  return launch_query_as<QueryConfig<256, TYPE>>(p, device, st, launches);
}

}  // namespace

QuerySpace query_space(int D) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int64_t rows = kQueryRows * query_tiles(D), chunks = kQueryCtas;
  QuerySpace s;
  // Decode attention's counters and error word come first, and what is zero between calls lies
  // behind them where it has nothing: one workspace can serve both, one call after another.
  constexpr int64_t counters = (kDecodeCtas + 1) * 4, next = (counters + 63) / 64 * 64;
  static_assert(next % 8 == 0 && next + 16 <= (counters + 255) / 256 * 256, "the counters lie before decode attention's parts");
  s.next = next;
  s.open = up(counters);
  s.parts = up(s.open + chunks * 16);
  s.bytes = up(s.parts + chunks * 2 * (rows * query_cols(D) + 2 * rows) * 4);
  return s;
}

int launch_query(const QueryParams &p, int device, void *stream, int *launches) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.e4m3) return launch_query_type<kQE4m3>(p, device, st, launches);
  if (p.bf16) return launch_query_type<kQBf16>(p, device, st, launches);
  return launch_query_type<kQFp16>(p, device, st, launches);
}

}  // namespace hicache
