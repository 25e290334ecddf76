// hicache_evict.cu -- the pages of each sequence with the least accumulated
// attention weight, and the page table without them.
//
// One CTA per sequence.  The count-th lowest key among the pages that may go is
// found by a radix select (four 8-bit digits of an order-preserving integer key,
// a shared-memory histogram each); then one pass over the pages in order splits
// them into those that leave and those that stay, each place worked out by a
// block-wide scan.  Among equal keys the first pages leave.  A page moves to
// its own place or an earlier one, and a chunk is written only once it has been
// read whole, so the outputs may be the inputs.

#include <cuda_runtime.h>

#include "hicache_serving.h"

namespace hicache {
namespace {

constexpr int kEvictThreads = 1024;

// Integers in the order of the weights: -0 as 0, NaN above infinity.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];              // digit, rank within it
  __shared__ unsigned long long warp_sum[32];
  const int64_t b = blockIdx.x;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int len = p.lens[b];
  const int64_t pages64 = len > 0 ? (int64_t(len) + p.P - 1) / p.P : 0;
  const int n = int(pages64 < p.max_pages ? pages64 : p.max_pages);
  const int keep = max(0, p.keep[b]);
  const int last = n - p.recent;            // pages in [sink, last) may go
  const int may = max(0, last - p.sink);
  const int count = min(min(max(0, n - keep), may), p.max_victims);
  const int32_t *table = p.table + b * p.t_sb;
  const float *weights = p.weights + b * p.w_sb;

  // the key of the last page that leaves, and how many pages with that key do
  uint32_t key = 0, mask = 0, need = uint32_t(count);
  if (count > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = p.sink + tid; i < last; i += kEvictThreads) {
        const uint32_t k = order_key(weights[i]);
        if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid < 32) {
        uint32_t c[8], sum = 0;
        for (int j = 0; j < 8; ++j) sum += c[j] = hist[tid * 8 + j];
        uint32_t before = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
          if (tid >= o) before += y;
        }
        before -= sum;
        for (int j = 0; j < 8; ++j) {
          if (before < need && need <= before + c[j]) {
            pick[0] = uint32_t(tid * 8 + j);
            pick[1] = need - before;
          }
          before += c[j];
        }
      }
      __syncthreads();
      key |= pick[0] << shift;
      mask |= 255u << shift;
      need = pick[1];
      __syncthreads();
    }
  }

  // pages in order: low word of a scan value = keys below, high word = equal keys
  uint32_t below0 = 0, equal0 = 0;
  for (int base = 0; base < n; base += kEvictThreads) {
    const int i = base + tid;
    const bool in = i < n;
    const int32_t page = in ? table[i] : 0;
    const float w = in ? weights[i] : 0.f;
    uint32_t below = 0, equal = 0;
    if (count > 0 && i >= p.sink && i < last) {
      const uint32_t k = order_key(w);
      below = k < key;
      equal = k == key;
    }
    unsigned long long v = below | (static_cast<unsigned long long>(equal) << 32);
    unsigned long long inc = v;
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      unsigned long long s = warp_sum[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    const unsigned long long ex = inc - v + (warp ? warp_sum[warp - 1] : 0ull);
    const unsigned long long total = warp_sum[31];
    const uint32_t nb = below0 + uint32_t(ex), ne = equal0 + uint32_t(ex >> 32);
    const uint32_t gone = nb + min(ne, need);       // pages before this one that leave
    if (in) {
      if (below || (equal && ne < need)) {
        p.victims[b * p.v_sb + gone] = page;
      } else {
        p.out_table[b * p.ot_sb + i - gone] = page;
        p.out_weights[b * p.ow_sb + i - gone] = w;
      }
    }
    below0 += uint32_t(total);
    equal0 += uint32_t(total >> 32);
    __syncthreads();
  }
  for (int i = n - count + tid; i < n; i += kEvictThreads) {
    p.out_table[b * p.ot_sb + i] = -1;
    p.out_weights[b * p.ow_sb + i] = 0.f;
  }
  if (tid == 0) {
    p.num_victims[b] = count;
    p.out_lens[b] = len - count * p.P;
  }
}

}  // namespace

int launch_evict(const EvictParams &p, void *stream) {
  evict_kernel<<<unsigned(p.B), kEvictThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return int(cudaGetLastError());
}

}  // namespace hicache
