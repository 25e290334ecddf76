// hicache_evict.cu -- the pages of each sequence with the least accumulated
// attention weight, and the page table without them.
//
// The count-th lowest key among the pages that may go is found by a radix select
// (four 8-bit digits of an order-preserving integer key, a histogram each); then the
// pages are split, in their order, into those that leave and those that stay, each
// place worked out by a scan.  Among equal keys the first pages leave.
//
// A cluster of CTAs takes a sequence, each CTA a part of its pages, which it reads
// once into shared memory; histograms and counts are summed over the cluster through
// distributed shared memory.  Everything has been read before anything is written,
// so the outputs may be the inputs.  Bound by the cluster's barriers: two sequences of
// 131,071 and 100,000 pages take 17 us (198 us by one CTA each).  Sequences too long
// for the cluster's shared memory (393,216 pages) take one CTA that walks them chunk by
// chunk: 400,000 pages 671 us.

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "hicache_serving.h"

namespace hicache {
namespace {

namespace cg = cooperative_groups;

constexpr int kEvictThreads = 1024;

// Integers in the order of the weights: -0 as 0, NaN above infinity.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// A sequence's pages: n in all, those present in [sink, last) may go, at most `count` of
// them do (how many are present is known with the first histogram).
struct EvictSeq {
  int len, n, last, count;
};
__device__ __forceinline__ EvictSeq evict_seq(const EvictParams &p, int64_t b) {
  EvictSeq s;
  s.len = p.lens[b];
  const int64_t pages = s.len > 0 ? (int64_t(s.len) + p.P - 1) / p.P : 0;
  s.n = int(pages < p.max_pages ? pages : p.max_pages);
  s.last = s.n - p.recent;
  s.count = evict_count(s.n, p.sink, p.recent, p.keep[b], p.max_victims);
  return s;
}

// The digit of the need-th lowest key in `hist` (256 counts; the last one if there are
// fewer), the rank left within it and whether that is all the keys with this digit, into
// pick[0..2], min(need, keys) into pick[3]; for one warp.
__device__ __forceinline__ void pick_digit(const uint32_t *hist, uint32_t need, uint32_t *pick, int lane) {
  uint32_t c[8], sum = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum += c[j] = hist[lane * 8 + j];
  uint32_t before = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  need = min(need, __shfl_sync(0xffffffffu, before, 31));
  if (lane == 0) pick[3] = need;
  before -= sum;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (before < need && need <= before + c[j]) {
      pick[0] = uint32_t(lane * 8 + j);
      pick[1] = need - before;
      pick[2] = need - before == c[j];
    }
    before += c[j];
  }
}

// `cap`: pages that a CTA's dynamic shared memory holds (8 bytes each).
__global__ void __launch_bounds__(kEvictThreads) evict_cluster_kernel(const __grid_constant__ EvictParams p, int cap) {
  extern __shared__ __align__(16) unsigned char pages_smem[];
  __shared__ uint32_t hist[2][256], total[256], pick[4];
  __shared__ uint32_t warp_below[32], warp_equal[32], cta_count[2], ahead[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call
  float *const w_s = reinterpret_cast<float *>(pages_smem);
  int32_t *const t_s = reinterpret_cast<int32_t *>(w_s + cap);
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int64_t b = blockIdx.x / unsigned(cs);
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  auto sync = [&]() {
    if (cs > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  const EvictSeq q = evict_seq(p, b);
  const int n = q.n;
  int count = q.count;
  const int slice = min(cap, ((n + cs - 1) / cs + 31) & ~31);
  const int lo = min(n, rank * slice), mine = min(n, lo + slice) - lo;
  int absent = 0;
#pragma unroll 4
  for (int i = tid; i < mine; i += kEvictThreads) {
    w_s[i] = p.weights[b * p.w_sb + lo + i];
    t_s[i] = p.table[b * p.t_sb + lo + i];
    absent |= t_s[i] < 0;
  }
  if (tid < 512) hist[tid >> 8][tid & 255] = 0;
  const bool all_present = !__syncthreads_or(absent);   // of this CTA's: the usual case

  // the leading digits (mask) of the key of the last page that leaves, and how many
  // pages with those digits do; once that is all of them, further digits do not matter
  uint32_t key = 0, mask = 0, need = uint32_t(count);
  if (count > 0) {
    const int from = max(0, p.sink - lo), to = min(mine, q.last - lo);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      uint32_t *h = hist[pass & 1];
      for (int i = from + tid; i < to; i += kEvictThreads) {
        const uint32_t k = order_key(w_s[i]);
        if ((k & mask) == key && (all_present || t_s[i] >= 0)) atomicAdd(&h[(k >> shift) & 255], 1u);
      }
      sync();
      if (tid < 256) {
        uint32_t sum = 0;
        for (int r = 0; r < cs; ++r) sum += cluster.map_shared_rank(h, r)[tid];
        total[tid] = sum;
        // the other histogram was last read before the barrier above
        hist[(pass & 1) ^ 1][tid] = 0;
      }
      __syncthreads();
      if (warp == 0) pick_digit(total, need, pick, lane);
      __syncthreads();
      if (pass == 0) count = int(pick[3]);
      if (count == 0) break;
      key |= pick[0] << shift;
      mask |= 255u << shift;
      need = pick[1];
      if (pick[2]) break;
    }
  }

  // keys below and equal: per warp (a run of pages each), CTA and cluster
  const int run = ((slice + kEvictThreads - 1) / kEvictThreads) * 32;
  const int w0 = min(mine, warp * run), w1 = min(mine, w0 + run);
  auto flags = [&](int i, bool *below, bool *equal) {
    *below = *equal = false;
    if (count > 0 && i < w1 && lo + i >= p.sink && lo + i < q.last && (all_present || t_s[i] >= 0)) {
      const uint32_t k = order_key(w_s[i]);
      *below = (k & mask) < key;
      *equal = (k & mask) == key;
    }
  };
  uint32_t below0 = 0, equal0 = 0;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    bool below, equal;
    flags(i, &below, &equal);
    below0 += __popc(__ballot_sync(0xffffffffu, below));
    equal0 += __popc(__ballot_sync(0xffffffffu, equal));
  }
  if (lane == 0) {
    warp_below[warp] = below0;
    warp_equal[warp] = equal0;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t x = warp_below[lane], y = warp_equal[lane];
    const uint32_t x0 = x, y0 = y;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t xo = __shfl_up_sync(0xffffffffu, x, o), yo = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += xo, y += yo;
    }
    warp_below[lane] = x - x0;
    warp_equal[lane] = y - y0;
    if (lane == 31) cta_count[0] = x, cta_count[1] = y;
  }
  sync();                                         // and every CTA has read its pages
  if (warp == 0) {
    uint32_t x = 0, y = 0;
    if (lane < rank) {
      const uint32_t *c = cluster.map_shared_rank(cta_count, lane);
      x = c[0];
      y = c[1];
    }
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    if (lane == 0) ahead[0] = x, ahead[1] = y;
  }
  __syncthreads();
  below0 = ahead[0] + warp_below[warp];
  equal0 = ahead[1] + warp_equal[warp];
  const uint32_t lower = (1u << lane) - 1u;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    bool below, equal;
    flags(i, &below, &equal);
    const uint32_t bm = __ballot_sync(0xffffffffu, below), em = __ballot_sync(0xffffffffu, equal);
    const uint32_t nb = below0 + __popc(bm & lower), ne = equal0 + __popc(em & lower);
    const uint32_t gone = nb + min(ne, need);     // pages before this one that leave
    if (i < w1) {
      if (below || (equal && ne < need)) {
        p.victims[b * p.v_sb + gone] = t_s[i];
      } else {
        p.out_table[b * p.ot_sb + lo + i - gone] = t_s[i];
        p.out_weights[b * p.ow_sb + lo + i - gone] = w_s[i];
      }
    }
    below0 += __popc(bm);
    equal0 += __popc(em);
  }
  for (int i = n - count + rank * kEvictThreads + tid; i < n; i += cs * kEvictThreads) {
    p.out_table[b * p.ot_sb + i] = -1;
    p.out_weights[b * p.ow_sb + i] = 0.f;
  }
  if (rank == 0 && tid == 0) {
    p.num_victims[b] = count;
    p.out_lens[b] = q.len - count * p.P;
  }
  if (cs > 1) cluster.sync();                     // nobody reads this CTA's memory any more
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[4];
  __shared__ unsigned long long warp_sum[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call
  const int64_t b = blockIdx.x;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const EvictSeq q = evict_seq(p, b);
  const int n = q.n, last = q.last;
  int count = q.count;
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
        if ((k & mask) == key && table[i] >= 0) atomicAdd(&hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) pick_digit(hist, need, pick, lane);
      __syncthreads();
      if (shift == 24) count = int(pick[3]);
      if (count == 0) break;
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
    if (count > 0 && i >= p.sink && i < last && page >= 0) {
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
    p.out_lens[b] = q.len - count * p.P;
  }
}

}  // namespace

int launch_evict(const EvictParams &p, int device, void *stream) {
  constexpr int kMaxDevices = 64;
  constexpr int kCap = 24576;                     // pages of a CTA: 192 KiB of shared memory
  constexpr int kCluster = 16;
  // One CTA a sequence up to 4,096 pages (one sequence of 4,000: 8.9 us, 7.7 by 16 CTAs;
  // but 5.6 against 7.5 at 1,000 pages and 10.2 against 83 for 64 sequences).  Beyond,
  // as many as let every sequence's cluster run at once: large clusters find few places
  // (8 sequences of 16,384 pages: 18.7 us by 16 CTAs each, 10.3 by 8, 22.0 by one;
  // 64: 97 by 16, 17.7 by 2, 23.8 by one).  And no fewer than hold the pages.
  int cs = 1;
  if (p.max_pages > 4096) cs = p.B <= 4 ? 16 : p.B <= 9 ? 8 : p.B <= 32 ? 4 : p.B <= 76 ? 2 : 1;
  while (cs < kCluster && int64_t(cs) * kCap < p.max_pages) cs *= 2;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(cs);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.blockDim = dim3(kEvictThreads);
  c.stream = static_cast<cudaStream_t>(stream);
  c.attrs = at;
  cudaError_t e;
  if (p.max_pages > kCluster * kCap) {
    c.gridDim = dim3(unsigned(p.B));
    c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, evict_kernel, p);
  } else {
    static std::atomic<bool> ready[kMaxDevices];
    if (device >= kMaxDevices || !ready[device].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(evict_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCap * 8);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(evict_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return int(e);
      if (device < kMaxDevices) ready[device].store(true, std::memory_order_release);
    }
    const int cap = ((p.max_pages + cs - 1) / cs + 31) & ~31;
    c.gridDim = dim3(unsigned(p.B) * unsigned(cs));
    c.dynamicSmemBytes = size_t(cap) * 8;
    c.numAttrs = 2;
    e = cudaLaunchKernelEx(&c, evict_cluster_kernel, p, cap);
  }
  return int(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace hicache
