// hicache_append.cu -- norms of the query and key heads, the position rotation
// and the store of K and V into the paged cache, in one pass.
//
// Nothing is used twice, so memory binds, once the arithmetic on the way (norm,
// rotation, conversions) is short enough.  A warp takes 4 heads of a token at a time,
// 8 lanes a head: a vector of each 128 bytes of it per lane, so that the sum of
// squares takes three shuffles however long the head, and every access is whole
// 128-byte lines.  What depends on the token alone (cosines, sines, norm weights) is
// read once for all its heads of a warp, and the next heads are on their way while
// these are worked on.
//
// Two kernels: the usual shapes, where partners half a rotation away can be had
// without shared memory, and any shape.  Measured, 8,191 tokens of 32 + 8 heads of
// 128 (206 MB): 36 us, 5.7 TB/s, 85% of the rate of a plain copy.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "hicache_serving.h"

namespace hicache {
namespace {

constexpr int kAppendThreads = 128;

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

constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kLanes = 8, kGroups = 32 / kLanes;  // lanes of a head, heads of a warp

__device__ __forceinline__ void load8(const float *p, float *x) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The cosines and (signed) sines of the eight elements e0.. of a rotation, and which
// of them belong to it.  WHOLE: all of them do, and they lie in one half.
template <bool WHOLE>
__device__ __forceinline__ uint32_t rotation8(const AppendParams &p, const float *row, int e0, float *cs, float *sn) {
  const int half = p.rot >> 1;
  if constexpr (WHOLE) {
    if (p.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4 *>(row + (e0 >> 1)));
      const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + (e0 >> 1)));
      cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
      sn[0] = -s.x, sn[1] = s.x, sn[2] = -s.y, sn[3] = s.y, sn[4] = -s.z, sn[5] = s.z, sn[6] = -s.w, sn[7] = s.w;
    } else {
      const bool second = e0 >= half;
      load8(row + (second ? e0 - half : e0), cs);
      load8(row + (second ? e0 : e0 + half), sn);
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = second ? sn[i] : -sn[i];
    }
    return 255u;
  } else {
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      if (e < 0 || e >= p.rot) continue;
      const bool second = p.interleaved ? (e & 1) : e >= half;
      const int j = p.interleaved ? e >> 1 : second ? e - half : e;
      in |= 1u << i;
      cs[i] = __ldg(row + j);
      sn[i] = second ? __ldg(row + half + j) : -__ldg(row + half + j);
    }
    return in;
  }
}

// ---- the usual shapes ------------------------------------------------------------
// Where the head is whole 64 elements (ITERS vectors a lane), the norm covers whole
// 64s and a vector's partners are one vector that the warp can reach without shared
// memory, the sum is regrouped: with a partner z of element y
//   out_y = r * (y * (w_y cos) + z * (w_z sin)),
// the two coefficients are worked out once per token and kind, and an element costs
// a multiply, a multiply-add, a multiply and its share of the sum of squares, all of
// them on pairs (fma.rn.f32x2).  Against the general kernel below: a prefill chunk of
// 8,191 tokens of 48 heads of 128 takes 36 us instead of 61.
enum : int { kSelf = 0, kAcross = 1, kInside = 2 };   // where partners are: ITERS / 2 vectors
                                                      // on, 4 lanes on, in the vector itself

// Every warp that the SMs hold at once takes an even share of all steps (a step: 4
// heads of one kind of a token), across tokens, so that none idles behind the last
// ones, and copies of its next steps run ahead through a ring in shared memory.
// Measured, 8,191 tokens of 32 + 8 heads of 128 and 4,096 of 16 + 1 heads of 576: a
// warp per token with one step ahead in registers 45 and 40 us, shared out 42 and 35,
// and 36 and 30 with the ring.
//   heads of 64:  5 CTAs an SM, 2 steps ahead: 23.5 us for the 8,191 (4 CTAs 25)
//            128: 4 CTAs, 3 steps: 35.6 (5 CTAs spill, 39; 3 CTAs 38.7; 2 steps 37.1)
//            256: 3 CTAs, 2 steps: 68.1 (4 steps 69.0)
//            576: 3 CTAs, 2 steps: 29.7 for the 4,096, 107 for 16,000 (4 CTAs spill, 28.9 and 118)
constexpr int append_ctas(int iters) { return iters == 1 ? 5 : iters == 2 ? 4 : 3; }
template <int ITERS>
constexpr int kAppendSlots = ITERS == 2 ? 3 : 2;

struct AppendDeal {
  int steps;                                      // of each warp, one more of the first `longer`
  uint32_t longer;
  FastDiv fd_steps;                               // by a token's steps
};

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// to two units of the last place
__device__ __forceinline__ float rsqrt_fast(float x) {
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  if constexpr (BF16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return pair(f.x, f.y);
}
__device__ __forceinline__ uint64_t swapped(uint64_t x) {
  const float2 f = unpair(x);
  return pair(f.y, f.x);
}

// E4M3: whether the cache is; the inlined divisions, in the way of the others, cost long
// heads a sixth of their time (35 against 29.5 us for the 4,096).
template <int ITERS, bool BF16, int MODE, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, append_ctas(ITERS))
    append_fast_kernel(const __grid_constant__ AppendParams p, const AppendDeal deal) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call
  constexpr bool HOLD = ITERS <= 4;               // coefficients of every vector in registers
  constexpr int SLOTS = kAppendSlots<ITERS>;
  const int warp = int(threadIdx.x) >> 5;
  const int sub = (int(threadIdx.x) & 31) / kLanes, lane = int(threadIdx.x) & (kLanes - 1);
  // a step: 4 heads of one kind
  const int q_steps = (p.q_heads + kGroups - 1) / kGroups, kv_steps = (p.kv_heads + kGroups - 1) / kGroups;
  const int all_steps = q_steps + kv_steps * (p.has_v ? 2 : 1);
  // this warp's steps: `count` of them from step `s` of token n on
  const uint32_t w = blockIdx.x * uint32_t(kAppendWarps) + uint32_t(warp);
  const int count = deal.steps + (w < deal.longer ? 1 : 0);
  const uint32_t past = w * uint32_t(deal.steps) + min(w, deal.longer);   // < 2^31 in all
  int64_t n = fast_div(past, deal.fd_steps);
  int s = int(past - uint32_t(n) * uint32_t(all_steps));
  // the step to fetch next: its source, the step its kind ends at, heads of the kind
  // from this one on
  const char *f_src = nullptr;
  int64_t f_step = 0;
  int64_t f_n = n;
  int f_s = s, f_end = 0, f_left = 0, f_count = count;
  auto seek = [&]() {
    const int kind = f_s < q_steps ? 0 : f_s < q_steps + kv_steps ? 1 : 2;
    const int begin = kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + kv_steps;
    const int64_t sh = kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh;
    const int h = (f_s - begin) * kGroups + sub;
    f_src = static_cast<const char *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
            2 * (f_n * (kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st) + h * sh) + lane * 16;
    f_step = 2 * kGroups * sh;
    f_end = begin + (kind == 0 ? q_steps : kv_steps);
    f_left = (kind == 0 ? p.q_heads : p.kv_heads) - h;
  };
  // a ring of steps; a lane reads only what it has copied itself
  __shared__ uint4 ring[kAppendWarps][SLOTS][ITERS][32];
  uint4 *const mine = &ring[warp][0][0][threadIdx.x & 31];
  int f_slot = 0;                                 // to be read, then to be fetched into
  auto fetch = [&]() {
    if (f_s == all_steps) f_s = f_end = 0, ++f_n;
    if (f_s >= f_end && f_count > 0) seek();
    const bool have = f_count > 0 && f_left > 0;
    if (have) {
      const uint32_t to = uint32_t(__cvta_generic_to_shared(mine + f_slot * (ITERS * 32)));
#pragma unroll
      for (int it = 0; it < ITERS; ++it)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + it * 512), "l"(f_src + it * (kLanes * 16))
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    f_slot = f_slot + 1 == SLOTS ? 0 : f_slot + 1;
    ++f_s;
    --f_count;
    f_left -= kGroups;
    f_src += f_step;
  };
  int64_t slot = -1;
  bool known = true;                              // whether the position is in the table
  const float *row = nullptr;
  auto place = [&]() {
    slot = p.kv_heads > 0 ? p.slots[n] : -1;
    if (slot >= p.num_slots) slot = -1;
    if (p.rot == 0) return;
    const int64_t pos = p.positions[n];
    known = pos >= 0 && pos < p.cos_sin_rows;
    row = p.cos_sin + pos * p.rot;
  };
  if (count > 0) place();
#pragma unroll 1
  for (int i = 0; i < SLOTS; ++i) fetch();
  // long heads: the weights in shared memory, where they cost no registers
  __shared__ uint4 weights[HOLD ? 1 : 2][HOLD ? 1 : kLanes * ITERS];
  if constexpr (!HOLD) {
    for (int i = int(threadIdx.x); i < kLanes * ITERS; i += kAppendThreads) {
      if (i * 8 < p.q_norm) weights[0][i] = __ldg(static_cast<const uint4 *>(p.q_weight) + i);
      if (i * 8 < p.k_norm) weights[1][i] = __ldg(static_cast<const uint4 *>(p.k_weight) + i);
    }
    __syncthreads();
  }
  if (count == 0) return;                         // the whole warp

  // coefficients of the current kind: of the element and of its partner
  uint64_t own[HOLD ? ITERS : 1][4], mate[HOLD ? ITERS : 1][4];
  float cs1[HOLD ? 1 : 8], sn1[HOLD ? 1 : 8];     // and the rotation of the one vector it turns
  int kind = 0, m = 0, s_end = 0, left = 0;       // the current kind, where it ends, heads from this one on
  float inv_m = 0.f;
  char *dst = nullptr;
  int64_t dst_step = 0;
  auto turned = [&](int it) {                     // whether vector `it` is rotated (the same in all lanes)
    return known && p.rot > 0 && it * 64 >= p.rot_off && it * 64 < p.rot_off + p.rot;
  };
  auto prepare = [&](int kind) {
    m = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : 0;
    inv_m = m > 0 ? 1.f / float(m) : 0.f;
    const uint4 *w = static_cast<const uint4 *>(kind == 0 ? p.q_weight : p.k_weight);
    if constexpr (HOLD) {
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int c = lane + it * kLanes;
        const bool turn = kind != 2 && turned(it);
        float a[8], z[8], cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = z[i] = cs[i] = 1.f, sn[i] = 0.f;
        if (it * 64 < m) {
          unpack8<BF16>(__ldg(w + c), a);
          if (MODE == kInside) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = a[i ^ 1];
          } else {
            unpack8<BF16>(__ldg(w + (MODE == kSelf ? c ^ (ITERS / 2 * kLanes) : c ^ 4)), z);
          }
        }
        if (turn) rotation8<true>(p, row, c * 8 - p.rot_off, cs, sn);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          own[it][i] = pair(a[2 * i] * cs[2 * i], a[2 * i + 1] * cs[2 * i + 1]);
          mate[it][i] = pair(z[2 * i] * sn[2 * i], z[2 * i + 1] * sn[2 * i + 1]);
        }
      }
    } else {
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        if (turned(it)) rotation8<true>(p, row, (lane + it * kLanes) * 8 - p.rot_off, cs1, sn1);
      }
    }
  };

#pragma unroll 1
  for (int i = 0; i < count; ++i, ++s) {
    if (s == all_steps) {                         // on to the next token
      s = s_end = 0;
      ++n;
      place();
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    uint4 raw[ITERS];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) raw[it] = mine[f_slot * (ITERS * 32) + it * 32];
    if (s >= s_end) {                             // on to the next kind: its coefficients and places
      kind = s < q_steps ? 0 : s < q_steps + kv_steps ? 1 : 2;
      const int begin = kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + kv_steps;
      s_end = begin + (kind == 0 ? q_steps : kv_steps);
      const int h = (s - begin) * kGroups + sub;
      left = !known ? 0 : kind == 0 ? p.q_heads - h : slot >= 0 ? p.kv_heads - h : 0;
      const int vec = kind != 0 && E4M3 ? 8 : 16;              // bytes that 8 elements take
      const int64_t sh = kind == 0 ? p.o_sh : p.D;
      const int64_t at = kind == 0 ? n * p.o_st + h * sh : slot * p.row + h * sh;
      dst = static_cast<char *>(kind == 0 ? p.q_out : kind == 1 ? p.k_cache : p.v_cache) + at * (vec / 8) + lane * vec;
      dst_step = kGroups * sh * (vec / 8);
      if (kind != 2 || E4M3) prepare(kind);
    }
    const bool live = left > 0;
    char *const to = dst;
    left -= kGroups;
    dst += dst_step;
    if (kind == 2 && !E4M3) {                   // as it came
#pragma unroll
      for (int it = 0; it < ITERS; ++it)
        if (live) reinterpret_cast<uint4 *>(to)[it * kLanes] = raw[it];
      fetch();
      continue;
    }
    uint64_t v[HOLD ? ITERS : 1][4];              // not held: widened again for the second pass
    uint64_t sq = 0;
    uint32_t across[HOLD && MODE == kAcross ? ITERS : 1][4];      // the partners, as they come
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const uint32_t w[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (HOLD) {
          v[it][i] = widen<BF16>(w[i]);
        } else if (it * 64 < m) {
          const uint64_t x = widen<BF16>(w[i]);
          sq = fma2(x, x, sq);
        }
        if constexpr (HOLD && MODE == kAcross) across[it][i] = __shfl_xor_sync(0xffffffffu, w[i], 4);
      }
    }
    fetch();                                      // into the slot just read
    float r = 1.f;
    if (m > 0) {
#pragma unroll
      for (int it = 0; it < ITERS; ++it)
        if (HOLD && it * 64 < m) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sq = fma2(v[HOLD ? it : 0][i], v[HOLD ? it : 0][i], sq);
        }
      const float2 f = unpair(sq);
      float sum = f.x + f.y;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrt_fast(fmaf(sum, inv_m, p.eps));
    }
    auto store = [&](int it, const float *x) {
      if (kind != 0 && E4M3)
        reinterpret_cast<uint2 *>(to)[it * kLanes] = pack8_e4m3(x, kind == 1 ? p.k_scale : p.v_scale);
      else
        reinterpret_cast<uint4 *>(to)[it * kLanes] = pack8<BF16>(x);
    };
    float out[HOLD ? ITERS : 1][8];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const float rr = it * 64 < m ? r : 1.f;
      const uint64_t r2 = pair(rr, rr);
      const bool turn = kind != 2 && turned(it);
      uint64_t x[4];
      if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(v[it][i], own[it][i]);
      } else {
        const uint32_t y[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
        const uint4 f = weights[kind == 0 ? 0 : 1][lane + it * kLanes];
        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = it * 64 < m ? mul2(widen<BF16>(y[i]), widen<BF16>(w[i])) : widen<BF16>(y[i]);
      }
      if (turn) {
        uint64_t z[4];
        if constexpr (MODE == kSelf) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = v[it ^ (ITERS / 2)][i];
        } else if constexpr (MODE == kInside) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = swapped(HOLD ? v[HOLD ? it : 0][i] : x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if constexpr (HOLD) {
              z[i] = widen<BF16>(across[it][i]);
            } else {
              const float2 f = unpair(x[i]);
              z[i] = pair(__shfl_xor_sync(0xffffffffu, f.x, 4), __shfl_xor_sync(0xffffffffu, f.y, 4));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if constexpr (HOLD)
            x[i] = fma2(z[i], mate[it][i], x[i]);
          else
            x[i] = fma2(z[i], pair(sn1[2 * i], sn1[2 * i + 1]), mul2(x[i], pair(cs1[2 * i], cs1[2 * i + 1])));
      }
      float *const y = out[HOLD ? it : 0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpair(mul2(x[i], r2));
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
      }
      if (!HOLD && live) store(it, y);
    }
    if (HOLD && live) {
#pragma unroll
      for (int it = 0; it < ITERS; ++it) store(it, out[HOLD ? it : 0]);
    }
  }
}

// The kernel for p's shape, or null where only the general one will do.
using AppendFast = void (*)(const AppendParams, const AppendDeal);
template <int ITERS, int MODE>
AppendFast fast_of(const AppendParams &p) {
  return p.bf16 ? (p.e4m3 ? append_fast_kernel<ITERS, true, MODE, true> : append_fast_kernel<ITERS, true, MODE, false>)
                : (p.e4m3 ? append_fast_kernel<ITERS, false, MODE, true> : append_fast_kernel<ITERS, false, MODE, false>);
}
AppendFast append_fast(const AppendParams &p) {
  if (p.D % 64 || reinterpret_cast<uintptr_t>(p.cos_sin) % 16) return nullptr;
  if (p.q_norm % 64 || p.k_norm % 64 || p.rot_off % 64) return nullptr;
  const bool every = (p.q_norm == 0 || p.q_norm == p.D) && (p.k_norm == 0 || p.k_norm == p.D);
  if (p.rot == 0 || (p.interleaved && p.rot % 64 == 0)) {
    if (p.D == 64) return fast_of<1, kInside>(p);
    if (p.D == 128) return fast_of<2, kInside>(p);
    if (p.D == 256) return fast_of<4, kInside>(p);
    if (p.D == 576 && p.rot <= 64) return fast_of<9, kInside>(p);
  } else if (!p.interleaved && p.rot == 64) {
    if (p.D == 64) return fast_of<1, kAcross>(p);
    if (p.D == 128) return fast_of<2, kAcross>(p);
    if (p.D == 256) return fast_of<4, kAcross>(p);
    if (p.D == 576) return fast_of<9, kAcross>(p);
  } else if (!p.interleaved && p.rot == p.D && every) {
    if (p.D == 128) return fast_of<2, kSelf>(p);
    if (p.D == 256) return fast_of<4, kSelf>(p);
  }
  return nullptr;
}

// ---- any shape -------------------------------------------------------------------
// ITERS: 16-byte vectors of a head per lane; `segments` tasks per token, `reps`
// times AHEAD heads of each group per task.  WHOLE: the rotation begins and ends at
// whole vectors in either half, and the table's rows at 16 bytes.
template <int ITERS, bool BF16, bool WHOLE>
__global__ void __launch_bounds__(kAppendThreads, ITERS <= 4 ? 4 : 3)
    append_kernel(const __grid_constant__ AppendParams p, int reps, FastDiv fd_segments) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call
  constexpr int AHEAD = ITERS == 1 ? 4 : ITERS == 2 ? 2 : 1;
  constexpr bool HOLD = ITERS <= 2;               // cosines, sines and weights in registers
  constexpr int UPPER = 32 * ITERS;
  __shared__ float4 stage_all[kAppendWarps][2 * 32 * ITERS];
  const int warp = int(threadIdx.x) >> 5;
  const uint32_t task = blockIdx.x * uint32_t(kAppendWarps) + uint32_t(warp);
  const uint32_t n = fast_div(task, fd_segments);
  if (int64_t(n) >= p.num_tokens) return;         // the whole warp
  const int sub = (int(threadIdx.x) & 31) / kLanes, lane = int(threadIdx.x) & (kLanes - 1);
  const int units = p.q_heads + p.kv_heads * (p.has_v ? 2 : 1);
  const int u_first = int(task - n * fd_segments.d) * kGroups * AHEAD * reps;
  const int u_end = min(units, u_first + kGroups * AHEAD * reps);
  const int chunks = p.D >> 3;
  const char *const q_n = static_cast<const char *>(p.q) + 2 * int64_t(n) * p.q_st;
  const char *const k_n = static_cast<const char *>(p.k) + 2 * int64_t(n) * p.k_st;
  const char *const v_n = static_cast<const char *>(p.v) + 2 * int64_t(n) * p.v_st;
  // the vectors of AHEAD heads; the next ones are fetched before these are used, the
  // first ones before anything that depends on the token's position or slot
  uint4 ahead[AHEAD][ITERS];
  auto fetch = [&](int u0) {
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int u = u0 + x * kGroups + sub;
      const bool is_q = u < p.q_heads, is_k = !is_q && u < p.q_heads + p.kv_heads;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          is_q ? q_n + 2 * u * p.q_sh
               : is_k ? k_n + 2 * (u - p.q_heads) * p.k_sh : v_n + 2 * (u - p.q_heads - p.kv_heads) * p.v_sh);
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int c = lane + it * kLanes;
        ahead[x][it] = u < u_end && c < chunks ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  int64_t pos = 0, slot = -1;
  if (p.kv_heads > 0) slot = p.slots[n];
  if (p.rot > 0) pos = p.positions[n];
  fetch(u_first);
  if (p.rot > 0 && (pos < 0 || pos >= p.cos_sin_rows)) return;   // the whole warp
  const bool store_kv = slot >= 0 && slot < p.num_slots;
  const float *row = p.cos_sin + pos * p.rot;
  const int half = p.rot >> 1;
  const bool exchange = half > 0 && !p.interleaved;

  float cs[HOLD ? ITERS : 1][8], sn[HOLD ? ITERS : 1][8], qw[HOLD ? ITERS : 1][8], kw[HOLD ? ITERS : 1][8];
  uint32_t turned[ITERS];                         // a bit per element
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int c = lane + it * kLanes, e0 = c * 8 - p.rot_off;
    turned[it] = c < chunks && e0 > -8 && e0 < p.rot ? 255u : 0u;
    if constexpr (HOLD) {
      if (turned[it]) turned[it] = rotation8<WHOLE>(p, row, e0, cs[it], sn[it]);
      if (c * 8 < p.q_norm) unpack8<BF16>(__ldg(static_cast<const uint4 *>(p.q_weight) + c), qw[it]);
      if (c * 8 < p.k_norm) unpack8<BF16>(__ldg(static_cast<const uint4 *>(p.k_weight) + c), kw[it]);
    }
  }
  // the group's head in shared memory: the lower and the upper four of each vector
  float4 *const stage = stage_all[warp] + sub * kLanes * ITERS;
  for (int u0 = u_first; u0 < u_end; u0 += kGroups * AHEAD) {
    uint4 raw[AHEAD][ITERS];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x)
#pragma unroll
      for (int it = 0; it < ITERS; ++it) raw[x][it] = ahead[x][it];
    if (u0 + kGroups * AHEAD < u_end) fetch(u0 + kGroups * AHEAD);
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      if (u0 + x * kGroups >= u_end) break;       // the whole warp
      const int u = u0 + x * kGroups + sub;
      const bool is_q = u < p.q_heads, is_k = !is_q && u < p.q_heads + p.kv_heads;
      const bool live = u < u_end && (is_q || store_kv);
      const int m = is_q ? p.q_norm : is_k ? p.k_norm : 0;
      float v[ITERS][8];
      float sum = 0.f;
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        unpack8<BF16>(raw[x][it], v[it]);
        if ((lane + it * kLanes) * 8 < m) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(v[it][i], v[it][i], sum);
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (m > 0) {
        const float r = rsqrtf(__fdividef(sum, float(m)) + p.eps);
#pragma unroll
        for (int it = 0; it < ITERS; ++it) {
          const int c = lane + it * kLanes;
          if (c * 8 >= m) continue;
          if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[it][i] *= r * (is_q ? qw[it][i] : kw[it][i]);
          } else {
            float w[8];
            unpack8<BF16>(__ldg(static_cast<const uint4 *>(is_q ? p.q_weight : p.k_weight) + c), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[it][i] *= r * w[i];
          }
        }
      }
      const bool turn = is_q || is_k;
      if (exchange) {
        __syncwarp();                             // the head before has been read
#pragma unroll
        for (int it = 0; it < ITERS; ++it)
          if (turned[it]) {
            stage[lane + it * kLanes] = make_float4(v[it][0], v[it][1], v[it][2], v[it][3]);
            stage[UPPER + lane + it * kLanes] = make_float4(v[it][4], v[it][5], v[it][6], v[it][7]);
          }
        __syncwarp();
      }
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        if (!turn || !turned[it]) continue;
        const int e0 = (lane + it * kLanes) * 8 - p.rot_off;
        float cl[8], sl[8];
        uint32_t in = turned[it];
        const float *cp = cl, *sp = sl;
        if constexpr (HOLD)
          cp = cs[it], sp = sn[it];
        else
          in = rotation8<WHOLE>(p, row, e0, cl, sl);
        float y[8];
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = v[it][i ^ 1];
        } else if constexpr (WHOLE) {
          const int at = ((e0 < half ? e0 + half : e0 - half) + p.rot_off) >> 3;
          const float4 a = stage[at], b = stage[UPPER + at];
          y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = e0 + i, at = ((in >> i) & 1u) ? (e < half ? e + half : e - half) + p.rot_off : 0;
            y[i] = ((in >> i) & 1u) ? reinterpret_cast<const float *>(stage + ((at & 4) ? UPPER : 0) + (at >> 3))[at & 3]
                                    : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (WHOLE || ((in >> i) & 1u)) v[it][i] = fmaf(v[it][i], cp[i], y[i] * sp[i]);
      }
      if (!live) continue;
      char *const dst = static_cast<char *>(p.q_out) + 2 * (int64_t(n) * p.o_st + int64_t(u) * p.o_sh);
      const int64_t at = slot * p.row + (is_k ? u - p.q_heads : u - p.q_heads - p.kv_heads) * int64_t(p.D);
      char *const buf = static_cast<char *>(is_k ? p.k_cache : p.v_cache);
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int c = lane + it * kLanes;
        if (c >= chunks) continue;
        if (is_q)
          reinterpret_cast<uint4 *>(dst)[c] = pack8<BF16>(v[it]);
        else if (p.e4m3)
          reinterpret_cast<uint2 *>(buf + at)[c] = pack8_e4m3(v[it], is_k ? p.k_scale : p.v_scale);
        else
          reinterpret_cast<uint4 *>(buf + 2 * at)[c] = pack8<BF16>(v[it]);
      }
    }
  }
}

using AppendKernel = void (*)(const AppendParams, int, FastDiv);
template <int ITERS>
AppendKernel append_kernel_of(const AppendParams &p) {
  const int half = p.rot / 2;
  const bool whole = p.rot_off % 8 == 0 && (p.interleaved ? p.rot : half) % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(p.cos_sin) % 16 == 0;
  return p.bf16 ? (whole ? append_kernel<ITERS, true, true> : append_kernel<ITERS, true, false>)
                : (whole ? append_kernel<ITERS, false, true> : append_kernel<ITERS, false, false>);
}

}  // namespace

int launch_append(const AppendParams &p, void *stream) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.blockDim = dim3(kAppendThreads);
  c.stream = static_cast<cudaStream_t>(stream);
  c.attrs = &at;
  c.numAttrs = 1;
  if (AppendFast k = append_fast(p)) {
    const int steps = (p.q_heads + kGroups - 1) / kGroups + (p.kv_heads + kGroups - 1) / kGroups * (p.has_v ? 2 : 1);
    const int64_t total = p.num_tokens * steps, most = 152 * append_ctas(p.D / 64);
    const int64_t ctas = (total + kAppendWarps - 1) / kAppendWarps;
    c.gridDim = dim3(unsigned(ctas < most ? ctas : most));
    const int64_t warps = int64_t(c.gridDim.x) * kAppendWarps;
    const AppendDeal deal{int(total / warps), uint32_t(total % warps), make_fastdiv(uint32_t(steps))};
    const cudaError_t e = cudaLaunchKernelEx(&c, k, p, deal);
    return int(e != cudaSuccess ? e : cudaGetLastError());
  }
  const int iters = (p.D / 8 + kLanes - 1) / kLanes;
  AppendKernel k = iters == 1   ? append_kernel_of<1>(p)
                   : iters == 2 ? append_kernel_of<2>(p)
                   : iters == 3 ? append_kernel_of<3>(p)
                   : iters == 4 ? append_kernel_of<4>(p)
                   : iters <= 9 ? append_kernel_of<9>(p)
                                : append_kernel_of<12>(p);
  // a warp per token, unless the SMs hold several: then its heads are dealt to as many
  // as there is room for, so that all tasks run at once.  One more than that, and the
  // last wait for the first: 900 tokens of 32 + 8 heads of 96 take 8.6 us, where three
  // tasks each took 11.4.
  const int step = kGroups * (iters == 1 ? 4 : iters == 2 ? 2 : 1);
  const int most = (p.q_heads + p.kv_heads * (p.has_v ? 2 : 1) + step - 1) / step;
  int64_t segments = int64_t(152) * kAppendWarps * (iters <= 4 ? 4 : 3) / p.num_tokens;
  segments = segments < 1 ? 1 : segments > most ? most : segments;
  const int per_task = int((most + segments - 1) / segments);
  segments = (most + per_task - 1) / per_task;
  c.gridDim = dim3(unsigned((p.num_tokens * segments + kAppendWarps - 1) / kAppendWarps));
  const cudaError_t e = cudaLaunchKernelEx(&c, k, p, per_task, make_fastdiv(uint32_t(segments)));
  return int(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace hicache
