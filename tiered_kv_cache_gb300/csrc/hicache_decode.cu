// hicache_decode.cu -- attention of one new token per sequence over its pages.
//
// K, V caches (decode_kv_kernel).  Every cached byte is used once per group of
// query heads, so reading the pages binds: at 4 heads a group the products are
// 4 multiply-adds per element.  The work of a call is cut into tiles of 16
// tokens of one kv head, and the tiles of all sequences, in order, into one
// equal contiguous range per warp, whatever the lengths: no warp of the GPU
// has more than one tile more than another.  A warp streams its range through a
// ring of its own in shared memory (cp.async, page numbers read one tile ahead,
// no block-wide barrier until the end) and keeps a running maximum and sum per
// head.  The products are mma.sync m16n8k16 with the group's heads as the 16
// rows (8 of them unused for groups up to 8): the tensor work is a fraction of
// the time the tile's bytes take, and the exponentials of a tile are already in
// the registers that the product with V wants them in.
//
// A warp that has all tiles of a (sequence, kv head) writes the result itself.
// The others leave a partial result, joined in tile order: first among the warps
// of a CTA in shared memory, then among CTAs in the workspace, by whichever
// CTA finishes last (a counter per CTA in which such a unit begins).  Which
// pieces exist depends on the lengths alone and they are added in order, so
// timing cannot change the result.
//
// Latent caches: hicache_decode_latent.cu.

#include <cuda_fp8.h>

#include <atomic>

#include "hicache_decode.cuh"

namespace hicache {
namespace {

// ---- K, V caches -----------------------------------------------------------------

enum : int { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };   // element types of the products

constexpr int kTok = 16;                          // tokens of a tile

template <int DP_, int TYPE_, int ROWS_>
struct KvConfig {
  static constexpr int DP = DP_;                  // head_dim, padded
  static constexpr int TYPE = TYPE_;
  static constexpr int ROWS = ROWS_;              // query heads of a unit
  static constexpr int ES = TYPE_ == kE4m3 ? 1 : 2;
  static constexpr int WARPS = DP_ == 256 && TYPE_ != kE4m3 ? 4 : 8;
  static constexpr int CH = DP_ * ES / 16;        // 16-byte chunks of a row
  static constexpr int ROWB = DP_ * ES;
  static constexpr int TILE_B = 2 * kTok * ROWB;  // K and V
  // 192 KiB of ring a CTA, one CTA per SM: all but one stage in flight
  static constexpr int RAW = 192 * 1024 / (WARPS * TILE_B);
  static constexpr int STAGES = RAW > 8 ? 8 : RAW;
  static constexpr int RING_B = STAGES * TILE_B;
  static constexpr int KS = DP_ / 16;             // k steps of q . k
  static constexpr int NT = DP_ / 8;              // n tiles of the output
  static constexpr int RH = ROWS_ / 8;            // 8-row halves in use
  static constexpr int PIECE = ROWS_ * DP_ + 2 * ROWS_;   // floats of a partial result: O, m, l
  static constexpr int SMEM = WARPS * RING_B;
  static_assert(STAGES >= 2 && RING_B >= ROWS_ * DP_ * 4, "ring");
};

__device__ __forceinline__ void ldmatrix4(uint32_t *r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t *r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// c += a b, 16 x 8 x 16.  RH == 1: rows 8..15 of a are zero and their sums unused.
template <bool BF16, int RH>
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  float x = 0.f, y = 0.f;
  float &c2 = RH == 2 ? c[2] : x, &c3 = RH == 2 ? c[3] : y;
  const uint32_t a1 = RH == 2 ? a[1] : 0u, a3 = RH == 2 ? a[3] : 0u;
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c2), "+f"(c3)
        : "r"(a[0]), "r"(a1), "r"(a[2]), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c2), "+f"(c3)
        : "r"(a[0]), "r"(a1), "r"(a[2]), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 unpack2(uint32_t u, bool bf16) {
  return bf16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u))
              : __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
// two e4m3 (the low or the high 16 bits of a word) -> two fp16, exactly
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(r) : "r"(w));
  return r;
}
// Where chunk c of row r lies in its row of shared memory.  2-byte types: eight
// rows at one chunk (ldmatrix) fall on eight different 16-byte bank groups.
// e4m3 K: 16-byte loads of four chunks of two rows; e4m3 V: 4-byte loads of
// eight words of rows 0, 2, 4, 6.
template <class C, bool V>
__device__ __forceinline__ int swizzle(int c, int r) {
  if constexpr (C::TYPE != kE4m3) return c ^ (r & 7);
  if constexpr (!V) return C::CH >= 8 ? c ^ ((r & 1) << 2) : c;
  return C::CH >= 8 ? c ^ (((r >> 1) & 3) << 1) : c ^ (((r >> 1) & 1) << 1);
}

// The output element (column of the head) of n tile `tile`, element e of a
// lane with c = lane % 4.
template <class C>
__device__ __forceinline__ int column(int tile, int e, int c) {
  if constexpr (C::TYPE != kE4m3) return tile * 8 + 2 * c + e;
  return 32 * (tile >> 2) + 8 * c + 4 * e + (tile & 3);
}

// A tile in a warp's ring.  flags: the tokens present (16 bits), then whether it
// is the first (16) or the last (17) of the warp's piece of its unit, and whether
// that piece begins (18) or ends (19) the unit.
struct TileMeta {
  uint32_t flags;
  int32_t b, u, t0;   // sequence, unit within it, first token
};

__device__ __forceinline__ int tiles_of(int start, int len) {
  return len > start ? (len + kTok - 1) / kTok - start / kTok : 0;
}

template <class C>
__global__ void __launch_bounds__(C::WARPS * 32, 1) decode_kv_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) unsigned char ring_all[];
  constexpr int THREADS = C::WARPS * 32, ROWS = C::ROWS, RH = C::RH, DP = C::DP;
  constexpr bool MMA_BF16 = C::TYPE == kBf16;
  __shared__ TileMeta meta_all[C::WARPS][C::STAGES];
  __shared__ long long prefix[THREADS + 1];
  __shared__ long long warp_tot[C::WARPS];
  // the CTA's pieces, two per warp: where O lies, m and l, the unit, and
  // (4: present, 1: begins its unit, 2: ends it)
  __shared__ const float *piece_o[C::WARPS][2];
  __shared__ float piece_m[C::WARPS][2][ROWS], piece_l[C::WARPS][2][ROWS];
  __shared__ int piece_b[C::WARPS][2], piece_u[C::WARPS][2], piece_state[C::WARPS][2];
  __shared__ int last_flag;

  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const int units = p.Hkv * p.QB;                 // units of a sequence

  // ---- the tiles before each sequence; thread i takes `per` sequences
  const int per = (p.B + THREADS - 1) / THREADS;
  long long mine = 0;
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
    int start, len;
    seq_range(p, b, &start, &len);
    mine += tiles_of(start, len);
  }
  if (lane < 2) piece_state[warp][lane] = 0;
  long long total = 0;
  const long long before = block_prefix<C::WARPS>(mine, warp_tot, &total);
  total *= units;
  prefix[tid] = before * units;
  if (tid == 0) prefix[THREADS] = total;
  __syncthreads();

  // sequences of which there is nothing to attend to
  for (int b = int(blockIdx.x); b < p.B; b += int(gridDim.x)) {
    int start, len;
    seq_range(p, b, &start, &len);
    if (len > start) continue;
    for (int i = tid; i < p.Hq * DP; i += THREADS) store_out(p, b, i / DP, i % DP, 0.f);
    for (int h = tid; h < p.Hq; h += THREADS) store_lse(p, b, h, 0.f, 0.f);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // with fewer tiles than CTAs, only as many CTAs take part: each has a tile then
  const long long n_cta = min((long long)gridDim.x, total);
  if (blockIdx.x >= n_cta) return;

  const long long W = n_cta * C::WARPS, w_id = (long long)blockIdx.x * C::WARPS + warp;
  const long long lo = total * w_id / W, hi = total * (w_id + 1) / W;

  unsigned char *ring = ring_all + warp * C::RING_B;
  const uint32_t ring_s = smem_u32(ring);
  TileMeta *meta = meta_all[warp];

  // ---- the tile to load next: sequence, unit, tile of lnt
  int lb = 0, lu = 0, lt = 0, lnt = 0, lstart = 0, llen = 0, lstage = 0;
  long long lnext = lo;
  int lpage = -1, lpg = 0;                        // this lane's token: page number, its place in the table
  auto tokens_of = [&](int b) {
    seq_range(p, b, &lstart, &llen);
    lnt = tiles_of(lstart, llen);
  };
  auto fetch_page = [&]() {                       // the page of this lane's token of the next tile
    const int t = (lstart / kTok + lt) * kTok + (lane & 15);
    lpage = -1;
    if (t >= lstart && t < llen) {
      lpg = int(fast_div(uint32_t(t), p.fd_page));
      lpage = __ldg(p.table + int64_t(lb) * p.t_sb + lpg);
    }
  };
  if (lo < hi) {
    int a = 0, z = THREADS;                       // prefix[a] <= lo < prefix[z]
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (prefix[mid] <= lo) a = mid; else z = mid;
    }
    long long rest = lo - prefix[a];
    lb = a * per;
    tokens_of(lb);
    while (rest >= (long long)lnt * units && lb + 1 < p.B) {
      rest -= (long long)lnt * units;
      tokens_of(++lb);
    }
    lu = int(rest / lnt);
    lt = int(rest - (long long)lu * lnt);
    fetch_page();
  }
  auto load = [&]() {                             // one tile into the ring, and on to the next
    const int t0 = (lstart / kTok + lt) * kTok;
    const int t = t0 + (lane & 15);
    const int kvh = lu / p.QB;
    const bool ok = page_present(lpage, p.num_pages);
    int64_t off = 0;
    if (ok) off = ((int64_t(lpage) * p.P + (t - lpg * p.P)) * p.row + int64_t(kvh) * p.D) * C::ES;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    const uint32_t base = ring_s + lstage * C::TILE_B;
    constexpr int RPI = C::CH <= 32 ? 32 / C::CH : 1;         // rows per instruction
    static_assert(C::CH <= 32, "a row is at most a warp of chunks");
    const int c = lane % C::CH;
    const bool in_d = c * 16 < p.D * C::ES;
    const char *kp = static_cast<const char *>(p.k), *vp = static_cast<const char *>(p.v);
#pragma unroll
    for (int i = 0; i < kTok / RPI; ++i) {
      const int r = i * RPI + lane / C::CH;
      const int64_t o = __shfl_sync(0xffffffffu, off, r);
      const bool have = in_d && ((mask >> r) & 1u);
      const int64_t at = have ? o + c * 16 : 0;
      cp_async16(base + r * C::ROWB + swizzle<C, false>(c, r) * 16, kp + at, have ? 16 : 0);
      cp_async16(base + kTok * C::ROWB + r * C::ROWB + swizzle<C, true>(c, r) * 16, vp + at, have ? 16 : 0);
    }
    if (lane == 0) {
      uint32_t f = mask;
      if (lnext == lo || lt == 0) f |= 1u << 16;
      if (lnext == hi - 1 || lt == lnt - 1) f |= 1u << 17;
      if (lnext - lt >= lo) f |= 1u << 18;
      if (lnext - lt + lnt <= hi) f |= 1u << 19;
      meta[lstage] = TileMeta{f, lb, lu, t0};
    }
    if (++lstage == C::STAGES) lstage = 0;
    if (++lnext < hi) {
      if (++lt == lnt) {
        lt = 0;
        if (++lu == units) {
          lu = 0;
          do tokens_of(++lb); while (lnt == 0 && lb + 1 < p.B);
        }
      }
      fetch_page();
    }
  };

  // ---- stream
#pragma unroll 1
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (lnext < hi) load();
    cp_commit();
  }
  uint32_t qf[C::KS][4];                          // q as the A operand
  float qmul[2] = {0.f, 0.f};                     // scale2, and for e4m3 the power of two taken out of q
  float o[C::NT][RH * 2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int h0 = 0, rows = 0, pieces = 0, stage = 0;
#pragma unroll 1
  for (long long it = lo; it < hi; ++it) {
    __syncwarp();                                 // everyone is done with the stage that is filled next
    if (lnext < hi) load();
    cp_commit();
    cp_wait<C::STAGES - 1>();
    __syncwarp();
    const TileMeta tm = meta[stage];
    if (tm.flags & (1u << 16)) {                  // a new piece: its q
      const int kvh = tm.u / p.QB, qb = tm.u - kvh * p.QB;
      h0 = kvh * p.G + qb * ROWS;
      rows = min(ROWS, p.G - qb * ROWS);
#pragma unroll
      for (int i = 0; i < C::NT; ++i)
#pragma unroll
        for (int j = 0; j < RH * 2; ++j) o[i][j] = 0.f;
#pragma unroll
      for (int x = 0; x < RH; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
        qmul[x] = p.scale2;
        const int r = g + 8 * x;
        const char *qp = static_cast<const char *>(p.q) + 2 * (int64_t(tm.b) * p.q_sb + int64_t(h0 + r) * p.q_sh);
        const bool live = r < rows;
        if constexpr (C::TYPE != kE4m3) {
#pragma unroll
          for (int s = 0; s < C::KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = s * 16 + e * 8 + 2 * c4;
              qf[s][x + 2 * e] = live && d < p.D ? __ldg(reinterpret_cast<const unsigned int *>(qp + 2 * d)) : 0u;
            }
        } else {
          // fp16, after the power of two that brings the head's largest element
          // into [1, 2): bf16 and fp16 queries keep every bit down to 2^-14
          // of it, and below that are off by 2^-25 of it at most
          float top = 0.f;
#pragma unroll
          for (int s = 0; s < C::KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = (s >> 2) * 64 + c4 * 16 + (s & 3) * 4 + 2 * e;
              const uint32_t u = live && d < p.D ? __ldg(reinterpret_cast<const unsigned int *>(qp + 2 * d)) : 0u;
              qf[s][x + 2 * e] = u;
              const float2 f = unpack2(u, p.bf16);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = top > 0.f && top < INFINITY ? max(-120, min(120, ilogbf(top))) : 0;
          const float down = ldexpf(1.f, -ex);
          qmul[x] = p.scale2 * ldexpf(1.f, ex);
#pragma unroll
          for (int s = 0; s < C::KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack2(qf[s][x + 2 * e], p.bf16);
              qf[s][x + 2 * e] = pack2<false>(f.x * down, f.y * down);
            }
        }
      }
    }

    // ---- scores: the unit's rows x 16 tokens
    float sc[2][4] = {};
    const uint32_t kb = ring_s + stage * C::TILE_B, vb = kb + kTok * C::ROWB;
    if constexpr (C::TYPE != kE4m3) {
      const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint32_t f[4];
        ldmatrix4(f, kb + r * C::ROWB + ((2 * s + cc) ^ (r & 7)) * 16);
        mma<MMA_BF16, RH>(sc[0], qf[s], f[0], f[1]);
        mma<MMA_BF16, RH>(sc[1], qf[s], f[2], f[3]);
      }
    } else {
      // a lane's 16 bytes of a token are the B operand of four k steps (which
      // element of the head a k index stands for is free, as long as q agrees)
#pragma unroll
      for (int kk = 0; kk < C::KS / 4; ++kk)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int r = g + nt * 8;
          const uint4 w = *reinterpret_cast<const uint4 *>(ring + stage * C::TILE_B + r * C::ROWB +
                                                           swizzle<C, false>(kk * 4 + c4, r) * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) mma<false, RH>(sc[nt], qf[kk * 4 + i], e4m3_lo(ws[i]), e4m3_hi(ws[i]));
        }
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int x = 0; x < RH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) sc[nt][2 * x + e] *= qmul[x];
    if ((tm.flags & 0xffffu) != 0xffffu) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!((tm.flags >> (nt * 8 + 2 * c4 + e)) & 1u)) {
#pragma unroll
            for (int x = 0; x < RH; ++x) sc[nt][2 * x + e] = -INFINITY;
          }
    }
    if (p.weights) {
#pragma unroll
      for (int x = 0; x < RH; ++x)
        if (g + 8 * x < rows) {
          float *d = p.scores + (int64_t(tm.b) * p.Hq + h0 + g + 8 * x) * p.score_row + tm.t0 + 2 * c4;
          __stcg(reinterpret_cast<float2 *>(d), make_float2(sc[0][2 * x], sc[0][2 * x + 1]));
          __stcg(reinterpret_cast<float2 *>(d + 8), make_float2(sc[1][2 * x], sc[1][2 * x + 1]));
        }
    }

    // ---- running maximum: raised only when a score passes it by as much (in log2)
    // as the products' type allows, so that the sums are rarely rescaled: fp16
    // ends at 2^16, bf16 has room for 2^40 and its sums
    constexpr float RAISE = MMA_BF16 ? 40.f : 14.f;
    uint32_t pf[4] = {0u, 0u, 0u, 0u};
    float top[2];
    bool raise = false;
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      float t = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      top[x] = t;
      raise |= t > m[x] + RAISE;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int x = 0; x < RH; ++x) {
        const float m2 = fmaxf(m[x], top[x]);
        const float f = m[x] == -INFINITY ? 0.f : exp2_fast(m[x] - m2);
        m[x] = m2;
        l[x] *= f;
#pragma unroll
        for (int i = 0; i < C::NT; ++i) {
          o[i][2 * x] *= f;
          o[i][2 * x + 1] *= f;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      const float mm = m[x] == -INFINITY ? 0.f : m[x];
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = exp2_fast(sc[i >> 1][2 * x + (i & 1)] - mm);
      l[x] += (e[0] + e[1]) + (e[2] + e[3]);
      // rounded to the product's type for the tensor cores; the sum above keeps
      // all bits, and the rounding errors of many tokens average out
      pf[x] = pack2<MMA_BF16>(e[0], e[1]);
      pf[x + 2] = pack2<MMA_BF16>(e[2], e[3]);
    }

    // ---- O += P V
    if constexpr (C::TYPE != kE4m3) {
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), cc = lane >> 4;
#pragma unroll
      for (int n = 0; n < C::NT; n += 2) {
        uint32_t f[4];
        ldmatrix4_trans(f, vb + r * C::ROWB + ((n + cc) ^ (r & 7)) * 16);
        mma<MMA_BF16, RH>(o[n], pf, f[0], f[1]);
        mma<MMA_BF16, RH>(o[n + 1], pf, f[2], f[3]);
      }
    } else {
      const unsigned char *vr = ring + stage * C::TILE_B + kTok * C::ROWB;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * c4 + (i & 1) + 8 * (i >> 1);
          w[i] = *reinterpret_cast<const uint32_t *>(vr + r * C::ROWB + swizzle<C, true>(2 * j + (g >> 2), r) * 16 +
                                                     (g & 3) * 4);
        }
        // 4 tokens x 4 columns transposed: tokens (2c, 2c+1) and (2c+8, 2c+9) side by side
        const uint32_t a01 = __byte_perm(w[0], w[1], 0x5140), a23 = __byte_perm(w[0], w[1], 0x7362);
        const uint32_t b01 = __byte_perm(w[2], w[3], 0x5140), b23 = __byte_perm(w[2], w[3], 0x7362);
        mma<false, RH>(o[4 * j + 0], pf, e4m3_lo(a01), e4m3_lo(b01));
        mma<false, RH>(o[4 * j + 1], pf, e4m3_hi(a01), e4m3_hi(b01));
        mma<false, RH>(o[4 * j + 2], pf, e4m3_lo(a23), e4m3_lo(b23));
        mma<false, RH>(o[4 * j + 3], pf, e4m3_hi(a23), e4m3_hi(b23));
      }
    }
    if (++stage == C::STAGES) stage = 0;

    // ---- the end of a piece
    if (tm.flags & (1u << 17)) {
      const int whole = int(tm.flags >> 18) & 3;
#pragma unroll
      for (int x = 0; x < RH; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      }
      if (whole == 3) {
#pragma unroll
        for (int x = 0; x < RH; ++x) {
          const int r = g + 8 * x;
          if (r >= rows) continue;
          const float inv = l[x] == 0.f ? 0.f : p.v_scale / l[x];
#pragma unroll
          for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) store_out(p, tm.b, h0 + r, column<C>(i, e, c4), o[i][2 * x + e] * inv);
          if (c4 == 0) store_lse(p, tm.b, h0 + r, m[x], l[x]);
        }
      } else {
        // the warp's last piece goes into its own ring, which nothing else will
        // fill; an earlier one (there is at most one) into the workspace
        const bool end = it == hi - 1;
        const int k = pieces++;
        float *dst = end ? reinterpret_cast<float *>(ring) : p.warp_parts + w_id * (ROWS * DP);
        if (end) {
          cp_wait<0>();
          __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < RH; ++x) {
          const int r = g + 8 * x;
#pragma unroll
          for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) dst[r * DP + column<C>(i, e, c4)] = o[i][2 * x + e];
          if (c4 == 0) {
            piece_m[warp][k][r] = m[x];
            piece_l[warp][k][r] = l[x];
          }
        }
        if (lane == 0) {
          piece_o[warp][k] = dst;
          piece_b[warp][k] = tm.b;
          piece_u[warp][k] = tm.u;
          piece_state[warp][k] = 4 | whole;
        }
      }
    }
  }
  cp_wait<0>();
  __syncthreads();

  // ---- join the CTA's pieces: runs of pieces of one unit, in order
  constexpr int PIECES = 2 * C::WARPS;
  const int *state = &piece_state[0][0];
  auto next = [&](int k) {                        // the first piece at or after k
    while (k < PIECES && !state[k]) ++k;
    return k;
  };
  int k0 = next(0);
  while (k0 < PIECES) {
    const int b = (&piece_b[0][0])[k0], u = (&piece_u[0][0])[k0];
    const bool begins = state[k0] & 1;
    int k1 = k0;                                  // the run's last piece
    while (!(state[k1] & 2) && next(k1 + 1) < PIECES) k1 = next(k1 + 1);
    const bool all = begins && (state[k1] & 2);
    const int kvh = u / p.QB, qb = u - kvh * p.QB;
    const int hh = kvh * p.G + qb * ROWS, nr = min(ROWS, p.G - qb * ROWS);
    float *part = p.cta_parts + (int64_t(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE;
    for (int i = tid; i < nr * DP; i += THREADS) {
      const int r = i / DP, d = i - r * DP;
      float mm = -INFINITY;
      for (int k = k0; k <= k1; ++k)
        if (state[k]) mm = fmaxf(mm, (&piece_m[0][0][0])[k * ROWS + r]);
      float acc = 0.f, sum = 0.f;
      for (int k = k0; k <= k1; ++k)
        if (state[k]) {
          const float mk = (&piece_m[0][0][0])[k * ROWS + r];
          const float f = mk == -INFINITY ? 0.f : exp2_fast(mk - mm);
          acc += f * (&piece_o[0][0])[k][i];
          sum += f * (&piece_l[0][0][0])[k * ROWS + r];
        }
      if (all) {
        store_out(p, b, hh + r, d, acc * (sum == 0.f ? 0.f : p.v_scale / sum));
        if (d == 0) store_lse(p, b, hh + r, mm, sum);
      } else {
        __stcg(part + i, acc);
        if (d == 0) {
          __stcg(part + ROWS * DP + r, mm);
          __stcg(part + ROWS * DP + ROWS + r, sum);
        }
      }
    }
    if (!all) {
      __threadfence();
      __syncthreads();
      // the unit's first tile, its tiles, and the CTAs they lie in
      int start, len;
      seq_range(p, b, &start, &len);
      const int nt = tiles_of(start, len);
      long long first = prefix[b / per];
      for (int x = b / per * per; x < b; ++x) {
        seq_range(p, x, &start, &len);
        first += (long long)tiles_of(start, len) * units;
      }
      first += (long long)u * nt;
      const int c0 = int(((first + 1) * n_cta - 1) / total), c1 = int(((first + nt) * n_cta - 1) / total);
      const int np = c1 - c0 + 1;
      if (tid == 0) {
        const unsigned int was = atomicAdd(p.counters + c0, 1u);
        last_flag = was == unsigned(np - 1);
        if (last_flag) p.counters[c0] = 0u;       // ready for the next call
      }
      __syncthreads();
      if (last_flag) {
        __threadfence();
        // piece x of the unit: CTA c0 + x, its second slot where the unit begins
        auto slot = [&](int x) { return p.cta_parts + (int64_t(c0 + x) * 2 + (x == 0 ? 1 : 0)) * C::PIECE; };
        for (int i = tid; i < nr * DP; i += THREADS) {
          const int r = i / DP, d = i - r * DP;
          float mm = -INFINITY;
          for (int x = 0; x < np; ++x) mm = fmaxf(mm, __ldcg(slot(x) + ROWS * DP + r));
          float acc = 0.f, sum = 0.f;
          for (int x = 0; x < np; ++x) {
            const float mx = __ldcg(slot(x) + ROWS * DP + r);
            const float f = mx == -INFINITY ? 0.f : exp2_fast(mx - mm);
            acc += f * __ldcg(slot(x) + i);
            sum += f * __ldcg(slot(x) + ROWS * DP + ROWS + r);
          }
          store_out(p, b, hh + r, d, acc * (sum == 0.f ? 0.f : p.v_scale / sum));
          if (d == 0) store_lse(p, b, hh + r, mm, sum);
        }
      }
      __syncthreads();
    }
    k0 = next(k1 + 1);
  }
}

// ---- page weights ----------------------------------------------------------------

// weights[b, p] <- decay * weights[b, p] + sum over heads and tokens of
// 2^(score - lse2).  A block takes as many whole pages as 256 tokens hold (one
// page if it is longer); each thread sums a token over the heads, then each
// page is summed in token order, so the result does not depend on timing.
constexpr int kWeightThreads = 256;

__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const __grid_constant__ DecodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the scores and lse of the kernel before
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

// The kernel's shared memory is raised once per device, on first use.
constexpr int kMaxDevices = 64;

template <class C>
int launch_kv(const DecodeParams &p, int grid, int device, cudaStream_t st) {
  static std::atomic<bool> ready[kMaxDevices];
  if (device >= kMaxDevices || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode_kv_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return int(e);
    if (device < kMaxDevices) ready[device].store(true, std::memory_order_release);
  }
  decode_kv_kernel<C><<<unsigned(grid), C::WARPS * 32, C::SMEM, st>>>(p);
  return int(cudaGetLastError());
}

template <int TYPE, int ROWS>
int launch_kv_dim(const DecodeParams &p, int grid, int device, cudaStream_t st) {
  if (p.D <= 64) return launch_kv<KvConfig<64, TYPE, ROWS>>(p, grid, device, st);
  if (p.D <= 128) return launch_kv<KvConfig<128, TYPE, ROWS>>(p, grid, device, st);
  return launch_kv<KvConfig<256, TYPE, ROWS>>(p, grid, device, st);
}

template <int ROWS>
int launch_kv_type(const DecodeParams &p, int grid, int device, cudaStream_t st) {
  if (p.e4m3) return launch_kv_dim<kE4m3, ROWS>(p, grid, device, st);
  if (p.bf16) return launch_kv_dim<kBf16, ROWS>(p, grid, device, st);
  return launch_kv_dim<kFp16, ROWS>(p, grid, device, st);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace

// Counters first, at the same place for calls of every shape: a call leaves
// them at zero for the next one, whatever its shape.
DecodeSpace decode_space(const DecodeParams &p, bool weights) {
  DecodeSpace s{};
  const int64_t grid = kDecodeCtas;
  int64_t at = round_up((grid + 1) * 4, 256);
  s.cta_parts = at;
  if (p.latent) {
    const int64_t rows = latent_rows(p.Hq);
    at = round_up(at + grid * 2 * (rows * 512 + 2 * rows) * 4, 256);
    s.seq_pieces = at;
    at = round_up(at + int64_t(p.B) * 8, 256);
  } else {
    const int64_t rows = decode_rows(p.G), dp = p.D <= 64 ? 64 : p.D <= 128 ? 128 : 256;
    at = round_up(at + grid * 2 * (rows * dp + 2 * rows) * 4, 256);
    s.warp_parts = at;
    at = round_up(at + grid * 8 * rows * dp * 4, 256);
  }
  s.score_row = round_up(int64_t(p.max_pages) * p.P, kTok);
  if (weights) {
    s.lse2 = at;
    at = round_up(at + int64_t(p.B) * p.Hq * 4, 256);
    s.scores = at;
    at += int64_t(p.B) * p.Hq * s.score_row * 4;
  }
  s.bytes = at;
  return s;
}

int launch_decode(const DecodeParams &p, int device, void *stream, int *launches) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int e = 0;
  if (p.latent) {
    e = launch_decode_latent(p, device, stream, launches);
  } else {
    e = decode_rows(p.G) == 8 ? launch_kv_type<8>(p, kDecodeCtas, device, st)
                              : launch_kv_type<16>(p, kDecodeCtas, device, st);
    *launches += e == 0;
  }
  if (e || !p.weights) return e;
  const int per = p.P < kWeightThreads ? kWeightThreads / p.P : 1;
  e = launch_dependent(weights_kernel, dim3(unsigned((p.max_pages + per - 1) / per), unsigned(p.B)), kWeightThreads, st,
                       p);
  *launches += e == 0;
  return e;
}

}  // namespace hicache
