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
// head.  The products are mma.sync m16n8k16 with the 16 tokens (for V: 16 elements
// of the head) as rows and the group's heads as columns, 8 at a time, so that a
// group of 4 costs half of what heads as rows would; one 8 x 8 transposition per
// 8 tokens takes the exponentials from one product to the other.  What scores are
// taken relative to follows the running maximum only when a score passes it by as
// much (in log2) as the products' type allows: the usual tile needs a vote and no
// reduction.
//
// A warp that has all tiles of a (sequence, kv head) writes the result itself.
// The others leave a partial result, joined in tile order: first among the warps
// of a CTA in shared memory, then among CTAs in the workspace, by whichever
// CTA finishes last (a counter per CTA in which such a unit begins).  Which
// pieces exist depends on the lengths alone and they are added in order, so
// timing cannot change the result.
//
// Measured: 16 sequences of 32,768 tokens, 32 heads on 8 of 128 in bf16 (2.15 GB),
// 335 us, 6.4 TB/s, 94% of a copy's rate; 64 sequences of 33 to 8,192 tokens, pages of
// 16, 84 us (59 streaming, the rest start, joins and SMs that get 12% less of HBM
// than others); one of 4,097, 11.3 us, all of it latency.
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
  // 192 KiB of ring a CTA, one CTA per SM, in as many warps as leave each three
  // tiles or more (with few bytes to a tile it is the warps' own latency that
  // binds) and registers enough: 128 e4m3 elements spill at 16 warps
  static constexpr int WARPS = DP_ * ES >= 512 ? 4 : DP_ * ES >= 256 ? 8 : TYPE_ == kE4m3 && DP_ == 128 ? 12 : 16;
  static constexpr int CH = DP_ * ES / 16;        // 16-byte chunks of a row
  static constexpr int ROWB = DP_ * ES;
  static constexpr int TILE_B = 2 * kTok * ROWB;  // K and V
  static constexpr int RAW = 192 * 1024 / (WARPS * TILE_B);
  static constexpr int STAGES = RAW > 8 ? 8 : RAW;
  static constexpr int RING_B = STAGES * TILE_B;
  static constexpr int KS = DP_ / 16;             // k steps of q . k
  static constexpr int MT = DP_ / 16;             // m tiles of the output
  static constexpr int NB = ROWS_ / 8;            // n tiles: 8 heads each
  static constexpr float RAISE = kRaise<TYPE_ != kBf16>, ABOVE = kAbove<TYPE_ != kBf16>;
  static constexpr int PIECE = ROWS_ * DP_ + 2 * ROWS_;   // floats of a partial result: O, m, l
  static constexpr int LD = DP_ + 4;              // floats of a row of a warp's: no bank twice
  static constexpr int SMEM = WARPS * RING_B;
  static_assert(STAGES >= 2 && RING_B >= ROWS_ * LD * 4, "ring");
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

// c += a b, 16 x 8 x 16
template <bool BF16>
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit elements, a row per 4 lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

// The elements of the head that rows g and g + 8 of m tile t are.
template <class C>
__device__ __forceinline__ int element(int t, int upper, int g) {
  if constexpr (C::TYPE != kE4m3) return 16 * t + 8 * upper + g;
  return 32 * (t >> 1) + 4 * g + 2 * (t & 1) + upper;
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
  constexpr int THREADS = C::WARPS * 32, ROWS = C::ROWS, NB = C::NB, DP = C::DP;
  constexpr bool MMA_BF16 = C::TYPE == kBf16;
  __shared__ TileMeta meta_all[C::WARPS][C::STAGES];
  __shared__ long long prefix[THREADS + 1];
  __shared__ long long warp_tot[C::WARPS];
  // the CTA's pieces, two per warp: where O lies, m and l, the unit, and
  // (4: present, 1: begins its unit, 2: ends it)
  __shared__ const float *piece_o[C::WARPS][2];
  __shared__ __align__(16) float piece_m[C::WARPS][2][ROWS], piece_l[C::WARPS][2][ROWS];
  __shared__ int piece_b[C::WARPS][2], piece_u[C::WARPS][2], piece_state[C::WARPS][2];
  // joining CTAs' pieces: the two open units (first CTA, pieces if it falls to this
  // CTA), and what the teams of threads beside the first have
  __shared__ int join_cta[2], join_n[2];
  __shared__ float4 team_o[THREADS];
  __shared__ float2 team_ml[3][ROWS];

  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const int units = p.Hkv * p.QB;                 // units of a sequence

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call

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
    const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    const uint32_t base = ring_s + lstage * C::TILE_B;
    constexpr int RPI = C::CH <= 32 ? 32 / C::CH : 1;         // rows per instruction
    static_assert(C::CH <= 32, "a row is at most a warp of chunks");
    const int c = lane % C::CH, r0 = lane / C::CH;
    const bool in_d = c * 16 < p.D * C::ES;
    const char *kp = static_cast<const char *>(p.k), *vp = static_cast<const char *>(p.v);
    int64_t off = 0;
    if (ok) off = ((int64_t(lpage) * p.P + (t - lpg * p.P)) * p.row + int64_t(kvh) * p.D) * C::ES;
    if (mask == 0xffffu && (p.P & 15) == 0) {     // one page, every row: rows at a fixed distance
      const int64_t first = __shfl_sync(0xffffffffu, off, 0) + r0 * p.row * C::ES + c * 16;
      const char *ks = kp + (in_d ? first : 0), *vs = vp + (in_d ? first : 0);
      const int64_t step = in_d ? RPI * p.row * C::ES : 0;
      const int n = in_d ? 16 : 0;
#pragma unroll
      for (int i = 0; i < kTok / RPI; ++i) {
        const int r = i * RPI + r0;
        cp_async16(base + r * C::ROWB + swizzle<C, false>(c, r) * 16, ks, n);
        cp_async16(base + kTok * C::ROWB + r * C::ROWB + swizzle<C, true>(c, r) * 16, vs, n);
        ks += step;
        vs += step;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kTok / RPI; ++i) {
        const int r = i * RPI + r0;
        const int64_t o = __shfl_sync(0xffffffffu, off, r);
        const bool have = in_d && ((mask >> r) & 1u);
        const int64_t at = have ? o + c * 16 : 0;
        cp_async16(base + r * C::ROWB + swizzle<C, false>(c, r) * 16, kp + at, have ? 16 : 0);
        cp_async16(base + kTok * C::ROWB + r * C::ROWB + swizzle<C, true>(c, r) * 16, vp + at, have ? 16 : 0);
      }
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
  uint32_t qf[C::KS][NB][2];                      // q as the B operand
  // of heads 8 n + 2 c4 and + 1: the scale (for e4m3 with the power of two taken out
  // of q), the reference, what scores are taken relative to (0 while there is none),
  // the sum
  float qmul[NB][2], m[NB][2], mu[NB][2], l[NB][2];
  float o[C::MT][NB][4];
  int h0 = 0, rows = 0, pieces = 0, stage = 0;
#pragma unroll 1
  for (long long it = lo; it < hi; ++it) {
    __syncwarp();                                 // everyone is done with the stage that is filled next
    if (lnext < hi) load();
    cp_commit();
    const TileMeta tm = meta[stage];              // written a turn ago or more
    if (tm.flags & (1u << 16)) {                  // a new piece: its q
      const int kvh = tm.u / p.QB, qb = tm.u - kvh * p.QB;
      h0 = kvh * p.G + qb * ROWS;
      rows = min(ROWS, p.G - qb * ROWS);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int t = 0; t < C::MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][n][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qmul[n][i] = p.scale2;
          m[n][i] = -INFINITY;
          mu[n][i] = 0.f;
          l[n][i] = 0.f;
        }
        const int r = 8 * n + g;
        const char *qp = static_cast<const char *>(p.q) + 2 * (int64_t(tm.b) * p.q_sb + int64_t(h0 + r) * p.q_sh);
        const bool live = r < rows;
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = C::TYPE != kE4m3 ? s * 16 + e * 8 + 2 * c4 : (s >> 2) * 64 + c4 * 16 + (s & 3) * 4 + 2 * e;
            qf[s][n][e] = live && d < p.D ? __ldg(reinterpret_cast<const unsigned int *>(qp + 2 * d)) : 0u;
          }
        if constexpr (C::TYPE == kE4m3) {
          // fp16, after the power of two that brings the head's largest element
          // into [1, 2): bf16 and fp16 queries keep every bit down to 2^-14
          // of it, and below that are off by 2^-25 of it at most
          float top = 0.f;
#pragma unroll
          for (int s = 0; s < C::KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack2(qf[s][n][e], p.bf16);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = top > 0.f && top < INFINITY ? max(-120, min(120, ilogbf(top))) : 0;
          const float down = ldexpf(1.f, -ex), up = p.scale2 * ldexpf(1.f, ex);
#pragma unroll
          for (int i = 0; i < 2; ++i) qmul[n][i] = __shfl_sync(0xffffffffu, up, (2 * c4 + i) * 4);
#pragma unroll
          for (int s = 0; s < C::KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack2(qf[s][n][e], p.bf16);
              qf[s][n][e] = pack2<false>(f.x * down, f.y * down);
            }
        }
      }
    }
    cp_wait<C::STAGES - 1>();
    __syncwarp();

    // ---- scores: 16 tokens x the unit's heads
    float sc[NB][4] = {};
    const uint32_t kb = ring_s + stage * C::TILE_B, vb = kb + kTok * C::ROWB;
    if constexpr (C::TYPE != kE4m3) {
      const int r = lane & 15, cc = lane >> 4;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint32_t f[4];
        ldmatrix4(f, kb + r * C::ROWB + ((2 * s + cc) ^ (r & 7)) * 16);
#pragma unroll
        for (int n = 0; n < NB; ++n) mma<MMA_BF16>(sc[n], f, qf[s][n][0], qf[s][n][1]);
      }
    } else {
      // a lane's 16 bytes of a token are the A operand of four k steps (which
      // element of the head a k index stands for is free, as long as q agrees)
#pragma unroll
      for (int kk = 0; kk < C::KS / 4; ++kk) {
        uint4 w[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
          w[x] = *reinterpret_cast<const uint4 *>(ring + stage * C::TILE_B + (g + 8 * x) * C::ROWB +
                                                  swizzle<C, false>(kk * 4 + c4, g + 8 * x) * 16);
        const uint32_t lo_w[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, hi_w[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f[4] = {e4m3_lo(lo_w[i]), e4m3_lo(hi_w[i]), e4m3_hi(lo_w[i]), e4m3_hi(hi_w[i])};
#pragma unroll
          for (int n = 0; n < NB; ++n) mma<false>(sc[n], f, qf[kk * 4 + i][n][0], qf[kk * 4 + i][n][1]);
        }
      }
    }
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][i] = fmaf(sc[n][i], qmul[n][i & 1], -mu[n][i & 1]);
    if ((tm.flags & 0xffffu) != 0xffffu) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (!((tm.flags >> (g + 8 * x)) & 1u)) {
#pragma unroll
          for (int n = 0; n < NB; ++n) sc[n][2 * x] = sc[n][2 * x + 1] = -INFINITY;
        }
    }
    if (p.weights) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (8 * n + 2 * c4 + i < rows) {
            float *d = p.scores + (int64_t(tm.b) * p.Hq + h0 + 8 * n + 2 * c4 + i) * p.score_row + tm.t0 + g;
            __stcg(d, sc[n][i] + mu[n][i]);
            __stcg(d + 8, sc[n][2 + i] + mu[n][i]);
          }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        raise |= fmaxf(sc[n][i], sc[n][2 + i]) > C::RAISE || m[n][i] == -INFINITY;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(sc[n][i], sc[n][2 + i]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
          const float m2 = fmaxf(m[n][i], top + mu[n][i] - C::ABOVE);
          const float f = m[n][i] == -INFINITY ? 0.f : exp2_fast(m[n][i] - m2);
          const float use = m2 == -INFINITY ? 0.f : m2, by = mu[n][i] - use;
          m[n][i] = m2;
          mu[n][i] = use;
          sc[n][i] += by;
          sc[n][2 + i] += by;
          l[n][i] *= f;
#pragma unroll
          for (int t = 0; t < C::MT; ++t) {
            o[t][n][i] *= f;
            o[t][n][2 + i] *= f;
          }
        }
    }
    uint32_t pf[NB][2];                           // the exponentials as the B operand
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][i] = exp2_fast(sc[n][i]);
      l[n][0] += sc[n][0] + sc[n][2];
      l[n][1] += sc[n][1] + sc[n][3];
      // rounded to the product's type for the tensor cores; the sum above keeps all
      // bits, and the rounding errors of many tokens average out (those of the smallest,
      // which become 0, do not: see kAbove)
#pragma unroll
      for (int x = 0; x < 2; ++x) pf[n][x] = transpose8(pack2<MMA_BF16>(sc[n][2 * x], sc[n][2 * x + 1]));
    }

    // ---- O^T += V^T P^T
    if constexpr (C::TYPE != kE4m3) {
      const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
      for (int t = 0; t < C::MT; ++t) {
        uint32_t f[4];
        ldmatrix4_trans(f, vb + r * C::ROWB + ((2 * t + cc) ^ (r & 7)) * 16);
#pragma unroll
        for (int n = 0; n < NB; ++n) mma<MMA_BF16>(o[t][n], f, pf[n][0], pf[n][1]);
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
        // 4 tokens x 4 elements transposed: tokens (2c, 2c+1) and (2c+8, 2c+9) side by side
        const uint32_t a01 = __byte_perm(w[0], w[1], 0x5140), a23 = __byte_perm(w[0], w[1], 0x7362);
        const uint32_t b01 = __byte_perm(w[2], w[3], 0x5140), b23 = __byte_perm(w[2], w[3], 0x7362);
        const uint32_t f0[4] = {e4m3_lo(a01), e4m3_hi(a01), e4m3_lo(b01), e4m3_hi(b01)};
        const uint32_t f1[4] = {e4m3_lo(a23), e4m3_hi(a23), e4m3_lo(b23), e4m3_hi(b23)};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma<false>(o[2 * j][n], f0, pf[n][0], pf[n][1]);
          mma<false>(o[2 * j + 1][n], f1, pf[n][0], pf[n][1]);
        }
      }
    }
    if (++stage == C::STAGES) stage = 0;

    // ---- the end of a piece
    if (tm.flags & (1u << 17)) {
      const int whole = int(tm.flags >> 18) & 3;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], w);
      if (whole == 3) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          float inv[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            inv[i] = l[n][i] == 0.f ? 0.f : p.v_scale / l[n][i];
            const int r = 8 * n + 2 * c4 + i;
            if (g == 0 && r < rows) store_lse(p, tm.b, h0 + r, m[n][i], l[n][i]);
          }
          if constexpr (C::TYPE != kE4m3) {       // a head's pairs of elements, by a transposition
            const int r = 8 * n + g;
            char *dst = static_cast<char *>(p.out) + 2 * (int64_t(tm.b) * p.o_sb + int64_t(h0 + r) * p.o_sh);
#pragma unroll
            for (int t = 0; t < C::MT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w =
                    transpose8(pack2<MMA_BF16>(o[t][n][2 * x] * inv[0], o[t][n][2 * x + 1] * inv[1]));
                const int d = 16 * t + 8 * x + 2 * c4;
                if (r < rows && d < p.D) *reinterpret_cast<uint32_t *>(dst + 2 * d) = w;
              }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 8 * n + 2 * c4 + i;
              char *dst = static_cast<char *>(p.out) + 2 * (int64_t(tm.b) * p.o_sb + int64_t(h0 + r) * p.o_sh);
#pragma unroll
              for (int j = 0; j < DP / 32; ++j) { // 4 elements in a row
                const int d = 32 * j + 4 * g;
                const float v0 = o[2 * j][n][i] * inv[i], v1 = o[2 * j][n][2 + i] * inv[i];
                const float v2 = o[2 * j + 1][n][i] * inv[i], v3 = o[2 * j + 1][n][2 + i] * inv[i];
                if (r < rows && d < p.D)
                  *reinterpret_cast<uint2 *>(dst + 2 * d) =
                      p.bf16 ? make_uint2(pack2<true>(v0, v1), pack2<true>(v2, v3))
                             : make_uint2(pack2<false>(v0, v1), pack2<false>(v2, v3));
              }
            }
          }
        }
      } else {
        // the warp's last piece goes into its own ring, which nothing else will
        // fill; an earlier one (there is at most one) into the workspace
        const bool end = it == hi - 1;
        const int k = pieces++;
        float *dst = end ? reinterpret_cast<float *>(ring) : p.warp_parts + w_id * (ROWS * C::LD);
        if (end) {
          cp_wait<0>();
          __syncwarp();
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * n + 2 * c4 + i;
#pragma unroll
            for (int t = 0; t < C::MT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) dst[r * C::LD + element<C>(t, x, g)] = o[t][n][2 * x + i];
            if (g == 0) {
              piece_m[warp][k][r] = m[n][i];
              piece_l[warp][k][r] = l[n][i];
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

  // ---- join the CTA's pieces.  A chain is a run of pieces of one unit: it starts
  // at a piece that begins its unit, or at the CTA's first piece.
  constexpr int PIECES = 2 * C::WARPS, COL4 = DP / 4;
  constexpr int COLS = ROWS * COL4 > THREADS ? 2 : 1;   // columns of 4 elements a thread takes at once
  static_assert(PIECES <= 32, "a lane for a piece");
  const int *state = &piece_state[0][0];
  const int mine_state = lane < PIECES ? state[lane] : 0;
  const uint32_t present = __ballot_sync(0xffffffffu, mine_state & 4);
  const uint32_t begin_m = __ballot_sync(0xffffffffu, mine_state & 1), end_m = __ballot_sync(0xffffffffu, mine_state & 2);
  const uint32_t starts = begin_m | (present & (~present + 1u));
  auto chain_of = [&](int k, int *k1) {           // the last piece of the chain that starts at k
    const uint32_t later = k < 31 ? starts & (~0u << (k + 1)) : 0u;
    const uint32_t upto = later ? (later & (~later + 1u)) - 1u : ~0u;
    *k1 = 31 - __clz(int(present & upto));
    return bool((begin_m >> k) & (end_m >> *k1) & 1u);
  };
  __shared__ unsigned char order[32];             // the pieces there are
  if (warp == 0 && (mine_state & 4)) order[__popc(present & ((1u << lane) - 1u))] = (unsigned char)lane;
  __syncthreads();
  int chain = 0;
  for (uint32_t left = starts; left; left &= left - 1u, ++chain) {
    // a warp's worth of chains at a time: warps take elements, not chains
    const int k0 = __ffs(int(left)) - 1;
    int k1;
    const bool all = chain_of(k0, &k1);
    const int u = (&piece_u[0][0])[k0], b = (&piece_b[0][0])[k0];
    const int kvh = u / p.QB, qb = u - kvh * p.QB;
    const int hh = kvh * p.G + qb * ROWS, nr = min(ROWS, p.G - qb * ROWS);
    float *part = p.cta_parts + (int64_t(blockIdx.x) * 2 + int((begin_m >> k0) & 1u)) * C::PIECE;
    const int x0 = __popc(present & ((1u << k0) - 1u)), x1 = __popc(present & (k1 < 31 ? (2u << k1) - 1u : ~0u)) - 1;
    const int cols = nr * COL4;
    const bool more = cols > THREADS;             // two columns a thread, else one
    for (int i0 = (tid + chain * 128) % THREADS; i0 < cols; i0 += COLS * THREADS) {
      float mm[COLS], sum[COLS];
      float4 acc[COLS];
      int r[COLS], d[COLS];
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const int i = min(i0 + c * THREADS, cols - 1);
        r[c] = i / COL4, d[c] = (i - r[c] * COL4) * 4;
        mm[c] = -INFINITY, sum[c] = 0.f;
        acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float *ms = &piece_m[0][0][0], *ls = &piece_l[0][0][0];
      for (int x = x0; x <= x1; ++x)
#pragma unroll
        for (int c = 0; c < COLS; ++c) mm[c] = fmaxf(mm[c], ms[order[x] * ROWS + r[c]]);
      for (int xb = x0; xb <= x1; xb += 4) {      // 4 at a time: some come back from the workspace
        float4 v[4][COLS];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (xb + x <= x1) {
            const float *o = (&piece_o[0][0])[order[xb + x]];
#pragma unroll
            for (int c = 0; c < COLS; ++c)
              if (c == 0 || more) v[x][c] = *reinterpret_cast<const float4 *>(o + r[c] * C::LD + d[c]);
          }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (xb + x <= x1) {
            const int k = order[xb + x] * ROWS;
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
              if (c > 0 && !more) break;
              const float mk = ms[k + r[c]];
              const float f = mk == -INFINITY ? 0.f : exp2_fast(mk - mm[c]);
              acc[c].x += f * v[x][c].x;
              acc[c].y += f * v[x][c].y;
              acc[c].z += f * v[x][c].z;
              acc[c].w += f * v[x][c].w;
              sum[c] += f * ls[k + r[c]];
            }
          }
      }
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        if (i0 + c * THREADS >= cols) continue;
        if (all) {
          store_out4(p, b, hh + r[c], d[c], acc[c], sum[c] == 0.f ? 0.f : p.v_scale / sum[c]);
          if (d[c] == 0) store_lse(p, b, hh + r[c], mm[c], sum[c]);
        } else {
          __stcg(reinterpret_cast<float4 *>(part + r[c] * DP + d[c]), acc[c]);
          if (d[c] == 0) {
            __stcg(part + ROWS * DP + r[c], mm[c]);
            __stcg(part + ROWS * DP + ROWS + r[c], sum[c]);
          }
        }
      }
    }
  }

  // ---- join the CTAs' parts: of the first chain if it does not begin its unit, of
  // the last if it does not end it.  Two warps see to the two counters at once.
  const int first_k = starts ? __ffs(int(starts)) - 1 : 0, last_k = starts ? 31 - __clz(int(starts)) : 0;
  int unused;
  const bool open_first = starts && !chain_of(first_k, &unused);
  const bool open_last = starts && last_k != first_k && !chain_of(last_k, &unused);
  if (!open_first && !open_last) return;
  int c0 = 0, c1 = 0;
  const bool counts = lane == 0 && (warp == 0 ? open_first : warp == 1 && open_last);
  if (counts) {
    // the unit's first tile, its tiles, and the CTAs they lie in
    const int k = warp == 0 ? first_k : last_k;
    const int b = (&piece_b[0][0])[k], u = (&piece_u[0][0])[k];
    int start, len;
    seq_range(p, b, &start, &len);
    const int nt = tiles_of(start, len);
    long long first = prefix[b / per];
    for (int x = b / per * per; x < b; ++x) {
      seq_range(p, x, &start, &len);
      first += (long long)tiles_of(start, len) * units;
    }
    first += (long long)u * nt;
    c0 = int(((first + 1) * n_cta - 1) / total);
    c1 = int(((first + nt) * n_cta - 1) / total);
  }
  __syncthreads();                                // the CTA's parts are written
  if (counts) {
    __threadfence();
    const unsigned int was = atomicAdd(p.counters + c0, 1u);
    const bool last = was == unsigned(c1 - c0);
    if (last) p.counters[c0] = 0u;                // ready for the next call
    __threadfence();
    join_cta[warp] = c0;
    join_n[warp] = last ? c1 - c0 + 1 : 0;
  }
  __syncthreads();
  for (int side = 0; side < 2; ++side) {
    if (!(side == 0 ? open_first : open_last)) continue;
    const int np = join_n[side], from = join_cta[side];
    if (np == 0) continue;
    const int k = side == 0 ? first_k : last_k;
    const int b = (&piece_b[0][0])[k], u = (&piece_u[0][0])[k];
    const int kvh = u / p.QB, qb = u - kvh * p.QB;
    const int hh = kvh * p.G + qb * ROWS, nr = min(ROWS, p.G - qb * ROWS);
    // piece x of the unit: CTA from + x, its second slot where the unit begins
    auto slot = [&](int x) { return p.cta_parts + (int64_t(from + x) * 2 + (x == 0 ? 1 : 0)) * C::PIECE; };
    // a thread takes four elements of a row, or twice four where there are 16 rows (one
    // sequence of 4,096 with 12 heads of 256 on each of 4: 41 -> 34 us; with 8 rows,
    // 8 heads on each, 28.1 -> 32); with threads to spare, every `teams`-th piece of
    // them.  Maximum, sum and O of 8 pieces are on their way together.
    constexpr int JOIN = ROWS > 8 ? COLS : 1;
    const int cols = nr * COL4, teams = max(1, min(4, THREADS / cols));
    const int team = teams > 1 ? tid / cols : 0;
    for (int i0 = 0; i0 < cols; i0 += JOIN * THREADS) {
      const int i = teams > 1 ? tid - team * cols : i0 + tid;
      float m_r[JOIN], l_r[JOIN];
      float4 acc[JOIN];
      auto add = [&](int c, float mx, float lx, const float4 &v) {
        const float now = fmaxf(m_r[c], mx);
        const float was = m_r[c] == -INFINITY ? 0.f : exp2_fast(m_r[c] - now);
        const float f = mx == -INFINITY ? 0.f : exp2_fast(mx - now);
        acc[c].x = acc[c].x * was + f * v.x;
        acc[c].y = acc[c].y * was + f * v.y;
        acc[c].z = acc[c].z * was + f * v.z;
        acc[c].w = acc[c].w * was + f * v.w;
        l_r[c] = l_r[c] * was + f * lx;
        m_r[c] = now;
      };
      bool mine[JOIN];
      int r[JOIN], d[JOIN];
#pragma unroll
      for (int c = 0; c < JOIN; ++c) {
        mine[c] = team < teams && i + c * THREADS < cols;
        const int j = min(i + c * THREADS, cols - 1);
        r[c] = j / COL4, d[c] = (j - r[c] * COL4) * 4;
        m_r[c] = -INFINITY, l_r[c] = 0.f;
        acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (int x0 = team; mine[0] && x0 < np; x0 += 8 * teams) {
        float4 v[8][JOIN];
        float mx[8][JOIN], lx[8][JOIN];
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x0 + x * teams < np) {
            const float *s = slot(x0 + x * teams);
#pragma unroll
            for (int c = 0; c < JOIN; ++c) {
              v[x][c] = __ldcg(reinterpret_cast<const float4 *>(s + r[c] * DP + d[c]));
              mx[x][c] = __ldcg(s + ROWS * DP + r[c]);
              lx[x][c] = __ldcg(s + ROWS * DP + ROWS + r[c]);
            }
          }
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x0 + x * teams < np)
#pragma unroll
            for (int c = 0; c < JOIN; ++c) add(c, mx[x][c], lx[x][c], v[x][c]);
      }
      if (teams > 1) {
        __syncthreads();
        if (mine[0] && team > 0) {
          team_o[(team - 1) * cols + i] = acc[0];
          if (d[0] == 0) team_ml[team - 1][r[0]] = make_float2(m_r[0], l_r[0]);
        }
        __syncthreads();
        if (mine[0] && team == 0)
          for (int t = 0; t + 1 < teams; ++t) add(0, team_ml[t][r[0]].x, team_ml[t][r[0]].y, team_o[t * cols + i]);
      }
#pragma unroll
      for (int c = 0; c < JOIN; ++c)
        if (mine[c] && team == 0) {
          store_out4(p, b, hh + r[c], d[c], acc[c], l_r[c] == 0.f ? 0.f : p.v_scale / l_r[c]);
          if (d[c] == 0) store_lse(p, b, hh + r[c], m_r[c], l_r[c]);
        }
    }
    __syncthreads();
  }
}

// ---- page weights ----------------------------------------------------------------

// weights[b, p] <- decay * weights[b, p] + sum over heads and tokens of
// 2^(score - lse2).  Bound by reading the scores (4 bytes a head and token).  A warp
// takes as many whole pages as 128 tokens hold, a lane four tokens, with the loads
// of 8 heads on their way together and no barrier with other warps; a longer page
// is dealt to the block's warps in chunks of 128 tokens.  Heads, then a page's
// tokens are added in an order that does not depend on timing.
constexpr int kWeightWarps = 4, kWeightTok = 128;

HC_HD int weight_pages(int page) { return page <= kWeightTok ? kWeightTok / page : 1; }
// blocks for a sequence of max_pages pages
HC_HD int weight_blocks(int page, int max_pages) {
  const int per = page <= kWeightTok ? kWeightWarps * weight_pages(page) : 1;
  return (max_pages - 1) / per + 1;
}

__global__ void __launch_bounds__(kWeightWarps * 32) weights_kernel(const __grid_constant__ DecodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the scores and lse of the kernel before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float val_all[kWeightWarps][kWeightTok];
  const int b = blockIdx.y, warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  float *const val = val_all[warp];
  const bool shared_page = p.P > kWeightTok;
  const int per = weight_pages(p.P);
  const int first = shared_page ? int(blockIdx.x) : (int(blockIdx.x) * kWeightWarps + warp) * per;
  int start, len;
  seq_range(p, b, &start, &len);
  const int pages = int(len > 0 ? fast_div(uint32_t(len - 1), p.fd_page) + 1 : 0);
  if (first >= pages) return;                     // the whole warp (of a long page: the whole block)
  const int t0 = first * p.P, t1 = int(min(int64_t(len), (int64_t(first) + per) * p.P));
  const float *lse2 = p.lse2 + int64_t(b) * p.Hq;
  const float *sc = p.scores + int64_t(b) * p.Hq * p.score_row;
  float *const weights = p.weights + b * p.w_sb + first;
  const int mine = min(per, pages - first);
  // the old weights, on their way with the scores
  const float old = lane < mine && !shared_page ? weights[lane] : 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int step = shared_page ? kWeightWarps * kWeightTok : kWeightTok;
  for (int base = t0 + (shared_page ? warp * kWeightTok : 0); base < t1; base += step) {
    for (int h0 = 0; h0 < p.Hq; h0 += 8) {
      float s[8][4], z[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        z[h] = h0 + h < p.Hq ? __ldg(lse2 + h0 + h) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = base + lane + 32 * j;
          s[h][j] = h0 + h < p.Hq && t >= start && t < t1 ? __ldcs(sc + (h0 + h) * p.score_row + t) : -INFINITY;
        }
      }
#pragma unroll
      for (int h = 0; h < 8; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += s[h][j] == -INFINITY ? 0.f : exp2_fast(s[h][j] - z[h]);
    }
  }
  if (shared_page) {
    float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) val[0] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.f;
      for (int w = 0; w < kWeightWarps; ++w) s += val_all[w][0];
      *weights = p.decay * *weights + s;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) val[lane + 32 * j] = acc[j];
  __syncwarp();
  if (p.P >= 16) {                                // the warp a page at a time (8 of them at most)
    for (int pg = 0; pg < mine; ++pg) {
      float s = 0.f;
      for (int i = lane; i < p.P; i += 32) s += val[pg * p.P + i];
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == pg) weights[pg] = p.decay * old + s;
    }
  } else {                                        // a page a lane
    for (int pg = lane; pg < mine; pg += 32) {
      float s = 0.f;
      for (int i = 0; i < p.P; ++i) s += val[pg * p.P + i];
      weights[pg] = p.decay * (pg < 32 ? old : weights[pg]) + s;
    }
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
  return launch_dependent(decode_kv_kernel<C>, dim3(unsigned(grid)), C::WARPS * 32, st, p, C::SMEM);
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
    at = round_up(at + grid * 16 * rows * (dp + 4) * 4, 256);
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
  e = launch_dependent(weights_kernel, dim3(unsigned(weight_blocks(p.P, p.max_pages)), unsigned(p.B)),
                       kWeightWarps * 32, st, p);
  *launches += e == 0;
  return e;
}

}  // namespace hicache
