// hicache_decode_latent.cu -- attention of one new token per sequence over a
// latent cache: rows of 576 elements, all of them the key, the first 512 the
// value, one row for every query head.
//
// A cached byte serves all heads, so with many heads this is a pair of matrix
// products: 16 heads do 30 multiply-adds per byte read, 128 heads 242.  The
// tensor cores (tcgen05) take them with the TOKENS as the rows and the heads as
// the columns:
//   S^T [64 tokens, heads] = K q^T        36 steps of 16 over the 576 elements
//   O^T [512, heads]      += V^T P^T      4 blocks of 128 rows, 4 steps of 16 tokens
// so that few heads cost few columns, and the cache tile, as it lies in shared
// memory (rows of 128 bytes, 128-byte swizzle), is the first operand of both:
// K-major for S, M-major for O.  Accumulators live in tensor memory: 4 blocks of
// `heads` columns for O, 2 for S.
//
// A tile is 64 tokens (72 KiB), so that two and more fit beside q and the copies
// of the next tile never stop for the products of this one.  S is double-buffered
// and the two products are issued by a warp each, as their operands arrive: S of
// tile n + 1 runs during the softmax of tile n, and a product with V whose P is
// ready never waits behind one whose tile is still on its way.
//
// Softmax: a set of four warps (two sets for 64 heads, 32 heads each) reads 16
// tokens a warp as 16 x 8 fragments (2 tokens x heads / 4 a thread).  What a head's
// scores are taken relative to follows the running maximum only when some score
// passes it by more than P's type can hold, so that the usual tile needs one barrier
// and no reduction; sums stay per thread until the piece ends.
//
// The work is cut into strips of 32 tokens; the strips of all sequences, in
// order, are dealt in equal contiguous ranges to the CTAs (one per SM; with more
// than 64 heads, CTAs in groups that walk the same range with 64 heads each, so
// that the cache is read from HBM once and from L2 after that).  A CTA's part of
// a sequence is a piece; whole sequences are written out directly, the other
// pieces go to the workspace and latent_join_kernel adds them in order.
//
// Warps: first the softmax and epilogue, one issues S, one O, four copy the cache
// and q into shared memory (cp.async, 16 bytes per lane, so any page size, absent
// pages as zeros), signalling by mbarrier.  The tile's rope block (elements
// 512..575) is free once S is there and then holds P.
//
// Measured, 32 sequences of 4,096 to 16,384 tokens (331 MB): 16 heads 66 us, of which
// 12 are start, epilogue and join, the rest HBM's rate; 128 heads 124 us, where the
// two tiles that fit beside 72 KiB of q take turns with products and softmax.  With
// tiles of 128 tokens, one and a bit of which fit, 16 heads took 83 us.
//
// Every wait has a limit of about two seconds, after which the CTA gives up,
// sets the workspace's error word and returns.

#include <atomic>

#include "hicache_decode.cuh"

namespace hicache {
namespace {

constexpr int kLatD = 576, kLatDv = 512;
constexpr int kTileTok = 64, kStrip = 32;
constexpr int kAtomB = kTileTok * 128;            // 64 elements of a tile's tokens
constexpr int kDuoB = 2 * kAtomB;                 // 128 elements
constexpr int kRopeB = kAtomB;                    // the last 64 elements

template <int NH_, bool BF16_>
struct LatConfig {
  static constexpr int NH = NH_;                  // heads (columns)
  static constexpr bool BF16 = BF16_;
  static constexpr int SETS = NH_ == 64 ? 2 : 1;  // of four softmax warps
  static constexpr int NS = NH_ / SETS;           // heads of a set
  static constexpr int S_WARP = 4 * SETS, O_WARP = S_WARP + 1, COPY_WARP = S_WARP + 2;
  static constexpr int WARPS = COPY_WARP + 4, THREADS = WARPS * 32;
  // A tile is 4 duos and a rope block; at least two tiles must fit.
  static constexpr int DUOS = NH_ == 64 ? 8 : NH_ == 32 ? 10 : 11;
  static constexpr int ROPES = NH_ == 16 ? 3 : 2;
  static constexpr int Q_B = 9 * NH_ * 128;
  static constexpr int SMEM = Q_B + DUOS * kDuoB + ROPES * kRopeB + 1024;
  static constexpr int COLS = NH_ == 16 ? 128 : NH_ == 32 ? 256 : 512;   // tensor memory
  static constexpr int PIECE = NH_ * kLatDv + 2 * NH_;                   // floats: O, m, l
  static constexpr float RAISE = kRaise<!BF16_>, ABOVE = kAbove<!BF16_>;
};

// ---- mbarriers and tcgen05 ------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("{.reg .b64 t; mbarrier.arrive.shared::cta.b64 t, [%0];}" ::"r"(bar) : "memory");
}
// arrives once all copies this thread has issued so far are in shared memory
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
constexpr long long kWaitClocks = 4000000000ll;   // about two seconds
// Waits for the phase `parity` to end; false once a wait of the CTA has run out (LAST:
// only once this one has).
template <bool LAST = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up) {
  long long since = 0;
  for (;;) {
    uint32_t done;
    asm volatile(
        "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if (!LAST && *gave_up) return false;
    const long long now = clock64();
    if (since == 0) since = now;
    if (now - since > kWaitClocks) {
      *gave_up = 1;
      return false;
    }
  }
}

// true in one lane of the (whole) warp, in a way the compiler can follow
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, float *v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const float *v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand, 128-byte swizzle.  lbo: bytes between blocks of 64
// elements along M (operands that are contiguous along M); sbo: between groups
// of 8 rows of 128 bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3fff) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// m x n, 32-bit sums; a_m, b_n: the operand is contiguous along M (N) instead of K
__device__ __forceinline__ constexpr uint32_t instr_desc(bool bf16, int m, int n, bool a_m, bool b_n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_m ? 1u << 15 : 0u) | (b_n ? 1u << 16 : 0u) |
         (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// barriers of the four warps of a softmax set
__device__ __forceinline__ void set_sync(int set) { asm volatile("bar.sync %0, 128;" ::"r"(1 + 2 * set) : "memory"); }
__device__ __forceinline__ bool set_any(int set, bool x) {
  int r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.s32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.s32 %0, 1, 0, q;}"
      : "=r"(r)
      : "r"(int(x)), "r"(2 + 2 * set)
      : "memory");
  return r != 0;
}

// The maximum or sum over a warp's 16 tokens of the columns a lane holds (8 n + 2 c
// + i, in v[2 n + i]) into out.
template <int NH, bool MAX>
__device__ __forceinline__ void reduce_columns(float *v, int lane, float *out) {
#pragma unroll
  for (int j = 0; j < NH / 4; ++j) {
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, v[j], w);
      v[j] = MAX ? fmaxf(v[j], y) : v[j] + y;
    }
    if (lane < 4) out[8 * (j >> 1) + 2 * lane + (j & 1)] = v[j];
  }
}

// 16 lanes (tokens) x 16 columns: v[0..1] row lane / 4, columns 2 (lane % 4) + {0, 1};
// v[2..3] row lane / 4 + 8; v[4..7] the same 8 columns on.
__device__ __forceinline__ void tc_ld_16x16(uint32_t addr, float *v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ int strips_of(int start, int len) {
  return len > start ? (len + kStrip - 1) / kStrip - start / kStrip : 0;
}

constexpr int kLens = 512;                        // lengths kept in shared memory

__device__ __forceinline__ void seq_range(const DecodeParams &p, const int *lens, int b, int *start, int *len) {
  if (b >= kLens) return seq_range(p, b, start, len);
  *len = lens[b];
  *start = p.window > 0 ? max(0, *len - p.window) : 0;
}

// The pieces of a CTA's range of strips, in order.
struct Pieces {
  const int *lens;
  long long pos, hi;
  long long skip;      // strips of sequence b before the range
  int b;
  // the current piece
  int t_lo, t_hi, start, tiles;   // tokens [t_lo, t_hi) from t_lo = a multiple of kStrip; first token attended to
  bool begins, ends;
  __device__ __forceinline__ bool next(const DecodeParams &p) {
    if (pos >= hi) return false;
    int len, n;
    for (;; ++b) {
      seq_range(p, lens, b, &start, &len);
      n = strips_of(start, len);
      if (skip < n || b + 1 >= p.B) break;
      skip -= n;
    }
    const long long x1 = min((long long)n, skip + (hi - pos));
    begins = skip == 0;
    ends = x1 == n;
    t_lo = (start / kStrip + int(skip)) * kStrip;
    t_hi = min(len, (start / kStrip + int(x1)) * kStrip);
    tiles = (int(x1 - skip) * kStrip + kTileTok - 1) / kTileTok;
    pos += max(1ll, x1 - skip);
    skip = 0;
    ++b;
    return true;
  }
  __device__ __forceinline__ int seq() const { return b - 1; }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) decode_latent_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ unsigned char smem_raw[];
  constexpr int NH = C::NH, NS = C::NS, THREADS = C::THREADS;
  __shared__ long long prefix[THREADS + 1];
  __shared__ unsigned long long scratch[C::WARPS];
  __shared__ int lens_s[kLens];
  __shared__ __align__(8) unsigned long long bars[4 + C::DUOS + C::ROPES + 9];
  // per head: the reference (and what scores are taken relative to: 0 while there is
  // none), the factor and the shift of the last raise
  __shared__ __align__(16) float m_s[NH], mu_s[NH], f_s[NH], d_s[NH];
  __shared__ float red[4][NH];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;

  const int tid = int(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_s = base, duo_s = base + C::Q_B, rope_s = duo_s + C::DUOS * kDuoB;
  unsigned char *const rope_p = smem_raw + (rope_s - smem_u32(smem_raw));
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  // a tile's copies have landed: one barrier (of 4: never more tiles in flight) for the
  // whole tile, since a wait and its fences cost the issuing warp what 8 to 14
  // products do; a duo, a rope block is free again: one each
  constexpr int FULL = 0, EMPTY = 4, REMPTY = EMPTY + C::DUOS, QFULL = REMPTY + C::ROPES, QEMPTY = QFULL + 1, SFULL = QFULL + 2, PFULL = QFULL + 4, PVDONE = QFULL + 6, LAST = QFULL + 8;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call

  // the strips before each sequence, and whether there are sequences without any
  const int per = (p.B + THREADS - 1) / THREADS;
  unsigned long long mine = 0, sum = 0;
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
    int start, len;
    seq_range(p, b, &start, &len);
    if (b < kLens) lens_s[b] = len;
    mine += len > start ? uint64_t(strips_of(start, len)) : kIdleSeq;
  }
  const long long ahead = strips_in(block_prefix<C::WARPS>(mine, scratch, &sum));
  const bool idle = idle_seqs(sum) > 0;
  const long long total = strips_in(sum);
  prefix[tid] = ahead;
  if (tid == 0) {
    prefix[THREADS] = total;
    gave_up = 0;
    for (int i = 0; i < 4; ++i) mbar_init(bar(FULL + i), 128);
    for (int i = 0; i < C::DUOS + C::ROPES; ++i) mbar_init(bar(EMPTY + i), 1);
    mbar_init(bar(QFULL), 128);
    mbar_init(bar(QEMPTY), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(SFULL + i), 1);
      mbar_init(bar(PFULL + i), 128 * C::SETS);
      mbar_init(bar(PVDONE + i), 1);
    }
    mbar_init(bar(LAST), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // sequences of which there is nothing to attend to
  for (int b = int(blockIdx.x); idle && b < p.B; b += int(gridDim.x)) {
    int start, len;
    seq_range(p, b, &start, &len);
    if (len > start) continue;
    for (int i = tid; i < p.Hq * kLatDv; i += THREADS) store_out(p, b, i / kLatDv, i % kLatDv, 0.f);
    for (int h = tid; h < p.Hq; h += THREADS) store_lse(p, b, h, 0.f, 0.f);
    if (tid == 0) p.seq_pieces[b] = make_int2(0, 0);
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // with few strips, only as many groups take part as have a tile (two strips) each
  const long long groups = min((long long)(gridDim.x / unsigned(p.QB)), (total + 1) / 2);
  const int group = int(blockIdx.x) / p.QB, qb = int(blockIdx.x) - group * p.QB;
  if (group >= groups) return;
  const int h0 = qb * NH, heads = min(NH, p.Hq - h0);

  if (warp == C::S_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "n"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
  const uint32_t tmem_o = tmem, tmem_sc = tmem + 4 * NH;

  Pieces pc;
  pc.lens = lens_s;
  pc.pos = total * group / groups;
  pc.hi = total * (group + 1) / groups;
  {
    int a = 0, z = THREADS;                   // prefix[a] <= pos < prefix[z]
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (prefix[mid] <= pc.pos) a = mid; else z = mid;
    }
    pc.b = a * per;
    pc.skip = pc.pos - prefix[a];
  }

  if (warp >= C::COPY_WARP) {
    // ---- copies: rows of 128 bytes, 8 lanes a row, 16 rows at a time
    const int pt = tid - C::COPY_WARP * 32, c = pt & 7, r0 = pt >> 3;
    const char *kp = static_cast<const char *>(p.k);
    int duo = 0, duo_ph = 1, rope = 0, rope_ph = 1, piece = 0, full = 0;
    bool ok = true;
    while (ok && pc.next(p)) {
      const int b = pc.seq();
      if (piece > 0) ok = mbar_wait(bar(QEMPTY), uint32_t(piece - 1) & 1u, &gave_up);
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < NH / 16; ++x) {
        const int r = x * 16 + r0;
        const bool have = r < heads;
        const char *src = static_cast<const char *>(p.q) +
                          (have ? 2 * (int64_t(b) * p.q_sb + int64_t(h0 + r) * p.q_sh) + c * 16 : 0);
        const uint32_t dst = q_s + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
        for (int blk = 0; blk < 9; ++blk)
          cp_async16(dst + blk * (NH * 128), src + (have ? blk * 128 : 0), have ? 16 : 0);
      }
      mbar_arrive_copies(bar(QFULL));
      ++piece;
      auto page_at = [&](int t, int *pg) {
        int page = -1;
        if (t >= pc.start && t < pc.t_hi) {
          *pg = int(fast_div(uint32_t(t), p.fd_page));
          page = __ldg(p.table + int64_t(b) * p.t_sb + *pg);
        }
        return page;
      };
      // page numbers are read two tiles ahead, and a tile's rows brought to the L2 cache
      // one tile ahead: shared memory holds two tiles and a bit, which is less than
      // HBM's latency times an SM's share of its bandwidth
      int pages[4], places[4], next_pages[4], next_places[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pages[i] = page_at(pc.t_lo + i * 16 + r0, &places[i]);
        next_pages[i] = page_at(pc.t_lo + kTileTok + i * 16 + r0, &next_places[i]);
      }
      for (int tile = 0; ok && tile < pc.tiles; ++tile) {
        const int t0 = pc.t_lo + tile * kTileTok;
        const char *src[4];
        int bytes[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + i * 16 + r0;
          const bool have = page_present(pages[i], p.num_pages);
          bytes[i] = have ? 16 : 0;
          src[i] = kp + (have ? (int64_t(pages[i]) * p.P + (t - places[i] * p.P)) * (kLatD * 2) + c * 16 : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pages[i] = next_pages[i];
          places[i] = next_places[i];
          if (page_present(pages[i], p.num_pages)) {
            const int t = t0 + kTileTok + i * 16 + r0;
            const char *row = kp + (int64_t(pages[i]) * p.P + (t - places[i] * p.P)) * (kLatD * 2);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c * 128));
            if (c == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 1024));
          }
          next_pages[i] = page_at(t0 + 2 * kTileTok + i * 16 + r0, &next_places[i]);
        }
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          if (ok) ok = mbar_wait(bar(EMPTY + duo), uint32_t(duo_ph), &gave_up);
          if (!ok) break;
          const uint32_t dst = duo_s + duo * kDuoB + r0 * 128 + ((c ^ (r0 & 7)) << 4);
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              cp_async16(dst + a * kAtomB + i * 2048, src[i] + (bytes[i] ? part * 256 + a * 128 : 0), bytes[i]);
          if (++duo == C::DUOS) {
            duo = 0;
            duo_ph ^= 1;
          }
        }
        if (ok) ok = mbar_wait(bar(REMPTY + rope), uint32_t(rope_ph), &gave_up);
        if (!ok) break;
        const uint32_t dst = rope_s + rope * kRopeB + r0 * 128 + ((c ^ (r0 & 7)) << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + i * 2048, src[i] + (bytes[i] ? 1024 : 0), bytes[i]);
        mbar_arrive_copies(bar(FULL + full));
        full = (full + 1) & 3;
        if (++rope == C::ROPES) {
          rope = 0;
          rope_ph ^= 1;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == C::S_WARP) {
    // ---- S^T = K q^T: the warp runs as one, and one elected lane issues (descriptors
    // that the compiler knows to be the same in all lanes cost 1/6 of the issue
    // time: with a branch on the lane an issue took 90 to 270 clocks)
    constexpr uint32_t kS = instr_desc(C::BF16, kTileTok, NH, false, false);
    int duo = 0, rope = 0, piece = 0;
    uint32_t tiles = 0;
    bool ok = true;
    while (ok && pc.next(p)) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(QFULL), uint32_t(piece) & 1u, &gave_up));
      ++piece;
      for (int tile = 0; ok && tile < pc.tiles; ++tile, ++tiles) {
        const uint32_t buf = tiles & 1u, s_at = tmem_sc + buf * NH;
        // the softmax two tiles back has read this buffer
        if (tiles >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar(PFULL + buf), ((tiles - 2) >> 1) & 1u, &gave_up));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(FULL + (tiles & 3u)), (tiles >> 2) & 1u, &gave_up));
        if (!ok) break;
        uint32_t a[4];
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          a[part] = __shfl_sync(0xffffffffu, duo_s + duo * kDuoB, 0);
          if (++duo == C::DUOS) duo = 0;
        }
        const uint32_t ra = __shfl_sync(0xffffffffu, rope_s + rope * kRopeB, 0);
        if (++rope == C::ROPES) rope = 0;
        proxy_fence();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < 36; ++x)
            tc_mma(s_at, smem_desc((x < 32 ? a[x >> 3] + ((x >> 2) & 1) * kAtomB : ra) + (x & 3) * 32, 16, 1024),
                   smem_desc(q_s + (x >> 2) * (NH * 128) + (x & 3) * 32, 16, 1024), kS, x > 0);
          if (tile == pc.tiles - 1) tc_commit(bar(QEMPTY));
          tc_commit(bar(SFULL + buf));
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(bar(LAST));
    __syncwarp();
  } else if (warp == C::O_WARP) {
    // ---- O^T += V^T P^T
    constexpr uint32_t kO = instr_desc(C::BF16, 128, NH, true, true);
    int duo = 0, rope = 0;
    uint32_t tiles = 0;
    bool ok = true;
    while (ok && pc.next(p)) {
      for (int tile = 0; tile < pc.tiles; ++tile, ++tiles) {
        const uint32_t buf = tiles & 1u;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(PFULL + buf), (tiles >> 1) & 1u, &gave_up));
        if (!ok) break;
        tc_fence_after();
        const uint32_t pb = __shfl_sync(0xffffffffu, rope_s + rope * kRopeB, 0);
        uint32_t a[4], done[4];
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          a[part] = __shfl_sync(0xffffffffu, duo_s + duo * kDuoB, 0);
          done[part] = __shfl_sync(0xffffffffu, bar(EMPTY + duo), 0);
          if (++duo == C::DUOS) duo = 0;
        }
        const uint32_t rope_done = __shfl_sync(0xffffffffu, bar(REMPTY + rope), 0);
        if (++rope == C::ROPES) rope = 0;
        if (elect_one()) {
#pragma unroll
          for (int part = 0; part < 4; ++part) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              tc_mma(tmem_o + part * NH, smem_desc(a[part] + x * 2048, kAtomB, 1024),
                     smem_desc(pb + x * 2048, 1024, 1024), kO, tile > 0 || x > 0);
            tc_commit(done[part]);
          }
          tc_commit(rope_done);
          tc_commit(bar(PVDONE + buf));
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(bar(LAST));
    __syncwarp();
  } else {
    // ---- softmax: token rows warp * 16 + g and + 8, heads 8 n + 2 c and + 1
    const int set = warp >> 2, st = tid & 127, col0 = set * NS;   // this set and its first head
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const int g = lane >> 2, c = lane & 3, row0 = (warp & 3) * 16 + g;
    uint32_t tiles = 0, rope = 0;
    bool fail = false;
    while (!fail && pc.next(p)) {
      const int b = pc.seq();
      float l[NS / 4];                            // sums of heads 8 (j / 2) + 2 c + j % 2
#pragma unroll
      for (int j = 0; j < NS / 4; ++j) l[j] = 0.f;
      if (st < NS) {
        m_s[col0 + st] = -INFINITY;
        mu_s[col0 + st] = 0.f;
      }
      bool unset = true;                          // a head has no reference yet
      set_sync(set);
      for (int tile = 0; tile < pc.tiles; ++tile, ++tiles) {
        const uint32_t buf = tiles & 1u;
        bool in[2], present[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = pc.t_lo + tile * kTileTok + row0 + 8 * x;
          in[x] = t >= pc.start && t < pc.t_hi;
          present[x] = in[x] && page_present(__ldg(p.table + int64_t(b) * p.t_sb + fast_div(uint32_t(t), p.fd_page)),
                                             p.num_pages);
        }
        fail = !mbar_wait(bar(SFULL + buf), (tiles >> 1) & 1u, &gave_up);
        // O of two tiles back (long done), so that the waits for it below see each phase
        if (!fail && tiles >= 2) fail = !mbar_wait(bar(PVDONE + buf), ((tiles - 2) >> 1) & 1u, &gave_up);
        tc_fence_after();
        float e[NS / 2];                          // scores less the references, in log2: [4 n + 2 x + i]
#pragma unroll
        for (int j = 0; j < NS; j += 16) tc_ld_16x16(tmem_sc + buf * NH + lanes + col0 + j, e + j / 2);
        tc_wait_ld();
        float over = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS / 8; ++n) {
          const float2 mu = *reinterpret_cast<const float2 *>(&mu_s[col0 + 8 * n + 2 * c]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float *v = e + 4 * n + 2 * x;
            v[0] = present[x] ? fmaf(v[0], p.scale2, -mu.x) : -INFINITY;
            v[1] = present[x] ? fmaf(v[1], p.scale2, -mu.y) : -INFINITY;
            over = fmaxf(over, fmaxf(v[0], v[1]));
          }
        }
        if (p.weights) {
          float *d = p.scores + (int64_t(b) * p.Hq + h0) * p.score_row + pc.t_lo + tile * kTileTok + row0;
#pragma unroll
          for (int n = 0; n < NS / 8; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int h = col0 + 8 * n + 2 * c + i;
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (h < heads && in[x]) __stcg(d + h * p.score_row + 8 * x, e[4 * n + 2 * x + i] + mu_s[h]);
            }
        }
        if (set_any(set, unset || over > C::RAISE || fail)) {
          // raise the references (all threads take this path, or none), once the
          // product with V of the piece's tile before has ended
          if (!fail && tile > 0) fail = !mbar_wait(bar(PVDONE + (buf ^ 1u)), ((tiles - 1) >> 1) & 1u, &gave_up);
          fail = set_any(set, fail);
          if (fail) break;
          tc_fence_after();
          float v[NS / 4];
#pragma unroll
          for (int j = 0; j < NS / 4; ++j)
            v[j] = fmaxf(e[4 * (j >> 1) + (j & 1)], e[4 * (j >> 1) + 2 + (j & 1)]);
          reduce_columns<NS, true>(v, lane, red[warp & 3] + col0);
          set_sync(set);
          float now = 0.f;
          if (st < NS) {
            const int h = col0 + st;
            const float mu = mu_s[h], old = m_s[h];
            const float top = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h])) + mu;
            now = fmaxf(old, top - C::ABOVE);
            f_s[h] = old == -INFINITY ? 0.f : exp2_fast(old - now);
            m_s[h] = now;
            const float use = now == -INFINITY ? 0.f : now;
            d_s[h] = mu - use;
            mu_s[h] = use;
          }
          unset = set_any(set, now == -INFINITY);
#pragma unroll
          for (int j = 0; j < NS / 4; ++j) {
            const int h = col0 + 8 * (j >> 1) + 2 * c + (j & 1);
            l[j] *= f_s[h];
            e[4 * (j >> 1) + (j & 1)] += d_s[h];
            e[4 * (j >> 1) + 2 + (j & 1)] += d_s[h];
          }
          if (tile > 0) {
#pragma unroll 1
            for (int j = 0; j < 4 * NS; j += 16) {
              const uint32_t at = tmem_o + lanes + (j / NS) * NH + col0 + j % NS;
              float o[16];
              tc_ld16(at, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f_s[col0 + j % NS + i];
              tc_st16(at, o);
            }
            tc_wait_st();
          }
        }
        // P, rounded to the cache's type for the tensor cores (the sums l keep all
        // bits), over the rope block: a row of heads per token
        unsigned char *prow = rope_p + rope * kRopeB + row0 * 128 + c * 4;
#pragma unroll
        for (int n = 0; n < NS / 8; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) e[4 * n + i] = exp2_fast(e[4 * n + i]);
          l[2 * n] += e[4 * n] + e[4 * n + 2];
          l[2 * n + 1] += e[4 * n + 1] + e[4 * n + 3];
          const int at = ((col0 / 8 + n) ^ (row0 & 7)) << 4;   // rows 8 apart share it
          *reinterpret_cast<uint32_t *>(prow + at) = pack2<C::BF16>(e[4 * n], e[4 * n + 1]);
          *reinterpret_cast<uint32_t *>(prow + at + 1024) = pack2<C::BF16>(e[4 * n + 2], e[4 * n + 3]);
        }
        if (++rope == C::ROPES) rope = 0;
        proxy_fence();
        tc_fence_before();
        mbar_arrive(bar(PFULL + buf));
      }
      if (fail) break;
      // ---- the piece's end
      reduce_columns<NS, false>(l, lane, red[warp & 3] + col0);
      fail = !mbar_wait(bar(PVDONE + ((tiles - 1) & 1u)), ((tiles - 1) >> 1) & 1u, &gave_up);
      tc_fence_after();
      fail = set_any(set, fail);
      if (fail) break;
      const bool whole = pc.begins && pc.ends;
      float *part = p.cta_parts + (int64_t(blockIdx.x) * 2 + (pc.begins ? 1 : 0)) * C::PIECE;
      if (st < NS) {
        const int h = col0 + st;
        const float sum = (red[0][h] + red[1][h]) + (red[2][h] + red[3][h]);
        f_s[h] = !whole ? 1.f : sum == 0.f ? 0.f : p.v_scale / sum;
        if (whole) {
          if (h < heads) store_lse(p, b, h0 + h, m_s[h], sum);
        } else {
          part[NH * kLatDv + h] = m_s[h];
          part[NH * kLatDv + NH + h] = sum;
        }
      }
      if (tid == 0 && qb == 0 && pc.begins) {
        // the group the sequence begins in, and the groups it lies in
        int start, len;
        seq_range(p, b, &start, &len);
        const long long n = strips_of(start, len);
        const long long first = pc.pos - max(1, (pc.t_hi + kStrip - 1) / kStrip - pc.t_lo / kStrip);
        const int last = int(((first + n) * groups - 1) / total);
        p.seq_pieces[b] = make_int2(group, whole ? 1 : last - group + 1);
      }
      set_sync(set);
      // a thread has one element of the head for 16 heads; neighbours exchange halves,
      // so that it has two for 8: even lanes the even heads, odd lanes the odd ones
      const int odd = lane & 1;
      const int64_t step = whole ? 4 * p.o_sh : 8 * kLatDv;      // bytes, two heads on
      const int size = whole ? 4 : 8;                            // bytes of two elements
#pragma unroll 1
      for (int j = 0; j < NS; j += 16) {
        const int h_even = col0 + j + odd;        // this lane's first head
        char *const row = whole ? static_cast<char *>(p.out) + 2 * (int64_t(b) * p.o_sb + int64_t(h0 + h_even) * p.o_sh)
                                : reinterpret_cast<char *>(part + h_even * kLatDv);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f_s[h_even + 2 * i];
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          float o[16];
          tc_ld16(tmem_o + lanes + blk * NH + col0 + j, o);
          tc_wait_ld();
          float2 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? o[2 * i] : o[2 * i + 1], 1);
            v[i] = odd ? make_float2(got, o[2 * i + 1]) : make_float2(o[2 * i], got);
          }
          char *at = row + ((blk * 128 + st) >> 1) * size;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i, at += step)
              if (h_even + 2 * i < heads) *reinterpret_cast<uint32_t *>(at) = pack2<C::BF16>(v[i].x * f[i], v[i].y * f[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i, at += step)
              if (h_even + 2 * i < heads) *reinterpret_cast<float2 *>(at) = v[i];
          }
        }
      }
      tc_fence_before();
      set_sync(set);                             // m_s, f_s, red are free
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == C::S_WARP) {
    // nothing is in flight when the tensor memory is given back, after a wait that ran
    // out neither: the products that were issued end by themselves
    mbar_wait<true>(bar(LAST), 0, &gave_up);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::COLS) : "memory");
    // every role has passed its waits, and this was the last one
    if (lane == 0 && *static_cast<volatile int *>(&gave_up)) p.counters[kDecodeCtas] = 1u;
  }
}

// Adds the pieces of a sequence that several groups of CTAs share; a block per
// sequence and head, 128 threads with 4 elements each for every PARTS-th piece.
template <int NH, int PARTS>
__global__ void __launch_bounds__(128 * PARTS) latent_join_kernel(const __grid_constant__ DecodeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int PIECE = NH * kLatDv + 2 * NH;
  __shared__ float4 acc_s[PARTS][128];
  __shared__ float m_s[PARTS], l_s[PARTS];
  const int b = int(blockIdx.x) / p.Hq, h = int(blockIdx.x) - b * p.Hq;
  const int2 at = __ldcg(p.seq_pieces + b);
  if (!pieces_to_join(at.x, at.y, p.QB)) return;
  const int qb = h / NH, r = h - qb * NH, tid = int(threadIdx.x) & 127, part = int(threadIdx.x) >> 7;
  auto slot = [&](int x) { return p.cta_parts + (int64_t((at.x + x) * p.QB + qb) * 2 + (x == 0 ? 1 : 0)) * PIECE; };
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float mx, float lx, float4 v) {
    const float now = fmaxf(m, mx);
    const float was = m == -INFINITY ? 0.f : exp2_fast(m - now), f = mx == -INFINITY ? 0.f : exp2_fast(mx - now);
    acc.x = acc.x * was + f * v.x;
    acc.y = acc.y * was + f * v.y;
    acc.z = acc.z * was + f * v.z;
    acc.w = acc.w * was + f * v.w;
    sum = sum * was + f * lx;
    m = now;
  };
  for (int x0 = part; x0 < at.y; x0 += 4 * PARTS) {           // 4 pieces on their way at a time
    float4 v[4];
    float mx[4], lx[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x0 + x * PARTS >= at.y) break;
      const float *s = slot(x0 + x * PARTS);
      v[x] = __ldcg(reinterpret_cast<const float4 *>(s + r * kLatDv) + tid);
      mx[x] = __ldcg(s + NH * kLatDv + r);
      lx[x] = __ldcg(s + NH * kLatDv + NH + r);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x0 + x * PARTS >= at.y) break;
      add(mx[x], lx[x], v[x]);
    }
  }
  if constexpr (PARTS > 1) {
    acc_s[part][tid] = acc;
    if (tid == 0) m_s[part] = m, l_s[part] = sum;
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int x = 1; x < PARTS; ++x) add(m_s[x], l_s[x], acc_s[x][tid]);
  }
  store_out4(p, b, h, tid * 4, acc, sum == 0.f ? 0.f : p.v_scale / sum);
  if (tid == 0) store_lse(p, b, h, m, sum);
}

constexpr int kMaxDevices = 64;

template <int NH, bool BF16>
int launch_lat(const DecodeParams &p, int device, cudaStream_t st) {
  using C = LatConfig<NH, BF16>;
  static std::atomic<bool> ready[kMaxDevices];
  if (device >= kMaxDevices || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode_latent_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return int(e);
    if (device < kMaxDevices) ready[device].store(true, std::memory_order_release);
  }
  const int e = launch_dependent(decode_latent_kernel<C>, dim3(unsigned(kDecodeCtas / p.QB * p.QB)), C::THREADS, st, p,
                                 C::SMEM);
  if (e) return e;
  // few rows are cut into many pieces each: four at a time then
  const unsigned rows = unsigned(p.B) * unsigned(p.Hq);
  return rows < 1024 ? launch_dependent(latent_join_kernel<NH, 4>, dim3(rows), 512, st, p)
                     : launch_dependent(latent_join_kernel<NH, 1>, dim3(rows), 128, st, p);
}

}  // namespace

int launch_decode_latent(const DecodeParams &p, int device, void *stream, int *launches) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rows = latent_rows(p.Hq);
  const int e = rows == 16   ? (p.bf16 ? launch_lat<16, true>(p, device, st) : launch_lat<16, false>(p, device, st))
                : rows == 32 ? (p.bf16 ? launch_lat<32, true>(p, device, st) : launch_lat<32, false>(p, device, st))
                             : (p.bf16 ? launch_lat<64, true>(p, device, st) : launch_lat<64, false>(p, device, st));
  if (e == 0) *launches += 2;
  return e;
}

}  // namespace hicache
