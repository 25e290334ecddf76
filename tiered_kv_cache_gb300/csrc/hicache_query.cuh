// hicache_query.cuh -- attention of many query tokens over a paged K, V cache:
// cross attention, chunks of prompts, and a prefix shared by a batch.
//
// The rows of a product are pairs of a query token and one of the G query heads of
// a kv head, 128 of them, so that a token of the cache serves all that need it:
//   S [128 rows, 128 tokens] = Q K^T      head_dim / 16 steps
//   O [128 rows, head_dim]  += P V        8 steps of 16 tokens
// on the tensor cores (tcgen05), sums in tensor memory.  Two such tiles of rows (a unit
// of 256) share every block of the cache: while one's scores become exponentials, the
// tensor cores work for the other.  P goes back to tensor memory in the place of its
// scores, as the first operand of the second product; K and V lie in shared memory as
// they came (rows of 128 bytes, 128-byte swizzle).  A head of more than 128 leaves room
// for one tile of rows and blocks of 64 tokens, and a unit of up to 128 rows has only
// one: there the two score buffers are filled in turn.
//
// Bounds: with N rows a byte of the cache takes N operations (2-byte elements, N / 2
// multiply-adds), so from 280 rows on the tensor cores bind, below that HBM.  8 sequences of 2,048
// queries over 4,001 tokens, 32 heads of 128 on 8: 695 us in a burst, 1,540 TFLOP/s, 81% of a large
// library product's burst rate, and 737 us once the power cap lowers the clock; 8,191 queries of
// one prompt at themselves: 415 and 420 us, 1,320 TFLOP/s.  A step of the tensor
// cores for 128 rows takes 64 clocks whatever its operands come from, and the exponentials of
// two tiles half of the products' time on the units that compute them, so each hides behind the other
// as long as nobody waits.
//
// Softmax: a thread per row, so that maximum and sum need no other thread.  What a row's
// scores are taken relative to follows the running maximum only when the sum of a block's
// exponentials passes what P's type can hold; O is rescaled then, and only then, by the same
// thread.  (With a maximum per block in place of that sum, 2,048 queries at 32,768
// tokens took 732 us when this took 691, now 655.)
//
// Units of one tile of rows (a decode batch's prefix, short queries) would leave the second set of
// softmax warps idle: the two sets share its blocks there, even and odd, with sums of
// their own, and join them at the end.
//
// The work of few units is cut into blocks; the blocks of all units (sequences, kv heads,
// groups of rows, in order) are dealt in contiguous ranges of equal cost, chunks, to the
// CTAs (one per SM), whatever the lengths.  A chunk's part of a unit is a piece; whole units are
// written out directly, the other pieces go to the workspace and query_join_kernel adds
// them in order, so that timing cannot change the result.  Of many units each CTA takes one
// after another from a counter: which CTA has a unit does not change its result either.
//
// Warps: softmax and epilogue (four for each tile of rows); four that copy the cache into
// shared memory; one that issues the products; one that makes what cp.async brought visible to
// them; one that plans, a few pieces ahead of the others, what this CTA does.  The copies are TMA
// boxes of 64 elements by 16 to 64 rows where the pages are whole boxes (see query_maps), else
// cp.async of 16 bytes a lane, so any page size, absent tokens as zeros; e4m3 comes through
// registers, to fp16.  Every wait has a limit of about two seconds, after which the CTA gives up,
// sets the workspace's error word and returns.
//
// The instruction cache is what this layout minds most: above about 128 KB of code whatever is
// not the inner loop runs at 8 clocks an instruction and more, hence the planner in one
// warp, loops that are not unrolled and prefix calls in kernels of their own.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <atomic>

#include "hicache_decode.cuh"
#include "hicache_tcgen05.cuh"

namespace hicache {
namespace {

enum : int { kQBf16 = 0, kQFp16 = 1, kQE4m3 = 2 };   // element types of the cache

// OWN: a prefix call's, whose units are the groups' prefixes and then the sequences' own
// tokens, with results in 32 bits for prefix_end_kernel; of its own, since the code for both in one
// kernel costs a call without groups 5 to 9% (8,192 queries at themselves: 411 -> 445 us).
template <int DP_, int TYPE_, bool OWN_ = false>
struct QueryConfig {
  static constexpr int DP = DP_;                  // head_dim, padded
  static constexpr int TYPE = TYPE_;
  static constexpr bool OWN = OWN_;
  static constexpr bool BF16 = TYPE_ == kQBf16;   // the products' type, else fp16
  static constexpr int ES = TYPE_ == kQE4m3 ? 1 : 2;
  static constexpr int QT = DP_ <= 128 ? 2 : 1;   // tiles of rows
  static constexpr int BN = DP_ <= 128 ? 128 : 64;
  static constexpr int ROWS = QT * kQueryRows;    // of a unit
  static constexpr int ATOMS = DP_ / 64;          // of 64 elements: 128 bytes a row
  static constexpr int QATOM_B = kQueryRows * 128, ATOM_B = BN * 128;
  static constexpr int QTILE_B = ATOMS * QATOM_B, TILE_B = ATOMS * ATOM_B;
  static constexpr int STAGES = query_stages(DP_);   // tiles of K or V
  static constexpr int SMEM = QT * QTILE_B + STAGES * TILE_B;
  static constexpr int SOFT_WARPS = 4 * QT, COPY_WARP = SOFT_WARPS, MMA_WARP = COPY_WARP + 4;
  static constexpr int WARPS = MMA_WARP + 4, THREADS = WARPS * 32;
  // Registers of a thread of each group of four warps: what the launch has, dealt anew.  The
  // softmax holds up to 64 scores, e4m3 copies two tiles' parts (with 88 registers for them 239 us
  // in place of 172, with 120 the same).
  static constexpr bool E4 = TYPE_ == kQE4m3;
  // Halves of a block whose scores are loaded together, and whose code is there twice: 4 to 6% for
  // what the products bind (2,048 queries at 32,768: 689 -> 659 us, 8 x 2,048 740 -> 695), but 23 to
  // 29% against what copies and starts do (32 ragged encoders 50 -> 64, e4m3 172 -> 212), for
  // the instruction cache.
  static constexpr int AT_ONCE = BN == 128 && DP_ == 128 && !E4 ? 2 : 1;
  static constexpr int SOFT_REGS = QT == 1 ? 240 : E4 ? 176 : 192, COPY_REGS = QT == 1 ? 152 : E4 ? 104 : 72,
                       MMA_REGS = QT == 1 ? 112 : 56;
  static_assert(4 * QT * SOFT_REGS + 4 * COPY_REGS + 4 * MMA_REGS <= WARPS * (65536 / THREADS / 8 * 8), "registers");
  static constexpr int O_COL = 2 * BN;            // tensor memory: two score buffers, then O of each tile
  static constexpr int PIECE = ROWS * DP_ + 2 * ROWS;   // floats: O [tile][element][row], m, l
  static constexpr float LIMIT = BF16 ? 1.f : 32768.f, ABOVE = kAbove<!BF16>;   // 2^kRaise
  static_assert(kRaise<false> == 0.f && kRaise<true> == 15.f, "the sums' limit");
  static_assert(O_COL + QT * DP_ <= 512, "tensor memory");
  static_assert(query_turns_hold(kQueryTurns, STAGES), "a parity wait of the copies could pass two phases early");
  static_assert(query_info_holds(kQueryInfo, kQueryTurns, STAGES), "what is present of a block could be overwritten");
};

// A shared-memory operand's descriptor in two halves (see smem_desc): the upper is the same
// for all, the lower moves by an address over 16, so that a product costs an addition.
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;   // 8 rows of 128 bytes, 128-byte swizzle
// d += a b in one lane of a warp that runs as one: predicated, not behind a branch, where the
// compiler takes each operand from vector registers
__device__ __forceinline__ void tc_mma_in(uint32_t lane, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{.reg .pred p, q; .reg .b64 x, y; setp.ne.u32 p, %5, 0; setp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc),
      "r"(add), "r"(lane)
      : "memory");
}
// the same with a in tensor memory
__device__ __forceinline__ void tc_mma_ta(uint32_t lane, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{.reg .pred p, q; .reg .b64 y; setp.ne.u32 p, %5, 0; setp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc),
      "r"(add), "r"(lane)
      : "memory");
}
__device__ __forceinline__ void tc_commit_in(uint32_t lane, uint32_t bar) {
  asm volatile(
      "{.reg .pred q; setp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];}" ::"r"(bar), "r"(lane)
      : "memory");
}
// 16 bytes of the cache, or zeros; issued here, not where they are first used
__device__ __forceinline__ uint4 load_or_zero(const void *at, bool yes) {
  uint4 v;
  asm volatile(
      "{.reg .pred p; setp.ne.u32 p, %5, 0; mov.u32 %0, 0; mov.u32 %1, 0; mov.u32 %2, 0; mov.u32 %3, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at), "r"(uint32_t(yes)));
  return v;
}
// what is the same in all lanes, in a register that the compiler knows to be
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t elected() {
  uint32_t r;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tc_ld32(uint32_t addr, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
// The loads so far are there; the registers pass through, so that no use of them moves up.
__device__ __forceinline__ void tc_loaded32(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
  asm volatile(""
               : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_st16u(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// two floats at a time
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t x, float *v) { asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int REGS, bool MORE>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
__device__ __forceinline__ uint32_t q_e4m3(uint32_t two) {   // two e4m3 in the low 16 bits -> two fp16, exactly
  uint32_t r;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ float2 q_unpack2(uint32_t u, bool bf16) {
  return bf16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u))
              : __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// The layer's buffers as TMA sees them, rows of elements of 2 bytes in boxes of 64 elements
// (128 bytes) by `box` rows; box 0: not at all.
// q, as [token, kv head, head of the group, element], in boxes of 64 elements by 128 rows of a
// tile; q_boxes 0: not at all.
struct QueryMaps {
  CUtensorMap k, v, q;
  int32_t box, q_boxes;
};
__device__ __forceinline__ void tma_box4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {   // and arrives
  asm volatile("{.reg .b64 t; mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;}" ::"r"(bar), "r"(bytes) : "memory");
}
// mbar_wait for what takes as long as the work in hand does: the limit runs from the last end of a
// phase of `moves`, a barrier that the work in hand ends again and again.
__device__ __forceinline__ bool mbar_wait_moving(uint32_t bar, uint32_t parity, uint32_t moves, volatile int *gave_up) {
  uint32_t turn = 0;
  long long since = 0;
  for (;;) {
    uint32_t done, moved;
    asm volatile(
        "{.reg .pred p, q; mbarrier.try_wait.parity.shared::cta.b64 p, [%2], %3; selp.u32 %0, 1, 0, p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 q, [%4], %5; selp.u32 %1, 1, 0, q;}"
        : "=r"(done), "=r"(moved)
        : "r"(bar), "r"(parity), "r"(moves), "r"(turn)
        : "memory");
    if (done) return true;
    if (*gave_up) return false;
    const long long now = clock64();
    if (since == 0 || moved) since = now;
    turn ^= moved;
    if (now - since > kWaitClocks) {
      *gave_up = int(bar);
      return false;
    }
  }
}

// A sequence's queries and tokens; starts that do not ascend, or leave the rows there
// are, hold no query.
struct QuerySeq {
  int32_t q0, nq, kv;
};
__device__ __forceinline__ QuerySeq query_seq(const QueryParams &p, int b) {
  QuerySeq s;
  s.q0 = min(max(__ldg(p.starts + b), 0), p.N);
  s.nq = min(max(__ldg(p.starts + b + 1), s.q0), p.N) - s.q0;
  s.kv = int(min(int64_t(max(0, __ldg(p.lens + b))), int64_t(p.max_pages) * p.P));
  return s;
}

// a / b of what is not negative, in 32 bits where they fit: a division of 64 takes 400 clocks
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
  return a / b;
}

// The pieces of a chunk, in order.  A unit counts its blocks and kQueryStart more, what
// beginning and ending it takes.
template <class C>
struct QueryPieces {
  long long pos, hi;
  int b, h, m, units, off;         // the unit: sequence, kv head, group of rows (of `units`); how much of it is done
  QuerySeq s;
  QueryUnit u;
  // the current piece: blocks [x0, x1) of the unit
  int x0, x1;
  __device__ __forceinline__ bool begins() const { return x0 == 0; }
  __device__ __forceinline__ bool ends() const { return x1 == u.blocks; }
  // one tile of rows, or two that share the blocks
  __device__ __forceinline__ bool dual() const { return C::QT == 2 && u.rows > kQueryRows; }
  __device__ __forceinline__ QueryUnit unit(const QueryParams &p, int i) const {
    return query_unit(i, s.nq, s.kv, p.fd_group, C::ROWS, C::BN, p.causal, p.window);
  }
  __device__ __forceinline__ void sequence(const QueryParams &p) {
    s = query_seq(p, b);
    units = query_units(s.nq, p.G, C::ROWS);
  }
  __device__ __forceinline__ int cost(const QueryParams &p, int i) const { return query_cost(unit(p, i).blocks); }
  // what a kv head of the sequence counts (a whole warp calls)
  __device__ __forceinline__ long long head(const QueryParams &p) const {
    const int lane = int(threadIdx.x) & 31;
    if (units == 0) return 0;
    long long n = 0;
#pragma unroll 1
    for (int i = lane; i < (p.causal ? units : 1); i += 32) n += cost(p, i);
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return p.causal ? n : n * units;              // alike, then
  }
  // at `at` of all, `rest` from the first of sequence b (a whole warp calls)
  __device__ __forceinline__ void start(const QueryParams &p, long long at, long long end, int b0, long long rest) {
    const int lane = int(threadIdx.x) & 31;
    pos = at;
    hi = end;
    b = b0;
    long long n;
    for (;; ++b) {
      sequence(p);
      n = head(p);
      if (rest < n * p.Hkv || b + 1 >= p.B) break;
      rest -= n * p.Hkv;
    }
    h = n > 0 ? int(quotient(rest, n)) : 0;
    rest -= h * n;
    m = 0;
    if (!p.causal) {
      const int each = units > 0 ? int(quotient(n, units)) : 0;   // (a head's count: of units that are alike)
      m = each > 0 ? int(quotient(rest, each)) : 0;
      rest -= (long long)m * each;
    } else {
#pragma unroll 1
      for (;; m += 32) {           // 32 units at a time
        const int mine = m + lane < units ? cost(p, m + lane) : 0;
        int inc = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const int all = __shfl_sync(0xffffffffu, inc, 31);
        if (rest >= all && m + 32 < units) {
          rest -= all;
          continue;
        }
        const unsigned past = __ballot_sync(0xffffffffu, inc > rest);
        const int at_lane = past ? __ffs(int(past)) - 1 : 31;
        rest -= __shfl_sync(0xffffffffu, inc - mine, at_lane);
        m += at_lane;
        break;
      }
    }
    u = unit(p, m);
    off = int(rest);
  }
  __device__ __forceinline__ bool next(const QueryParams &p) {
    do {
      if (pos >= hi) return false;
      while (off >= query_cost(u.blocks)) {
        if (++m >= units) {
          m = 0;
          if (++h >= p.Hkv) {
            h = 0;
            do {
              if (++b >= p.B) return false;
              sequence(p);
            } while (units == 0 || s.kv == 0);
          }
        }
        u = unit(p, m);
        off = 0;
      }
      const int end = int(min((long long)query_cost(u.blocks), off + (hi - pos)));
      pos += end - off;
      x0 = max(0, off - kQueryStart);
      x1 = max(0, end - kQueryStart);
      off = end;
    } while (x1 == x0);
    return true;
  }
};

// A piece as the roles see it; n == 0: there is none any more.
struct alignas(16) QueryPiece {
  int32_t b, h, n, t0;             // sequence, kv head, blocks, the first one's first token
  int32_t row0, rows, q0, nq;      // rows of the unit; the sequence's first query and their number
  int32_t kv, lo, hi, flags;       // tokens of the sequence; those [lo, hi) that some row of the unit sees
};
enum : int { kTwoTiles = 1, kBegins = 2, kWhole = 4, kOwn = 8 };   // kOwn: over the sequence's own tokens
constexpr int kPieceRing = kQueryPieces;

// The output's row of row r of a unit: the query token and head.
struct QueryRow {
  int64_t token;
  int head;
  int i;                           // query of the sequence
};
__device__ __forceinline__ QueryRow query_row(const QueryParams &p, int q0, int h, int r) {
  QueryRow x;
  x.i = int(fast_div(uint32_t(r), p.fd_group));
  x.token = int64_t(q0) + x.i;
  x.head = h * p.G + (r - x.i * p.G);
  return x;
}
__device__ __forceinline__ void query_lse(const QueryParams &p, const QueryRow &x, float m, float l) {
  const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
  if (p.lse2) p.lse2[x.token * p.Hq + x.head] = lse2;
  else if (p.lse) p.lse[x.token * p.lse_st + x.head] = lse2 * kLn2;
}
// the call's type is the cache's, but for e4m3
template <class C>
__device__ __forceinline__ uint4 query_pack8(const QueryParams &p, const float *v) {
  if (C::TYPE == kQE4m3 ? p.bf16 : C::BF16)
    return make_uint4(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]), pack2<true>(v[4], v[5]), pack2<true>(v[6], v[7]));
  return make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]), pack2<false>(v[6], v[7]));
}
// 8 elements of a row from a multiple of 8 on
__device__ __forceinline__ void query_store8(const QueryParams &p, const QueryRow &x, int col, const float *v) {
  if (p.out32) {
    float4 *at = reinterpret_cast<float4 *>(p.out32 + (x.token * p.Hq + x.head) * p.D + col);
    at[0] = make_float4(v[0], v[1], v[2], v[3]);
    at[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  char *at = static_cast<char *>(p.out) + 2 * (x.token * p.o_st + int64_t(x.head) * p.o_sh + col);
  *reinterpret_cast<uint4 *>(at) = p.bf16 ? query_pack8<QueryConfig<64, kQBf16>>(p, v) : query_pack8<QueryConfig<64, kQFp16>>(p, v);
}

// The boxes of V in `rows` row by row, zeros beyond [lo, hi); by one warp.  Not inlined: it is rare,
// and with it inlined what the products bind loses 2% (8 x 2,048 queries 695 -> 710 us).
__device__ __noinline__ void copy_cut_boxes(uint32_t rows, const char *v, int64_t pitch, int y, int box_r, int box_c, int box, int d,
                                            uint32_t at, uint32_t atom, int t_lo, int t_hi) {
  const int lane = int(threadIdx.x) & 31;
#pragma unroll 1
  for (; rows; rows &= rows - 1u) {
    const int src = __ffs(int(rows)) - 1;
    const int64_t y0 = __shfl_sync(0xffffffffu, y, src);
    const int r0 = __shfl_sync(0xffffffffu, box_r, src), c0 = __shfl_sync(0xffffffffu, box_c, src);
    const int c = lane & 7, col = c0 + c * 8;     // 8 lanes a row of 128 bytes
#pragma unroll 1
    for (int i = lane >> 3; i < box; i += 4) {
      const int x = r0 + i;
      const bool in = x >= t_lo && x < t_hi;
      if (col < d)
        cp_async16(at + uint32_t(c0 >> 6) * atom + x * 128 + ((c ^ (x & 7)) << 4), in ? v + (y0 + i) * pitch + col * 2 : v,
                   in ? 16 : 0);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  proxy_fence();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) query_kernel(const __grid_constant__ QueryParams p, const __grid_constant__ QueryMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  constexpr int BN = C::BN, THREADS = C::THREADS, WORDS = BN / 32, INFO = kQueryInfo, PARTS = BN / 64;
  __shared__ long long scratch[C::WARPS], units_of[C::WARPS];
  __shared__ long long first_rest;                // where the chunk starts: blocks from the first of a sequence on
  __shared__ int first_seq;
  __shared__ __align__(8) unsigned long long bars[3 * C::STAGES + INFO + 16 + 2 * kPieceRing];
  __shared__ int64_t offs[2][BN];                 // the rows a block's tokens lie in; -1: absent
  __shared__ uint32_t there[INFO][WORDS];         // which of them are present
  __shared__ QueryPiece ring_of_pieces[kPieceRing];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  // (static variables, up to the tiles' alignment)
  static_assert(C::SMEM + (sizeof(scratch) + sizeof(units_of) + sizeof(bars) + sizeof(offs) + sizeof(there) +
                           sizeof(ring_of_pieces) + 64 + 1023) / 1024 * 1024 <= 227 * 1024, "a block's shared memory");

  const int tid = int(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t q_s = smem_u32(smem_raw), ring_s = q_s + C::QT * C::QTILE_B;
  unsigned char *const q_p = smem_raw, *const ring_p = smem_raw + C::QT * C::QTILE_B;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  // A stage is full, its copies are visible to the products, it is empty; what of a block
  // is present; Q of a tile is there; a lane's scores, exponentials are there, their product with V
  // is done; the last product; the copying warps are together; a piece is there, is read.
  // A lane is a score buffer, of a tile of rows, or, in a unit with one tile, of every other
  // block: the two sets of softmax warps share its blocks then, each with sums of its own,
  // which the first set adds up when the second has put its (OTHER) and until when it leaves
  // them (ADDED).
  constexpr int FULL = 0, EMPTY = C::STAGES, READY = 2 * C::STAGES, KNOWN = 3 * C::STAGES, QFULL = KNOWN + INFO,
                SFULL = QFULL + 2, PFULL = SFULL + 2, PVDONE = PFULL + 4, LAST = PVDONE + 4, GROUP = LAST + 1,
                OTHER = GROUP + 1, ADDED = OTHER + 1, PIECE = ADDED + 1,
                TAKEN = PIECE + kPieceRing;       // PFULL, PVDONE: + 2 for a block's second half
  // rows that cp.async brings tile after tile: a warp makes them visible to the products
  const bool relayed = C::TYPE != kQE4m3 && maps.box == 0;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the work before this call

  // ---- what lies before each sequence; thread i takes `per` sequences
  const int per = (p.B + THREADS - 1) / THREADS;
  long long mine = 0, units = 0;
  bool zero = false;                              // a sequence has rows that no unit holds
#pragma unroll 1
  for (int x = 0; x < per; ++x) {
    const int b = tid * per + x;
    QueryPieces<C> t;
    t.s = b < p.B ? query_seq(p, b) : QuerySeq{0, 0, 0};
    t.units = query_units(t.s.nq, p.G, C::ROWS);
    long long n = 0;
    const bool many = p.causal && t.units > 4;    // counted by the whole warp
#pragma unroll 1
    for (int i = 0; !many && i < (p.causal ? t.units : min(t.units, 1)); ++i) n += t.cost(p, i);
    if (!p.causal) n *= t.units;
#pragma unroll 1
    for (unsigned todo = __ballot_sync(0xffffffffu, many); todo; todo &= todo - 1u) {
      const int src = __ffs(int(todo)) - 1;
      QueryPieces<C> o;
      o.s.nq = __shfl_sync(0xffffffffu, t.s.nq, src);
      o.s.kv = __shfl_sync(0xffffffffu, t.s.kv, src);
      o.units = __shfl_sync(0xffffffffu, t.units, src);
      const long long all = o.head(p);
      if (lane == src) n = all;
    }
    mine += n * p.Hkv;
    units += (long long)t.units * p.Hkv;
    zero |= t.s.nq > 0 && (t.s.kv == 0 || (p.causal && t.s.nq > t.s.kv));
  }
  long long total = 0, all_units = 0;
  const bool zeros = __syncthreads_or(zero);
  for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
  if (lane == 0) units_of[warp] = units;          // read behind block_prefix's barrier
  const long long ahead = block_prefix<C::WARPS>(mine, scratch, &total);
  for (int w = 0; w < C::WARPS; ++w) all_units += units_of[w];
  // with less than that for each CTA, only as many CTAs take part
  const long long chunks = min((long long)gridDim.x, total);
  // With many units to a CTA, whole units one after another (see the planner)
  const bool whole_units = all_units >= kQueryWhole * (long long)gridDim.x;
  if (blockIdx.x < chunks) {
    const long long lo = quotient(total * int(blockIdx.x), chunks);
    if (ahead <= lo && lo < ahead + mine) {       // one thread
      first_seq = tid * per;
      first_rest = lo - ahead;
    }
  }
  if (tid == 0) {
    gave_up = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(bar(FULL + i), 128);
      mbar_init(bar(EMPTY + i), 1);
      mbar_init(bar(READY + i), 1);
    }
    for (int i = 0; i < INFO; ++i) mbar_init(bar(KNOWN + i), 4);
    for (int i = 0; i < 2; ++i) mbar_init(bar(QFULL + i), maps.q_boxes > 0 ? 1 : 4);
    mbar_init(bar(OTHER), 4);
    mbar_init(bar(ADDED), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(SFULL + i), 1);
      for (int part = 0; part < 4; part += 2) {
        mbar_init(bar(PFULL + part + i), 4);
        mbar_init(bar(PVDONE + part + i), 1);
      }
    }
    mbar_init(bar(LAST), 1);
    mbar_init(bar(GROUP), 4);
    for (int i = 0; i < kPieceRing; ++i) {
      mbar_init(bar(PIECE + i), 1);
      mbar_init(bar(TAKEN + i), C::SOFT_WARPS + 5 + int(relayed));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    p.open[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  // rows of which there is nothing to attend to and that no unit holds: of sequences
  // without tokens, and of queries before the first token
#pragma unroll 1
  for (int b = int(blockIdx.x); zeros && b < p.B; b += int(gridDim.x)) {
    const QuerySeq s = query_seq(p, b);
    uint32_t rows = uint32_t(s.nq) * p.G;         // times Hkv under 2^31, as N * Hq is
    if (s.kv > 0) rows = p.causal ? uint32_t(max(0, min(s.nq, s.nq - s.kv))) * p.G / C::ROWS * C::ROWS : 0;
#pragma unroll 1
    for (uint32_t i = tid; i < rows * p.Hkv; i += THREADS) {
      const QueryRow x = query_row(p, s.q0, int(i / rows), int(i % rows));
      char *const at = C::OWN ? reinterpret_cast<char *>(p.out32 + (x.token * p.Hq + x.head) * p.D)
                              : static_cast<char *>(p.out) + 2 * (x.token * p.o_st + int64_t(x.head) * p.o_sh);
#pragma unroll 1
      for (int c = 0; c < p.D * (C::OWN ? 4 : 2); c += 16) *reinterpret_cast<uint4 *>(at + c) = make_uint4(0u, 0u, 0u, 0u);
      query_lse(p, x, 0.f, 0.f);
    }
  }
  if (C::OWN) {                                   // rows of no sequence
    const int s0 = p.B > 0 ? min(max(__ldg(p.starts), 0), p.N) : 0;
    const int s1 = p.B > 0 ? min(max(__ldg(p.starts + p.B), s0), p.N) : 0;
#pragma unroll 1
    for (uint32_t i = blockIdx.x * THREADS + tid; i < uint32_t(p.N) * p.Hq; i += gridDim.x * THREADS)
      if (int(i / p.Hq) < s0 || int(i / p.Hq) >= s1) p.lse2[i] = -INFINITY;
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (blockIdx.x >= chunks && !C::OWN) return;
  if (q_s & 1023u) {                              // the tiles' swizzle counts on it
    if (tid == 0) *p.error = 1u;
    return;
  }

  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_base);

  const int d16 = (p.D + 15) & ~15;
  // The next piece, in order: every warp but the planner's takes each of them.
  uint32_t taken = 0;
  bool ok = true;
  auto took = [&](QueryPiece &x, bool there_is) {
    const uint32_t i = taken % kPieceRing;
    ok = __all_sync(0xffffffffu, there_is);
    if (!ok) return false;
    x = ring_of_pieces[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(TAKEN + i));
    ++taken;
    return __any_sync(0xffffffffu, x.n > 0) != 0;
  };
  auto take = [&](QueryPiece &x) {
    return took(x, mbar_wait(bar(PIECE + taken % kPieceRing), (taken / kPieceRing) & 1u, &gave_up));
  };

  if (warp >= C::MMA_WARP) {
    set_registers<C::MMA_REGS, false>();
    if (warp == C::MMA_WARP) {
      // ---- the products: the warp runs as one, one elected lane issues.  In the order
      // QK(0) QK(1) PV(0) QK(2) PV(1) QK(3) ...: products of one CTA run in order, so
      // QK(s + 2) may overwrite the buffer that PV(s) reads.
      const uint32_t s_desc = instr_desc(C::BF16, kQueryRows, BN, false, false);
      const uint32_t o_desc = instr_desc(C::BF16, kQueryRows, d16, false, true);
      const int ksteps = d16 / 16;
      const uint32_t one = elected();             // all products and commits are this lane's
      int kst = 0, kph = 0, vst = 1, vph = 0;     // stage and phase of the next block's K, V
      uint32_t used0 = 0, used1 = 0, duals = 0, pieces = 0;
      auto wait = [&](int b, uint32_t parity) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1u, &gave_up));
      };
      auto arrived = [&](int stage, int parity) { wait((relayed ? READY : FULL) + stage, uint32_t(parity)); };
      QueryPiece pc;
      while (take(pc)) {
        const bool dual = __all_sync(0xffffffffu, pc.flags & kTwoTiles);
        const int steps = int(uniform(uint32_t(pc.n))) << int(dual);
        uint32_t k_at = 0, v_at = 0;              // of the block's K, V
        // PV(s), QK(s + 2) with score buffer x
        auto step = [&](int s, int x) {
          const bool last_of_tile = !dual || x == 1, more = s + 2 < steps;
          const uint32_t s_at = tmem + x * BN, o_at = tmem + C::O_COL + (C::QT == 2 ? x : 0) * C::DP;
          // what two tiles share is waited for ahead of the exponentials, so that PV(s) and
          // QK(s + 2) follow one another without a pause
          if (!dual || x == 0) {
            if (s >= 0) {
              arrived(vst, vph);
              v_at = uniform(desc_low(ring_s + vst * C::TILE_B, C::ATOM_B));
            }
            if (ok && dual && more) {
              arrived(kst, kph);
              k_at = uniform(desc_low(ring_s + kst * C::TILE_B, 16));
            }
          }
          if (s >= 0) {
            const uint32_t turn = (x == 0 ? used0 : used1) + uint32_t(s >> 1);
            const uint32_t add = s >= C::QT;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              if (ok) wait(PFULL + 2 * part + x, turn);
              if (!ok) return;
              tc_fence_after();
#pragma unroll
              for (int i = 4 * part; i < 4 * part + 4; ++i)
                tc_mma_ta(one, o_at, s_at + i * 8, v_at + i * (2048 >> 4), o_desc, i > 0 ? 1u : add);
              tc_commit_in(one, bar(PVDONE + 2 * part + x));
            }
            if (last_of_tile) {
              tc_commit_in(one, bar(EMPTY + vst));
              if ((vst += 2) >= C::STAGES) vst -= C::STAGES, vph ^= 1;
            }
          }
          if (!ok || !more) return;
          if (!dual) {
            arrived(kst, kph);
            if (!ok) return;
            k_at = uniform(desc_low(ring_s + kst * C::TILE_B, 16));
          }
          tc_fence_after();
          const uint32_t q_at = desc_low(q_s + (dual ? x : 0) * C::QTILE_B, 16);
          auto product = [&](int i) {
            tc_mma_in(one, s_at, q_at + ((i >> 2) * C::QATOM_B + (i & 3) * 32) / 16, k_at + ((i >> 2) * C::ATOM_B + (i & 3) * 32) / 16,
                      s_desc, i > 0);
          };
          if (ksteps == C::DP / 16) {
#pragma unroll
            for (int i = 0; i < C::DP / 16; ++i) product(i);
          } else {
#pragma unroll 1
            for (int i = 0; i < ksteps; ++i) product(i);
          }
          tc_commit_in(one, bar(SFULL + x));
          if (last_of_tile) {
            tc_commit_in(one, bar(EMPTY + kst));
            if ((kst += 2) >= C::STAGES) kst -= C::STAGES, kph ^= 1;
          }
        };
#pragma unroll 1
        for (int s = -2; ok && s < steps; s += 2) {
          if (s < 0) {
            wait(QFULL, pieces++);
            if (!ok) break;
          }
          step(s, 0);
          if (!ok || s + 1 >= steps) break;
          if (s < 0 && dual) {
            wait(QFULL + 1, duals++);
            if (!ok) break;
          }
          step(s + 1, 1);
        }
        if (!ok) break;
        used0 += uint32_t(steps + 1) >> 1;
        used1 += uint32_t(steps) >> 1;
      }
      tc_commit_in(one, bar(LAST));
      __syncwarp();
    } else if (relayed && warp == C::MMA_WARP + 1) {
      // ---- copies that have landed are made visible to the products: the fence takes
      // hundreds of clocks, which the warp that issues them does not have
      int stage = 0, phase = 0;
      QueryPiece pc;
      while (take(pc)) {
        for (int x = 0; ok && x < 2 * pc.n; ++x) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(FULL + stage), uint32_t(phase), &gave_up));
          if (!ok) break;
          proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(READY + stage));
          if (++stage == C::STAGES) stage = 0, phase ^= 1;
        }
        if (!ok) break;
      }
    } else if (warp == C::MMA_WARP + 2) {
      // ---- the planner: this CTA's pieces, a few ahead of the other warps.  (With this in
      // every role the kernel was 200 KB, more than the instruction cache holds: whatever was
      // not the inner loop ran at 8 clocks an instruction and more.)
      // Few units: the chunk's pieces.  Many: whole units, taken from a counter as they are
      // needed, those of one kv head one after another, so that the CTAs read the same part of
      // the cache at the same time, the longest first; which CTA has a unit does not change
      // its result.
      QueryPieces<C> pc;
      int list = 0;                               // 1: of the sequences' own tokens, when the prefixes are dealt
      int base = -32, part = 0;                   // the sequences of this and 31 more, one a lane; kOwnTokens of them
      long long before = 0, upto = 0;             // units before them; this lane's and those before it
      QuerySeq seq{0, 0, 0};
      const int own_units = query_units(1, p.G, C::ROWS);
      auto group = [&]() {
        const int b = base + lane;
        seq = QuerySeq{0, 0, 0};
        if (!C::OWN || list == 0) {
          if (b < p.B) seq = query_seq(p, b);
          upto = (long long)query_units(seq.nq, p.G, C::ROWS) * p.Hkv;
        } else {
          if (b < p.N) seq = QuerySeq{b, 1, int(min(int64_t(max(0, __ldg(p.own_lens + b))), int64_t(p.own_pages) * p.P))};
          upto = (long long)own_parts(seq.kv) * own_units * p.Hkv;
        }
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
      };
      auto claim = [&]() {                        // the next whole unit with something to attend to
        for (;;) {
          long long at = lane == 0 ? (long long)atomicAdd(p.next + (C::OWN ? list : 0), 1ull) : 0;
          at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll 1
          for (;;) {
            const long long here = __shfl_sync(0xffffffffu, upto, 31);   // 0 at first
            if (at < before + here) break;
            before += here;
            base += 32;
            if (base >= (!C::OWN || list == 0 ? p.B : p.N)) return false;
            group();
          }
          const int src = __ffs(int(__ballot_sync(0xffffffffu, before + upto > at))) - 1;
          pc.b = base + src;
          pc.s.q0 = __shfl_sync(0xffffffffu, seq.q0, src);
          pc.s.nq = __shfl_sync(0xffffffffu, seq.nq, src);
          pc.s.kv = __shfl_sync(0xffffffffu, seq.kv, src);
          pc.x0 = 0;
          const int parts = C::OWN ? own_parts(pc.s.kv) : 0;
          pc.units = !C::OWN || list == 0 ? query_units(pc.s.nq, p.G, C::ROWS) : own_units * parts;
          const int i = int(at - (before + __shfl_sync(0xffffffffu, upto, src) - (long long)pc.units * p.Hkv));
          pc.h = i / pc.units;
          const int m = i - pc.h * pc.units;
          part = !C::OWN || list == 0 ? 0 : m / own_units;
          pc.m = !C::OWN || list == 0 ? pc.units - 1 - m : m - part * own_units;
          pc.u = pc.unit(p, pc.m);
          if (C::OWN && list == 1) {
            pc.u.blk0 = part * (kOwnTokens / BN);
            pc.u.blocks = (own_end(part * kOwnTokens, pc.s.kv) - part * kOwnTokens + BN - 1) / BN;
          }
          pc.x1 = pc.u.blocks;
          if (pc.x1 > 0) return true;
        }
      };
      pc.pos = pc.hi = 0;
      if (!whole_units && blockIdx.x < chunks)
        pc.start(p, quotient(total * int(blockIdx.x), chunks), quotient(total * (int(blockIdx.x) + 1), chunks), first_seq, first_rest);
      bool more = true;
#pragma unroll 1
      for (uint32_t i = 0; more; ++i) {
        const uint32_t slot = i % kPieceRing;
#pragma unroll 1
        for (;;) {
          const bool counted = whole_units || (C::OWN && list == 1);
          // a whole unit is taken when the one before it is begun, so that none waits at the
          // end for a CTA that has another to do
          const uint32_t ahead = counted ? 1 : kPieceRing, j = i - ahead;
          // (for as long as a piece takes, which nothing bounds)
          if (i >= ahead)
            ok = __all_sync(0xffffffffu, mbar_wait_moving(bar(TAKEN + j % kPieceRing), (j / kPieceRing) & 1u, bar(EMPTY), &gave_up));
          if (!ok) break;
          more = __any_sync(0xffffffffu, counted ? claim() : pc.next(p)) != 0;
          if (!C::OWN || more || list == 1) break;
          list = 1, base = -32, before = upto = 0;
        }
        if (!ok) break;
        if (lane == 0) {
          QueryPiece x{};
          if (more) {
            const bool begins = pc.begins(), whole = begins && pc.ends();
            int unused;
            query_sees(int(fast_div(uint32_t(pc.u.row0), p.fd_group)), pc.s.nq, pc.s.kv, p.causal, p.window, &x.lo, &unused);
            query_sees(int(fast_div(uint32_t(pc.u.row0 + pc.u.rows - 1), p.fd_group)), pc.s.nq, pc.s.kv, p.causal,
                       p.window, &unused, &x.hi);
            x.b = pc.b;
            x.h = pc.h;
            x.n = pc.x1 - pc.x0;
            x.t0 = (pc.u.blk0 + pc.x0) * BN;
            x.row0 = pc.u.row0;
            x.rows = pc.u.rows;
            x.q0 = pc.s.q0;
            x.nq = pc.s.nq;
            x.kv = pc.s.kv;
            x.flags = (pc.dual() ? kTwoTiles : 0) | (begins ? kBegins : 0) | (whole ? kWhole : 0);
            if (C::OWN && list == 1) {
              x.flags |= kOwn;
              x.lo = part * kOwnTokens;
              x.hi = own_end(x.lo, pc.s.kv);
            }
            if (begins && !whole) {
              // the chunks that the unit lies in
              const long long first = pc.pos - pc.off;
              const int last = int(quotient((first + query_cost(pc.u.blocks)) * chunks - 1, total));
              p.open[blockIdx.x] = make_int4(pc.b, pc.h, pc.m, last - int(blockIdx.x) + 1);
            }
          }
          ring_of_pieces[slot] = x;
          mbar_arrive(bar(PIECE + slot));
        }
        __syncwarp();
      }
    }
  } else if (warp >= C::COPY_WARP) {
    set_registers<C::COPY_REGS, false>();
    // ---- copies
    const int pt = tid - C::COPY_WARP * 32;
    // boxes: lane i takes rows from box_r on, 64 elements from box_c on.  A block's take a
    // warp 2,500 clocks, so three take turns.  (No more: see query_turns_hold.)
    const int columns = (p.D + 63) >> 6, box_r = lane / columns * maps.box, box_c = lane % columns * 64;
    const int boxes_all = maps.box > 0 ? BN / maps.box * columns : 0;
    int stage = 0, phase = 1;
    uint32_t blk = 0, turns = 0;
    auto advance = [&]() {
      if (++stage == C::STAGES) stage = 0, phase ^= 1;
    };
    auto together = [&]() {                       // the four warps, with a limit as for every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(GROUP));
      ok = __all_sync(0xffffffffu, mbar_wait(bar(GROUP), turns++ & 1u, &gave_up));
    };
    QueryPiece pc;
    // (a warp that has no block's boxes to bring is there a piece ahead of the others, for as long as theirs takes)
    while (took(pc, mbar_wait_moving(bar(PIECE + taken % kPieceRing), (taken / kPieceRing) & 1u, bar(EMPTY), &gave_up))) {
      int page = -1, pg = 0;
      auto lookup = [&](int t) {
        page = -1;
        if (t >= pc.lo && t < pc.hi) {
          pg = int(fast_div(uint32_t(t), p.fd_page));
          const bool own = C::OWN && (pc.flags & kOwn);
          page = __ldg((own ? p.own_table : p.table) + int64_t(pc.b) * (own ? p.own_t_sb : p.t_sb) + pg);
        }
      };
      // By TMA, boxes present or not (one that is not lies behind the rows and reads as zeros).
      // Where the range of tokens cuts a box, what it holds beyond the range is masked in K, but V
      // there might be no number, and 0 times that is none either: that box of V comes row by row,
      // zeros beyond the range, by the warp whose turn it is (by all four together, which had to
      // meet for it, 32 ragged encoders took 53 us in place of 49; heads of 256, whose boxes are the largest, lose 2%).
      const bool by_box = C::TYPE != kQE4m3 && maps.box > 0;
      if (!by_box) lookup(pc.t0 + pt);
      if constexpr (C::TYPE == kQE4m3) {
        // Through registers, where a tile waits for its stage while the next one is on its
        // way: a tile after the other, each load waited for, was what bound the kernel (chunks of up
        // 1,000 queries, a window of 4,000, e4m3: 197 -> 172 us).
        constexpr int RC = C::DP / 16, RP = 128 / RC, LOADS = BN / RP;   // 16-byte chunks of a row, rows at a time
        const int c = pt % RC, r0 = pt / RC;
        const bool mine = c * 16 < p.D;
        uint4 wk[LOADS], wv[LOADS];
        auto fetch = [&](const void *from, uint32_t b, uint4 *w) {
          if (!mine) return;
          const char *src = static_cast<const char *>(from) + int64_t(pc.h) * p.D + c * 16;
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            const int64_t y = offs[b & 1u][i * RP + r0];
            w[i] = load_or_zero(src + (y >= 0 ? y * p.row : 0), y >= 0);
          }
        };
        auto place = [&](const uint4 *w) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(EMPTY + stage), uint32_t(phase), &gave_up));
          if (!ok) return;
          unsigned char *const dst = ring_p + stage * C::TILE_B + (c >> 2) * C::ATOM_B;
          if (mine) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
              const int r = i * RP + r0, j = 2 * (c & 3);
              *reinterpret_cast<uint4 *>(dst + r * 128 + ((j ^ (r & 7)) << 4)) =
                  make_uint4(q_e4m3(w[i].x), q_e4m3(w[i].x >> 16), q_e4m3(w[i].y), q_e4m3(w[i].y >> 16));
              *reinterpret_cast<uint4 *>(dst + r * 128 + (((j + 1) ^ (r & 7)) << 4)) =
                  make_uint4(q_e4m3(w[i].z), q_e4m3(w[i].z >> 16), q_e4m3(w[i].w), q_e4m3(w[i].w >> 16));
            }
          }
          proxy_fence();
          mbar_arrive(bar(FULL + stage));
          advance();
        };
#pragma unroll 1
        for (int x = 0; ok && x <= pc.n; ++x) {
          if (x < pc.n) {
            const int t0 = pc.t0 + x * BN;
            const bool have = pt < BN && page_present(page, p.num_pages);
            if (pt < BN) offs[blk & 1u][pt] = have ? int64_t(page) * p.P + (t0 + pt - pg * p.P) : -1;
            const uint32_t word = __ballot_sync(0xffffffffu, have);
            if (lane == 0) {
              if (pt < BN) there[blk % INFO][pt >> 5] = word;
              mbar_arrive(bar(KNOWN + blk % INFO));
            }
            // the places of two blocks ago were read before this barrier of the last block
            together();
            if (!ok) break;
            if (x + 1 < pc.n) lookup(t0 + BN + pt);
            fetch(p.k, blk, wk);
          }
          if (x > 0) place(wv);
          if (!ok || x == pc.n) break;
          fetch(p.v, blk, wv);
          place(wk);
          ++blk;
        }
        if (!ok) break;
        continue;
      }
      for (int x = 0; ok && x < pc.n; ++x, ++blk) {
        const int t0 = pc.t0 + x * BN;
        if (by_box) {
          if (blk % uint32_t(kQueryTurns) == uint32_t(pt >> 5)) {
            // the page of the box's first token that is in the range
            const int t = max(t0 + box_r, pc.lo);
            page = -1;
            if (lane < boxes_all && t < t0 + box_r + maps.box) lookup(t);
            const bool have = page_present(page, p.num_pages);
            const int y = have ? int(int64_t(page) * p.P + (t0 + box_r - pg * p.P)) : int(p.num_pages * p.P);
            const uint32_t bits = __ballot_sync(0xffffffffu, have);
            if (lane < WORDS) {                   // tokens lane * 32 on
              const int at = lane * 32 / maps.box * columns;
              uint32_t word = (bits >> at) & 1u ? ~0u : 0u;
              if (maps.box == 16) word = (word & 0xffffu) | ((bits >> (at + columns)) & 1u ? 0xffff0000u : 0u);
              there[blk % INFO][lane] = word;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(KNOWN + blk % INFO), 4);
            const uint32_t cut = __ballot_sync(0xffffffffu, have && (t0 + box_r < pc.lo || t0 + box_r + maps.box > pc.hi));
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(EMPTY + stage), uint32_t(phase), &gave_up));
              if (!ok) break;
              uint32_t rows = kv ? cut : 0u;      // boxes that come row by row
              const uint32_t full = bar(FULL + stage), at = ring_s + stage * C::TILE_B;
              if (lane == 0) mbar_expect(full, uint32_t(boxes_all - __popc(rows)) * uint32_t(maps.box) * 128u);
              if (lane == 1 && !rows) mbar_arrive(full, 127);
              __syncwarp();
              if (lane < boxes_all && !(rows >> lane & 1u))
                tma_box(at + (box_c >> 6) * C::ATOM_B + box_r * 128, kv ? &maps.v : &maps.k, pc.h * p.D + box_c, y, full);
              if (rows) {
                copy_cut_boxes(rows, static_cast<const char *>(p.v) + int64_t(pc.h) * p.D * 2, p.row * 2, y, box_r, box_c, maps.box,
                               p.D, at, C::ATOM_B, pc.lo - t0, pc.hi - t0);
                mbar_arrive(full, lane == 0 ? 3 : 4);
              }
              advance();
            }
          } else {
            advance();
            advance();
          }
          if (!ok) break;
          continue;
        }
        const bool have = pt < BN && page_present(page, p.num_pages);
        int64_t *const at = offs[blk & 1u];
        if (pt < BN) at[pt] = have ? int64_t(page) * p.P + (t0 + pt - pg * p.P) : -1;
        const uint32_t word = __ballot_sync(0xffffffffu, have);
        if (lane == 0) {
          if (pt < BN) there[blk % INFO][pt >> 5] = word;
          mbar_arrive(bar(KNOWN + blk % INFO));
        }
        together();
        if (x + 1 < pc.n) lookup(t0 + BN + pt);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(EMPTY + stage), uint32_t(phase), &gave_up));
          if (!ok) break;
          const char *src = static_cast<const char *>(kv ? p.v : p.k) + int64_t(pc.h) * p.D * C::ES;
          if constexpr (C::TYPE != kQE4m3) {
            const int c = pt & 7, r0 = pt >> 3;   // 8 lanes a row of 128 bytes, 16 rows at a time
            const uint32_t dst = ring_s + stage * C::TILE_B + r0 * 128 + ((c ^ (r0 & 7)) << 4);
#pragma unroll
            for (int i = 0; i < BN / 16; ++i) {
              const int64_t y = at[i * 16 + r0], o = y * p.row * 2;
#pragma unroll
              for (int a = 0; a < C::ATOMS; ++a) {
                const int col = a * 64 + c * 8;
                if (col < d16) {
                  const bool in = y >= 0 && col < p.D;
                  cp_async16(dst + a * C::ATOM_B + i * 2048, src + (in ? o + col * 2 : 0), in ? 16 : 0);
                }
              }
            }
            mbar_arrive_copies(bar(FULL + stage));
          }
          advance();
        }
      }
      if (!ok) break;
    }
    if constexpr (C::TYPE != kQE4m3) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      // after a wait that ran out, boxes may be on their way still: the last of each stage
#pragma unroll 1
      for (int i = 0; !ok && i < C::STAGES; ++i) {
        mbar_wait<true>(bar(FULL + stage), uint32_t(phase), &gave_up);
        advance();
      }
    }
  } else {
    set_registers<C::SOFT_REGS, true>();
    // ---- softmax: a thread per row
    const int tile = warp >> 2, r = tid & 127, w0 = (warp & 3) * 32;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t o_at = tmem + C::O_COL + tile * C::DP + lanes;
    uint32_t used0 = 0, used1 = 0, blk = 0;       // uses of this set's lane (of one set: of both); blocks before the piece
    uint32_t shares = 0;                          // pieces whose blocks the sets shared
    int row = 0;
    QueryPiece pc{};
    bool more = false, live = false;
    // where this thread's row lies in out and in lse, or in out32 and lse2: in local memory,
    // since the blocks need every register
    volatile int64_t places[2] = {0, 0};
    int lo = 0, hi = 0;                           // the tokens it sees
    uint32_t asked = 0;                           // tiles of Q by TMA
    // The next piece's row, and its Q into shared memory (the products that read the one
    // before it are done: their scores were there).  Returns the scores' factor.
    auto begin = [&]() {
      const bool two = pc.flags & kTwoTiles;
      row = two ? tile * kQueryRows + r : r;
      live = more && row < pc.rows;
      float mul = 0.f;
      int64_t q_at = -1;
      lo = 0, hi = INT32_MAX;                     // of no row: nothing to mask, and 0 times its scores
      if (live) {
        const QueryRow x = query_row(p, pc.q0, pc.h, pc.row0 + row);
        q_at = x.token * p.q_st + int64_t(x.head) * p.q_sh;
        if constexpr (C::OWN) {
          places[0] = (int64_t(pc.flags & kOwn ? 1 + pc.t0 / kOwnTokens : 0) * p.N + x.token) * p.Hq + x.head;
        } else {
          places[0] = x.token * p.o_st + int64_t(x.head) * p.o_sh;
          places[1] = x.token * p.lse_st + x.head;
        }
        query_sees(x.i, pc.nq, pc.kv, p.causal, p.window, &lo, &hi);
        mul = p.scale2;
      }
      const bool loads = tile == 0 || two;        // one tile's Q is the first set's to bring
      if (!more || !(loads || (C::TYPE == kQE4m3 && p.bf16))) return mul;
      if (loads && maps.q_boxes > 0) {
        if (r == 0) {
          mbar_expect(bar(QFULL + tile), uint32_t(maps.q_boxes) * C::QATOM_B);
          const int token = pc.q0 + (pc.row0 + tile * kQueryRows) / p.G;   // a whole number of queries
          for (int a = 0; a < maps.q_boxes; ++a)
            tma_box4(q_s + tile * C::QTILE_B + a * C::QATOM_B, &maps.q, a * 64, 0, pc.h, token, bar(QFULL + tile));
        }
        ++asked;
        __syncwarp();
        return mul;
      }
      // row by row, LPR lanes each: every lane knows where its own lies, and the others ask it
      constexpr int LPR = C::DP / 8, RPI = 32 / LPR, QI = 32 / RPI;
      const int qc = lane % LPR, qr = lane / LPR;
#pragma unroll 4
      for (int i = 0; i < QI; ++i) {
        const int rr = i * RPI + qr;
        const int64_t at = __shfl_sync(0xffffffffu, (long long)q_at, rr);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (at >= 0 && qc * 8 < p.D) w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(p.q) + 2 * at + qc * 16));
        if (C::TYPE == kQE4m3 && p.bf16) {
          // fp16, after the power of two that brings the row's largest element into [1, 2):
          // queries keep every bit down to 2^-14 of it, and below that are off by 2^-25 of
          // it at most
          float top = 0.f;
          uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = q_unpack2(y[k], true);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int ex = top < INFINITY ? max(-120, min(120, (__float_as_int(top) >> 23) - 127)) : 0;
          const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = q_unpack2(y[k], true);
            y[k] = pack2<false>(f.x * down, f.y * down);
          }
          w = make_uint4(y[0], y[1], y[2], y[3]);
          const int mine = __shfl_sync(0xffffffffu, ex, lane % RPI * LPR);
          if (i == lane / RPI) mul *= __int_as_float((127 + mine) << 23);
        }
        if (loads && qc * 8 < d16)
          *reinterpret_cast<uint4 *>(q_p + tile * C::QTILE_B + (qc >> 3) * C::QATOM_B + (w0 + rr) * 128 + (((qc & 7) ^ (rr & 7)) << 4)) = w;
      }
      if (!loads) return mul;                     // it needed the rows' factors alone
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(QFULL + tile));
      return mul;
    };
    // One pass per piece, the first for the first piece's Q alone: the code is here once.
    bool any = false, dual = false, begins = false, whole = false;
    int n = 0, t_first = 0;
    float mul = 0.f, m = 0.f, l = 0.f;
    for (;;) {
      // this set's blocks: j0, j0 + each, ...; of one tile with two sets every other
      const bool shared = C::QT == 2 && !dual;
      const int j0 = shared ? tile : 0, each = shared ? 2 : 1;
      // the lane of block j, and how often it was used before
      auto way = [&](int j) { return C::QT == 2 ? tile : j & 1; };
      auto turn = [&](int j) {
        return C::QT == 2 ? used0 + uint32_t(shared ? j >> 1 : j) : ((j & 1) ? used1 : used0) + (uint32_t(j) >> 1);
      };
      m = live ? -INFINITY : 0.f, l = 0.f;
      float mu = live ? 0.f : 1000.f;             // (no row: exponentials of 0)
      bool unset = true;                          // a row of the warp has no reference yet
#pragma unroll 1
      for (int j = j0; j < n; j += each) {
        const uint32_t info = (blk + uint32_t(j)) % INFO;
        bool mask = false;
        const int t0 = t_first + j * BN;
        if (any) {                                // what this row does not see
          ok = __all_sync(0xffffffffu, mbar_wait(bar(KNOWN + info), ((blk + uint32_t(j)) / INFO) & 1u, &gave_up));
          mask = lo > t0 || hi < t0 + BN;
#pragma unroll
          for (int w = 0; w < WORDS; ++w) {
            mask |= there[info][w] != ~0u;
          }
          mask = __any_sync(0xffffffffu, mask);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(SFULL + way(j)), turn(j) & 1u, &gave_up));
        if (!ok) break;
        if (!any) {
          if (lane < PARTS) mbar_arrive(bar(PFULL + 2 * lane + way(j)));
          continue;
        }
        tc_fence_after();
        const uint32_t s_at = tmem + way(j) * BN + lanes;
        // 64 tokens at a time, whose product with V starts while the next ones are taken.  No
        // maximum is looked for in the usual 64: an exponential above 2^RAISE shows in their sum,
        // and only then (or while a row has no reference) the scores are gone through again,
        // a reference put kAbove from the maximum, and the exponentials taken anew.
        float e_all[C::AT_ONCE * 64];             // scores less the reference, in log2
#pragma unroll C::AT_ONCE
        for (int part = 0; part < PARTS; ++part) {
          float *const e = e_all + part % C::AT_ONCE * 64;
          if (part % C::AT_ONCE == 0) {
#pragma unroll
            for (int w = 0; w < 2 * C::AT_ONCE; ++w) tc_ld32(s_at + 64 * part + 32 * w, e_all + 32 * w);
#pragma unroll
            for (int w = 0; w < 2 * C::AT_ONCE; ++w) tc_loaded32(e_all + 32 * w);
          }
          const uint64_t times = f32x2(mul, mul), less = f32x2(-mu, -mu);
#pragma unroll
          for (int i = 0; i < 64; i += 2) unpack(fma2(f32x2(e[i], e[i + 1]), times, less), e + i);
          if (__builtin_expect(mask, 0)) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int a = min(32, max(0, lo - t0 - 64 * part - 32 * w)), z = min(32, max(0, hi - t0 - 64 * part - 32 * w));
              const uint32_t in = there[info][2 * part + w] & uint32_t((uint64_t(1) << z) - 1u) & ~uint32_t((uint64_t(1) << a) - 1u);
#pragma unroll
              for (int i = 0; i < 32; ++i) e[32 * w + i] = (in >> i) & 1u ? e[32 * w + i] : -INFINITY;
            }
          }
          float all;
          for (bool again = unset;;) {
            if (__builtin_expect(again, 0)) {
              float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int i = 0; i < 64; i += 2) top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], e[i], e[i + 1]);
              const float now = fmaxf(m, fmaxf(max3(top[0], top[1], top[2]), top[3]) + mu - C::ABOVE);
              const float f = m == -INFINITY ? 0.f : exp2_fast(m - now), use = now == -INFINITY ? 0.f : now, by = mu - use;
              m = now;
              mu = use;
              l *= f;
#pragma unroll
              for (int i = 0; i < 64; ++i) e[i] += by;
              unset = __any_sync(0xffffffffu, m == -INFINITY);
              if (j > j0 || part > 0) {           // O, once the product with V before this is done
                const int last = part > 0 ? j : j - each;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(PVDONE + (part > 0 ? 0 : 2 * PARTS - 2) + way(last)), turn(last) & 1u, &gave_up));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < d16; c += 16) {
                  float o[16];
                  tc_ld16(o_at + c, o);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= f;
                  tc_st16(o_at + c, o);
                }
              }
            }
            // P, rounded to the products' type as in decode attention, since the tensor cores take 16-bit
            // operands of one type (outputs in bf16 are 0.0024 off in place of 0.0017, in fp16 0.0003
            // in place of 0.0002); the sums keep all bits.  P of word w takes half of the place of the
            // scores of word w / 2
            uint64_t sum[2] = {0, 0};             // two pairs of sums
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float a = exp2_fast(e[32 * w + 2 * i]), z = exp2_fast(e[32 * w + 2 * i + 1]);
                sum[i & 1] = add2(sum[i & 1], f32x2(a, z));
                pk[i] = pack2<C::BF16>(a, z);
              }
              tc_st16u(s_at + (2 * part + w) * 16, pk);
            }
            float x[2];
            unpack(add2(sum[0], sum[1]), x);
            all = x[0] + x[1];
            if (again) break;
            again = __any_sync(0xffffffffu, all > C::LIMIT);
            if (__builtin_expect(!again, 1)) break;
          }
          if (!ok) break;
          l += all;
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PFULL + 2 * part + way(j)));
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- the piece's end; the next one's first products run meanwhile
      const int mine = (n - j0 + each - 1) / each, j1 = j0 + (mine - 1) * each;   // blocks, the last one
      const int last_way = way(j1);
      const uint32_t last_turn = turn(j1);
      used0 += uint32_t(C::QT == 2 ? mine : (n + 1) >> 1);
      used1 += uint32_t(dual ? n : n >> 1);       // of the second lane, whoever's
      blk += uint32_t(n);
      const bool was_live = live, was_any = any;
      const int was_row = row;
      const int64_t was_out = places[0], was_lse = places[C::OWN ? 0 : 1];
      float take0 = 1.f, take1 = 0.f;             // of O, of the other set's
      // The next piece begins, its Q on its way, before the wait for the last product; but the
      // second set of a unit with one tile leaves its sums where its next Q would come.  (A
      // loop of two turns, so that the code is here once.)
      const bool early = !(shared && tile == 1);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        if ((k == 0) == early) {
          // of one tile, Q is still read for the other set's last block
          if (shared && n > 1 && !(n & 1) && tile == 0)
            ok = __all_sync(0xffffffffu, mbar_wait(bar(SFULL + 1), (used1 - 1u) & 1u, &gave_up));
          if (!ok) break;
          more = take(pc);
          mul = begin();
        }
        if (!ok) break;
        if (k == 1) continue;
        if (mine > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(PVDONE + 2 * PARTS - 2 + last_way), last_turn & 1u, &gave_up));
        tc_fence_after();
        if (!(ok && shared && n > 0)) continue;
        float2 *const other = reinterpret_cast<float2 *>(q_p + C::QTILE_B) + r;   // in the place of a second tile's Q
        if (tile == 1) {
          *other = make_float2(m, l);
          proxy_fence();                          // before the next piece's Q comes there by TMA
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(OTHER));
          ok = __all_sync(0xffffffffu, mbar_wait(bar(ADDED), shares & 1u, &gave_up));
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(OTHER), shares & 1u, &gave_up));
          tc_fence_after();
          if (n > 1) {
            const float2 x = *other;
            const float now = fmaxf(m, x.x), base = now == -INFINITY ? 0.f : now;
            take0 = exp2_fast(m - base);
            take1 = exp2_fast(x.x - base);
            l = l * take0 + x.y * take1;
            m = now;
          }
        }
        ++shares;
      }
      if (!ok) break;
      if (was_any && !(shared && tile == 1)) {
        // a row that saw nothing is 0, whatever 0 times V was
        const bool none = whole && __any_sync(0xffffffffu, was_live && l == 0.f);
        const float f = whole ? (l == 0.f ? 0.f : p.v_scale / l) : 1.f;
        const uint64_t f2 = f32x2(f * take0, f * take0), g2 = f32x2(f * take1, f * take1);
        const bool both = shared && n > 1;
        float *part = p.parts + (int64_t(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE + tile * C::DP * kQueryRows + r;
        char *const line = C::OWN ? reinterpret_cast<char *>(p.out32 + was_out * p.D) : static_cast<char *>(p.out) + 2 * was_out;
#pragma unroll 1
        for (int c = 0; c < d16; c += 32) {
          float o[32];
          __syncwarp();
          tc_ld32(o_at + c, o);
          tc_loaded32(o);
#pragma unroll
          for (int i = 0; i < 32; i += 2) unpack(mul2(f32x2(o[i], o[i + 1]), f2), o + i);
          if (both) {
            float z[32];
            tc_ld32(o_at + C::DP + c, z);
            tc_loaded32(z);
#pragma unroll
            for (int i = 0; i < 32; i += 2) unpack(fma2(f32x2(z[i], z[i + 1]), g2, f32x2(o[i], o[i + 1])), o + i);
          }
          if (__builtin_expect(none, 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i];
          }
          if (!was_live) continue;
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(part + i * kQueryRows, o[i]);
            part += 32 * kQueryRows;
          } else if (C::OWN) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (c + i < p.D) *reinterpret_cast<float4 *>(line + 4 * (c + i)) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (c + i < p.D) *reinterpret_cast<uint4 *>(line + 2 * (c + i)) = query_pack8<C>(p, o + i);
          }
        }
        tc_fence_before();
        if (was_live && whole) {
          const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
          if (C::OWN) p.lse2[was_lse] = lse2;
          else if (p.lse) p.lse[was_lse] = lse2 * kLn2;
        } else if (was_live) {
          float *const ml = p.parts + (int64_t(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE + C::ROWS * C::DP + was_row;
          __stcg(ml, m);
          __stcg(ml + C::ROWS, l);
        }
      }
      if (shared && tile == 0 && n > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ADDED));
      }
      if (!more) break;
      dual = pc.flags & kTwoTiles;
      begins = pc.flags & kBegins;
      whole = pc.flags & kWhole;
      n = pc.n;
      t_first = pc.t0;
      any = __any_sync(0xffffffffu, live);        // of a warp without rows, nothing is looked at
    }
    // after a wait that ran out, a tile of Q may be on its way still
    if (!ok && asked > 0 && r == 0) mbar_wait<true>(bar(QFULL + tile), (asked - 1u) & 1u, &gave_up);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == C::MMA_WARP) {
    // nothing is in flight when the tensor memory is given back, after a wait that ran
    // out neither: the products that were issued end by themselves
    mbar_wait<true>(bar(LAST), 0, &gave_up);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
    // every role has passed its waits, and this was the last one
    const int which = *static_cast<volatile int *>(&gave_up);
    if (lane == 0 && which) *p.error = 1u + ((uint32_t(which) - bar0) >> 3) + (blockIdx.x << 8);
  }
}

// Adds the pieces of the units that several chunks share: a block per chunk in which
// such a unit may begin, tile of rows and 8 elements; a thread per row.
template <int DP, int QT>
__global__ void __launch_bounds__(kQueryRows) query_join_kernel(const __grid_constant__ QueryParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int ROWS = QT * kQueryRows, PIECE = ROWS * DP + 2 * ROWS, BN = DP <= 128 ? 128 : 64;
  const int chunk = int(blockIdx.x), col = int(blockIdx.y) * 8;
  if (chunk == 0 && col == 0 && blockIdx.z == 0 && threadIdx.x == 0) p.next[0] = p.next[1] = 0ull;   // ready for the next call
  if (col >= p.D) return;
  const int4 at = __ldcg(p.open + chunk);
  if (!query_open(chunk, at.w, int(gridDim.x)) || at.x < 0 || at.x >= p.B || at.y < 0 || at.y >= p.Hkv || at.z < 0) return;
  const QuerySeq s = query_seq(p, at.x);
  if (at.z >= query_units(s.nq, p.G, ROWS)) return;
  const QueryUnit u = query_unit(at.z, s.nq, s.kv, p.fd_group, ROWS, BN, p.causal, p.window);
  const int row = int(blockIdx.z) * kQueryRows + int(threadIdx.x);
  if (row >= u.rows) return;
  auto slot = [&](int x) { return p.parts + (int64_t(chunk + x) * 2 + (x == 0 ? 1 : 0)) * PIECE; };
  float m = -INFINITY, sum = 0.f, acc[8] = {};
  constexpr int AT_ONCE = 4;
  for (int x0 = 0; x0 < at.w; x0 += AT_ONCE) {
    float v[AT_ONCE][8], mx[AT_ONCE], lx[AT_ONCE];
#pragma unroll
    for (int x = 0; x < AT_ONCE; ++x) {
      mx[x] = -INFINITY;
      if (x0 + x >= at.w) continue;
      const float *d = slot(x0 + x);
      mx[x] = __ldcg(d + ROWS * DP + row);
      lx[x] = __ldcg(d + ROWS * DP + ROWS + row);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[x][i] = __ldcg(d + (int(blockIdx.z) * DP + col + i) * kQueryRows + int(threadIdx.x));
    }
#pragma unroll
    for (int x = 0; x < AT_ONCE; ++x) {
      if (mx[x] == -INFINITY) {                   // nothing seen there (or only NaN, which its sum then is)
        if (x0 + x < at.w && lx[x] != lx[x]) sum = lx[x];
        continue;
      }
      const float now = fmaxf(m, mx[x]);
      const float was = m == -INFINITY ? 0.f : exp2_fast(m - now), f = exp2_fast(mx[x] - now);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = acc[i] * was + f * v[x][i];
      sum = sum * was + f * lx[x];
      m = now;
    }
  }
  const float f = sum == 0.f ? 0.f : p.v_scale / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = sum == 0.f ? 0.f : acc[i] * f;
  const QueryRow out = query_row(p, s.q0, at.y, u.row0 + row);
  query_store8(p, out, col, acc);
  if (col == 0) query_lse(p, out, m, sum);
}

// Joins the prefix's part of a row with those of its own tokens; a thread for 4 elements.
constexpr int kEndThreads = 256;
template <bool BF16>
__global__ void __launch_bounds__(kEndThreads) prefix_end_kernel(const __grid_constant__ QueryParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t at = int64_t(blockIdx.x) * kEndThreads + threadIdx.x, vecs = p.D / 4;
  const int64_t rows = int64_t(p.N) * p.Hq, row = at / vecs;
  if (row >= rows) return;
  const int col = int(at - row * vecs) * 4, b = int(row / p.Hq), h = int(row - int64_t(b) * p.Hq);
  const int kv = int(min(int64_t(max(0, __ldg(p.own_lens + b))), int64_t(p.own_pages) * p.P));
  const int parts = own_parts(kv);
  // weights over a power of two (exactly): the sum of as many parts near the largest bf16 would leave
  // 32 bits, though their mean does not
  const float unit = __int_as_float((127 - (32 - __clz(parts))) << 23);
  float m = __ldcg(p.lse2 + row), sum = m == -INFINITY ? 0.f : unit;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (m != -INFINITY) acc = __ldcg(reinterpret_cast<const float4 *>(p.out32 + row * p.D + col));
  acc = make_float4(acc.x * unit, acc.y * unit, acc.z * unit, acc.w * unit);
  for (int i = 0; i < parts; ++i) {
    const int64_t x = int64_t(1 + i) * rows + row;
    const float z = __ldcg(p.lse2 + x);
    if (z == -INFINITY) continue;
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.out32 + x * p.D + col));
    const float now = fmaxf(m, z), was = m == -INFINITY ? 0.f : exp2_fast(m - now), f = unit * exp2_fast(z - now);
    acc = make_float4(acc.x * was + f * v.x, acc.y * was + f * v.y, acc.z * was + f * v.z, acc.w * was + f * v.w);
    sum = sum * was + f;
    m = now;
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2 *>(static_cast<char *>(p.out) + 2 * (b * p.o_st + h * p.o_sh + col)) =
      make_uint2(pack2<BF16>(acc.x * f, acc.y * f), pack2<BF16>(acc.z * f, acc.w * f));
  if (p.lse && col == 0) p.lse[b * p.lse_st + h] = sum == 0.f ? -INFINITY : (m + log2f(sum / unit)) * kLn2;
}

template <class... A, class... B>
int query_launch(void (*kernel)(A...), dim3 grid, unsigned threads, cudaStream_t st, size_t smem, const B &...args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
  return int(e != cudaSuccess ? e : cudaGetLastError());
}

// The driver's call that describes a tensor to TMA, or null.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_call() {
  static const PFN_cuTensorMapEncodeTiled_v12000 call = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r);
    if (e != cudaSuccess || r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return call;
}

// Describes q and the layer's buffers to TMA where its boxes fit: pages of whole boxes of 16 rows
// or more (32 ragged encoders on pages of 16: 50 us, 70 row by row; 64 sequences on a prefix
// of 32,768: 91, 100; with fewer rows a block would take more requests than a warp has lanes), heads that the products'
// steps of 16 cover (what a box holds behind the head is not used), rows within a
// coordinate.  Else, or where the driver will not, the copies go row by row.
inline void query_maps(const QueryParams &p, int block, bool cache, QueryMaps *m) {
  const CUtensorMapDataType type = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const PFN_cuTensorMapEncodeTiled_v12000 call = tensor_map_call();
  m->box = m->q_boxes = 0;
  if (!call) return;
  // Q: groups that fill a tile's rows, queries that the products take as they are.  (A
  // dimension of one has a stride that nothing uses.)
  if (kQueryRows % p.G == 0 && !(p.e4m3 && p.bf16)) {
    const int64_t sh = p.Hq > 1 ? p.q_sh : p.D, st = p.N > 1 ? p.q_st : int64_t(p.Hq) * sh;
    const cuuint64_t dims[4] = {cuuint64_t(p.D), cuuint64_t(p.G), cuuint64_t(p.Hkv), cuuint64_t(p.N)};
    const cuuint64_t strides[3] = {cuuint64_t(sh) * 2, cuuint64_t(sh) * 2 * p.G, cuuint64_t(st) * 2};
    const cuuint32_t sizes[4] = {64, cuuint32_t(p.G), 1, cuuint32_t(kQueryRows / p.G)}, steps[4] = {1, 1, 1, 1};
    if (sh > 0 && st > 0 &&
        call(&m->q, type, 4, const_cast<void *>(p.q), dims, strides, sizes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
      m->q_boxes = (p.D + 63) / 64;
  }
  if (!cache) return;
  int box = 1;
  while (box < 64 && p.P % (2 * box) == 0) box *= 2;
  const int64_t rows = p.num_pages * p.P;
  if (box < 16 || p.D % 16 || rows >= INT32_MAX) return;
  const cuuint64_t dims[2] = {cuuint64_t(p.row), cuuint64_t(rows)}, strides[1] = {cuuint64_t(p.row) * 2};
  const cuuint32_t sizes[2] = {64, cuuint32_t(box < block ? box : block)}, steps[2] = {1, 1};
  for (int i = 0; i < 2; ++i)
    if (call(i ? &m->v : &m->k, type, 2, const_cast<void *>(i ? p.v : p.k), dims, strides, sizes, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return;
  m->box = int(sizes[1]);
}

constexpr int kQueryDevices = 64;

// The kernel (its shared memory is raised once per device, on first use) and the join.
template <class C>
int launch_query_as(const QueryParams &p, int device, cudaStream_t st, int *launches) {
  static std::atomic<bool> ready[kQueryDevices];
  if (device >= kQueryDevices || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(query_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return int(e);
    if (device < kQueryDevices) ready[device].store(true, std::memory_order_release);
  }
  QueryMaps maps{};
  query_maps(p, C::BN, C::TYPE != kQE4m3, &maps);
  int e = query_launch(query_kernel<C>, dim3(kQueryCtas), C::THREADS, st, C::SMEM, p, maps);
  if (e) return e;
  ++*launches;
  e = query_launch(query_join_kernel<C::DP, C::QT>, dim3(kQueryCtas, C::DP / 8, C::QT), kQueryRows, st, 0, p);
  *launches += e == 0;
  return e;
}

}  // namespace
}  // namespace hicache
