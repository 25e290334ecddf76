// hicache_serving.h -- kernel parameters shared by the operators on the device
// pages (hicache_append.cu, hicache_decode.cu, hicache_query.cu, hicache_merge.cu,
// hicache_evict.cu) and their argument checks (hicache_serving.cpp).  Not part of
// the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <vector_types.h>

#include "hicache_internal.h"

namespace hicache {

struct AppendParams {
  const void *q, *k, *v;
  void *q_out;
  const void *q_weight, *k_weight;
  const int64_t *slots, *positions;
  const float *cos_sin;
  void *k_cache, *v_cache;    // the layer's buffers
  int64_t q_st, q_sh, o_st, o_sh, k_st, k_sh, v_st, v_sh;   // token and head strides
  int64_t num_tokens, cos_sin_rows, num_slots;
  int64_t row;                // elements of a cache row
  int32_t q_heads, kv_heads, D;
  int32_t q_norm, k_norm, rot, rot_off;
  int32_t interleaved, has_v;
  int32_t bf16, e4m3;
  float eps, k_scale, v_scale;
};
int launch_append(const AppendParams &p, void *stream);

struct DecodeParams {
  const void *q, *k, *v;      // k, v: the layer's buffers (v == k for a latent)
  void *out;
  const int32_t *table, *lens;
  float *lse;                 // natural logarithm, or null
  float *weights;             // or null
  int64_t q_sb, q_sh, o_sb, o_sh, t_sb, lse_sb, w_sb;
  int64_t row;                // elements of a cache row
  int64_t num_pages;          // device pages
  int32_t QB;                 // units of a kv head: its G query heads by decode_rows(G)
  // workspace
  unsigned int *counters;     // kDecodeCtas, zero between calls; then the error word
  int2 *seq_pieces;           // latent: per sequence, the group it begins in and its pieces
  float *cta_parts, *warp_parts;
  float *scores;              // [batch, q_heads, score_row] in units of log2, if weights
  float *lse2;                // [batch, q_heads] base-2 logarithm, if weights
  int64_t score_row;
  int32_t B, Hq, Hkv, G, D, Dv, P, max_pages, window;
  int32_t bf16, e4m3, latent;
  FastDiv fd_page;            // tokens per page
  float scale2;               // scale * k_scale * log2(e)
  float v_scale, decay;
};
// Query heads of a unit of work (the rows of a product), and the CTAs of a
// launch: one on each of a GB300's 152 SMs.
HC_HD int decode_rows(int group) { return group <= 8 ? 8 : 16; }
constexpr int kDecodeCtas = 152;
// The heads (columns of a product) of a CTA over a latent cache.
HC_HD int latent_rows(int q_heads) { return q_heads <= 16 ? 16 : q_heads <= 32 ? 32 : 64; }
// The workspace of a call: byte offsets of its parts (from the sizes in p).
struct DecodeSpace {
  int64_t cta_parts, warp_parts, seq_pieces, lse2, scores, bytes;
  int64_t score_row;
};
DecodeSpace decode_space(const DecodeParams &p, bool weights);
int launch_decode(const DecodeParams &p, int device, void *stream, int *launches);
int launch_decode_latent(const DecodeParams &p, int device, void *stream, int *launches);

// A sum over sequences of their strips of work, in which a sequence without any
// counts kIdleSeq: unsigned, so that 65,535 of them and 2^48 - 1 strips fit.
constexpr uint64_t kIdleSeq = uint64_t(1) << 48;
HC_HD uint64_t idle_seqs(uint64_t sum) { return sum / kIdleSeq; }
HC_HD int64_t strips_in(uint64_t sum) { return int64_t(sum % kIdleSeq); }

// Whether a latent sequence's pieces are those of several of the call's groups of
// CTAs, QB CTAs each: `first` the one it begins in, `count` of them.  A call that gave
// up leaves the words of sequences it did not reach as another shape's call left them.
HC_HD bool pieces_to_join(int32_t first, int32_t count, int32_t QB) {
  const int32_t groups = kDecodeCtas / QB;
  return count >= 2 && first >= 0 && first < groups && count <= groups - first;
}

// Whether a page table's entry is a page of the cache (else it counts as absent).
HC_HD bool page_present(int32_t page, int64_t num_pages) { return page >= 0 && page < num_pages; }

// ---- many queries: hicache_query_attention, hicache_prefix_attention ----------------

struct QueryParams {
  const void *q, *k, *v;      // k, v: the layer's buffers
  void *out;
  const int32_t *starts, *table, *lens;
  float *lse;                 // natural logarithm, or null
  // Calls over prefixes: the sequences above are the groups, their queries one of each
  // sequence, which has tokens of its own besides.  Results in 32 bits and their base-2
  // logarithms, to be joined: [0] of the prefix [N, Hq, D], [1 + i] of each kOwnTokens of the
  // sequence's own.
  float *out32, *lse2;        // else null
  const int32_t *own_table, *own_lens;
  int64_t own_t_sb;
  int32_t own_pages;          // max_pages of own_table
  int64_t q_st, q_sh, o_st, o_sh, t_sb, lse_st;
  int64_t row;                // elements of a cache row
  int64_t num_pages;          // device pages
  // workspace
  unsigned int *error;        // set by a call that gave up waiting
  // The next whole unit, the next of the sequences' own; zero between calls.  In 64 bits: own parts
  // of up to 2^19 for each kv head of 65,535 sequences are more units than 32 bits count, and starts
  // that descend let sequences share queries.
  unsigned long long *next;
  int4 *open;                 // per chunk of work: the unit that begins in it and goes on, and in how many chunks it lies
  float *parts;               // two per chunk
  int32_t B, N, Hq, Hkv, G, D, P, max_pages, window, causal;
  int32_t bf16, e4m3;
  FastDiv fd_page, fd_group;  // tokens per page, query heads per kv head
  float scale2;               // scale * k_scale * log2(e)
  float v_scale;
};
// The rows of a product (query tokens times their heads of one kv head), products
// that share a tile of the cache, and tokens of that tile.
constexpr int kQueryRows = 128;
HC_HD int query_tiles(int D) { return D <= 128 ? 2 : 1; }
HC_HD int query_block(int D) { return D <= 128 ? 128 : 64; }
HC_HD int query_cols(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Who may be how far ahead of whom: stages of K or V tiles in shared memory, blocks whose present
// tokens are kept, copying warps that take turns, pieces that are planned ahead.
constexpr int query_stages(int D) { return D <= 64 ? 8 : 5; }   // what fits beside Q (2 x 32 KB + 5 x 32 KB at 128)
constexpr int kQueryInfo = 8;
constexpr int kQueryTurns = 3;
constexpr int kQueryPieces = 4;
// A copying warp waits for the stages of its own blocks only, by a phase's parity, which tells one
// phase from the next but not from the one after that.  At block b it has seen the tile 2 (b - turns) + 1 -
// stages used up, its last one's, and next waits for tile 2 b - stages: tile 2 b - 2 stages, which used
// that stage before it, must be known to be used up by then.
constexpr bool query_turns_hold(int turns, int stages) { return 2 * (-turns) + 1 - stages >= -2 * stages; }
// What it writes of block b must not be read as block b - info's any more.  If the tile it has seen used
// up is K's (an odd number of stages), the products with V two blocks before that are done, if V's, its own.
constexpr bool query_info_holds(int info, int turns, int stages) {
  return info >= turns + (stages % 2 ? (stages - 1) / 2 + 2 : stages / 2);
}
constexpr int kQueryCtas = 152;                   // one on each of a GB300's SMs
// What beginning and ending a unit takes, in blocks: without it CTAs with many short units end
// last (32 ragged encoders 66 us, 50 with 4, 52 with 8; chunks of up to 1,000 queries at e4m3 188,
// 172, 175).
constexpr int kQueryStart = 4;
HC_HD int32_t query_cost(int32_t blocks) { return blocks > 0 ? blocks + kQueryStart : 0; }
// The tokens of a unit over a sequence's own: 16 sequences of 8,000 to 20,000, 32 heads on 8, take
// 198 us with 1,024, 177 with 4,096, 206 with 32,768; 200 of 100 to 6,000 306, 278, 280.
constexpr int kOwnTokens = 4096;
// The parts of so many, and the end of the one that begins at `lo`: no step leaves 32 bits, up to
// the longest table's 2^31 - 1,025 tokens.
HC_HD int32_t own_parts(int32_t tokens) { return tokens / kOwnTokens + (tokens % kOwnTokens != 0); }
HC_HD int32_t own_end(int32_t lo, int32_t tokens) { return tokens - lo < kOwnTokens ? tokens : lo + kOwnTokens; }
// From so many units for each of them on, CTAs take whole units.  8 x 2,048 queries of 32 heads
// on 8 (13 for each): 768 us in chunks, 695 whole; unequal units can lose (16 prompts of 200 to
// 2,000 queries at up to 9,000 tokens, 425 in chunks, 449 whole).  With 2 as the limit 1,500 queries of
// heads of 256 on 6,001 tokens (2.5 for each) would take 255 us in place of 217, chunks at
// e4m3 222 in place of 172.
constexpr int kQueryWhole = 4;
struct QuerySpace {
  int64_t next, open, parts, bytes;
};
QuerySpace query_space(int D);
int launch_query(const QueryParams &p, int device, void *stream, int *launches);
int launch_prefix(const QueryParams &p, int device, void *stream, int *launches);

// A unit of work: rows [row0, row0 + rows) of a sequence's nq * G query rows, over
// blocks [blk0, blk0 + blocks) of the tokens.  Causal: query i of nq sees the tokens up
// to kv - nq + i, the last `window` of them if window > 0.
struct QueryUnit {
  int32_t row0, rows, blk0, blocks;
};
HC_HD int32_t query_units(int32_t nq, int32_t G, int32_t unit_rows) { return (nq * G + unit_rows - 1) / unit_rows; }
// The tokens [lo, hi) that query i sees.
HC_HD void query_sees(int32_t i, int32_t nq, int32_t kv, int32_t causal, int32_t window, int32_t *lo, int32_t *hi) {
  const int32_t end = causal ? kv - nq + i + 1 : kv;
  *hi = end < 0 ? 0 : end;
  *lo = window > 0 && end > window ? end - window : 0;
}
HC_HD QueryUnit query_unit(int32_t m, int32_t nq, int32_t kv, const FastDiv &group, int32_t unit_rows, int32_t block,
                           int32_t causal, int32_t window) {
  QueryUnit u;
  const int32_t all = nq * int32_t(group.d);
  u.row0 = m * unit_rows;
  u.rows = all - u.row0 < unit_rows ? all - u.row0 : unit_rows;
  int32_t lo, hi, unused;
  query_sees(int32_t(fast_div(uint32_t(u.row0), group)), nq, kv, causal, window, &lo, &unused);
  query_sees(int32_t(fast_div(uint32_t(u.row0 + u.rows - 1), group)), nq, kv, causal, window, &unused, &hi);
  u.blk0 = lo / block;
  u.blocks = hi > lo ? (hi + block - 1) / block - u.blk0 : 0;
  return u;
}
// Whether a record of the workspace is a unit of this call to join: its pieces lie in
// chunks of it.
HC_HD bool query_open(int32_t chunk, int32_t pieces, int32_t chunks) {
  return pieces >= 2 && chunk >= 0 && chunk < chunks && pieces <= chunks - chunk;
}

constexpr int kMergeParts = 8;
struct MergeParams {
  const void *outs[kMergeParts];
  const float *lses[kMergeParts];
  int64_t o_st[kMergeParts], o_sh[kMergeParts], l_st[kMergeParts];
  void *out;
  float *lse;
  int64_t out_st, out_sh, lse_st;
  int64_t rows;               // tokens times heads
  int32_t parts, heads, D, bf16;
  FastDiv fd_heads, fd_vecs;
};
int launch_merge(const MergeParams &p, void *stream);

struct EvictParams {
  const int32_t *table;
  const float *weights;
  const int32_t *lens, *keep;
  int32_t *victims, *num_victims, *out_table, *out_lens;
  float *out_weights;
  int64_t t_sb, w_sb, v_sb, ot_sb, ow_sb;
  int32_t P, B, max_pages, max_victims, sink, recent;
};
int launch_evict(const EvictParams &p, int device, void *stream);

// How many of a sequence's n pages leave: those in [sink, n - recent) may.  No step
// leaves 32 bits: none of n, sink and recent is negative, and the second difference is
// taken only where it is positive.
HC_HD int32_t evict_count(int32_t n, int32_t sink, int32_t recent, int32_t keep, int32_t max_victims) {
  const int32_t last = n - recent, may = last > sink ? last - sink : 0, over = n - (keep > 0 ? keep : 0);
  const int32_t most = over < 0 ? 0 : may < over ? may : over;
  return most < max_victims ? most : max_victims;
}

}  // namespace hicache
