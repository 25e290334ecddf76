// hicache_serving.h -- kernel parameters shared by the operators on the device
// pages (hicache_append.cu, hicache_decode.cu, hicache_evict.cu) and their
// argument checks (hicache_serving.cpp).  Not part of the public ABI.
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
