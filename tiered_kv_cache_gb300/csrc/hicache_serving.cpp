// hicache_serving.cpp -- argument checks and launches of the operators on the
// device pages: hicache_append_kv, hicache_decode_attention and
// hicache_evict_pages.  The kernels are in hicache_append.cu, hicache_decode.cu
// and hicache_evict.cu.
//
// No call allocates, waits for the GPU or reads device memory.  Like every
// call of the library, each checks its arguments before it enqueues anything.

#include "hicache_serving.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdlib>

#include "hicache.h"
#include "hicache_host.h"

using hicache::Shape;
using hicache::check_desc;
using hicache::clear_error;
using hicache::cuda_error;
using hicache::set_error;

namespace {

bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool positive(float x) { return std::isfinite(x) && x > 0.f; }

// Batch sizes and strides stay below 2^40 elements, so that no offset worked
// out here or in a kernel leaves 64 bits.
constexpr int64_t kMaxStride = int64_t(1) << 40;
bool stride_ok(int64_t s) { return s >= 0 && s < kMaxStride; }
// The stride of a dimension of n: of one element (or none) it is never used, and
// tensors have all kinds there.
int64_t used(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

// The shape and the layer's buffers of an operator on the device pages.
int check_pages(const hicache_device_kv *kv, const hicache_pool_desc *desc, int32_t layer, Shape *s,
                void **k, void **v) {
  int rc = check_desc(desc, s, true);
  if (rc) return rc;
  if (!kv || !kv->buf_ptrs) return set_error(HICACHE_ERR_INVALID_ARG, "device KV is NULL");
  if (kv->device_num_pages < 1 || kv->device_num_pages >= INT32_MAX)
    return set_error(HICACHE_ERR_INVALID_ARG, "device_num_pages = %lld must be in [1, 2^31)",
                     (long long)kv->device_num_pages);
  if (layer < 0 || layer >= s->L)
    return set_error(HICACHE_ERR_INVALID_ARG, "layer_id %d outside [0, %lld)", layer, (long long)s->L);
  if (s->B > 2) return set_error(HICACHE_ERR_INVALID_ARG, "num_buffers must be 2 (K, V) or 1 (latent)");
  if (s->es != 1 && s->es != 2)
    return set_error(HICACHE_ERR_INVALID_ARG, "elem_bytes must be 2 (dtype) or 1 (e4m3), is %lld", (long long)s->es);
  *k = kv->buf_ptrs[layer];
  *v = s->B == 2 ? kv->buf_ptrs[s->L + layer] : *k;
  if (!*k || !*v) return set_error(HICACHE_ERR_INVALID_ARG, "a device buffer of layer %d is NULL", layer);
  if (!aligned(*k, 16) || !aligned(*v, 16))
    return set_error(HICACHE_ERR_ALIGNMENT, "a device buffer of layer %d is not 16-byte aligned", layer);
  return HICACHE_OK;
}

int check_scales(const Shape &s, float k_scale, float v_scale) {
  if (!positive(k_scale) || !positive(v_scale))
    return set_error(HICACHE_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  if (s.es != 1 && (k_scale != 1.f || v_scale != 1.f))
    return set_error(HICACHE_ERR_INVALID_ARG, "k_scale and v_scale belong to 1-byte caches: they must be 1");
  return HICACHE_OK;
}

// A [n, h, d] tensor of 2-byte elements that kernels access by 16-byte vectors.
int check_heads(const char *name, const void *p, int64_t st, int64_t sh) {
  if (!p) return set_error(HICACHE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!stride_ok(st) || !stride_ok(sh))
    return set_error(HICACHE_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
  if (!aligned(p, 16) || st % 8 || sh % 8)
    return set_error(HICACHE_ERR_ALIGNMENT, "%s: address and strides must be multiples of 16 bytes", name);
  return HICACHE_OK;
}

// Whether no two (i, j) of [n, h] rows of d elements share an element.
bool rows_disjoint(int64_t n, int64_t st, int64_t h, int64_t sh, int64_t d) {
  if (n <= 1 && h <= 1) return true;
  if (n <= 1) return sh >= d;
  if (h <= 1) return st >= d;
  if (st >= sh) return sh >= d && st >= (h - 1) * sh + d;      // h <= 2^20, sh < 2^40
  return st >= d && (sh - d) / st >= n - 1;
}

int check_grid(const char *what, int64_t n, int64_t most) {
  if (n < 0 || n > most)
    return set_error(HICACHE_ERR_INVALID_ARG, "%s = %lld must be in [0, %lld]", what, (long long)n, (long long)most);
  return HICACHE_OK;
}

int launched(int e, int n, const char *what) {
  hicache::g_launches.fetch_add(n, std::memory_order_relaxed);
  return e ? cuda_error(cudaError_t(e), what) : HICACHE_OK;
}

// Checks a call's sizes and fills them in.
int decode_sizes(const Shape &s, int64_t batch, int64_t q_heads, int64_t head_dim, int64_t v_dim, int64_t max_pages,
                 hicache::DecodeParams *p) {
  int rc = check_grid("batch", batch, 65535);
  if (rc) return rc;
  if (q_heads < 1 || q_heads > 4096 || head_dim < 1 || v_dim < 1 || max_pages < 1)
    return set_error(HICACHE_ERR_INVALID_ARG,
                     "q_heads (in [1, 4096]), head_dim, v_dim and max_pages must be >= 1 (%lld, %lld, %lld, %lld)",
                     (long long)q_heads, (long long)head_dim, (long long)v_dim, (long long)max_pages);
  if (max_pages * s.P > INT32_MAX - 1024)
    return set_error(HICACHE_ERR_INVALID_ARG, "max_pages * page_size = %lld must be < 2^31 - 1024",
                     (long long)(max_pages * s.P));
  if (s.B == 1) {
    if (s.es != 2 || s.R != 576 || head_dim != 576 || v_dim != 512)
      return set_error(HICACHE_ERR_INVALID_ARG,
                       "a latent cache has rows of 576 elements of 2 bytes, head_dim 576 and v_dim 512 "
                       "(row_elems %lld, elem_bytes %lld, head_dim %lld, v_dim %lld)",
                       (long long)s.R, (long long)s.es, (long long)head_dim, (long long)v_dim);
  } else if (const int64_t unit = 16 / s.es; head_dim > 256 || head_dim % unit || v_dim != head_dim) {
    return set_error(HICACHE_ERR_INVALID_ARG, "head_dim %lld must be a multiple of %lld up to 256, v_dim %lld the same",
                     (long long)head_dim, (long long)unit, (long long)v_dim);
  } else if (s.R % head_dim || q_heads % (s.R / head_dim)) {
    return set_error(HICACHE_ERR_INVALID_ARG,
                     "rows of %lld elements must hold whole heads of %lld, and q_heads %lld be a multiple of their number",
                     (long long)s.R, (long long)head_dim, (long long)q_heads);
  }
  // tiles of 16 tokens per head, counted in 64 bits with room for the number of warps
  if ((max_pages * s.P / 16 + 1) * batch > (int64_t(1) << 48) / q_heads)
    return set_error(HICACHE_ERR_INVALID_ARG, "batch * max_pages * page_size * q_heads must be < 2^52");
  p->B = int32_t(batch);
  p->Hq = int32_t(q_heads);
  p->D = int32_t(head_dim);
  p->Dv = int32_t(v_dim);
  p->row = s.R;
  p->Hkv = int32_t(s.R / head_dim);
  p->G = p->Hq / p->Hkv;
  const int rows = s.B == 1 ? hicache::latent_rows(p->Hq) : hicache::decode_rows(p->G);
  p->QB = (p->G + rows - 1) / rows;
  p->P = int32_t(s.P);
  p->max_pages = int32_t(max_pages);
  p->e4m3 = s.es == 1;
  p->latent = s.B == 1;
  return HICACHE_OK;
}

}  // namespace

extern "C" {

int hicache_append_kv(const hicache_device_kv *kv, const hicache_pool_desc *desc, int32_t layer_id,
                      const hicache_append_desc *a, void *stream) {
  clear_error();
  Shape s{};
  void *k = nullptr, *v = nullptr;
  int rc = check_pages(kv, desc, layer_id, &s, &k, &v);
  if (rc) return rc;
  if (!a) return set_error(HICACHE_ERR_INVALID_ARG, "the append descriptor is NULL");
  if (a->dtype != HICACHE_BF16 && a->dtype != HICACHE_FP16)
    return set_error(HICACHE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if ((rc = check_scales(s, a->k_scale, a->v_scale))) return rc;
  const int64_t D = a->head_dim, N = a->num_tokens;
  if (a->q_heads < 0 || a->kv_heads < 0 || a->q_heads + int64_t(a->kv_heads) < 1)
    return set_error(HICACHE_ERR_INVALID_ARG, "q_heads and kv_heads must be >= 0, and not both 0");
  if (D < 8 || D > 768 || D % 8 || (s.es == 1 && D % 16))
    return set_error(HICACHE_ERR_INVALID_ARG, "head_dim %lld must be a multiple of %d in [8, 768]", (long long)D,
                     s.es == 1 ? 16 : 8);
  const bool has_v = a->kv_heads > 0 && s.B == 2;
  const int64_t units = a->q_heads + int64_t(a->kv_heads) * (has_v ? 2 : 1);
  if (units > (int64_t(1) << 20) || N < 0 || N > ((int64_t(1) << 31) - 4096) / units)
    return set_error(HICACHE_ERR_INVALID_ARG, "num_tokens = %lld times %lld heads must be in [0, 2^31 - 4096]",
                     (long long)N, (long long)units);
  if (a->kv_heads > 0 && (a->kv_heads * D != s.R || (s.B == 1 && a->kv_heads != 1)))
    return set_error(HICACHE_ERR_INVALID_ARG,
                     "kv_heads * head_dim = %lld is not the cache's row of %lld elements (one head in a latent cache)",
                     (long long)(a->kv_heads * D), (long long)s.R);
  for (const int32_t m : {a->q_norm_dim, a->k_norm_dim})
    if (m < 0 || m > D || m % 8)
      return set_error(HICACHE_ERR_INVALID_ARG, "norm dims must be multiples of 8 in [0, head_dim], one is %d", m);
  if (!std::isfinite(a->eps) || a->eps < 0.f) return set_error(HICACHE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (a->rot_dim < 0 || a->rot_dim % 2 || a->rot_offset < 0 || a->rot_offset % 2 ||
      int64_t(a->rot_offset) + a->rot_dim > D)
    return set_error(HICACHE_ERR_INVALID_ARG, "rot_dim %d and rot_offset %d must be even, >= 0 and within head_dim",
                     a->rot_dim, a->rot_offset);
  if (a->rot_dim > 0 && (!a->positions || !a->cos_sin || a->cos_sin_rows < 1 || a->cos_sin_rows >= kMaxStride))
    return set_error(HICACHE_ERR_INVALID_ARG, "a rotation needs positions and cos_sin with at least one row");
  if (a->rot_dim > 0 && (!aligned(a->positions, 8) || !aligned(a->cos_sin, 4)))
    return set_error(HICACHE_ERR_ALIGNMENT, "positions or cos_sin is not aligned to its elements");
  if (N == 0) return HICACHE_OK;
  const int64_t q_st = used(a->q_token_stride, N), q_sh = used(a->q_head_stride, a->q_heads);
  const int64_t o_st = used(a->q_out_token_stride, N), o_sh = used(a->q_out_head_stride, a->q_heads);
  const int64_t k_st = used(a->k_token_stride, N), k_sh = used(a->k_head_stride, a->kv_heads);
  const int64_t v_st = used(a->v_token_stride, N), v_sh = used(a->v_head_stride, a->kv_heads);
  if (a->q_heads > 0) {
    if ((rc = check_heads("q", a->q, q_st, q_sh))) return rc;
    if ((rc = check_heads("q_out", a->q_out, o_st, o_sh))) return rc;
    if (!rows_disjoint(N, o_st, a->q_heads, o_sh, D))
      return set_error(HICACHE_ERR_INVALID_ARG, "q_out: heads overlap one another");
    if (a->q_out == a->q && (o_st != q_st || o_sh != q_sh))
      return set_error(HICACHE_ERR_INVALID_ARG, "q_out is q with other strides");
    if (a->q_norm_dim > 0 && (!a->q_weight || !aligned(a->q_weight, 16)))
      return set_error(a->q_weight ? HICACHE_ERR_ALIGNMENT : HICACHE_ERR_INVALID_ARG,
                       "q_weight is NULL or not 16-byte aligned");
  }
  if (a->kv_heads > 0) {
    if ((rc = check_heads("k", a->k, k_st, k_sh))) return rc;
    if (has_v && (rc = check_heads("v", a->v, v_st, v_sh))) return rc;
    if (!has_v && a->v) return set_error(HICACHE_ERR_INVALID_ARG, "a latent cache takes no v");
    if (!a->slots) return set_error(HICACHE_ERR_INVALID_ARG, "slots is NULL");
    if (!aligned(a->slots, 8)) return set_error(HICACHE_ERR_ALIGNMENT, "slots is not aligned to its elements");
    if (a->k_norm_dim > 0 && (!a->k_weight || !aligned(a->k_weight, 16)))
      return set_error(a->k_weight ? HICACHE_ERR_ALIGNMENT : HICACHE_ERR_INVALID_ARG,
                       "k_weight is NULL or not 16-byte aligned");
  }
  hicache::AppendParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_out = a->q_out;
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.slots = a->slots;
  p.positions = a->positions;
  p.cos_sin = a->cos_sin;
  p.k_cache = k;
  p.v_cache = v;
  p.q_st = q_st;
  p.q_sh = q_sh;
  p.o_st = o_st;
  p.o_sh = o_sh;
  p.k_st = k_st;
  p.k_sh = k_sh;
  p.v_st = v_st;
  p.v_sh = v_sh;
  p.num_tokens = N;
  p.cos_sin_rows = a->cos_sin_rows;
  p.num_slots = kv->device_num_pages * s.P;
  p.row = s.R;
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.D = a->head_dim;
  p.q_norm = a->q_heads > 0 ? a->q_norm_dim : 0;    // the kernels read the weights of a norm
  p.k_norm = a->kv_heads > 0 ? a->k_norm_dim : 0;   // wherever there is one
  p.rot = a->rot_dim;
  p.rot_off = a->rot_offset;
  p.interleaved = a->interleaved != 0;
  p.has_v = has_v;
  p.bf16 = a->dtype == HICACHE_BF16;
  p.e4m3 = s.es == 1;
  p.eps = a->eps;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  const int e = hicache::launch_append(p, stream);
  return launched(e, e == 0, "append kernel launch");
}

int hicache_decode_workspace(const hicache_pool_desc *desc, int32_t batch, int32_t q_heads, int32_t head_dim,
                             int32_t v_dim, int32_t max_pages, int32_t with_weights, int64_t *bytes) {
  clear_error();
  Shape s{};
  int rc = check_desc(desc, &s, true);
  if (rc) return rc;
  if (!bytes) return set_error(HICACHE_ERR_INVALID_ARG, "bytes is NULL");
  hicache::DecodeParams p{};
  if ((rc = decode_sizes(s, batch, q_heads, head_dim, v_dim, max_pages, &p))) return rc;
  *bytes = hicache::decode_space(p, with_weights != 0).bytes;
  return HICACHE_OK;
}

int hicache_decode_attention(const hicache_device_kv *kv, const hicache_pool_desc *desc, int32_t layer_id,
                             const hicache_decode_desc *a, void *stream) {
  clear_error();
  Shape s{};
  void *k = nullptr, *v = nullptr;
  int rc = check_pages(kv, desc, layer_id, &s, &k, &v);
  if (rc) return rc;
  if (!a) return set_error(HICACHE_ERR_INVALID_ARG, "the decode descriptor is NULL");
  if (a->dtype != HICACHE_BF16 && a->dtype != HICACHE_FP16)
    return set_error(HICACHE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->reserved != 0) return set_error(HICACHE_ERR_INVALID_ARG, "reserved must be 0");
  if ((rc = check_scales(s, a->k_scale, a->v_scale))) return rc;
  hicache::DecodeParams p{};
  if ((rc = decode_sizes(s, a->batch, a->q_heads, a->head_dim, a->v_dim, a->max_pages, &p))) return rc;
  if (!std::isfinite(a->scale) || !std::isfinite(a->decay))
    return set_error(HICACHE_ERR_INVALID_ARG, "scale and decay must be finite");
  p.scale2 = float(double(a->scale) * double(a->k_scale) * 1.4426950408889634);
  if (!std::isfinite(p.scale2)) return set_error(HICACHE_ERR_INVALID_ARG, "scale * k_scale leaves 32 bits");
  if (a->window < 0) return set_error(HICACHE_ERR_INVALID_ARG, "window must be >= 0");
  if (a->batch == 0) return HICACHE_OK;
  p.q_sb = used(a->q_batch_stride, a->batch);
  p.q_sh = used(a->q_head_stride, a->q_heads);
  p.o_sb = used(a->out_batch_stride, a->batch);
  p.o_sh = used(a->out_head_stride, a->q_heads);
  p.t_sb = used(a->table_stride, a->batch);
  p.lse_sb = used(a->lse_stride, a->batch);
  p.w_sb = used(a->weights_stride, a->batch);
  if ((rc = check_heads("q", a->q, p.q_sb, p.q_sh))) return rc;
  if ((rc = check_heads("out", a->out, p.o_sb, p.o_sh))) return rc;
  if (!rows_disjoint(a->batch, p.o_sb, a->q_heads, p.o_sh, a->v_dim))
    return set_error(HICACHE_ERR_INVALID_ARG, "out: heads overlap one another");
  if (!a->page_table || !a->seq_lens || !a->workspace)
    return set_error(HICACHE_ERR_INVALID_ARG, "page_table, seq_lens or workspace is NULL");
  if (!stride_ok(p.t_sb)) return set_error(HICACHE_ERR_INVALID_ARG, "table_stride must be in [0, 2^40)");
  if (a->lse && (!stride_ok(p.lse_sb) || !rows_disjoint(a->batch, p.lse_sb, 1, 0, a->q_heads)))
    return set_error(HICACHE_ERR_INVALID_ARG, "lse_stride must be at least q_heads");
  if (a->weights && (!stride_ok(p.w_sb) || !rows_disjoint(a->batch, p.w_sb, 1, 0, a->max_pages)))
    return set_error(HICACHE_ERR_INVALID_ARG, "weights_stride must be at least max_pages");
  if (!aligned(a->page_table, 4) || !aligned(a->seq_lens, 4) || !aligned(a->lse, 4) || !aligned(a->weights, 4))
    return set_error(HICACHE_ERR_ALIGNMENT, "page_table, seq_lens, lse or weights is not aligned to its elements");
  if (!aligned(a->workspace, 256)) return set_error(HICACHE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  const hicache::DecodeSpace sp = hicache::decode_space(p, a->weights != nullptr);
  if (a->workspace_bytes < sp.bytes)
    return set_error(HICACHE_ERR_INVALID_ARG, "workspace of %lld bytes is below the %lld needed",
                     (long long)a->workspace_bytes, (long long)sp.bytes);
  char *ws = static_cast<char *>(a->workspace);
  p.q = a->q;
  p.k = k;
  p.v = v;
  p.out = a->out;
  p.table = a->page_table;
  p.lens = a->seq_lens;
  p.lse = a->lse;
  p.weights = a->weights;
  p.num_pages = kv->device_num_pages;
  p.counters = reinterpret_cast<unsigned int *>(ws);
  p.cta_parts = reinterpret_cast<float *>(ws + sp.cta_parts);
  p.seq_pieces = reinterpret_cast<int2 *>(ws + sp.seq_pieces);
  p.warp_parts = reinterpret_cast<float *>(ws + sp.warp_parts);
  p.lse2 = reinterpret_cast<float *>(ws + sp.lse2);
  p.scores = reinterpret_cast<float *>(ws + sp.scores);
  p.score_row = sp.score_row;
  p.window = a->window;
  p.bf16 = a->dtype == HICACHE_BF16;
  p.fd_page = hicache::make_fastdiv(uint32_t(s.P));
  p.v_scale = a->v_scale;
  p.decay = a->decay;
  int n = 0, device = 0;
  const cudaError_t de = cudaGetDevice(&device);
  if (de != cudaSuccess) return cuda_error(de, "cudaGetDevice");
  const int e = hicache::launch_decode(p, device, stream, &n);
  return launched(e, n, "decode kernel launch");
}

int hicache_decode_status(void *workspace, int32_t *gave_up, int32_t clear) {
  clear_error();
  if (!workspace || !gave_up) return set_error(HICACHE_ERR_INVALID_ARG, "workspace or gave_up is NULL");
  if (!aligned(workspace, 256)) return set_error(HICACHE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  unsigned int *word = static_cast<unsigned int *>(workspace) + hicache::kDecodeCtas, x = 0;
  // a copy on the default stream alone would pass calls on streams that do not block it
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&x, word, sizeof(x), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && clear) e = cudaMemset(word, 0, sizeof(x));
  if (e == cudaSuccess && clear) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_error(e, "decode status");
  *gave_up = x != 0;
  return HICACHE_OK;
}

int hicache_evict_pages(const hicache_evict_desc *a, void *stream) {
  clear_error();
  if (!a) return set_error(HICACHE_ERR_INVALID_ARG, "the evict descriptor is NULL");
  int rc = check_grid("batch", a->batch, (1 << 28) - 1);
  if (rc) return rc;
  if (a->page_size < 1 || a->max_pages < 1 || a->max_victims < 0 || a->sink < 0 || a->recent < 1)
    return set_error(HICACHE_ERR_INVALID_ARG,
                     "page_size %d, max_pages %d and recent %d must be >= 1, max_victims %d and sink %d >= 0",
                     a->page_size, a->max_pages, a->recent, a->max_victims, a->sink);
  if (int64_t(a->max_pages) * a->page_size > INT32_MAX - 1024)
    return set_error(HICACHE_ERR_INVALID_ARG, "max_pages * page_size = %lld must be < 2^31 - 1024",
                     (long long)a->max_pages * a->page_size);
  if (a->batch == 0) return HICACHE_OK;
  if (!a->page_table || !a->weights || !a->seq_lens || !a->keep || !a->num_victims || !a->out_table ||
      !a->out_weights || !a->out_lens || (!a->victims && a->max_victims > 0))
    return set_error(HICACHE_ERR_INVALID_ARG, "an array is NULL");
  for (const void *q : {static_cast<const void *>(a->page_table), static_cast<const void *>(a->weights),
                        static_cast<const void *>(a->seq_lens), static_cast<const void *>(a->keep),
                        static_cast<const void *>(a->victims), static_cast<const void *>(a->num_victims),
                        static_cast<const void *>(a->out_table), static_cast<const void *>(a->out_weights),
                        static_cast<const void *>(a->out_lens)})
    if (!aligned(q, 4)) return set_error(HICACHE_ERR_ALIGNMENT, "an array is not aligned to its elements");
  hicache::EvictParams p{};
  p.t_sb = used(a->table_stride, a->batch);
  p.w_sb = used(a->weights_stride, a->batch);
  p.v_sb = used(a->victims_stride, a->batch);
  p.ot_sb = used(a->out_table_stride, a->batch);
  p.ow_sb = used(a->out_weights_stride, a->batch);
  for (const int64_t t : {p.t_sb, p.w_sb, p.v_sb, p.ot_sb, p.ow_sb})
    if (!stride_ok(t)) return set_error(HICACHE_ERR_INVALID_ARG, "strides must be in [0, 2^40)");
  if (a->batch > 1 && (p.v_sb < a->max_victims || p.ot_sb < a->max_pages || p.ow_sb < a->max_pages))
    return set_error(HICACHE_ERR_INVALID_ARG, "the rows of an output overlap");
  if ((a->out_table == a->page_table && p.ot_sb != p.t_sb) || (a->out_weights == a->weights && p.ow_sb != p.w_sb))
    return set_error(HICACHE_ERR_INVALID_ARG, "an output is its input with another stride");
  p.table = a->page_table;
  p.weights = a->weights;
  p.lens = a->seq_lens;
  p.keep = a->keep;
  p.victims = a->victims;
  p.num_victims = a->num_victims;
  p.out_table = a->out_table;
  p.out_lens = a->out_lens;
  p.out_weights = a->out_weights;
  p.P = a->page_size;
  p.B = a->batch;
  p.max_pages = a->max_pages;
  p.max_victims = a->max_victims;
  p.sink = a->sink;
  p.recent = a->recent;
  int device = 0;
  const cudaError_t de = cudaGetDevice(&device);
  if (de != cudaSuccess) return cuda_error(de, "cudaGetDevice");
  const int e = hicache::launch_evict(p, device, stream);
  return launched(e, e == 0, "evict kernel launch");
}

}  // extern "C"
