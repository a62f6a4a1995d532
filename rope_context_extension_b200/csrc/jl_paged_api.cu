// C ABI of the paged-cache operators: argument checks, scratch layout,
// tensor-map encoding and kernel launches.  See include/jl_api.h.
#include <algorithm>
#include <cstring>

#include "../../include/jl_api.h"
#include "jl_host.h"
#include "jl_paged.cuh"

namespace {

using jl::aligned16;
using jl::round_up;

constexpr int64_t kMaxLen = int64_t(1) << 30;
constexpr int kMaxBatch = 65535;  // a grid's y dimension

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int shape_checks(int B, int Hq, int Hkv, int D, double rope_base) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return JL_ERR_INVALID_ARG;
  if (!(rope_base > 0.0) || !std::isfinite(rope_base)) return JL_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return JL_ERR_UNSUPPORTED;
  if (B > kMaxBatch || Hkv > kMaxBatch || Hq > (1 << 20) || (int64_t)B * Hkv > (1 << 30)) return JL_ERR_UNSUPPORTED;
  return JL_OK;
}

int rule_checks(int w0, int w_pretrained, int mode) {
  if (w0 < 0 || w_pretrained < 1) return JL_ERR_INVALID_ARG;
  // the prefill flags mean nothing here, as in the other decode calls
  if ((mode & ~(JL_QSHIFT_SELF_EXTEND | JL_PREFILL_FP16 | JL_PREFILL_KEYS_IN_KERNEL)) != 0) return JL_ERR_INVALID_ARG;
  if ((mode & JL_PREFILL_FP16) && (mode & JL_PREFILL_KEYS_IN_KERNEL)) return JL_ERR_INVALID_ARG;
  return JL_OK;
}

int page_size_checks(int page_size, int64_t max_pages) {
  if (page_size < 1 || max_pages < 1) return JL_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || page_size > 1024 || max_pages > kMaxLen / page_size) return JL_ERR_UNSUPPORTED;
  return JL_OK;
}

// A cache whose pages, rows and heads do not overlap.
int cache_checks(const jl_paged_kv* c, int Hkv, int D, int64_t max_pages, bool need_v) {
  if (!c || !c->k || (need_v && !c->v) || c->num_pages < 1) return JL_ERR_INVALID_ARG;
  const int st = page_size_checks(c->page_size, max_pages);
  if (st != JL_OK) return st;
  if (c->num_pages > INT32_MAX) return JL_ERR_UNSUPPORTED;
  const int64_t limit = int64_t(1) << 38;  // elements: a tensor map's strides stay below 2^40 bytes
  if (c->page_stride < 1 || c->row_stride < 1 || c->head_stride < 1) return JL_ERR_INVALID_ARG;
  if (c->page_stride > limit || c->row_stride > limit || c->head_stride > limit) return JL_ERR_UNSUPPORTED;
  if (c->page_stride % 8 || c->row_stride % 8 || c->head_stride % 8) return JL_ERR_ALIGNMENT;
  const int64_t rows = (c->page_size - 1) * c->row_stride, heads = (Hkv - 1) * c->head_stride;
  const bool by_row = c->head_stride >= D && c->row_stride >= heads + D;   // a row holds all heads
  const bool by_head = c->row_stride >= D && c->head_stride >= rows + D;   // a head holds all rows
  if (!by_row && !by_head) return JL_ERR_INVALID_ARG;
  if (c->page_stride < rows + heads + D) return JL_ERR_INVALID_ARG;
  if (!aligned16(c->k) || (need_v && !aligned16(c->v))) return JL_ERR_ALIGNMENT;
  return JL_OK;
}

jl::PagedView view_of(const jl_paged_kv* c) {
  jl::PagedView v;
  v.k = reinterpret_cast<__nv_bfloat16*>(c->k);
  v.v = reinterpret_cast<__nv_bfloat16*>(c->v);
  v.num_pages = c->num_pages;
  v.page_stride = c->page_stride;
  v.row_stride = c->row_stride;
  v.head_stride = c->head_stride;
  v.page_size = c->page_size;
  return v;
}

// 5-D map over (64 dims, page rows, D / 64, Hkv, pages) of the cache's strides with
// a {64, 16, D / 64, 1, 1} box and 128-byte swizzle: 16 rows of one head of one page
// in one copy.
bool encode_pages(CUtensorMap* map, const void* base, const jl_paged_kv* c, int Hkv, int D) {
  auto fn = jl::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[5] = {64, (cuuint64_t)c->page_size, (cuuint64_t)(D / 64), (cuuint64_t)Hkv, (cuuint64_t)c->num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)c->row_stride * 2, 128, (cuuint64_t)c->head_stride * 2,
                           (cuuint64_t)c->page_stride * 2};
  cuuint32_t box[5] = {64, 16, (cuuint32_t)(D / 64), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Args>
void set_turns(Args& a, int D, double rope_base) {
  const jl::TurnTable& t = jl::turn_table(D, rope_base);
  std::memcpy(a.u_hi, t.hi, sizeof(t.hi));
  std::memcpy(a.u_lo, t.lo, sizeof(t.lo));
}

int norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
              const void* q_weight, const void* k_weight, float eps, const int32_t* seq_ids, const int32_t* positions,
              int T, void* q_out, void* k_out, const jl_paged_kv* cache, const int32_t* block_table,
              int64_t max_pages, int B, int Hq, int Hkv, int D, double rope_base, int* dev_error, void* stream) {
  int st = shape_checks(B, Hq, Hkv, D, rope_base);
  if (st != JL_OK) return st;
  if (T < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return JL_ERR_INVALID_ARG;
  if (!q || !k || !positions || !q_out) return JL_ERR_INVALID_ARG;
  const bool append = cache != nullptr;
  if (append) {
    if (!v || !seq_ids || !block_table) return JL_ERR_INVALID_ARG;
    st = cache_checks(cache, Hkv, D, max_pages, true);
    if (st != JL_OK) return st;
  } else if (!k_out) {
    return JL_ERR_INVALID_ARG;
  }
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || (append && v_stride < (int64_t)Hkv * D))
    return JL_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || (append && v_stride % 8)) return JL_ERR_ALIGNMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !aligned4(positions) || (append && (!aligned16(v) || !aligned4(seq_ids) ||
                                                                   !aligned4(block_table))))
    return JL_ERR_ALIGNMENT;
  jl::NormRopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.qw = reinterpret_cast<const __nv_bfloat16*>(q_weight);
  a.kw = reinterpret_cast<const __nv_bfloat16*>(k_weight);
  a.eps = eps;
  a.positions = positions;
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  if (append) {
    a.v = reinterpret_cast<const __nv_bfloat16*>(v);
    a.v_stride = v_stride;
    a.seq_ids = seq_ids;
    a.pages = view_of(cache);
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.B = B;
  }
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dev_error = dev_error;
  std::memcpy(a.turn, jl::turn_table(D, rope_base).fixed, sizeof(a.turn));
  if (jl::launch_norm_rope(a, D, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return JL_ERR_CUDA;
  return JL_OK;
}

struct PagedDecodeLayout {
  size_t counters, cta, warp, total;
};
PagedDecodeLayout paged_decode_layout(int r, int D) {
  const size_t ctas = jl::decode_paged_max_ctas(), part = jl::decode_partial_floats(r, D) * sizeof(float);
  PagedDecodeLayout lay;
  lay.counters = 0;
  lay.cta = round_up(ctas * sizeof(unsigned));
  lay.warp = lay.cta + round_up(ctas * 2 * part);
  lay.total = lay.warp + round_up(ctas * jl::decode_paged_warps() * part);
  return lay;
}

int decode_paged(const void* q, const jl_paged_kv* cache, const int32_t* block_table, int64_t max_pages,
                 const int32_t* seq_lens, bool sparse, const int32_t* page_list, int64_t list_stride,
                 const int32_t* page_counts, void* o, float* lse, int B, int Hq, int Hkv, int D, int w0,
                 int w_pretrained, double rope_base, float softmax_scale, int mode, void* workspace,
                 size_t workspace_bytes, int* dev_error, void* stream) {
  int st = shape_checks(B, Hq, Hkv, D, rope_base);
  if (st != JL_OK) return st;
  st = rule_checks(w0, w_pretrained, mode);
  if (st != JL_OK) return st;
  if (!std::isfinite(softmax_scale)) return JL_ERR_INVALID_ARG;
  if (!q || !o || !block_table || !seq_lens) return JL_ERR_INVALID_ARG;
  if (sparse && (!page_list || !page_counts || list_stride < 1)) return JL_ERR_INVALID_ARG;
  st = cache_checks(cache, Hkv, D, max_pages, true);
  if (st != JL_OK) return st;
  if (Hq / Hkv > 8) return JL_ERR_UNSUPPORTED;
  if (sparse && list_stride > kMaxLen / cache->page_size) return JL_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(page_list) || !aligned4(page_counts))
    return JL_ERR_ALIGNMENT;
  const PagedDecodeLayout lay = paged_decode_layout(Hq / Hkv, D);
  if (!workspace || workspace_bytes < lay.total) return JL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return JL_ERR_ALIGNMENT;
  CUtensorMap tk, tv;
  if (!encode_pages(&tk, cache->k, cache, Hkv, D) || !encode_pages(&tv, cache->v, cache, Hkv, D)) return JL_ERR_CUDA;
  jl::PagedDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  char* ws = reinterpret_cast<char*>(workspace);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.counters = reinterpret_cast<unsigned*>(ws + lay.counters);
  a.cta_parts = reinterpret_cast<float*>(ws + lay.cta);
  a.warp_parts = reinterpret_cast<float*>(ws + lay.warp);
  a.dev_error = dev_error;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.page_list = sparse ? page_list : nullptr;
  a.page_counts = sparse ? page_counts : nullptr;
  a.max_pages = max_pages;
  a.list_stride = list_stride;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.r = Hq / Hkv;
  a.w0 = w0;
  a.w_pretrained = w_pretrained;
  a.qshift = mode & JL_QSHIFT_SELF_EXTEND;
  a.scale_log2 = jl::resolve_scale(softmax_scale, D) * 1.4426950408889634f;
  std::memcpy(a.turn, jl::turn_table(D, rope_base).fixed, sizeof(a.turn));
  if (jl::launch_decode_paged(tk, tv, a, D, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return JL_ERR_CUDA;
  return JL_OK;
}

}  // namespace

extern "C" {

int jl_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* q_weight,
                    const void* k_weight, float eps, const int32_t* positions, void* q_out, void* k_out, int T,
                    int Hq, int Hkv, int head_dim, double rope_base, int* dev_error, void* stream) {
  return norm_rope(q, q_stride, k, k_stride, nullptr, 0, q_weight, k_weight, eps, nullptr, positions, T, q_out, k_out,
                   nullptr, nullptr, 0, 1, Hq, Hkv, head_dim, rope_base, dev_error, stream);
}

int jl_qk_norm_rope_append_paged(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                                 const int32_t* seq_ids, const int32_t* positions, void* q_out, void* k_out,
                                 const jl_paged_kv* cache, const int32_t* block_table, int64_t max_pages, int T,
                                 int B, int Hq, int Hkv, int head_dim, double rope_base, int* dev_error,
                                 void* stream) {
  if (cache == nullptr) return JL_ERR_INVALID_ARG;
  return norm_rope(q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, seq_ids, positions, T, q_out,
                   k_out, cache, block_table, max_pages, B, Hq, Hkv, head_dim, rope_base, dev_error, stream);
}

size_t jl_decode_paged_workspace_bytes(int Hq, int Hkv, int head_dim) {
  if (Hq < 1 || Hkv < 1 || head_dim < 1 || Hq % Hkv != 0 || Hq / Hkv > 8) return 0;
  return paged_decode_layout(Hq / Hkv, head_dim).total;
}

int jl_bifocal_decode_paged(const void* q, const jl_paged_kv* cache, const int32_t* block_table, int64_t max_pages,
                            const int32_t* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int head_dim,
                            int w0, int w_pretrained, double rope_base, float softmax_scale, int mode,
                            void* workspace, size_t workspace_bytes, int* dev_error, void* stream) {
  return decode_paged(q, cache, block_table, max_pages, seq_lens, false, nullptr, 0, nullptr, o, lse, B, Hq, Hkv,
                      head_dim, w0, w_pretrained, rope_base, softmax_scale, mode, workspace, workspace_bytes,
                      dev_error, stream);
}

int jl_bifocal_decode_paged_sparse(const void* q, const jl_paged_kv* cache, const int32_t* block_table,
                                   int64_t max_pages, const int32_t* seq_lens, const int32_t* page_list,
                                   int64_t list_stride, const int32_t* page_counts, void* o, float* lse, int B,
                                   int Hq, int Hkv, int head_dim, int w0, int w_pretrained, double rope_base,
                                   float softmax_scale, int mode, void* workspace, size_t workspace_bytes,
                                   int* dev_error, void* stream) {
  return decode_paged(q, cache, block_table, max_pages, seq_lens, true, page_list, list_stride, page_counts, o, lse,
                      B, Hq, Hkv, head_dim, w0, w_pretrained, rope_base, softmax_scale, mode, workspace,
                      workspace_bytes, dev_error, stream);
}

int jl_page_summaries(const jl_paged_kv* cache, const int32_t* block_table, int64_t max_pages, const int32_t* starts,
                      const int32_t* seq_lens, int max_new, void* summaries, int B, int Hkv, int head_dim,
                      double rope_base, int* dev_error, void* stream) {
  int st = shape_checks(B, Hkv, Hkv, head_dim, rope_base);
  if (st != JL_OK) return st;
  if (!block_table || !starts || !seq_lens || !summaries || max_new < 1) return JL_ERR_INVALID_ARG;
  st = cache_checks(cache, Hkv, head_dim, max_pages, false);
  if (st != JL_OK) return st;
  if (!aligned16(summaries) || !aligned4(block_table) || !aligned4(starts) || !aligned4(seq_lens))
    return JL_ERR_ALIGNMENT;
  jl::PageSummaryArgs a;
  std::memset(&a, 0, sizeof(a));
  a.pages = view_of(cache);
  a.block_table = block_table;
  a.starts = starts;
  a.seq_lens = seq_lens;
  a.summaries = reinterpret_cast<__nv_bfloat16*>(summaries);
  a.max_pages = max_pages;
  a.B = B;
  a.Hkv = Hkv;
  // max_new tokens that begin anywhere in a page touch at most this many pages
  a.pages_per_seq = (int)std::min<int64_t>(((int64_t)max_new + 2 * cache->page_size - 2) / cache->page_size,
                                           max_pages);
  a.dev_error = dev_error;
  std::memcpy(a.turn, jl::turn_table(head_dim, rope_base).fixed, sizeof(a.turn));
  if (jl::launch_page_summaries(a, head_dim, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return JL_ERR_CUDA;
  return JL_OK;
}

namespace {
struct SelectLayout {
  size_t scores, bounds, pages, exact, total;
  int64_t tiles;
};
SelectLayout select_layout(int B, int Hkv, int64_t max_pages) {
  const size_t rows = (size_t)B * Hkv, each = round_up(rows * max_pages * sizeof(float));
  SelectLayout lay;
  lay.tiles = (max_pages + 15) / 16;
  lay.scores = 0;
  lay.pages = each;
  lay.exact = 2 * each;
  lay.bounds = 3 * each;
  lay.total = lay.bounds + round_up(rows * lay.tiles * sizeof(float));
  return lay;
}
}  // namespace

size_t jl_select_pages_workspace_bytes(int B, int Hkv, int64_t max_pages) {
  if (B < 1 || Hkv < 1 || max_pages < 1 || max_pages > kMaxLen) return 0;
  return select_layout(B, Hkv, max_pages).total;
}

int jl_select_pages(const void* q, const void* summaries, int64_t num_pages, int page_size,
                    const int32_t* block_table, int64_t max_pages, const int32_t* seq_lens, int sink_pages, int top_k,
                    int32_t* page_list, int64_t list_stride, int32_t* page_counts, int B, int Hq, int Hkv,
                    int head_dim, int w0, int w_pretrained, double rope_base, int mode, void* workspace,
                    size_t workspace_bytes, int* dev_error, void* stream) {
  int st = shape_checks(B, Hq, Hkv, head_dim, rope_base);
  if (st != JL_OK) return st;
  st = rule_checks(w0, w_pretrained, mode);
  if (st != JL_OK) return st;
  if (!q || !summaries || !block_table || !seq_lens || !page_list || !page_counts) return JL_ERR_INVALID_ARG;
  if (num_pages < 1 || sink_pages < 0 || top_k < 0) return JL_ERR_INVALID_ARG;
  st = page_size_checks(page_size, max_pages);
  if (st != JL_OK) return st;
  if (Hq / Hkv > 8 || num_pages > INT32_MAX) return JL_ERR_UNSUPPORTED;
  // room for every page that a sequence can keep
  const int64_t band = ((int64_t)w0 + page_size - 1) / page_size + 1;
  if (list_stride < std::min<int64_t>(max_pages, (int64_t)sink_pages + top_k + band)) return JL_ERR_INVALID_ARG;
  if (list_stride > kMaxLen / page_size) return JL_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(summaries) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(page_list) || !aligned4(page_counts))
    return JL_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < jl_select_pages_workspace_bytes(B, Hkv, max_pages)) return JL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return JL_ERR_ALIGNMENT;
  jl::PageSelectArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.summaries = reinterpret_cast<const __nv_bfloat16*>(summaries);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  const SelectLayout lay = select_layout(B, Hkv, max_pages);
  char* ws = reinterpret_cast<char*>(workspace);
  a.scores = reinterpret_cast<float*>(ws + lay.scores);
  a.amb_pages = reinterpret_cast<int*>(ws + lay.pages);
  a.amb_scores = reinterpret_cast<float*>(ws + lay.exact);
  a.bounds = reinterpret_cast<float*>(ws + lay.bounds);
  a.bound_tiles = lay.tiles;
  a.page_list = page_list;
  a.page_counts = page_counts;
  a.max_pages = max_pages;
  a.list_stride = list_stride;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.r = Hq / Hkv;
  a.w0 = w0;
  a.w_pretrained = w_pretrained;
  a.qshift = mode & JL_QSHIFT_SELF_EXTEND;
  a.sink_pages = sink_pages;
  a.top_k = top_k;
  a.dev_error = dev_error;
  set_turns(a, head_dim, rope_base);
  std::memcpy(a.turn, jl::turn_table(head_dim, rope_base).fixed, sizeof(a.turn));
  if (jl::launch_page_select(a, head_dim, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return JL_ERR_CUDA;
  return JL_OK;
}

}  // extern "C"
