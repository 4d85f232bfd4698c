// cache_api.cu -- the C ABI of the key-value cache: argument validation and dispatch.  Everything here
// runs on the host before any launch.
#include <math.h>

#include <algorithm>

#include "cache_common.cuh"

static_assert(sizeof(kda_rotary_params_t) == 72, "kda_rotary_params_t layout is part of the ABI");
static_assert(sizeof(kda_cache_params_t) == 128, "kda_cache_params_t layout is part of the ABI");
static_assert(sizeof(kda_cache_rows_params_t) == 20, "kda_cache_rows_params_t layout is part of the ABI");

namespace {

bool is_dtype(int32_t d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
kda_status_t to_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
bool workspace_ok(const void* ws, size_t bytes, size_t need) { return ws && bytes >= need && aligned(ws, 256); }

constexpr int64_t kMaxStride = int64_t{1} << 40;
constexpr int kMaxHead = 1024, kMaxAttentionHead = 256, kMaxWindow = 64;
constexpr int64_t kMaxRow = 1 << 22;                          // elements of a token's heads

// row strides are 0 (dense) or at least the row
bool stride_ok(int64_t stride, int64_t cols) { return stride == 0 || (stride >= cols && stride <= kMaxStride); }
int64_t or_dense(int64_t stride, int64_t cols) { return stride ? stride : cols; }

bool rotation_ok(int32_t R, int32_t d, float magnitude) {
  return R >= 0 && R % 2 == 0 && R <= d && isfinite(magnitude);
}

// The heads of the pages do not overlap: of pages, rows and heads, in whatever order, each is as far apart as what lies
// between two of it spans (in fp64: strides of 2^40 times extents of 2^31).
bool pages_ok(const kda_cache_params_t* p) {
  struct Extent {
    int64_t stride, size;
  } e[3] = {{p->page_head_stride, p->num_kv_heads}, {p->page_row_stride, p->page_size}, {p->page_stride, p->num_pages}};
  for (const Extent& x : e)
    if (x.stride < 1 || x.stride > kMaxStride) return false;
  std::sort(e, e + 3, [](const Extent& x, const Extent& y) { return x.stride < y.stride; });
  double span = p->head_dim;
  for (const Extent& x : e) {
    if (x.size <= 1) continue;
    if (static_cast<double>(x.stride) < span) return false;
    span += static_cast<double>(x.stride) * (x.size - 1);
  }
  return true;
}

kda_status_t check_cache(const kda_cache_params_t* p) {
  if (!p || p->num_seqs < 0 || p->num_kv_heads < 1 || p->num_q_heads < 0 || p->head_dim < 1) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(p->dtype) || p->page_size < 1 || p->max_pages < 0 || p->num_pages < 0) return KDA_ERR_INVALID_ARG;
  const int64_t d = p->head_dim;
  if ((p->num_q_heads + 2 * static_cast<int64_t>(p->num_kv_heads)) * d > kMaxRow) return KDA_ERR_UNSUPPORTED;
  if (!pages_ok(p) || !stride_ok(p->q_row_stride, p->num_q_heads * d)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status_t check_attention(const kda_cache_params_t* p) {
  const kda_status_t s = check_cache(p);
  if (s != KDA_OK) return s;
  if (p->num_q_heads < 1 || p->num_q_heads % p->num_kv_heads || !is_dtype(p->o_dtype)) return KDA_ERR_INVALID_ARG;
  if (p->window < 1 || p->span < 0 || !isfinite(p->scale) || !isfinite(p->softcap) || p->softcap < 0.f)
    return KDA_ERR_INVALID_ARG;
  const int64_t piece = 16 / static_cast<int64_t>(kda::dtype_bytes(p->dtype));
  if (p->window > kMaxWindow || p->head_dim > kMaxAttentionHead || p->head_dim % piece) return KDA_ERR_UNSUPPORTED;
  // the units of work are counted in 32 bits: tiles of 32 keys and more, and 3 for each (sequence, key head, 8 rows)
  const double rows = static_cast<double>(p->window) * (p->num_q_heads / p->num_kv_heads) / 2 + 1;
  if (p->num_seqs * static_cast<double>(p->num_kv_heads) * rows * (static_cast<double>(p->max_pages) * p->page_size / 32 + 4) >=
      2147483648.0)
    return KDA_ERR_UNSUPPORTED;
  if (p->page_stride % piece || p->page_row_stride % piece || p->page_head_stride % piece || p->q_row_stride % piece)
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status_t check_rows(const kda_cache_rows_params_t* p) {
  if (!p || p->rows < 0 || p->rows_out < 0 || p->max_pages < 0 || p->page_size < 1 || p->num_pages < 0)
    return KDA_ERR_INVALID_ARG;
  if (p->num_pages > (1 << 28) || p->rows > (1 << 24) || p->rows_out > (1 << 24)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status_t rotary(const kda_rotary_params_t* p, const void* q, const void* k, const void* positions,
                    const double* freq, void* q_out, void* k_out, void* stream, int transpose) {
  if (!p || p->tokens < 0 || p->num_q_heads < 0 || p->num_k_heads < 0 || p->head_dim < 1 || !is_dtype(p->dtype))
    return KDA_ERR_INVALID_ARG;
  if (p->rot_dim < 1 || !rotation_ok(p->rot_dim, p->head_dim, p->magnitude)) return KDA_ERR_INVALID_ARG;
  const int64_t d = p->head_dim, nq = p->num_q_heads * d, nk = p->num_k_heads * d;
  if (p->head_dim > kMaxHead || nq + nk > kMaxRow || p->tokens > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(p->q_row_stride, nq) || !stride_ok(p->k_row_stride, nk) || !stride_ok(p->q_out_row_stride, nq) ||
      !stride_ok(p->k_out_row_stride, nk))
    return KDA_ERR_INVALID_ARG;
  if (p->tokens == 0 || nq + nk == 0) return KDA_OK;
  const size_t e = kda::dtype_bytes(p->dtype);
  if ((nq && (!q || !q_out)) || (nk && (!k || !k_out)) || !positions || !freq) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(freq, 8) ||
      !aligned(positions, p->wide_positions ? 8 : 4))
    return KDA_ERR_INVALID_ARG;
  kda::RotaryArgs a{};
  a.q = nq ? q : nullptr;
  a.k = nk ? k : nullptr;
  a.q_out = nq ? q_out : nullptr;
  a.k_out = nk ? k_out : nullptr;
  a.positions = positions;
  a.freq = freq;
  a.q_stride = or_dense(p->q_row_stride, nq);
  a.k_stride = or_dense(p->k_row_stride, nk);
  a.q_out_stride = or_dense(p->q_out_row_stride, nq);
  a.k_out_stride = or_dense(p->k_out_row_stride, nk);
  a.T = p->tokens;
  a.H = p->num_q_heads;
  a.HK = p->num_k_heads;
  a.D = p->head_dim;
  a.R = p->rot_dim;
  a.P = 1;
  a.wide = p->wide_positions != 0;
  a.interleaved = p->interleaved != 0;
  a.transpose = transpose;
  a.magnitude = p->magnitude;
  return to_status(kda::launch_rotary(a, p->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

kda_status_t kda_rotary_fwd(const kda_rotary_params_t* p, const void* q, const void* k, const void* positions,
                            const double* frequencies, void* q_out, void* k_out, void* stream) {
  return rotary(p, q, k, positions, frequencies, q_out, k_out, stream, 0);
}

kda_status_t kda_rotary_bwd(const kda_rotary_params_t* p, const void* d_q, const void* d_k, const void* positions,
                            const double* frequencies, void* dq_out, void* dk_out, void* stream) {
  return rotary(p, d_q, d_k, positions, frequencies, dq_out, dk_out, stream, 1);
}

kda_status_t kda_cache_append(const kda_cache_params_t* p, const void* q, const void* k, const void* v,
                              const double* frequencies, void* key_pages, void* value_pages,
                              const int32_t* block_table, const int32_t* start, const uint32_t* input_row_offsets,
                              void* q_out, void* stream) {
  const kda_status_t s = check_cache(p);
  if (s != KDA_OK) return s;
  if (!rotation_ok(p->rot_dim, p->head_dim, p->magnitude) || p->tokens < 0) return KDA_ERR_INVALID_ARG;
  const int64_t d = p->head_dim, nq = p->num_q_heads * d, nk = p->num_kv_heads * d;
  if (p->head_dim > kMaxHead || p->tokens > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(p->k_row_stride, nk) || !stride_ok(p->v_row_stride, nk) || !stride_ok(p->q_out_row_stride, nq))
    return KDA_ERR_INVALID_ARG;
  if (!input_row_offsets && p->tokens != p->num_seqs) return KDA_ERR_INVALID_ARG;
  if (p->tokens == 0 || p->num_seqs == 0) return KDA_OK;
  const size_t e = kda::dtype_bytes(p->dtype);
  if ((nq && (!q || !q_out)) || !k || !v || !key_pages || !value_pages || !block_table || !start ||
      (p->rot_dim > 0) != (frequencies != nullptr))
    return KDA_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(q_out, e) || !aligned(key_pages, e) ||
      !aligned(value_pages, e) || !aligned(frequencies, 8) || !aligned(block_table, 4) || !aligned(start, 4) ||
      !aligned(input_row_offsets, 4))
    return KDA_ERR_INVALID_ARG;
  kda::RotaryArgs a{};
  a.q = nq ? q : nullptr;
  a.k = k;
  a.v = v;
  a.q_out = nq ? q_out : nullptr;
  a.k_out = key_pages;
  a.v_out = value_pages;
  a.freq = frequencies;
  a.table = block_table;
  a.start = start;
  a.offsets = input_row_offsets;
  a.q_stride = or_dense(p->q_row_stride, nq);
  a.k_stride = or_dense(p->k_row_stride, nk);
  a.v_stride = or_dense(p->v_row_stride, nk);
  a.q_out_stride = or_dense(p->q_out_row_stride, nq);
  a.page_stride = p->page_stride;
  a.page_row_stride = p->page_row_stride;
  a.page_head_stride = p->page_head_stride;
  a.T = p->tokens;
  a.B = p->num_seqs;
  a.H = p->num_q_heads;
  a.HK = a.HV = p->num_kv_heads;
  a.D = p->head_dim;
  a.R = p->rot_dim;
  a.P = p->page_size;
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.interleaved = p->interleaved != 0;
  a.magnitude = p->magnitude;
  a.err = kda::layer_error_word();
  if (!a.err) return KDA_ERR_CUDA;
  return to_status(kda::launch_rotary(a, p->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_attention_workspace_size(const kda_cache_params_t* p, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status_t s = check_attention(p);
  if (s != KDA_OK) return s;
  *bytes = kda::cache_attention_workspace(*p);
  return KDA_OK;
}

kda_status_t kda_cache_attention(const kda_cache_params_t* p, const void* q, const void* key_pages,
                                 const void* value_pages, const int32_t* block_table, const int32_t* lens,
                                 const float* slopes, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const kda_status_t s = check_attention(p);
  if (s != KDA_OK) return s;
  if (p->num_seqs == 0) return KDA_OK;
  if (!q || !key_pages || !value_pages || (!block_table && p->max_pages) || !lens || !o) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(key_pages, 16) || !aligned(value_pages, 16) || !aligned(block_table, 4) ||
      !aligned(lens, 4) || !aligned(slopes, 4) || !aligned(o, kda::dtype_bytes(p->o_dtype)) || !aligned(lse, 4))
    return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::cache_attention_workspace(*p))) return KDA_ERR_WORKSPACE;
  kda::AttentionArgs a{};
  a.q = q;
  a.k = key_pages;
  a.v = value_pages;
  a.table = block_table;
  a.lens = lens;
  a.slopes = slopes;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  a.q_stride = or_dense(p->q_row_stride, static_cast<int64_t>(p->num_q_heads) * p->head_dim);
  a.page_stride = p->page_stride;
  a.page_row_stride = p->page_row_stride;
  a.page_head_stride = p->page_head_stride;
  a.B = p->num_seqs;
  a.W = p->window;
  a.H = p->num_q_heads;
  a.HK = p->num_kv_heads;
  a.D = p->head_dim;
  a.P = p->page_size;
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.span = p->span;
  a.scale = p->scale != 0.f ? p->scale : 1.f / sqrtf(static_cast<float>(p->head_dim));
  a.softcap = p->softcap;
  a.err = kda::layer_error_word();
  if (!a.err) return KDA_ERR_CUDA;
  return to_status(kda::launch_cache_attention(a, p->dtype == KDA_DTYPE_BF16, p->o_dtype == KDA_DTYPE_BF16,
                                               static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_rows_workspace_size(const kda_cache_rows_params_t* p, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const kda_status_t s = check_rows(p);
  if (s != KDA_OK) return s;
  *bytes = kda::cache_rows_workspace(*p);
  return KDA_OK;
}

kda_status_t kda_cache_update(const kda_cache_rows_params_t* p, const int32_t* block_table, const int32_t* lens,
                              const int32_t* refs, const int32_t* parent, const int32_t* new_lens, int32_t* out_table,
                              int32_t* out_lens, int32_t* out_refs, int32_t* kept, int32_t* copy_src,
                              int32_t* copy_dst, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status_t s = check_rows(p);
  if (s != KDA_OK) return s;
  const bool in = p->rows > 0, out = p->rows_out > 0, pages = p->num_pages > 0, wide = p->max_pages > 0;
  if ((in && !lens) || (in && wide && !block_table) || (pages && (!refs || !out_refs)) || (out && wide && !out_table) ||
      (out && (!new_lens || !out_lens || !kept || !copy_src || !copy_dst)) || (out && !parent && p->rows != p->rows_out))
    return KDA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(lens), static_cast<const void*>(refs),
                        static_cast<const void*>(parent), static_cast<const void*>(new_lens),
                        static_cast<const void*>(out_table), static_cast<const void*>(out_lens),
                        static_cast<const void*>(out_refs), static_cast<const void*>(kept),
                        static_cast<const void*>(copy_src), static_cast<const void*>(copy_dst)})
    if (!aligned(x, 4)) return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::cache_rows_workspace(*p))) return KDA_ERR_WORKSPACE;
  kda::RowsArgs a{};
  a.table = block_table;
  a.lens = lens;
  a.refs = refs;
  a.parent = parent;
  a.new_lens = new_lens;
  a.out_table = out_table;
  a.out_lens = out_lens;
  a.out_refs = out_refs;
  a.kept = kept;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.scratch = static_cast<int32_t*>(workspace);
  a.S = p->rows;
  a.S_out = p->rows_out;
  a.width = p->max_pages;
  a.P = p->page_size;
  a.N = p->num_pages;
  a.err = kda::layer_error_word();
  if (!a.err) return KDA_ERR_CUDA;
  return to_status(kda::launch_cache_update(a, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_compact(const kda_cache_rows_params_t* p, const int32_t* block_table, const int32_t* lens,
                               const int32_t* refs, int32_t* out_table, int32_t* out_refs, int32_t* page_map,
                               int32_t* copy_src, int32_t* copy_dst, void* workspace, size_t workspace_bytes,
                               void* stream) {
  const kda_status_t s = check_rows(p);
  if (s != KDA_OK) return s;
  const bool in = p->rows > 0, pages = p->num_pages > 0, wide = p->max_pages > 0;
  if ((in && !lens) || (in && wide && (!block_table || !out_table)) || (pages && (!refs || !out_refs || !page_map)) ||
      (p->num_pages > 1 && (!copy_src || !copy_dst)))
    return KDA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(lens), static_cast<const void*>(refs),
                        static_cast<const void*>(out_table), static_cast<const void*>(out_refs),
                        static_cast<const void*>(page_map), static_cast<const void*>(copy_src),
                        static_cast<const void*>(copy_dst)})
    if (!aligned(x, 4)) return KDA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, kda::cache_rows_workspace(*p))) return KDA_ERR_WORKSPACE;
  kda::RowsArgs a{};
  a.table = block_table;
  a.lens = lens;
  a.refs = refs;
  a.out_table = out_table;
  a.out_refs = out_refs;
  a.page_map = page_map;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.scratch = static_cast<int32_t*>(workspace);
  a.S = p->rows;
  a.width = p->max_pages;
  a.P = p->page_size;
  a.N = p->num_pages;
  a.err = kda::layer_error_word();
  if (!a.err) return KDA_ERR_CUDA;
  return to_status(kda::launch_cache_compact(a, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_copy(void* const* pools, const int64_t* page_bytes, const int64_t* page_strides,
                            int32_t num_pools, const int32_t* src, const int32_t* dst, int64_t n, int32_t num_pages,
                            void* stream) {
  if (num_pools < 0 || n < 0 || num_pages < 0) return KDA_ERR_INVALID_ARG;
  if (num_pools == 0 || n == 0 || num_pages == 0) return KDA_OK;
  if (!pools || !page_bytes || !page_strides || !src || !dst || !aligned(src, 4) || !aligned(dst, 4))
    return KDA_ERR_INVALID_ARG;
  if (n > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  for (int i = 0; i < num_pools; ++i)
    if ((!pools[i] && page_bytes[i] > 0) || page_bytes[i] < 0 || page_bytes[i] > kMaxStride ||
        (num_pages > 1 && page_strides[i] < page_bytes[i]) || page_strides[i] > kMaxStride)
      return KDA_ERR_INVALID_ARG;
  int32_t* err = kda::layer_error_word();
  if (!err) return KDA_ERR_CUDA;
  return to_status(kda::launch_cache_copy(pools, page_bytes, page_strides, num_pools, src, dst, n, num_pages, err,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
