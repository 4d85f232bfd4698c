// cache_common.cuh -- what the kernels of the key-value cache share (rotary.cu, cache_attention.cu,
// cache_rows.cu): division by a number that is fixed for a launch, and the launchers behind
// cache_api.cu.
#pragma once

#include "layer_common.cuh"

namespace kda {

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994): with l = ceil(log2 d) and m = ceil(2^(31 + l) / d), n / d = n m >> (31 + l).
struct FastDiv {
  uint32_t m, d;
  int32_t shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_) {
    int l = 0;
    while (l < 31 && (1u << l) < d) ++l;
    shift = 31 + l;
    m = static_cast<uint32_t>(((uint64_t{1} << shift) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> shift);
  }
};

// the rows that rotary.cu reads and where they go
struct RotaryArgs {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;               // k_out, v_out: the pages where `table` is set
  const void* positions;                     // [T] int32 or int64; null with `table`
  const double* freq;                        // [R / 2] radians per position, or null: nothing is turned
  const int32_t *table, *start;
  const uint32_t* offsets;                   // [B + 1], or null: token s is sequence s
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t page_stride, page_row_stride, page_head_stride;
  int64_t T;
  int32_t B, H, HK, HV, D, R, P, max_pages, num_pages;
  int32_t wide, interleaved, transpose;
  float magnitude;
  int32_t* err;
};
cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t st);

struct AttentionArgs {
  const void *q, *k, *v;
  const int32_t *table, *lens;
  const float* slopes;                       // [H] or null
  void* o;
  float* lse;                                // [B W, H] or null
  void* workspace;
  int64_t q_stride, page_stride, page_row_stride, page_head_stride;
  int32_t B, W, H, HK, D, P, max_pages, num_pages, span;
  float scale, softcap;
  int32_t* err;
};
size_t cache_attention_workspace(const kda_cache_params_t& p);
cudaError_t launch_cache_attention(const AttentionArgs& a, bool bf16, bool bf16_out, cudaStream_t st);

struct RowsArgs {
  const int32_t *table, *lens, *refs, *parent, *new_lens;
  int32_t *out_table, *out_lens, *out_refs, *kept, *page_map, *copy_src, *copy_dst;
  int32_t* scratch;
  int32_t S, S_out, width, P, N;
  int32_t* err;
};
size_t cache_rows_workspace(const kda_cache_rows_params_t& p);
cudaError_t launch_cache_update(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_cache_compact(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_cache_copy(void* const* pools, const int64_t* bytes, const int64_t* strides, int num_pools,
                              const int32_t* src, const int32_t* dst, int64_t n, int num_pages, int32_t* err,
                              cudaStream_t st);

}  // namespace kda
