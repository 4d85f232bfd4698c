// gemm.cuh -- the matrix product behind the projections (linear.cu, linear_tc.cu):
//
//     out[j, i] = residual[j, i] + scale act(sum_c A(i, c) B(j, c) + bias[i])
//
// with i the contiguous dimension of every [J, I] array.  The forward takes A = w, B = x over
// c = k; dx takes A = w^T, B = dz over c = n; dw takes A = x^T, B = dz^T over c = t.
#pragma once

#include "layer_common.cuh"

namespace kda {

struct GemmOperand {
  const void* p;
  int64_t ld;      // elements between rows of the stored matrix
  bool mn;         // false: rows are i (or j) and c is contiguous; true: rows are c
};

struct GemmEpilogue {
  const float* bias;   // [I] or null
  const void* res;     // [J, I] or null
  void* out;           // [J, I]
  void* z;             // [J, I] or null: the sum before the activation
  int64_t res_ld, out_ld, z_ld;
  float scale;
  int32_t act;
  bool res_bf, out_bf, z_bf;
};

struct Gemm {
  GemmOperand A, B;
  int64_t I, J, C;
  bool bf16;           // operand type: bf16 or fp32
  GemmEpilogue epi;
  int32_t* err;
};

__device__ __forceinline__ float ld_any(const void* p, bool bf, int64_t i) {
  return bf ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void st_any(void* p, bool bf, int64_t i, float v) {
  if (bf) static_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
  else static_cast<float*>(p)[i] = v;
}

// one element of the result; `acc` is the finished sum over c
__device__ __forceinline__ void epilogue_store(const GemmEpilogue& E, int64_t j, int64_t i, float acc) {
  if (E.bias) acc += __ldg(E.bias + i);
  if (E.z) st_any(E.z, E.z_bf, j * E.z_ld + i, acc);
  float y = E.scale * (E.out_bf ? act_f<true>(E.act, acc) : act_f<false>(E.act, acc));
  if (E.res) y += ld_any(E.res, E.res_bf, j * E.res_ld + i);
  st_any(E.out, E.out_bf, j * E.out_ld + i, y);
}

cudaError_t launch_gemm_simt(const Gemm& g, cudaStream_t st);

// A and B K-major and J at most kRowsMax: CUDA cores, any alignment.
constexpr int kRowsMax = 8;
cudaError_t launch_gemm_rows(const Gemm& g, cudaStream_t st);

// The tensor-core product: operands are 16-byte aligned bf16 rows, `planes` (1, or 3 for the parts
// of fp32) planes of rows * ld elements one after another.  C >= 1.
cudaError_t launch_gemm_tc(const Gemm& g, int planes, cudaStream_t st);
// rows of `cols` elements copied into rows of `padded(cols)`: bf16 as they are, fp32 as three planes
// of bf16 parts.  The rows are whole 128-byte lines, so that a box's rows cross none.
inline int64_t padded(int64_t cols) { return (cols + 63) / 64 * 64; }
size_t repacked_bytes(int64_t rows, int64_t cols, bool bf16);
struct Repack {
  const void* src;
  int64_t src_ld, rows, cols;
  void* dst;
};
cudaError_t launch_repack(const Repack* arrays, int count, bool bf16, cudaStream_t st);   // up to 3

// the three bf16 parts of an fp32 value
__device__ __forceinline__ void split3(float x, uint16_t (&p)[3]) {
  // rounded to nearest at each step; a finite x whose rounding would overflow is cut instead
  p[0] = f32_to_bf16_bits(x);
  if ((p[0] & 0x7fff) == 0x7f80) p[0] = static_cast<uint16_t>(__float_as_uint(x) >> 16);
  const float hi = bf16_bits_to_f32(p[0]);
  const float r = (p[0] & 0x7f80) == 0x7f80 ? 0.f : x - hi;     // infinities and NaN have no rest
  p[1] = f32_to_bf16_bits(r);
  p[2] = f32_to_bf16_bits(r - bf16_bits_to_f32(p[1]));
}


}  // namespace kda
