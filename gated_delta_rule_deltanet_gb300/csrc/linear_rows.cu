// linear_rows.cu -- the projection of a few tokens (decode): out[j, i] for j < 2, or j < 8 where the
// tensor cores would need a copy of the weight.
//
// Bound by HBM: every weight is read once for at most 8 multiply-adds, which the CUDA cores do as
// fp32 pairs.  A warp owns R = 4 rows of the weight (4 outputs a token) and walks them together, 16
// bytes a lane and row, so that 4 weight loads a lane are in flight beside the tokens' elements,
// which come from L1; where there are too few rows for the SMs, 2 to 8 warps of a block share a
// group of rows and split k, adding their sums in warp order.  Compared with the tensor-core
// kernel, whose set-up (tensor maps, tensor memory, barriers, a cluster's sum) costs more than
// the arithmetic at these sizes: 2048 -> 6144 for one token 8.5 -> 4.8 us (6.3 us with the weight
// in HBM rather than L2).  The sums are fp32 in a fixed order; fp32 weights are read as they are.
#include <algorithm>

#include "gemm.cuh"

namespace kda {

namespace {

constexpr int kR = 4;

template <bool BF, bool VEC, int NT>
__global__ void __launch_bounds__(256) gemm_rows_kernel(const Gemm g, const int split) {
  __shared__ float s_part[8][kR * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = 8 / split;                  // groups of rows in a block
  const int64_t grp = static_cast<int64_t>(blockIdx.x) * groups + warp / split;
  const int part = warp % split;
  const int64_t i0 = grp * kR;
  const int K = static_cast<int>(g.C), J = static_cast<int>(g.J);
  const int es = BF ? 2 : 4;
  // this warp's share of k, in steps of 256
  const int steps = (K + 255) / 256;
  const int k0 = static_cast<int>(static_cast<int64_t>(steps) * part / split) * 256;
  const int k1 = min(K, static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / split) * 256);
  const char* wrow[kR];
  const char* xrow[NT];
#pragma unroll
  for (int r = 0; r < kR; ++r)
    wrow[r] = static_cast<const char*>(g.A.p) + std::min<int64_t>(i0 + r, g.I - 1) * g.A.ld * es;
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = static_cast<const char*>(g.B.p) + min(t, J - 1) * g.B.ld * es;
  float2 acc[kR][NT];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = make_float2(0.f, 0.f);
  if (i0 < g.I) {
#pragma unroll 2
    for (int k = k0; k < k1; k += 256) {
      const int n = min(256, k1 - k);
      Raw8<BF> w[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) w[r] = load_chunk<BF, VEC>(wrow[r] + static_cast<int64_t>(k) * es, lane, 32, n);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Raw8<BF> x = load_chunk<BF, VEC>(xrow[t] + static_cast<int64_t>(k) * es, lane, 32, n);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 xv = make_float2(x.f32(e), x.f32(e + 1));
#pragma unroll
          for (int r = 0; r < kR; ++r) acc[r][t] = fma2(make_float2(w[r].f32(e), w[r].f32(e + 1)), xv, acc[r][t]);
        }
      }
    }
  }
  // lane r * NT + t keeps the sum of row r and token t (kR * NT <= 32)
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float s = warp_sum(acc[r][t].x + acc[r][t].y);
      if (lane == r * NT + t) mine = s;
    }
  const int t = lane % NT;
  const int64_t i = i0 + lane / NT;
  const bool out = lane < kR * NT && t < J && i < g.I;
  if (split > 1) {
    if (lane < kR * NT) s_part[warp][lane] = mine;
    __syncthreads();
    if (part == 0 && lane < kR * NT)
      for (int p = 1; p < split; ++p) mine += s_part[warp + p][lane];
  }
  if (part == 0 && out) epilogue_store(g.epi, t, i, mine);
}

template <bool BF, bool VEC>
cudaError_t launch_rows_t(const Gemm& g, cudaStream_t st) {
  const int64_t groups = (g.I + kR - 1) / kR;
  // 12 warps an SM and at least two steps of k a warp
  int split = 1;
  while (split < 8 && groups * split < static_cast<int64_t>(sm_count()) * 12 && g.C >= 512 * split * 2) split *= 2;
  const int64_t blocks = (groups + 8 / split - 1) / (8 / split);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned n = static_cast<unsigned>(blocks);
  if (g.J == 1) gemm_rows_kernel<BF, VEC, 1><<<n, 256, 0, st>>>(g, split);
  else if (g.J == 2) gemm_rows_kernel<BF, VEC, 2><<<n, 256, 0, st>>>(g, split);
  else if (g.J <= 4) gemm_rows_kernel<BF, VEC, 4><<<n, 256, 0, st>>>(g, split);
  else gemm_rows_kernel<BF, VEC, 8><<<n, 256, 0, st>>>(g, split);
  return cudaGetLastError();
}

}  // namespace

// A and B K-major, J <= 8; any alignment and strides
cudaError_t launch_gemm_rows(const Gemm& g, cudaStream_t st) {
  if (g.I == 0 || g.J == 0) return cudaSuccess;
  const int es = g.bf16 ? 2 : 4;
  auto vec16 = [&](const GemmOperand& X) {
    return (reinterpret_cast<uintptr_t>(X.p) & 15) == 0 && X.ld * es % 16 == 0;
  };
  const bool vec = g.C % 8 == 0 && vec16(g.A) && vec16(g.B);
  if (g.bf16) return vec ? launch_rows_t<true, true>(g, st) : launch_rows_t<true, false>(g, st);
  return vec ? launch_rows_t<false, true>(g, st) : launch_rows_t<false, false>(g, st);
}

}  // namespace kda
