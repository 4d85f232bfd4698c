// linear_tc.cu -- the tensor-core product's forward form (K-major operands), the choice of form,
// and the aligned copies of operands.  The kernels are in linear_tc.cuh; each operand layout is
// compiled in a file of its own.
#include "linear_tc.cuh"

namespace kda {

cudaError_t launch_gemm_tc_dx(const Gemm& g, int planes, cudaStream_t st);
cudaError_t launch_gemm_tc_dw(const Gemm& g, int planes, cudaStream_t st);

namespace {

// ------------------------------------------------------------------ aligned copies

// rows of `cols` elements copied into rows of ld elements: bf16 as they are, fp32 as three planes
// of parts; blockIdx.y picks the array
struct RepackArgs {
  struct {
    const void* src;
    uint16_t* dst;
    int64_t src_ld, rows, cols, ld;
  } a[3];
};

// Bound by HBM.  A warp copies 256 elements of a row, two a lane and step, four steps in flight.  bf16
// rows that start in the middle of a 4-byte word are read as the words that hold them (each
// holds at least one element of the row) and shifted by one element against the next lane's word.
template <bool BF>
__global__ void __launch_bounds__(256) repack_kernel(const RepackArgs R) {
  const auto& a = R.a[blockIdx.y];
  const int64_t plane = a.rows * a.ld;
  const int64_t cb = (a.cols + 255) / 256;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < a.rows * cb; u += warps) {
    const int64_t r = u / cb;
    const int64_t c0 = (u - r * cb) * 256 + 2 * lane;
    if constexpr (BF) {
      const uint16_t* row = static_cast<const uint16_t*>(a.src) + r * a.src_ld;
      const int odd = (reinterpret_cast<uintptr_t>(row) >> 1) & 1;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(row - odd);
      const int64_t nw = (a.cols + odd + 1) / 2;       // words that hold elements of the row
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t w = (c0 >> 1) + e * 32;
        lo[e] = w < nw ? words[w] : 0;
        hi[e] = odd && lane == 31 && w + 1 < nw ? words[w + 1] : 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (odd) {                                     // the same for the whole warp
          const uint32_t next = __shfl_down_sync(0xffffffffu, lo[e], 1);
          lo[e] = (lo[e] >> 16) | ((lane == 31 ? hi[e] : next) << 16);
        }
        const int64_t c = c0 + e * 64;
        if (c < a.cols) *reinterpret_cast<uint32_t*>(a.dst + r * a.ld + c) = lo[e];   // (the padding takes the rest)
      }
    } else {
      const float* row = static_cast<const float*>(a.src) + r * a.src_ld;
      float x[4][2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t c = c0 + e * 64;
        x[e][0] = c < a.cols ? row[c] : 0.f;
        x[e][1] = c + 1 < a.cols ? row[c + 1] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t c = c0 + e * 64;
        if (c >= a.cols) continue;
        uint16_t p[3], q[3];
        split3(x[e][0], p);
        split3(x[e][1], q);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint32_t*>(a.dst + k * plane + r * a.ld + c) = p[k] | static_cast<uint32_t>(q[k]) << 16;
      }
    }
  }
}

}  // namespace

size_t repacked_bytes(int64_t rows, int64_t cols, bool bf16) {
  return static_cast<size_t>(rows) * padded(cols) * 2 * (bf16 ? 1 : 3);
}

cudaError_t launch_repack(const Repack* arrays, int count, bool bf16, cudaStream_t st) {
  RepackArgs R{};
  int64_t units = 0;
  for (int i = 0; i < count; ++i) {
    const Repack& a = arrays[i];
    R.a[i] = {a.src, static_cast<uint16_t*>(a.dst), a.src_ld, a.rows, a.cols, padded(a.cols)};
    units = std::max(units, (a.rows * ((a.cols + 255) / 256) + 7) / 8);   // blocks of eight warps
  }
  if (units == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(units, static_cast<int64_t>(sm_count()) * 16)),
                  static_cast<unsigned>(count));
  if (bf16) repack_kernel<true><<<grid, 256, 0, st>>>(R);
  else repack_kernel<false><<<grid, 256, 0, st>>>(R);
  return cudaGetLastError();
}

// g.A and g.B: 16-byte aligned bf16 rows, `planes` (1 or 3) planes of them one after another.  An
// MN-major A (a gradient) has no bias, activation, residual or pre-activation.
cudaError_t launch_gemm_tc(const Gemm& g, int planes, cudaStream_t st) {
  if (g.I == 0 || g.J == 0) return cudaSuccess;
  if (!g.A.mn) return g.B.mn ? cudaErrorInvalidValue : launch_shape<false, false>(g, planes, st);
  return g.B.mn ? launch_gemm_tc_dw(g, planes, st) : launch_gemm_tc_dx(g, planes, st);
}

}  // namespace kda
