// layer_common.cuh -- pieces shared by the kernels of the layer around the recurrence
// (linear.cu, norms.cu): eight-element chunks of a row in either dtype, the activations and
// their derivatives, and the fixed-order sum over partial rows.
#pragma once

#include <atomic>

#include "kda_common.cuh"

namespace kda {

// The device error word of the current device (null when CUDA reports an error).
int32_t* layer_error_word();

inline size_t dtype_bytes(int32_t dt) { return dt == KDA_DTYPE_BF16 ? 2 : 4; }

// ---------------------------------------------------------------- launches

// The kernel's dynamic shared-memory limit, raised once for each device to the most that any call takes: the
// limit belongs to the process, so a call that set its own could lower another thread's between that one's
// setting and launch.
template <typename Kernel>
inline cudaError_t raise_smem(Kernel k, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------- eight elements of a row

// VEC: elements [8 c, 8 c + 8) as 16-byte vectors (rows of a multiple of 8 elements, 16-byte
// aligned).  Otherwise: elements c, c + step, c + 2 step, ... below n, each loaded by itself,
// so that rows of any length and alignment are read with consecutive lanes on consecutive
// elements.
template <bool VEC>
__device__ __forceinline__ int chunk_index(int c, int step, int e) {
  return VEC ? 8 * c + e : c + e * step;
}

template <bool BF>
struct Raw8 {               // the chunk as loaded: no arithmetic waits on it until f32() is called
  uint32_t w[BF ? 4 : 8];
  __device__ __forceinline__ float f32(int e) const {
    if constexpr (BF)
      return (e & 1) ? __uint_as_float(w[e >> 1] & 0xffff0000u) : __uint_as_float(w[e >> 1] << 16);
    else
      return __uint_as_float(w[e]);
  }
  __device__ __forceinline__ float2 f2(int e) const { return make_float2(f32(2 * e), f32(2 * e + 1)); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF ? 4 : 8); ++i) w[i] = 0;
  }
};

template <bool BF, bool VEC>
__device__ __forceinline__ Raw8<BF> load_chunk(const void* row, int c, int step, int n) {
  Raw8<BF> r;
  if constexpr (VEC) {
    if (8 * c < n) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) +
                                                      static_cast<int64_t>(c) * (BF ? 16 : 32));
      const uint4 a = p[0];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
      if constexpr (!BF) {
        const uint4 b = p[1];
        r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
      }
    } else {
      r.zero();
    }
  } else {
    r.zero();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e * step;
      if (i < n) {
        if constexpr (BF)
          r.w[e >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << (16 * (e & 1));
        else
          r.w[e] = __float_as_uint(static_cast<const float*>(row)[i]);
      }
    }
  }
  return r;
}

// rounds to nearest even where the row is bf16
template <bool BF, bool VEC>
__device__ __forceinline__ void store_chunk(void* row, int c, int step, int n, const float (&x)[8]) {
  if constexpr (VEC) {
    if (8 * c >= n) return;
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(row) + static_cast<int64_t>(c) * (BF ? 16 : 32));
    if constexpr (BF) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
      p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      p[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      p[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e * step;
      if (i < n) {
        if constexpr (BF) static_cast<uint16_t*>(row)[i] = f32_to_bf16_bits(x[e]);
        else static_cast<float*>(row)[i] = x[e];
      }
    }
  }
}

// eight fp32 parameters of a chunk's columns (cached: every row reads them)
template <bool VEC>
__device__ __forceinline__ void load_params(const float* p, int c, int step, int n, float (&x)[8]) {
  if constexpr (VEC) {
    if (8 * c < n) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p) + 2 * c);
      const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 2 * c + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e * step;
      x[e] = i < n ? __ldg(p + i) : 0.f;
    }
  }
}

// aligned forms on pairs
__device__ __forceinline__ void load_params2(const float* p, int c, int n, float2 (&x)[4]) {
  float v[8];
  load_params<true>(p, c, 0, n, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float2(v[2 * e], v[2 * e + 1]);
}
template <bool BF>
__device__ __forceinline__ void store_pairs(void* row, int c, int n, const float2 (&x)[4]) {
  const float v[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
  store_chunk<BF, true>(row, c, 0, n, v);
}

// ---------------------------------------------------------------- activations

// sigmoid(z).  FAST (bf16 results, and the fp32 gradients that are formed from bf16 inputs with them: dbias,
// gated_norm's d_o and d_weight): __expf's error, 2 + 1.2 |z| ulp, stays far below the bf16
// rounding; otherwise expf.  The quotient is 0 where exp(-z) overflows.
template <bool FAST>
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.f, 1.f + (FAST ? __expf(-z) : expf(-z)));
}

// Phi(z) = erfc(-z / sqrt 2) / 2 and e = exp(-z^2 / 2).  FAST (bf16 results): erfc(x) = (a1 t + .. +
// a6 t^6) exp(-x^2), t = 1 / (1 + p x), x >= 0, the form of 7.1.26 in Abramowitz and Stegun, "Handbook of
// Mathematical Functions", with coefficients fitted (minimax) so that the error is within 1e-7 and
// within 1e-4 of the value up to x = 9.5, where erfc leaves fp32: the far negative side, Phi(z) itself,
// then rounds to bf16 as the exact value does (half a step is 2e-3 and more; the handbook's
// coefficients are off by 2.5e-3 at z = -5.5, 6.5e-3 at -7).  A third of erfcf's instructions, which set the
// pace of the persistent product's epilogue.
template <bool FAST>
__device__ __forceinline__ void normal_cdf(float z, float& phi, float& e) {
  if constexpr (FAST) {
    const float x = 0.70710678f * fabsf(z);
    e = __expf(-x * x);
    const float t = __fdividef(1.f, 1.f + 0.41f * x);
    const float poly =
        t * (0.23381889f +
             t * (0.20009884f + t * (0.36317647f + t * (-0.19286337f + t * (0.57457983f - t * 0.17881072f)))));
    const float tail = 0.5f * poly * e;             // of the side away from zero
    phi = z < 0.f ? tail : 1.f - tail;
  } else {
    phi = 0.5f * erfcf(-0.70710678f * z);
    e = expf(-0.5f * z * z);
  }
}

template <bool FAST>
__device__ __forceinline__ float act_f(int act, float z) {
  switch (act) {
    case KDA_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);   // a NaN stays one
    case KDA_ACT_SILU: return z == -INFINITY ? 0.f : z * sigmoid_f<FAST>(z);
    case KDA_ACT_GELU: {
      if (z < -20.f) return 0.f;                    // z Phi(z) below 1e-87; also -infinity
      float phi, e;
      normal_cdf<FAST>(z, phi, e);
      return z * phi;
    }
    case KDA_ACT_SIGMOID: return sigmoid_f<FAST>(z);
    default: return z;
  }
}

// p = sigmoid(z) and q = 1 - p from one exponential of -|z|: neither cancels
template <bool FAST>
__device__ __forceinline__ void sigmoid_pair(float z, float& p, float& q) {
  const float e = FAST ? __expf(-fabsf(z)) : expf(-fabsf(z));
  const float r = __fdividef(1.f, 1.f + e);
  p = z < 0.f ? e * r : r;
  q = z < 0.f ? r : e * r;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_grad_f(float z) {
  if constexpr (ACT == KDA_ACT_RELU) {
    return z > 0.f ? 1.f : (z == z ? 0.f : z);
  } else if constexpr (ACT == KDA_ACT_SILU || ACT == KDA_ACT_SIGMOID) {
    float p, q;
    sigmoid_pair<FAST>(z, p, q);
    if constexpr (ACT == KDA_ACT_SIGMOID) return p * q;
    return fabsf(z) > 100.f ? p : p * (1.f + z * q);      // 0 / 1 at the infinities
  } else if constexpr (ACT == KDA_ACT_GELU) {
    if (fabsf(z) > 20.f) return z > 0.f ? 1.f : 0.f;
    float phi, e;
    normal_cdf<FAST>(z, phi, e);
    return phi + 0.39894228f * z * e;
  } else {
    return 1.f;
  }
}

// ---------------------------------------------------------------- partial rows

// Partial rows of `segments` (at most 3) stretches of `cols` columns each: outs.p[s][c] =
// alpha * sum_{p < parts} part[(p * segments + s) * cols + c], added in a fixed order; stretches
// with a null output are skipped.
struct SumOuts {
  float* p[3];
};
cudaError_t launch_sum_parts(const float* part, int parts, int64_t cols, int segments, float alpha,
                             const SumOuts& outs, cudaStream_t st);

}  // namespace kda
