// gated_norm.cu -- the output norm of the recurrence: the RMS norm of every token's and head's row
// of o, times weight, times act(gate), forward and backward (rms' as in norms.cu).
//
// Bound by HBM: 8 bytes an element forward with an fp32 o and bf16 gate and y, 14 backward.  32768
// tokens x 32 heads x 128: 172 us, 92% of the measured copy rate; backward of 16384 x 16 x 128: 87 us,
// 80% (59% of the issue slots, most of them for the gate's exponential and the conversions; three blocks an
// SM leave 80 registers a thread, with 36 bytes spilled there and up to 112 in fp32).
#include <algorithm>

#include "layer_common.cuh"

namespace kda {

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct GatedNormArgs {
  const void* o;
  const void* gate;
  const float* w;
  const void* dy;
  void* out;                // forward: y; backward: d_o
  void* dgate;
  float* part;              // [grid][D]
  int64_t gate_stride;      // elements between tokens
  uint32_t rows;            // T * H
  int32_t H, D, act, lpr;   // lpr: lanes of a row, a power of two <= 32
  float eps, inv_d;
};

// A row is read by `lpr` lanes of a warp (8 elements a lane and chunk, VPL chunks a lane), so a
// warp works on 32 / lpr rows at a time and U such groups at once: with the head size 128 that
// is 8 rows, 12 16-byte loads a lane in flight (o fp32, gate bf16) before the first reduction.
// LPR = 16 (head sizes 65..128) fixes the lane count at compile time; LPR = 0 reads it from the
// arguments (other head sizes).
template <int LPR>
__device__ __forceinline__ float row_sum(float v, int lpr) {
  if constexpr (LPR > 0) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  } else {
    for (int off = lpr / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

// act(gate) and its derivative; the gate itself for KDA_ACT_NONE
template <int ACT, bool FAST>
__device__ __forceinline__ float gate_f(float z) {
  if constexpr (ACT == KDA_ACT_NONE) return z;
  const float p = sigmoid_f<FAST>(z);
  if constexpr (ACT == KDA_ACT_SIGMOID) return p;
  return z < -100.f ? 0.f : z * p;              // below e^-95: also -infinity
}
template <int ACT, bool FAST>
__device__ __forceinline__ void gate_grad_f(float z, float& a, float& da) {
  if constexpr (ACT == KDA_ACT_NONE) {
    a = z;
    da = 1.f;
  } else {
    float p, q;
    sigmoid_pair<FAST>(z, p, q);
    if constexpr (ACT == KDA_ACT_SIGMOID) {
      a = p;
      da = p * q;
    } else {
      a = z < -100.f ? 0.f : z * p;
      da = fabsf(z) > 100.f ? p : p * (1.f + z * q);
    }
  }
}

template <bool OBF, bool GBF, bool YBF, int ACT, int LPR, int VPL, bool VEC>
__global__ void __launch_bounds__(256) gated_norm_kernel(GatedNormArgs A) {
  constexpr int U = VPL == 1 ? 4 : 1;
  const int lpr = LPR > 0 ? LPR : A.lpr;
  const int lane = threadIdx.x & 31;
  const int rpw = 32 / lpr, sub = lane / lpr, c0 = lane % lpr;
  const int D = A.D, step = VPL * lpr;
  float w[VPL][8];
#pragma unroll
  for (int v = 0; v < VPL; ++v) load_params<VEC>(A.w, c0 + v * lpr, step, D, w[v]);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (rpw * U); base < A.rows;
       base += warps * (rpw * U)) {
    Raw8<OBF> o[U][VPL];
    Raw8<GBF> g[U][VPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u * rpw + sub;
      const bool in = row < A.rows;
      const uint32_t r = in ? static_cast<uint32_t>(row) : 0u;
      const uint32_t t = r / static_cast<uint32_t>(A.H);
      const int64_t go = t * A.gate_stride + static_cast<int64_t>(r - t * A.H) * D;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        o[u][v] = load_chunk<OBF, VEC>(static_cast<const char*>(A.o) + static_cast<int64_t>(r) * D * (OBF ? 2 : 4),
                                       c0 + v * lpr, step, in ? D : 0);
        g[u][v] = load_chunk<GBF, VEC>(static_cast<const char*>(A.gate) + go * (GBF ? 2 : 4), c0 + v * lpr, step, in ? D : 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u * rpw + sub;
      float sq = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += o[u][v].f32(e) * o[u][v].f32(e);
      sq = row_sum<LPR>(sq, lpr);
      const float rs = 1.f / sqrtf(sq * A.inv_d + A.eps);
      if (row < A.rows) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = o[u][v].f32(e) * rs * w[v][e] * gate_f<ACT, YBF>(g[u][v].f32(e));
          store_chunk<YBF, VEC>(static_cast<char*>(A.out) + row * D * (YBF ? 2 : 4), c0 + v * lpr, step, D, y);
        }
      }
    }
  }
}

template <bool OBF, bool GBF, bool YBF, int ACT, int LPR, int VPL, bool VEC>
__global__ void __launch_bounds__(256, VPL == 1 && VEC ? 3 : 1) gated_norm_bwd_kernel(GatedNormArgs A) {
  constexpr int U = VPL == 1 ? 2 : 1;
  __shared__ float s_dw[1024];
  const int lpr = LPR > 0 ? LPR : A.lpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rpw = 32 / lpr, sub = lane / lpr, c0 = lane % lpr;
  const int D = A.D, step = VPL * lpr;
  float w[VPL][8], aw[VPL][8];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    load_params<VEC>(A.w, c0 + v * lpr, step, D, w[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[v][e] = 0.f;
  }
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * (rpw * U); base < A.rows;
       base += warps * (rpw * U)) {
    Raw8<OBF> o[U][VPL];
    Raw8<GBF> g[U][VPL];
    Raw8<YBF> dy[U][VPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u * rpw + sub;
      const bool in = row < A.rows;
      const uint32_t r = in ? static_cast<uint32_t>(row) : 0u;
      const uint32_t t = r / static_cast<uint32_t>(A.H);
      const int64_t go = t * A.gate_stride + static_cast<int64_t>(r - t * A.H) * D;
      const int n = in ? D : 0;                // rows past the end add zeros
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int c = c0 + v * lpr;
        o[u][v] = load_chunk<OBF, VEC>(static_cast<const char*>(A.o) + static_cast<int64_t>(r) * D * (OBF ? 2 : 4), c, step, n);
        g[u][v] = load_chunk<GBF, VEC>(static_cast<const char*>(A.gate) + go * (GBF ? 2 : 4), c, step, n);
        dy[u][v] = load_chunk<YBF, VEC>(static_cast<const char*>(A.dy) + static_cast<int64_t>(r) * D * (YBF ? 2 : 4), c, step, n);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u * rpw + sub;
      const bool in = row < A.rows;
      float dn[VPL][8], dg[VPL][8];            // d act(gate), then its product with weight
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float oo = o[u][v].f32(e), gg = g[u][v].f32(e), d = dy[u][v].f32(e);
          float a, da;
          gate_grad_f<ACT, GBF && YBF>(gg, a, da);
          sq += oo * oo;
          dn[v][e] = d * a;
          dot += dn[v][e] * w[v][e] * oo;
          dg[v][e] = d * da * w[v][e] * oo;
        }
      sq = row_sum<LPR>(sq, lpr);
      dot = row_sum<LPR>(dot, lpr);
      const float rs = 1.f / sqrtf(sq * A.inv_d + A.eps);
      const float m = dot * A.inv_d * rs * rs;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float d_o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float oo = o[u][v].f32(e);
          aw[v][e] += dn[v][e] * (oo * rs);
          d_o[e] = rs * (dn[v][e] * w[v][e] - oo * m);
          dg[v][e] *= rs;
        }
        if (in) {
          store_chunk<OBF, VEC>(static_cast<char*>(A.out) + row * D * (OBF ? 2 : 4), c0 + v * lpr, step, D, d_o);
          store_chunk<GBF, VEC>(static_cast<char*>(A.dgate) + row * D * (GBF ? 2 : 4), c0 + v * lpr, step, D, dg[v]);
        }
      }
    }
  }
  // this block's partial row of d_weight: lanes of the same columns, then the warps in order
  for (int wv = 0; wv < 8; ++wv) {
    if (warp == wv) {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float t = aw[v][e];
          for (int off = lpr; off < 32; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
          const int i = chunk_index<VEC>(c0 + v * lpr, step, e);
          if (sub == 0 && i < D) s_dw[i] = wv == 0 ? t : s_dw[i] + t;
        }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < D; i += blockDim.x) A.part[static_cast<int64_t>(blockIdx.x) * D + i] = s_dw[i];
}

static int lanes_per_row(int D) {
  int l = 1;
  while (l < 32 && l * 8 < D) l *= 2;
  return l;
}

static int gated_grid(int64_t rows, int D, bool bwd) {
  const int lpr = lanes_per_row(D);
  const int64_t per_block = static_cast<int64_t>(32 / lpr) * 8 * (D <= 256 ? (bwd ? 2 : 4) : 1);
  const int64_t blocks = (rows + per_block - 1) / per_block;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, static_cast<int64_t>(sm_count()) * (bwd ? 3 : 8))));
}

template <bool OBF, bool GBF, bool YBF, int ACT, int LPR, int VPL, bool VEC>
static cudaError_t run_gated(const GatedNormArgs& A, bool bwd, cudaStream_t st) {
  const int grid = gated_grid(A.rows, A.D, bwd);
  if (bwd) gated_norm_bwd_kernel<OBF, GBF, YBF, ACT, LPR, VPL, VEC><<<grid, 256, 0, st>>>(A);
  else gated_norm_kernel<OBF, GBF, YBF, ACT, LPR, VPL, VEC><<<grid, 256, 0, st>>>(A);
  return cudaGetLastError();
}

template <bool OBF, bool GBF, bool YBF, int ACT>
static cudaError_t pick_gated_act(const GatedNormArgs& A, bool bwd, cudaStream_t st) {
  const bool vec = A.D % 8 == 0 && al16(A.o) && al16(A.gate) && al16(A.w) && al16(A.dy) && al16(A.out) &&
                   al16(A.dgate) && A.gate_stride * (GBF ? 2 : 4) % 16 == 0;
  if (A.D > 256) {
    if (vec) return run_gated<OBF, GBF, YBF, ACT, 0, 4, true>(A, bwd, st);
    return run_gated<OBF, GBF, YBF, ACT, 0, 4, false>(A, bwd, st);
  }
  if (!vec) return run_gated<OBF, GBF, YBF, ACT, 0, 1, false>(A, bwd, st);
  if (A.lpr == 16) return run_gated<OBF, GBF, YBF, ACT, 16, 1, true>(A, bwd, st);
  return run_gated<OBF, GBF, YBF, ACT, 0, 1, true>(A, bwd, st);
}

template <bool OBF, bool GBF, bool YBF>
static cudaError_t pick_gated(const GatedNormArgs& A, bool bwd, cudaStream_t st) {
  switch (A.act) {
    case KDA_ACT_SILU: return pick_gated_act<OBF, GBF, YBF, KDA_ACT_SILU>(A, bwd, st);
    case KDA_ACT_SIGMOID: return pick_gated_act<OBF, GBF, YBF, KDA_ACT_SIGMOID>(A, bwd, st);
    default: return pick_gated_act<OBF, GBF, YBF, KDA_ACT_NONE>(A, bwd, st);
  }
}

static cudaError_t launch_gated(const kda_norm_params_t& p, GatedNormArgs A, bool bwd, cudaStream_t st) {
  A.rows = static_cast<uint32_t>(p.tokens * p.num_heads);
  A.H = p.num_heads; A.D = p.features; A.act = p.activation;
  A.lpr = lanes_per_row(p.features);
  A.gate_stride = p.gate_row_stride ? p.gate_row_stride : static_cast<int64_t>(p.num_heads) * p.features;
  A.eps = p.eps; A.inv_d = 1.f / static_cast<float>(p.features);
  const bool ob = p.x_dtype == KDA_DTYPE_BF16, gb = p.gate_dtype == KDA_DTYPE_BF16, yb = p.y_dtype == KDA_DTYPE_BF16;
  if (ob) {
    if (gb) return yb ? pick_gated<true, true, true>(A, bwd, st) : pick_gated<true, true, false>(A, bwd, st);
    return yb ? pick_gated<true, false, true>(A, bwd, st) : pick_gated<true, false, false>(A, bwd, st);
  }
  if (gb) return yb ? pick_gated<false, true, true>(A, bwd, st) : pick_gated<false, true, false>(A, bwd, st);
  return yb ? pick_gated<false, false, true>(A, bwd, st) : pick_gated<false, false, false>(A, bwd, st);
}

cudaError_t launch_gated_norm(const kda_norm_params_t& p, const void* o, const void* gate,
                              const float* w, void* y, cudaStream_t st) {
  GatedNormArgs A{};
  A.o = o; A.gate = gate; A.w = w; A.out = y;
  return launch_gated(p, A, false, st);
}

size_t gated_norm_bwd_workspace(const kda_norm_params_t& p) {
  return static_cast<size_t>(gated_grid(p.tokens * p.num_heads, p.features, true)) * p.features * 4;
}

cudaError_t launch_gated_norm_bwd(const kda_norm_params_t& p, const void* o, const void* gate,
                                  const float* w, const void* dy, void* d_o, void* dgate, float* dw,
                                  void* workspace, cudaStream_t st) {
  GatedNormArgs A{};
  A.o = o; A.gate = gate; A.w = w; A.dy = dy; A.out = d_o; A.dgate = dgate;
  A.part = static_cast<float*>(workspace);
  const cudaError_t e = launch_gated(p, A, true, st);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(A.part, gated_grid(p.tokens * p.num_heads, p.features, true), p.features, 1,
                          1.f, SumOuts{{dw, nullptr, nullptr}}, st);
}

}  // namespace kda
