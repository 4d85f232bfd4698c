// norms.cu -- the norms around the recurrence: residual_norm (norm of the block's output, gate,
// residual scale, residual add and the norm before the next block in one pass) and gated_norm
// (the per-head norm of the recurrence's output times its gate), forward and backward.
//
// With rms(a) = a r, r = 1 / sqrt(mean(a^2) + eps), and d the gradient w.r.t. rms(a),
//
//     rms'(a)^T d = r (d - rms(a) mean(d rms(a))),
//
// so a row's gradient needs the row's two sums, sum a^2 and sum d a, before any element.
//
// All four are bound by HBM: about ten fp32 operations an element against 6 to 20 bytes.  A row
// of residual_norm belongs to one CTA that keeps it in registers from the load to the store, so
// every array crosses HBM once; a thread holds 8 to 32 elements as 16-byte vectors, all loaded
// before the first reduction, and several CTAs share an SM so that one's loads cover another's
// reductions.  The column sums (gradients of weights and of a learned gate) are kept in
// registers over all rows of a CTA and written once as partial rows, which a second kernel adds
// in a fixed order: no atomics, the same bits every time.  Sums and norms are fp32.
#include <algorithm>

#include "layer_common.cuh"

namespace kda {

// ---------------------------------------------------------------- partial rows

__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts,
                                                        int64_t cols, float alpha, SumOuts outs) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  float* out = outs.p[blockIdx.y];
  if (!out) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t stride = cols * gridDim.y;
  const float* src = part + blockIdx.y * cols + c;
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
  if (c < cols) {
    int p = row;
    for (; p + 24 < parts; p += 32) {
      a0 += src[p * stride];
      a1 += src[(p + 8) * stride];
      a2 += src[(p + 16) * stride];
      a3 += src[(p + 24) * stride];
    }
    for (; p < parts; p += 8) a0 += src[p * stride];
  }
  s[row][lane] = (a0 + a1) + (a2 + a3);
  __syncthreads();
  if (row == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i][lane];
    out[c] = alpha * t;
  }
}

cudaError_t launch_sum_parts(const float* part, int parts, int64_t cols, int segments, float alpha,
                             const SumOuts& outs, cudaStream_t st) {
  bool any = false;
  for (int i = 0; i < segments; ++i) any = any || outs.p[i];
  if (!any || cols == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), static_cast<unsigned>(segments));
  sum_parts_kernel<<<grid, 256, 0, st>>>(part, parts, cols, alpha, outs);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- residual_norm

struct ResidualNormArgs {
  const void* x;
  const void* res;          // forward: residual; backward: h
  const void* gate;         // [N] fp32, or [T, N] of x's dtype, or null
  const float* post_w;
  const float* w;
  const void* dy;
  const void* dh;
  void* out_h;              // forward: h; backward: d_residual
  void* out_y;              // forward: y; backward: dx
  void* dgate;              // backward, per token
  float* part;              // backward: [grid][3][N] partial rows: d_weight, d_post_weight, d_gate
  int64_t T, gate_stride;
  int32_t N, gate_per_token;
  float eps, scale, inv_n;
};

// Sums of K values over the block, the same in every thread.  Buffers alternate between calls,
// so one barrier a call is enough: a buffer is rewritten only after the next call's barrier.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float (*buf)[K]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int i = 0; i < nw; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += buf[i][k];
  }
}

template <bool XBF, bool HBF, int V, bool VEC>
__global__ void __launch_bounds__(V == 1 ? 128 : V == 2 ? 256 : 512)
residual_norm_kernel(ResidualNormArgs A) {
  __shared__ float s_buf[2][16][1];
  const int nt = blockDim.x, tid = threadIdx.x, step = V * nt;
  const int N = A.N;
  int par = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x) {
    const char* xr = static_cast<const char*>(A.x) + t * N * (XBF ? 2 : 4);
    Raw8<XBF> x[V], g[V];
    Raw8<HBF> r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = load_chunk<XBF, VEC>(xr, tid + v * nt, step, N);
    if (A.res) {
      const char* rr = static_cast<const char*>(A.res) + t * N * (HBF ? 2 : 4);
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] = load_chunk<HBF, VEC>(rr, tid + v * nt, step, N);
    }
    if (A.gate_per_token) {
      const char* gr = static_cast<const char*>(A.gate) + t * A.gate_stride * (XBF ? 2 : 4);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = load_chunk<XBF, VEC>(gr, tid + v * nt, step, N);
    }
    float h[V][8];
    float a = A.scale;
    if (A.post_w) {
      float sum[1] = {0.f};
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] += x[v].f32(e) * x[v].f32(e);
      block_sums<1>(sum, s_buf[par]);
      par ^= 1;
      a *= 1.f / sqrtf(sum[0] * A.inv_n + A.eps);
    }
    float sq[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = a * x[v].f32(e);
      if (A.post_w) {
        load_params<VEC>(A.post_w, c, step, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= p[e];
      }
      if (A.gate_per_token) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= g[v].f32(e);
      } else if (A.gate) {
        load_params<VEC>(static_cast<const float*>(A.gate), c, step, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= p[e];
      }
      if (A.res) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] += r[v].f32(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq[0] += h[v][e] * h[v][e];
      if (A.out_h)
        store_chunk<HBF, VEC>(static_cast<char*>(A.out_h) + t * N * (HBF ? 2 : 4), c, step, N, h[v]);
    }
    if (A.out_y) {
      block_sums<1>(sq, s_buf[par]);
      par ^= 1;
      const float rh = 1.f / sqrtf(sq[0] * A.inv_n + A.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tid + v * nt;
        float p[8], y[8];
        load_params<VEC>(A.w, c, step, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[v][e] * rh * p[e];
        store_chunk<XBF, VEC>(static_cast<char*>(A.out_y) + t * N * (XBF ? 2 : 4), c, step, N, y);
      }
    }
  }
}

template <bool XBF, bool HBF, int V, bool VEC>
__global__ void __launch_bounds__(V == 1 ? 128 : V == 2 ? 256 : 512)
residual_norm_bwd_kernel(ResidualNormArgs A) {
  __shared__ float s_buf[2][16][3];
  const int nt = blockDim.x, tid = threadIdx.x, step = V * nt;
  const int N = A.N;
  const bool need_x = A.post_w || A.gate;
  const bool chan = A.gate && !A.gate_per_token;
  float aw[V][8], ap[V][8], ag[V][8];          // this CTA's column sums
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[v][e] = ap[v][e] = ag[v][e] = 0.f;
  int par = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x) {
    const int64_t xo = t * N * (XBF ? 2 : 4), ho = t * N * (HBF ? 2 : 4);
    Raw8<XBF> x[V], dy[V], g[V];
    Raw8<HBF> h[V], dh[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
      if (A.dy) {
        h[v] = load_chunk<HBF, VEC>(static_cast<const char*>(A.res) + ho, c, step, N);
        dy[v] = load_chunk<XBF, VEC>(static_cast<const char*>(A.dy) + xo, c, step, N);
      }
      if (A.dh) dh[v] = load_chunk<HBF, VEC>(static_cast<const char*>(A.dh) + ho, c, step, N);
      if (need_x) x[v] = load_chunk<XBF, VEC>(static_cast<const char*>(A.x) + xo, c, step, N);
      if (A.gate_per_token)
        g[v] = load_chunk<XBF, VEC>(static_cast<const char*>(A.gate) + t * A.gate_stride * (XBF ? 2 : 4), c, step, N);
    }
    float s3[3] = {0.f, 0.f, 0.f};             // sum h^2, sum dy w h, sum x^2
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (A.dy) {
        float p[8];
        load_params<VEC>(A.w, tid + v * nt, step, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float hh = h[v].f32(e);
          s3[0] += hh * hh;
          s3[1] += dy[v].f32(e) * p[e] * hh;
        }
      }
      if (A.post_w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s3[2] += x[v].f32(e) * x[v].f32(e);
      }
    }
    block_sums<3>(s3, s_buf[par]);
    par ^= 1;
    const float rh = 1.f / sqrtf(s3[0] * A.inv_n + A.eps);
    const float mh = s3[1] * A.inv_n * rh * rh;            // mean(d rms(h)) r
    const float rx = A.post_w ? 1.f / sqrtf(s3[2] * A.inv_n + A.eps) : 1.f;
    float d[V][8];                                         // dh, then du post_weight
    float sx[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[v][e] = 0.f;
      if (A.dy) {
        load_params<VEC>(A.w, c, step, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float hh = h[v].f32(e), dd = dy[v].f32(e);
          aw[v][e] += dd * (hh * rh);
          d[v][e] = rh * (dd * p[e] - hh * mh);
        }
      }
      if (A.dh) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[v][e] += dh[v].f32(e);
      }
      if (A.out_h) store_chunk<HBF, VEC>(static_cast<char*>(A.out_h) + ho, c, step, N, d[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[v][e] *= A.scale;
      float pw[8];
      if (A.post_w) {
        load_params<VEC>(A.post_w, c, step, N, pw);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) pw[e] = 1.f;
      }
      if (A.gate) {                                        // d_gate = scale dh u, du = scale dh gate
        float dg[8], gg[8];
        if (chan) load_params<VEC>(static_cast<const float*>(A.gate), c, step, N, gg);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dg[e] = d[v][e] * (x[v].f32(e) * rx * pw[e]);
          if (chan) ag[v][e] += dg[e];
          else gg[e] = g[v].f32(e);
          d[v][e] *= gg[e];
        }
        if (!chan) store_chunk<XBF, VEC>(static_cast<char*>(A.dgate) + xo, c, step, N, dg);
      }
      if (A.post_w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xx = x[v].f32(e);
          ap[v][e] += d[v][e] * (xx * rx);
          d[v][e] *= pw[e];
          sx[0] += d[v][e] * xx;
        }
      } else {
        store_chunk<XBF, VEC>(static_cast<char*>(A.out_y) + xo, c, step, N, d[v]);
      }
    }
    if (A.post_w) {
      block_sums<3>(sx, s_buf[par]);
      par ^= 1;
      const float mx = sx[0] * A.inv_n * rx * rx;
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[v][e] = rx * (d[v][e] - x[v].f32(e) * mx);
        store_chunk<XBF, VEC>(static_cast<char*>(A.out_y) + xo, tid + v * nt, step, N, d[v]);
      }
    }
  }
  float* part = A.part + static_cast<int64_t>(blockIdx.x) * 3 * N;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = tid + v * nt;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = chunk_index<VEC>(c, step, e);
      if (i < N) {
        if (A.dy) part[i] = aw[v][e];
        if (A.post_w) part[N + i] = ap[v][e];
        if (chan) part[2 * N + i] = ag[v][e];
      }
    }
  }
}

// Threads and elements a thread: rows up to 1024 take one chunk a thread, up to 4096 two, up to
// 16384 four (two chunks of each array in flight a thread, with 64 registers and four CTAs of 256
// an SM, cover HBM's latency where one chunk and 512 threads did not).
struct RowShape {
  int V, threads;
};
static RowShape row_shape(int N) {
  const int chunks = (N + 7) / 8;
  const int V = chunks <= 128 ? 1 : chunks <= 512 ? 2 : 4;
  const int th = ((chunks + V - 1) / V + 31) / 32 * 32;
  return {V, th};
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static int residual_norm_bwd_grid(int64_t T, int N) {
  const RowShape s = row_shape(N);
  const int per_sm = std::max(1, 512 / s.threads);
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(T, 1), static_cast<int64_t>(sm_count()) * per_sm));
}

static bool residual_vec(const ResidualNormArgs& A, bool xbf) {
  const int64_t es = xbf ? 2 : 4;
  return A.N % 8 == 0 && al16(A.x) && al16(A.res) && al16(A.gate) && al16(A.post_w) && al16(A.w) &&
         al16(A.dy) && al16(A.dh) && al16(A.out_h) && al16(A.out_y) && al16(A.dgate) &&
         (!A.gate_per_token || A.gate_stride * es % 16 == 0);
}

template <bool XBF, bool HBF, int V, bool VEC>
static cudaError_t run_residual_norm(const ResidualNormArgs& A, bool bwd, int threads, cudaStream_t st) {
  if (bwd) {
    residual_norm_bwd_kernel<XBF, HBF, V, VEC><<<residual_norm_bwd_grid(A.T, A.N), threads, 0, st>>>(A);
  } else {
    const int64_t cap = static_cast<int64_t>(sm_count()) * std::max(1, 2048 / threads);
    residual_norm_kernel<XBF, HBF, V, VEC><<<static_cast<unsigned>(std::min(A.T, cap)), threads, 0, st>>>(A);
  }
  return cudaGetLastError();
}

template <bool XBF, bool HBF>
static cudaError_t pick_residual_norm(const ResidualNormArgs& A, bool bwd, cudaStream_t st) {
  const RowShape s = row_shape(A.N);
  if (residual_vec(A, XBF)) {
    if (s.V == 1) return run_residual_norm<XBF, HBF, 1, true>(A, bwd, s.threads, st);
    if (s.V == 2) return run_residual_norm<XBF, HBF, 2, true>(A, bwd, s.threads, st);
    return run_residual_norm<XBF, HBF, 4, true>(A, bwd, s.threads, st);
  }
  if (s.V == 1) return run_residual_norm<XBF, HBF, 1, false>(A, bwd, s.threads, st);
  if (s.V == 2) return run_residual_norm<XBF, HBF, 2, false>(A, bwd, s.threads, st);
  return run_residual_norm<XBF, HBF, 4, false>(A, bwd, s.threads, st);
}

static cudaError_t launch_residual(const ResidualNormArgs& A, bool xbf, bool hbf, bool bwd, cudaStream_t st) {
  if (xbf) return hbf ? pick_residual_norm<true, true>(A, bwd, st) : pick_residual_norm<true, false>(A, bwd, st);
  return hbf ? pick_residual_norm<false, true>(A, bwd, st) : pick_residual_norm<false, false>(A, bwd, st);
}

cudaError_t launch_residual_norm(const kda_norm_params_t& p, const void* x, const void* res,
                                 const void* gate, const float* post_w, const float* w, void* h,
                                 void* y, cudaStream_t st) {
  ResidualNormArgs A{};
  A.x = x; A.res = res; A.gate = gate; A.post_w = post_w; A.w = w; A.out_h = h; A.out_y = y;
  A.T = p.tokens; A.N = p.features;
  A.gate_per_token = gate && p.gate_per_token;
  A.gate_stride = p.gate_row_stride ? p.gate_row_stride : p.features;
  A.eps = p.eps; A.scale = p.scale; A.inv_n = 1.f / static_cast<float>(p.features);
  return launch_residual(A, p.x_dtype == KDA_DTYPE_BF16, p.h_dtype == KDA_DTYPE_BF16, false, st);
}

size_t residual_norm_bwd_workspace(const kda_norm_params_t& p) {
  return static_cast<size_t>(residual_norm_bwd_grid(p.tokens, p.features)) * 3 * p.features * 4;
}

cudaError_t launch_residual_norm_bwd(const kda_norm_params_t& p, const void* x, const void* h,
                                     const void* gate, const float* post_w, const float* w,
                                     const void* dy, const void* dh, void* dx, void* dres,
                                     void* dgate, float* dpost_w, float* dw, void* workspace,
                                     cudaStream_t st) {
  ResidualNormArgs A{};
  A.x = x; A.res = h; A.gate = gate; A.post_w = post_w; A.w = w; A.dy = dy; A.dh = dh;
  A.out_h = dres; A.out_y = dx;
  A.T = p.tokens; A.N = p.features;
  A.gate_per_token = gate && p.gate_per_token;
  A.dgate = A.gate_per_token ? dgate : nullptr;
  A.gate_stride = p.gate_row_stride ? p.gate_row_stride : p.features;
  A.eps = p.eps; A.scale = p.scale; A.inv_n = 1.f / static_cast<float>(p.features);
  A.part = static_cast<float*>(workspace);
  if (p.tokens == 0) {                          // sums over no tokens
    const size_t bytes = static_cast<size_t>(p.features) * 4;
    cudaError_t z = cudaSuccess;
    if (w) z = cudaMemsetAsync(dw, 0, bytes, st);
    if (z == cudaSuccess && post_w) z = cudaMemsetAsync(dpost_w, 0, bytes, st);
    if (z == cudaSuccess && gate && !p.gate_per_token) z = cudaMemsetAsync(dgate, 0, bytes, st);
    return z;
  }
  cudaError_t e = launch_residual(A, p.x_dtype == KDA_DTYPE_BF16, p.h_dtype == KDA_DTYPE_BF16, true, st);
  if (e != cudaSuccess) return e;
  const int parts = residual_norm_bwd_grid(p.tokens, p.features);
  const SumOuts outs{{dy ? dw : nullptr, post_w ? dpost_w : nullptr,
                      gate && !A.gate_per_token ? static_cast<float*>(dgate) : nullptr}};
  return launch_sum_parts(A.part, parts, p.features, 3, 1.f, outs, st);
}

// ---------------------------------------------------------------- gated_norm

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

template <bool OBF, bool GBF, bool YBF, int LPR, int VPL, bool VEC>
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
            y[e] = o[u][v].f32(e) * rs * w[v][e] * act_f<YBF>(A.act, g[u][v].f32(e));
          store_chunk<YBF, VEC>(static_cast<char*>(A.out) + row * D * (YBF ? 2 : 4), c0 + v * lpr, step, D, y);
        }
      }
    }
  }
}

template <bool OBF, bool GBF, bool YBF, int LPR, int VPL, bool VEC>
__global__ void __launch_bounds__(256) gated_norm_bwd_kernel(GatedNormArgs A) {
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
          if (A.act == KDA_ACT_NONE) {
            a = gg; da = 1.f;
          } else {
            const float p = sigmoid_f<GBF>(gg), q = sigmoid_f<GBF>(-gg);
            const bool silu = A.act == KDA_ACT_SILU;
            a = silu ? (gg == -INFINITY ? 0.f : gg * p) : p;
            da = silu ? (fabsf(gg) > 3e38f ? p : p * (1.f + gg * q)) : p * q;
          }
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
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, static_cast<int64_t>(sm_count()) * (bwd ? 4 : 8))));
}

template <bool OBF, bool GBF, bool YBF, int LPR, int VPL, bool VEC>
static cudaError_t run_gated(const GatedNormArgs& A, bool bwd, cudaStream_t st) {
  const int grid = gated_grid(A.rows, A.D, bwd);
  if (bwd) gated_norm_bwd_kernel<OBF, GBF, YBF, LPR, VPL, VEC><<<grid, 256, 0, st>>>(A);
  else gated_norm_kernel<OBF, GBF, YBF, LPR, VPL, VEC><<<grid, 256, 0, st>>>(A);
  return cudaGetLastError();
}

template <bool OBF, bool GBF, bool YBF>
static cudaError_t pick_gated(const GatedNormArgs& A, bool bwd, cudaStream_t st) {
  const bool vec = A.D % 8 == 0 && al16(A.o) && al16(A.gate) && al16(A.w) && al16(A.dy) && al16(A.out) &&
                   al16(A.dgate) && A.gate_stride * (GBF ? 2 : 4) % 16 == 0;
  if (A.D > 256) return vec ? run_gated<OBF, GBF, YBF, 0, 4, true>(A, bwd, st) : run_gated<OBF, GBF, YBF, 0, 4, false>(A, bwd, st);
  if (!vec) return run_gated<OBF, GBF, YBF, 0, 1, false>(A, bwd, st);
  return A.lpr == 16 ? run_gated<OBF, GBF, YBF, 16, 1, true>(A, bwd, st) : run_gated<OBF, GBF, YBF, 0, 1, true>(A, bwd, st);
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
