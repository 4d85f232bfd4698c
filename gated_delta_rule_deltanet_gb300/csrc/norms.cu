// norms.cu -- residual_norm: the norm of a block's output, its gate and residual scale, the
// residual add and the norm before the next block in one pass, forward and backward.
//
// With rms(a) = a r, r = 1 / sqrt(mean(a^2) + eps), and d the gradient w.r.t. rms(a),
//
//     rms'(a)^T d = r (d - rms(a) mean(d rms(a))),
//
// so a row's gradient needs the row's two sums, sum a^2 and sum d a, before any element.
//
// Bound by HBM: some ten fp32 operations an element forward (25 backward) against 8 to 20 bytes.  A
// row belongs to one CTA and crosses HBM once: it waits in shared memory (RowRing) or registers
// from its load to its store.  The column sums (gradients of weights and of a learned gate) are
// kept in registers over all rows of a CTA and written once as partial rows, which a second
// kernel adds in a fixed order: no atomics, the same bits every time.  Sums and norms are fp32.
// Residual add and norm of 32768 x 4096 bf16: 161 us, 98% of the measured copy rate; backward of
// 16384 x 2048 with a norm after the block and a gate a token: 112 us, 71%.
#include <algorithm>

#include "layer_common.cuh"
#include "tc_utils.cuh"

namespace kda {

// ---------------------------------------------------------------- partial rows

// the stretches that have an output, and their places in a partial row
struct LiveOuts {
  float* p[3];
  int at[3];
};

// A block adds 8 columns (one sector of each partial row) with 32 row lanes: some 20 loads a thread
// for the 608 partial rows of 2048 columns (up to 2432 rows of 256), 8 of them in flight (15 us with 32 columns and
// 8 row lanes, 4 us so).
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts,
                                                        int64_t cols, int segments, float alpha,
                                                        LiveOuts outs) {
  __shared__ float s[32][9];
  const int col = threadIdx.x & 7, row = threadIdx.x >> 3;
  float* out = outs.p[blockIdx.y];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + col;
  const int64_t stride = cols * segments;
  const float* src = part + outs.at[blockIdx.y] * cols + c;
  float a = 0.f;
  if (c < cols) {
    for (int p = row; p < parts; p += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = p + 32 * u < parts ? src[(p + 32 * u) * stride] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
  }
  s[row][col] = a;
  __syncthreads();
  if (row == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][col];
    out[c] = alpha * t;
  }
}

cudaError_t launch_sum_parts(const float* part, int parts, int64_t cols, int segments, float alpha,
                             const SumOuts& outs, cudaStream_t st) {
  LiveOuts live{};
  int n = 0;
  for (int i = 0; i < segments; ++i)
    if (outs.p[i]) {
      live.p[n] = outs.p[i];
      live.at[n++] = i;
    }
  if (n == 0 || cols == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((cols + 7) / 8), static_cast<unsigned>(n));
  sum_parts_kernel<<<grid, 256, 0, st>>>(part, parts, cols, segments, alpha, live);
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
  int32_t* err;
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

// ---------------------------------------------------------------- rows through a shared-memory ring

// Rows of a multiple of 8 elements, 16-byte aligned: a CTA walks its rows through a ring of 2 to 4
// stages, each holding one row of every input array, filled by bulk copies that one thread
// issues a full ring ahead.  HBM's latency is hidden by the ring instead of by registers and
// occupancy: with the row in registers the forward took 186 us instead of 161 (32768 x 4096), the
// backward 194 instead of 112 (16384 x 2048).
struct RowRing {
  uint32_t x, r, g, dy, dh;      // byte offsets inside a stage
  uint32_t stage;                // bytes of a stage
  uint32_t xrow, hrow;           // bytes of a row of x's and of h's type
  int32_t stages;
  int32_t* err;
};
constexpr int kMaxStages = 4;
constexpr size_t kRingBytes = 208 * 1024;
#ifndef KDA_ROW_WAIT
#define KDA_ROW_WAIT (1u << 22)
#endif
constexpr uint32_t kRowWait = KDA_ROW_WAIT;      // polls of a wait for a row (tests compile one that gives up)
constexpr uint32_t kDrainWait = 1u << 22;        // and of a wait for copies in flight after one gave up

template <bool BF>
__device__ __forceinline__ Raw8<BF> smem_chunk(const unsigned char* row, int c, int n) {
  Raw8<BF> r;
  if (8 * c < n) {
    const uint4* p = reinterpret_cast<const uint4*>(row + c * (BF ? 16 : 32));
    const uint4 a = p[0];
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    if constexpr (!BF) {
      const uint4 b = p[1];
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
  } else {
    r.zero();
  }
  return r;
}

// One thread's copies of row t into a stage.
template <bool BWD>
__device__ __forceinline__ void fetch_row(const ResidualNormArgs& A, const RowRing& R, int64_t t, uint32_t at,
                                          bool need_x, uint64_t* bar) {
  auto row = [&](const void* base, int64_t bytes) { return static_cast<const char*>(base) + t * bytes; };
  uint32_t bytes = 0;
  if (!BWD || need_x) bytes += R.xrow;
  if (BWD ? A.dy != nullptr : A.res != nullptr) bytes += R.hrow;
  if (A.gate_per_token) bytes += R.xrow;
  if (BWD && A.dy) bytes += R.xrow;
  if (BWD && A.dh) bytes += R.hrow;
  tc::mbar_arrive_expect_tx(bar, bytes);
  if (!BWD || need_x) tc::bulk_load(at + R.x, row(A.x, R.xrow), R.xrow, bar);
  if (BWD ? A.dy != nullptr : A.res != nullptr) tc::bulk_load(at + R.r, row(A.res, R.hrow), R.hrow, bar);
  if (A.gate_per_token) tc::bulk_load(at + R.g, row(A.gate, A.gate_stride * (R.xrow / A.N)), R.xrow, bar);
  if (BWD && A.dy) tc::bulk_load(at + R.dy, row(A.dy, R.xrow), R.xrow, bar);
  if (BWD && A.dh) tc::bulk_load(at + R.dh, row(A.dh, R.hrow), R.hrow, bar);
}

// The ring's part of a row loop: `full` holds the row, `empty` says every warp has read it.
struct RingState {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int fail;
  int fetched;                   // rows requested so far (thread 0's)
};

template <bool BWD>
__device__ __forceinline__ void ring_start(const ResidualNormArgs& A, const RowRing& R, RingState& S, uint32_t smem,
                                           bool need_x) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < R.stages; ++s) {
      tc::mbar_init(&S.full[s], 1);
      tc::mbar_init(&S.empty[s], blockDim.x >> 5);
    }
    S.fail = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t t = blockIdx.x;
    int s = 0;
    for (; s < R.stages && t < A.T; ++s, t += gridDim.x)
      fetch_row<BWD>(A, R, t, smem + s * R.stage, need_x, &S.full[s]);
    S.fetched = s;
  }
}

// Before row `it` (stage s): the stage that row it - 1 left is refilled, then row `it` awaited.  A
// wait that gives up raises the error word and ends the waiting of the whole block, whose
// remaining rows are then incomplete.
template <bool BWD>
__device__ __forceinline__ void ring_row(const ResidualNormArgs& A, const RowRing& R, RingState& S, uint32_t smem,
                                         bool need_x, int64_t t, int it, int s, uint32_t ph) {
  volatile int* fail = &S.fail;
  if (*fail) return;
  bool ok = true;
  if (threadIdx.x == 0 && it > 0) {
    const int64_t next = t + static_cast<int64_t>(R.stages - 1) * gridDim.x;
    if (next < A.T) {
      const int p = s == 0 ? R.stages - 1 : s - 1;
      ok = tc::mbar_wait_bounded(&S.empty[p], s == 0 ? ph ^ 1 : ph, kRowWait);
      if (ok) {
        fetch_row<BWD>(A, R, next, smem + p * R.stage, need_x, &S.full[p]);
        ++S.fetched;
      }
    }
  }
  if (!(tc::mbar_wait_bounded(&S.full[s], ph, kRowWait) && ok)) {
    raise_device_error(R.err, KDA_DEVERR_TIMEOUT);
    *fail = 1;
  }
}

// After the last row.  Every copy has been awaited then, unless a wait gave up: the thread that
// issued the copies stays until the last ones have landed, as the block's shared memory is someone
// else's once its threads are gone.
__device__ __forceinline__ void ring_end(const RowRing& R, RingState& S) {
  volatile int* fail = &S.fail;
  if (threadIdx.x != 0 || !*fail) return;
  for (int j = S.fetched > R.stages ? S.fetched - R.stages : 0; j < S.fetched; ++j)
    tc::mbar_wait_bounded(&S.full[j % R.stages], (j / R.stages) & 1, kDrainWait);
}

template <bool XBF, bool HBF, int V>
__global__ void __launch_bounds__(V == 1 ? 128 : V == 2 ? 256 : 512)
residual_norm_ring_kernel(const ResidualNormArgs A, const RowRing R) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float s_buf[2][16][1];
  __shared__ __align__(8) RingState S;
  const int nt = blockDim.x, tid = threadIdx.x;
  const int N = A.N;
  const uint32_t smem = tc::smem_u32(ring);
  ring_start<false>(A, R, S, smem, true);
  int par = 0, it = 0, s = 0;
  uint32_t ph = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x, ++it) {
    ring_row<false>(A, R, S, smem, true, t, it, s, ph);
    const unsigned char* st = ring + s * R.stage;
    float h[V][8];
    float a = A.scale;
    if (A.post_w) {
      float sum[1] = {0.f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Raw8<XBF> x = smem_chunk<XBF>(st + R.x, tid + v * nt, N);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] += x.f32(e) * x.f32(e);
      }
      block_sums<1>(sum, s_buf[par]);
      par ^= 1;
      a *= 1.f / sqrtf(sum[0] * A.inv_n + A.eps);
    }
    float sq[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
      const Raw8<XBF> x = smem_chunk<XBF>(st + R.x, c, N);
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = a * x.f32(e);
      if (A.post_w) {
        load_params<true>(A.post_w, c, 0, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= p[e];
      }
      if (A.gate_per_token) {
        const Raw8<XBF> g = smem_chunk<XBF>(st + R.g, c, N);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= g.f32(e);
      } else if (A.gate) {
        load_params<true>(static_cast<const float*>(A.gate), c, 0, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= p[e];
      }
      if (A.res) {
        const Raw8<HBF> r = smem_chunk<HBF>(st + R.r, c, N);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] += r.f32(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq[0] += h[v][e] * h[v][e];
      if (A.out_h)
        store_chunk<HBF, true>(static_cast<char*>(A.out_h) + t * N * (HBF ? 2 : 4), c, 0, N, h[v]);
    }
    __syncwarp();
    if ((tid & 31) == 0) tc::mbar_arrive(&S.empty[s]);
    if (A.out_y) {
      block_sums<1>(sq, s_buf[par]);
      par ^= 1;
      const float rh = 1.f / sqrtf(sq[0] * A.inv_n + A.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tid + v * nt;
        float p[8], y[8];
        load_params<true>(A.w, c, 0, N, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[v][e] * rh * p[e];
        store_chunk<XBF, true>(static_cast<char*>(A.out_y) + t * N * (XBF ? 2 : 4), c, 0, N, y);
      }
    }
    if (++s == R.stages) {
      s = 0;
      ph ^= 1;
    }
  }
  ring_end(R, S);
}

template <bool XBF, bool HBF, int V>
__global__ void __launch_bounds__(V == 1 ? 128 : V == 2 ? 256 : 512, V == 1 ? 4 : V == 2 ? 2 : 1)
residual_norm_bwd_ring_kernel(const ResidualNormArgs A, const RowRing R) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float s_buf[2][16][3];
  __shared__ __align__(8) RingState S;
  const int nt = blockDim.x, tid = threadIdx.x;
  const int N = A.N;
  const bool need_x = A.post_w || A.gate;
  const bool chan = A.gate && !A.gate_per_token;
  const uint32_t smem = tc::smem_u32(ring);
  ring_start<true>(A, R, S, smem, need_x);
  float2 aw[V][4], ap[V][4], ag[V][4];         // this CTA's column sums
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) aw[v][e] = ap[v][e] = ag[v][e] = make_float2(0.f, 0.f);
  int par = 0, it = 0, s = 0;
  uint32_t ph = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x, ++it) {
    ring_row<true>(A, R, S, smem, need_x, t, it, s, ph);
    const unsigned char* st = ring + s * R.stage;
    const int64_t xo = t * N * (XBF ? 2 : 4), ho = t * N * (HBF ? 2 : 4);
    // the row's arithmetic runs on fp32 pairs (f2: two elements an instruction)
    float2 q0 = make_float2(0.f, 0.f), q1 = q0, q2 = q0;   // sum h^2, sum dy w h, sum x^2
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
      if (A.dy) {
        const Raw8<HBF> h = smem_chunk<HBF>(st + R.r, c, N);
        const Raw8<XBF> dy = smem_chunk<XBF>(st + R.dy, c, N);
        float2 p[4];
        load_params2(A.w, c, N, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q0 = fma2(h.f2(e), h.f2(e), q0);
          q1 = fma2(mul2(dy.f2(e), p[e]), h.f2(e), q1);
        }
      }
      if (A.post_w) {
        const Raw8<XBF> x = smem_chunk<XBF>(st + R.x, c, N);
#pragma unroll
        for (int e = 0; e < 4; ++e) q2 = fma2(x.f2(e), x.f2(e), q2);
      }
    }
    float s3[3] = {q0.x + q0.y, q1.x + q1.y, q2.x + q2.y};
    block_sums<3>(s3, s_buf[par]);
    par ^= 1;
    const float rh = 1.f / sqrtf(s3[0] * A.inv_n + A.eps);
    const float mh = s3[1] * A.inv_n * rh * rh;            // mean(d rms(h)) r
    const float rx = A.post_w ? 1.f / sqrtf(s3[2] * A.inv_n + A.eps) : 1.f;
    const float2 rh2 = make_float2(rh, rh), mh2 = make_float2(-mh, -mh), rx2 = make_float2(rx, rx);
    const float2 scale2 = make_float2(A.scale, A.scale);
    float2 d[V][4];                                        // dh, then du post_weight
    float2 qx = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * nt;
#pragma unroll
      for (int e = 0; e < 4; ++e) d[v][e] = make_float2(0.f, 0.f);
      if (A.dy) {
        const Raw8<HBF> h = smem_chunk<HBF>(st + R.r, c, N);
        const Raw8<XBF> dy = smem_chunk<XBF>(st + R.dy, c, N);
        float2 p[4];
        load_params2(A.w, c, N, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 hh = h.f2(e), dd = dy.f2(e);
          aw[v][e] = fma2(dd, mul2(hh, rh2), aw[v][e]);
          d[v][e] = mul2(rh2, fma2(hh, mh2, mul2(dd, p[e])));
        }
      }
      if (A.dh) {
        const Raw8<HBF> dh = smem_chunk<HBF>(st + R.dh, c, N);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[v][e] = add2(d[v][e], dh.f2(e));
      }
      if (A.out_h) store_pairs<HBF>(static_cast<char*>(A.out_h) + ho, c, N, d[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[v][e] = mul2(d[v][e], scale2);
      if (need_x) {
        const Raw8<XBF> x = smem_chunk<XBF>(st + R.x, c, N);
        float2 xn[4], pw[4];                               // rms(x) (x without a norm)
#pragma unroll
        for (int e = 0; e < 4; ++e) xn[e] = mul2(x.f2(e), rx2);
        if (A.post_w) load_params2(A.post_w, c, N, pw);
        if (A.gate) {                                      // d_gate = scale dh u, du = scale dh gate
          float2 dg[4], gg[4];
          if (chan) {
            load_params2(static_cast<const float*>(A.gate), c, N, gg);
          } else {
            const Raw8<XBF> g = smem_chunk<XBF>(st + R.g, c, N);
#pragma unroll
            for (int e = 0; e < 4; ++e) gg[e] = g.f2(e);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dg[e] = mul2(d[v][e], A.post_w ? mul2(xn[e], pw[e]) : xn[e]);
            if (chan) ag[v][e] = add2(ag[v][e], dg[e]);
            d[v][e] = mul2(d[v][e], gg[e]);
          }
          if (!chan) store_pairs<XBF>(static_cast<char*>(A.dgate) + xo, c, N, dg);
        }
        if (A.post_w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ap[v][e] = fma2(d[v][e], xn[e], ap[v][e]);
            d[v][e] = mul2(d[v][e], pw[e]);
            qx = fma2(d[v][e], x.f2(e), qx);
          }
        }
      }
      if (!A.post_w) store_pairs<XBF>(static_cast<char*>(A.out_y) + xo, c, N, d[v]);
    }
    if (A.post_w) {
      float sx[3] = {qx.x + qx.y, 0.f, 0.f};
      block_sums<3>(sx, s_buf[par]);
      par ^= 1;
      const float mx = -sx[0] * A.inv_n * rx * rx;
      const float2 mx2 = make_float2(mx, mx);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tid + v * nt;
        const Raw8<XBF> x = smem_chunk<XBF>(st + R.x, c, N);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[v][e] = mul2(rx2, fma2(x.f2(e), mx2, d[v][e]));
        store_pairs<XBF>(static_cast<char*>(A.out_y) + xo, c, N, d[v]);
      }
    }
    __syncwarp();
    if ((tid & 31) == 0) tc::mbar_arrive(&S.empty[s]);
    if (++s == R.stages) {
      s = 0;
      ph ^= 1;
    }
  }
  ring_end(R, S);
  float* part = A.part + static_cast<int64_t>(blockIdx.x) * 3 * N;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = tid + v * nt;
    if (A.dy) store_pairs<false>(part, c, N, aw[v]);
    if (A.post_w) store_pairs<false>(part + N, c, N, ap[v]);
    if (chan) store_pairs<false>(part + 2 * N, c, N, ag[v]);
  }
}

// Threads and elements a thread: rows up to 1024 take one chunk a thread, up to 4096 two, up to
// 16384 four, so that a row's two reductions cross few warps (backward of 16384 x 2048 with one
// chunk and twice the threads: 116 against 106 us).
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

// CTAs an SM that walk the rows: bounded by registers (64 a thread forward, 128 backward)
static int rows_per_sm(int N, bool bwd) { return std::max(1, (bwd ? 512 : 1024) / row_shape(N).threads); }

static int residual_norm_bwd_grid(int64_t T, int N) {
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(T, 1), static_cast<int64_t>(sm_count()) * rows_per_sm(N, true)));
}

static bool residual_vec(const ResidualNormArgs& A, bool xbf) {
  const int64_t es = xbf ? 2 : 4;
  return A.N % 8 == 0 && al16(A.x) && al16(A.res) && al16(A.gate) && al16(A.post_w) && al16(A.w) &&
         al16(A.dy) && al16(A.dh) && al16(A.out_h) && al16(A.out_y) && al16(A.dgate) &&
         (!A.gate_per_token || A.gate_stride * es % 16 == 0);
}

// The ring of a call, or stages = 0 where rows are better read directly: with fewer than three
// rows a CTA there is nothing to run ahead of (256 bf16 rows of 4096 with a norm, a gate and an fp32 stream:
// 4.6 us directly, 5.6 us through the ring), and a stage has to fit twice.  Backward rows above 4096
// columns take the ring whenever a stage fits at all, though nothing runs ahead with one: beside the column
// sums, four chunks a thread do not fit the registers, and a row that waits in shared memory spills
// least (8192 bf16 rows of 8192 with a norm and a gate a token 329 us, 471 directly; of 16384 685 and 971).
static RowRing row_ring(const ResidualNormArgs& A, bool xbf, bool hbf, bool bwd, int grid) {
  RowRing R{};
  R.xrow = static_cast<uint32_t>(A.N) * (xbf ? 2 : 4);
  R.hrow = static_cast<uint32_t>(A.N) * (hbf ? 2 : 4);
  R.err = A.err;
  uint32_t at = 0;
  auto take = [&](bool yes, uint32_t bytes) {
    const uint32_t here = at;
    if (yes) at += bytes;
    return here;
  };
  R.x = take(!bwd || A.post_w || A.gate, R.xrow);
  R.r = take(bwd ? A.dy != nullptr : A.res != nullptr, R.hrow);
  R.g = take(A.gate_per_token, R.xrow);
  R.dy = take(bwd && A.dy, R.xrow);
  R.dh = take(bwd && A.dh, R.hrow);
  R.stage = (at + 127) / 128 * 128;
  const size_t share = kRingBytes / rows_per_sm(A.N, bwd);
  R.stages = static_cast<int>(std::min<size_t>(kMaxStages, share / R.stage));
  if (bwd && row_shape(A.N).V == 4) return R;
  if (R.stages < 2 || A.T < 3 * static_cast<int64_t>(grid)) R.stages = 0;
  return R;
}

template <typename Kernel>
static cudaError_t launch_ring(Kernel k, std::atomic<uint64_t>& raised, unsigned grid, int threads,
                               const ResidualNormArgs& A, const RowRing& R, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(R.stage) * R.stages;      // at most kRingBytes (row_ring)
  const cudaError_t e = raise_smem(k, kRingBytes, raised);
  if (e != cudaSuccess) return e;
  k<<<grid, threads, smem, st>>>(A, R);
  return cudaGetLastError();
}

template <bool XBF, bool HBF, int V, bool VEC>
static cudaError_t run_residual_norm(const ResidualNormArgs& A, bool bwd, int threads, cudaStream_t st) {
  const int grid = bwd ? residual_norm_bwd_grid(A.T, A.N)
                       : static_cast<int>(std::min<int64_t>(A.T, static_cast<int64_t>(sm_count()) * rows_per_sm(A.N, false)));
  if constexpr (VEC) {
    const RowRing R = row_ring(A, XBF, HBF, bwd, grid);
    static std::atomic<uint64_t> raised[2];      // of this instance's two kernels
    if (R.stages)
      return bwd ? launch_ring(residual_norm_bwd_ring_kernel<XBF, HBF, V>, raised[1], grid, threads, A, R, st)
                 : launch_ring(residual_norm_ring_kernel<XBF, HBF, V>, raised[0], grid, threads, A, R, st);
  }
  if (bwd) {
    residual_norm_bwd_kernel<XBF, HBF, V, VEC><<<grid, threads, 0, st>>>(A);
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
                                 void* y, int32_t* err, cudaStream_t st) {
  ResidualNormArgs A{};
  A.x = x; A.res = res; A.gate = gate; A.post_w = post_w; A.w = w; A.out_h = h; A.out_y = y;
  A.T = p.tokens; A.N = p.features;
  A.gate_per_token = gate && p.gate_per_token;
  A.gate_stride = p.gate_row_stride ? p.gate_row_stride : p.features;
  A.eps = p.eps; A.scale = p.scale; A.inv_n = 1.f / static_cast<float>(p.features);
  A.err = err;
  return launch_residual(A, p.x_dtype == KDA_DTYPE_BF16, p.h_dtype == KDA_DTYPE_BF16, false, st);
}

size_t residual_norm_bwd_workspace(const kda_norm_params_t& p) {
  return static_cast<size_t>(residual_norm_bwd_grid(p.tokens, p.features)) * 3 * p.features * 4;
}

cudaError_t launch_residual_norm_bwd(const kda_norm_params_t& p, const void* x, const void* h,
                                     const void* gate, const float* post_w, const float* w,
                                     const void* dy, const void* dh, void* dx, void* dres,
                                     void* dgate, float* dpost_w, float* dw, void* workspace,
                                     int32_t* err, cudaStream_t st) {
  ResidualNormArgs A{};
  A.x = x; A.res = h; A.gate = gate; A.post_w = post_w; A.w = w; A.dy = dy; A.dh = dh;
  A.out_h = dres; A.out_y = dx;
  A.T = p.tokens; A.N = p.features;
  A.gate_per_token = gate && p.gate_per_token;
  A.dgate = A.gate_per_token ? dgate : nullptr;
  A.gate_stride = p.gate_row_stride ? p.gate_row_stride : p.features;
  A.eps = p.eps; A.scale = p.scale; A.inv_n = 1.f / static_cast<float>(p.features);
  A.err = err;
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

}  // namespace kda
