// linear.cu -- projections with their epilogue (y = residual + scale act(x w^T + bias)) and their
// gradients: the fp32 product on CUDA cores, the element-wise gradient of the epilogue with the
// bias's column sums, and the choice of path.  The tensor-core product is in linear_tc.cu.
#include <algorithm>
#include <type_traits>

#include "gemm.cuh"

namespace kda {

// ---------------------------------------------------------------- fp32 product on CUDA cores

// 128 x 128 tiles of the result, 16 steps of c at a time in shared memory, 8 x 8 sums a thread
// held as fp32 pairs.  Bound by the CUDA cores' fp32 rate and its shared-memory feed (4 16-byte
// loads for 64 multiply-adds a thread and step): 32768 x 4096 x 4096 32 ms, 34 TFLOP/s.  For
// KDA_FLAG_CUDA_CORES and for sums over no tokens.  Takes any stride and alignment: every element
// is loaded by itself, consecutive lanes on consecutive addresses.
constexpr int kTile = 128, kStep = 16, kPad = kTile + 4;

template <bool BF, bool MN>
__device__ __forceinline__ void simt_fetch(const GemmOperand& X, int64_t r0, int64_t R, int64_t c0,
                                           int64_t C, float (&v)[8]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t r = r0 + (MN ? tid % kTile : tid / kStep + 16 * u);
    const int64_t c = c0 + (MN ? tid / kTile + 2 * u : tid % kStep);
    v[u] = (r < R && c < C) ? load_elem<BF>(X.p, MN ? c * X.ld + r : r * X.ld + c) : 0.f;
  }
}

template <bool MN>
__device__ __forceinline__ void simt_put(float (*s)[kPad], const float (&v)[8]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if constexpr (MN) s[tid / kTile + 2 * u][tid % kTile] = v[u];
    else s[tid % kStep][tid / kStep + 16 * u] = v[u];
  }
}

template <bool BF, bool AMN, bool BMN>
__global__ void __launch_bounds__(256) gemm_simt_kernel(Gemm g) {
  __shared__ __align__(16) float sa[2][kStep][kPad], sb[2][kStep][kPad];
  const int64_t ti = (g.I + kTile - 1) / kTile;
  const int64_t i0 = (blockIdx.x % ti) * kTile, j0 = (blockIdx.x / ti) * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float2 acc[8][4];
#pragma unroll
  for (int a = 0; a < 8; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = make_float2(0.f, 0.f);
  float va[8], vb[8];
  const int64_t nc = (g.C + kStep - 1) / kStep;
  if (nc > 0) {
    simt_fetch<BF, AMN>(g.A, i0, g.I, 0, g.C, va);
    simt_fetch<BF, BMN>(g.B, j0, g.J, 0, g.C, vb);
  }
  for (int64_t k = 0; k < nc; ++k) {
    const int buf = k & 1;
    simt_put<AMN>(sa[buf], va);
    simt_put<BMN>(sb[buf], vb);
    __syncthreads();                         // the other buffer's readers passed the last barrier
    if (k + 1 < nc) {
      simt_fetch<BF, AMN>(g.A, i0, g.I, (k + 1) * kStep, g.C, va);
      simt_fetch<BF, BMN>(g.B, j0, g.J, (k + 1) * kStep, g.C, vb);
    }
#pragma unroll
    for (int c = 0; c < kStep; ++c) {
      const float4 a0 = *reinterpret_cast<const float4*>(&sa[buf][c][tx * 4]);
      const float4 a1 = *reinterpret_cast<const float4*>(&sa[buf][c][64 + tx * 4]);
      const float4 b0 = *reinterpret_cast<const float4*>(&sb[buf][c][ty * 4]);
      const float4 b1 = *reinterpret_cast<const float4*>(&sb[buf][c][64 + ty * 4]);
      const float2 av[4] = {{a0.x, a0.y}, {a0.z, a0.w}, {a1.x, a1.y}, {a1.z, a1.w}};
      const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fma2(make_float2(bv[a], bv[a]), av[b], acc[a][b]);
    }
  }
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    const int64_t j = j0 + (a >> 2) * 64 + ty * 4 + (a & 3);
    if (j >= g.J) continue;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t i = i0 + (b >> 1) * 64 + tx * 4 + (b & 1) * 2;
      if (i < g.I) epilogue_store(g.epi, j, i, acc[a][b].x);
      if (i + 1 < g.I) epilogue_store(g.epi, j, i + 1, acc[a][b].y);
    }
  }
}

cudaError_t launch_gemm_simt(const Gemm& g, cudaStream_t st) {
  const int64_t tiles = ((g.I + kTile - 1) / kTile) * ((g.J + kTile - 1) / kTile);
  if (tiles == 0) return cudaSuccess;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned n = static_cast<unsigned>(tiles);
  const int sel = (g.bf16 ? 4 : 0) | (g.A.mn ? 2 : 0) | (g.B.mn ? 1 : 0);
  switch (sel) {
    case 0: gemm_simt_kernel<false, false, false><<<n, 256, 0, st>>>(g); break;
    case 1: gemm_simt_kernel<false, false, true><<<n, 256, 0, st>>>(g); break;
    case 2: gemm_simt_kernel<false, true, false><<<n, 256, 0, st>>>(g); break;
    case 3: gemm_simt_kernel<false, true, true><<<n, 256, 0, st>>>(g); break;
    case 4: gemm_simt_kernel<true, false, false><<<n, 256, 0, st>>>(g); break;
    case 5: gemm_simt_kernel<true, false, true><<<n, 256, 0, st>>>(g); break;
    case 6: gemm_simt_kernel<true, true, false><<<n, 256, 0, st>>>(g); break;
    default: gemm_simt_kernel<true, true, true><<<n, 256, 0, st>>>(g); break;
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient of the epilogue

// dz = act'(z) d_y (the scale is applied to the sums), rounded to the operand type where a
// product reads it, or as the three parts of fp32, and the column sums of the unrounded dz for the
// bias.  The rounding is a choice: the tensor cores take bf16 operands, and keeping dz's rest in a
// second plane would double both products.  It costs a rounding beside the results' own: dx and dw of
// 4096 x 2048 -> 4096 with SiLU are 2.35e-3 of their norm off instead of 1.66e-3.  A caller who wants the
// rest passes fp32 operands.
// Bound by HBM without an activation: d_y read once (the sums alone over 16384 x 6144: 43 us, 4.7
// TB/s); with one, by issue slots too (71 % of them; SiLU with dz written 106 us, 5.4 TB/s, gelu's sums alone
// 139 us).  A block walks 256 columns (8 a lane) with eight row lanes whose sums meet in shared
// memory; it writes one partial row, added in a fixed order afterwards.
struct DzArgs {
  const void* dy;
  const void* z;        // null: no activation
  void* dz;             // null: only the column sums
  int64_t plane;        // > 0: dz is three planes of bf16 parts, this many elements apart
  float* part;          // [gridDim.y][N] or null
  int64_t T, dy_ld, dz_ld;
  int32_t N, act;
};

// The activation is fixed at compile time; without one (the sums alone, or a copy) eight rows are in
// flight instead of four.
template <bool DYBF, bool ZBF, bool VEC, int ACT>
__global__ void __launch_bounds__(256) dz_kernel(DzArgs A) {
  __shared__ float s[8][256 + 8];
  const int lane = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n0 = blockIdx.x * 256, n = min(256, A.N - n0);
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  const int64_t stride = static_cast<int64_t>(gridDim.y) * 8;
  constexpr int U = ACT != KDA_ACT_NONE ? 4 : 8;
  for (int64_t t = static_cast<int64_t>(blockIdx.y) * 8 + ry; t < A.T; t += U * stride) {
    Raw8<DYBF> dy[U];
    Raw8<ZBF> z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * stride;
      const int m = tu < A.T ? n : 0;
      const int64_t tt = tu < A.T ? tu : 0;
      dy[u] = load_chunk<DYBF, VEC>(static_cast<const char*>(A.dy) + (tt * A.dy_ld + n0) * (DYBF ? 2 : 4), lane, 32, m);
      if constexpr (ACT != KDA_ACT_NONE)
        z[u] = load_chunk<ZBF, VEC>(static_cast<const char*>(A.z) + (tt * A.N + n0) * (ZBF ? 2 : 4), lane, 32, m);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * stride;
      if (tu >= A.T) break;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = dy[u].f32(e);
        if constexpr (ACT != KDA_ACT_NONE) d[e] *= act_grad_f<ACT, ZBF>(z[u].f32(e));
        sum[e] += chunk_index<VEC>(lane, 32, e) < n ? d[e] : 0.f;
      }
      if (A.dz && (ZBF || A.plane == 0)) {
        store_chunk<ZBF, VEC>(static_cast<char*>(A.dz) + (tu * A.dz_ld + n0) * (ZBF ? 2 : 4), lane, 32, n, d);
      } else if (A.dz) {
        float part[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint16_t q[3];
          split3(d[e], q);
#pragma unroll
          for (int p = 0; p < 3; ++p) part[p][e] = bf16_bits_to_f32(q[p]);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
          store_chunk<true, VEC>(static_cast<uint16_t*>(A.dz) + p * A.plane + tu * A.dz_ld + n0, lane, 32, n, part[p]);
      }
    }
  }
  if (!A.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) s[ry][chunk_index<VEC>(lane, 32, e)] = sum[e];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < n) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) t += s[r][c];
    A.part[static_cast<int64_t>(blockIdx.y) * A.N + n0 + c] = t;
  }
}

static int dz_rows(int64_t T, int N) {                    // blocks along the tokens
  const int64_t cols = (N + 255) / 256;
  const int64_t want = std::max<int64_t>(1, static_cast<int64_t>(sm_count()) * 6 / cols);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, (T + 7) / 8)));
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ZBF: the operand type (of z and dz)
template <bool DYBF, bool ZBF>
static cudaError_t launch_dz_t(const DzArgs& A, cudaStream_t st) {
  const bool vec = A.N % 8 == 0 && al16(A.dy) && al16(A.z) && al16(A.dz) &&
                   A.dy_ld * (DYBF ? 2 : 4) % 16 == 0 && A.dz_ld * (ZBF ? 2 : 4) % 16 == 0 && A.plane % 8 == 0;
  const dim3 grid(static_cast<unsigned>((A.N + 255) / 256), static_cast<unsigned>(dz_rows(A.T, A.N)));
  auto run = [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    if (vec) dz_kernel<DYBF, ZBF, true, ACT><<<grid, 256, 0, st>>>(A);
    else dz_kernel<DYBF, ZBF, false, ACT><<<grid, 256, 0, st>>>(A);
  };
  switch (A.z ? A.act : KDA_ACT_NONE) {
    case KDA_ACT_RELU: run(std::integral_constant<int, KDA_ACT_RELU>()); break;
    case KDA_ACT_SILU: run(std::integral_constant<int, KDA_ACT_SILU>()); break;
    case KDA_ACT_GELU: run(std::integral_constant<int, KDA_ACT_GELU>()); break;
    case KDA_ACT_SIGMOID: run(std::integral_constant<int, KDA_ACT_SIGMOID>()); break;
    default: run(std::integral_constant<int, KDA_ACT_NONE>()); break;
  }
  return cudaGetLastError();
}

static cudaError_t launch_dz(const DzArgs& A, bool dybf, bool zbf, cudaStream_t st) {
  if (dybf) return zbf ? launch_dz_t<true, true>(A, st) : launch_dz_t<true, false>(A, st);
  return zbf ? launch_dz_t<false, true>(A, st) : launch_dz_t<false, false>(A, st);
}

// ---------------------------------------------------------------- path and workspace

static int64_t or_dense(int64_t stride, int64_t dense) { return stride ? stride : dense; }
static size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// What a call keeps in the workspace (offsets; kNone: nothing).  The tensor cores read aligned
// bf16 rows: bf16 operands as they are where their rows and base are 16-byte aligned, else a
// copy; fp32 operands always as three planes of parts.  The CUDA cores' forward of few tokens
// reads everything in place.
constexpr size_t kNone = ~static_cast<size_t>(0);
struct LinearLayout {
  bool rows, tc;             // few tokens; tensor cores
  size_t part, dz, x, w, total;
  int64_t dz_ld, dz_plane;
};
static LinearLayout linear_layout(const kda_linear_params_t& p, bool bwd) {
  const int64_t T = p.tokens, K = p.in_features, N = p.out_features;
  const bool bf = p.dtype == KDA_DTYPE_BF16;
  LinearLayout L{};
  const bool copy_x = !bf || (p.flags & KDA_FLAG_UNALIGNED_X) || or_dense(p.x_row_stride, K) % 8;
  const bool copy_w = !bf || (p.flags & KDA_FLAG_UNALIGNED_W) || or_dense(p.w_row_stride, K) % 8;
  // Few tokens: from three on the tensor cores' ring streams an aligned bf16 weight faster (4 x 4096 ->
  // 16384 from HBM: 33 against 28 us), but a copy of the weight would cost more than reading it.
  L.rows = !bwd && !(p.flags & KDA_FLAG_CUDA_CORES) && (T <= 2 || (T <= kRowsMax && copy_w));
  L.tc = !L.rows && !(p.flags & KDA_FLAG_CUDA_CORES);
  size_t at = 0;
  auto take = [&](bool yes, size_t bytes) {
    if (!yes) return kNone;
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  L.x = take(L.tc && copy_x, repacked_bytes(T, K, bf));
  L.w = take(L.tc && copy_w, repacked_bytes(N, K, bf));
  L.dz = L.part = kNone;
  if (bwd) {
    L.part = take(true, static_cast<size_t>(dz_rows(T, p.out_features)) * N * 4);
    // dz is formed unless the products can read d_y itself
    const bool unaligned = L.tc && bf && ((p.flags & KDA_FLAG_UNALIGNED_DY) || or_dense(p.y_row_stride, N) % 8);
    L.dz_ld = padded(N);
    L.dz_plane = L.tc && !bf ? T * L.dz_ld : 0;
    L.dz = take(p.activation != KDA_ACT_NONE || p.y_dtype != p.dtype || unaligned || L.dz_plane,
                L.dz_plane ? repacked_bytes(T, N, false) : static_cast<size_t>(T) * L.dz_ld * dtype_bytes(p.dtype));
  }
  L.total = at;
  return L;
}

size_t linear_workspace_bytes(const kda_linear_params_t& p, bool bwd) { return linear_layout(p, bwd).total; }

// The operands as the products read them: copied into the workspace where the layout says so, in
// one launch.
struct Stage {
  Repack a[2];
  int n = 0;
  void add(GemmOperand* X, size_t at, char* ws, int64_t rows, int64_t cols) {
    if (at == kNone) return;
    a[n++] = {X->p, X->ld, rows, cols, ws + at};
    X->p = ws + at;
    X->ld = padded(cols);
  }
  cudaError_t run(bool bf16, cudaStream_t st) const { return n ? launch_repack(a, n, bf16, st) : cudaSuccess; }
};

static cudaError_t run_gemm(const Gemm& g, bool tc, cudaStream_t st) {
  return tc && g.C > 0 ? launch_gemm_tc(g, g.bf16 ? 1 : 3, st) : launch_gemm_simt(g, st);
}

cudaError_t launch_linear_fwd(const kda_linear_params_t& p, const void* x, const void* w, const float* bias,
                              const void* res, void* y, void* z, void* workspace, int32_t* err,
                              cudaStream_t st) {
  const int64_t T = p.tokens, K = p.in_features, N = p.out_features;
  if (T == 0) return cudaSuccess;
  const LinearLayout L = linear_layout(p, false);
  char* ws = static_cast<char*>(workspace);
  cudaError_t e;
  Gemm g{};
  g.bf16 = p.dtype == KDA_DTYPE_BF16;
  g.A = {w, or_dense(p.w_row_stride, K), false};
  g.B = {x, or_dense(p.x_row_stride, K), false};
  Stage copies;
  copies.add(&g.A, L.w, ws, N, K);
  copies.add(&g.B, L.x, ws, T, K);
  if ((e = copies.run(g.bf16, st)) != cudaSuccess) return e;
  g.I = N; g.J = T; g.C = K;
  g.epi = {bias, res, y, z, or_dense(p.residual_row_stride, N), or_dense(p.y_row_stride, N), N, p.scale,
           p.activation, p.residual_dtype == KDA_DTYPE_BF16, p.y_dtype == KDA_DTYPE_BF16, g.bf16};
  g.err = err;
  return L.rows ? launch_gemm_rows(g, st) : run_gemm(g, L.tc, st);
}

cudaError_t launch_linear_bwd(const kda_linear_params_t& p, const void* x, const void* w, const void* z,
                              const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                              int32_t* err, cudaStream_t st) {
  const int64_t T = p.tokens, K = p.in_features, N = p.out_features;
  const bool bf = p.dtype == KDA_DTYPE_BF16, any = T > 0;
  const LinearLayout L = linear_layout(p, true);
  char* ws = static_cast<char*>(workspace);
  GemmOperand dz{dy, or_dense(p.y_row_stride, N), false};
  cudaError_t e;
  const bool form = L.dz != kNone && (dx || dw) && any;
  if (form || dbias) {
    DzArgs A{};
    A.dy = dy; A.z = p.activation != KDA_ACT_NONE ? z : nullptr;
    A.dz = form ? ws + L.dz : nullptr;
    A.part = dbias ? reinterpret_cast<float*>(ws + L.part) : nullptr;
    A.T = T; A.dy_ld = dz.ld; A.dz_ld = L.dz_ld; A.N = p.out_features; A.act = p.activation;
    A.plane = L.dz_plane;
    if ((e = launch_dz(A, p.y_dtype == KDA_DTYPE_BF16, bf, st)) != cudaSuccess) return e;
    if (dbias && (e = launch_sum_parts(A.part, dz_rows(T, p.out_features), N, 1, p.scale,
                                       SumOuts{{dbias, nullptr, nullptr}}, st)) != cudaSuccess)
      return e;
    if (form) dz = {ws + L.dz, L.dz_ld, false};
  }
  GemmOperand wt{w, or_dense(p.w_row_stride, K), true}, xt{x, or_dense(p.x_row_stride, K), true};
  Stage copies;
  if (dx && any) copies.add(&wt, L.w, ws, N, K);
  if (dw && any) copies.add(&xt, L.x, ws, T, K);
  if ((e = copies.run(bf, st)) != cudaSuccess) return e;
  Gemm g{};
  g.bf16 = bf;
  g.err = err;
  g.epi = {nullptr, nullptr, nullptr, nullptr, 0, K, 0, p.scale, KDA_ACT_NONE, false, bf, false};
  if (dx && any) {
    g.A = wt;
    g.B = dz;
    g.I = K; g.J = T; g.C = N;
    g.epi.out = dx;
    if ((e = run_gemm(g, L.tc, st)) != cudaSuccess) return e;
  }
  if (dw) {
    g.A = xt;
    g.B = {dz.p, dz.ld, true};
    g.I = K; g.J = N; g.C = T;
    g.epi.out = dw;
    g.epi.out_bf = p.dw_dtype == KDA_DTYPE_BF16;
    if ((e = run_gemm(g, L.tc, st)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
