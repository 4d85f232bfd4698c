// rotary.cu -- rotary positions of queries and keys, their gradients' way back, and the same with the keys
// and values written into the pages of a cache.
//
// A pair (a, b) of a head's channels -- (i, i + R/2) or (2i, 2i + 1), i < R/2 -- at position p becomes
//
//     m (a cos - b sin),   m (b cos + a sin)       angle = p f_i
//
// the rotation of Su et al., "RoFormer" (2021), m a factor of the caller's; the channels from R on pass.  It
// is orthogonal up to m, so the gradients take the same form with -angle.
//
// The angle.  p f_i in fp32 is off by up to p 2^-24: 0.06 rad at p = 10^6.  Whole turns do not matter and p
// is an integer, so f_i / 2 pi is kept as a fraction of a turn in 64-bit fixed point and multiplied by p modulo
// 2^64: two integer multiplications, off by no more than p 2^-64 turns beside f_i's own rounding.  The two top bits
// give the quadrant, the rest an argument of at most an eighth of a turn for sincospif.
//
// Bound by HBM: every value is read and written once, and the sines (R/2 for each token, whatever its heads) are
// formed once into shared memory by the block that turns the token's heads.
#include <algorithm>

#include "cache_common.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256, kUnroll = 4;
constexpr int kMaxTokens = 16;               // of one block
constexpr int kTableBytes = 16384;           // its sines and cosines

struct Shape {                               // of the launch
  FastDiv slots, rows;                       // slots of a row, rows of a token
  int32_t pair_slots;                        // slots that turn; the rest copy
  int32_t tokens;                            // of a block
};

// VE consecutive elements as loaded
template <bool BF, int VE>
struct Vec {
  static constexpr int kBytes = VE * (BF ? 2 : 4);
  uint32_t w[(kBytes + 3) / 4];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const char* p = static_cast<const char*>(base) + i * (BF ? 2 : 4);
    if constexpr (kBytes == 16) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (kBytes == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    char* p = static_cast<char*>(base) + i * (BF ? 2 : 4);
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
  }
  __device__ __forceinline__ float f32(int e) const {
    if constexpr (BF) return (e & 1) ? __uint_as_float(w[e >> 1] & 0xffff0000u) : __uint_as_float(w[e >> 1] << 16);
    else return __uint_as_float(w[e]);
  }
  // rounds to nearest even where the row is bf16
  __device__ __forceinline__ void set(const float (&x)[VE]) {
    if constexpr (!BF) {
#pragma unroll
      for (int e = 0; e < VE; ++e) w[e] = __float_as_uint(x[e]);
    } else if constexpr (VE == 1) {
      w[0] = f32_to_bf16_bits(x[0]);
    } else {
#pragma unroll
      for (int e = 0; e < VE / 2; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
    }
  }
};

// m (cos, sin) of p turns / 2^64 of a turn each
__device__ __forceinline__ float2 turned(int64_t p, uint64_t turn, float m) {
  const int32_t x = static_cast<int32_t>((static_cast<uint64_t>(p) * turn) >> 32);
  const uint32_t quadrant = (static_cast<uint32_t>(x) + (1u << 29)) >> 30;
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(x) - (quadrant << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  if (quadrant & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quadrant & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(m * c, m * s);
}

// the sequence that holds token t: the last one whose first token is at most t
__device__ __forceinline__ int sequence_of(const uint32_t* offsets, int B, int64_t t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(offsets[mid]) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

enum { kSkipQ = 1, kSkipKV = 2 };

// HALF: pairs (i, i + R/2), a slot being VE of the first halves with their partners; otherwise pairs
// (2i, 2i + 1), a slot being max(VE, 2) consecutive elements.  A slot is read whole before it is written, and no other
// thread touches it, so the outputs may be the inputs.
template <bool BF, int VE, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const Shape sh) {
  constexpr int kSpan = HALF ? VE : (VE < 2 ? 2 : VE);   // elements of a turning slot (of each half)
  constexpr int kVecs = HALF ? 2 : kSpan / VE;           // vectors of a turning slot
  extern __shared__ float2 sines[];                      // [tokens][R / 2]
  __shared__ int64_t position[kMaxTokens], page_at[kMaxTokens];
  __shared__ int32_t skip[kMaxTokens];
  const int half_r = a.R / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * sh.tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(sh.tokens), a.T - t0));
  const uint32_t per_token = sh.slots.d * sh.rows.d, units = per_token * tokens;

  if (threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t p = 0, at = 0;
    int sk = 0;
    if (a.table) {
      int s = static_cast<int>(t);
      int64_t bos = t, eos = t + 1;
      if (a.offsets) {
        s = sequence_of(a.offsets, a.B, t);
        bos = a.offsets[s];
        eos = a.offsets[s + 1];
        if (bos > t || static_cast<int64_t>(a.offsets[a.B]) > a.T || a.offsets[0] != 0) {
          raise_device_error(a.err, KDA_DEVERR_OFFSETS);
          eos = 0;
        }
      }
      if (t >= eos) {                        // behind the last sequence: a padded batch
        sk = kSkipQ | kSkipKV;
      } else {
        p = static_cast<int64_t>(a.start[s]) + (t - bos);
        int32_t page = -1;
        if (p >= 0 && p < static_cast<int64_t>(a.max_pages) * a.P)
          page = a.table[static_cast<int64_t>(s) * a.max_pages + p / a.P];
        if (page < 0 || page >= a.num_pages) {
          raise_device_error(a.err, KDA_DEVERR_PAGE);
          sk = kSkipKV;
        } else {
          at = page * a.page_stride + (p % a.P) * a.page_row_stride;
        }
      }
    } else {
      p = a.wide ? static_cast<const int64_t*>(a.positions)[t] : static_cast<const int32_t*>(a.positions)[t];
    }
    position[threadIdx.x] = p;
    page_at[threadIdx.x] = at;
    skip[threadIdx.x] = sk;
  }
  __syncthreads();
  if (a.freq) {
    for (int i = threadIdx.x; i < half_r; i += kThreads) {
      const double x = a.freq[i] * 0.15915494309189533577;     // turns per position: 1 / 2 pi
      const double fraction = x - floor(x);
      // fraction < 1, but its product with 2^64 may round up to 2^64, a whole turn
      const uint64_t turn = fraction * 0x1p64 >= 0x1p64 ? 0 : static_cast<uint64_t>(fraction * 0x1p64);
      for (int j = 0; j < tokens; ++j) {
        float2 cs = turned(position[j], turn, a.magnitude);
        if (a.transpose) cs.y = -cs.y;
        sines[j * half_r + i] = cs;
      }
    }
    __syncthreads();
  }

  const uint32_t step = kThreads * gridDim.y;
  for (uint32_t u0 = blockIdx.y * kThreads + threadIdx.x; u0 < units; u0 += step * kUnroll) {
    Vec<BF, VE> x[kUnroll][kVecs];
    void* out[kUnroll];
    int64_t to[kUnroll];
    int token[kUnroll], slot[kUnroll];
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const uint32_t u = u0 + n * step;
      out[n] = nullptr;
      if (u >= units) continue;
      const uint32_t row_of_all = sh.slots.div(u);
      slot[n] = static_cast<int>(u - row_of_all * sh.slots.d);
      token[n] = static_cast<int>(sh.rows.div(row_of_all));
      int row = static_cast<int>(row_of_all - token[n] * sh.rows.d);
      const int64_t t = t0 + token[n];
      const void* from;
      int64_t at;
      if (row < a.H) {
        if (skip[token[n]] & kSkipQ) continue;
        from = a.q;
        at = t * a.q_stride + row * a.D;
        out[n] = a.q_out;
        to[n] = t * a.q_out_stride + row * a.D;
      } else {
        if (skip[token[n]] & kSkipKV) continue;
        row -= a.H;
        const bool value = row >= a.HK;
        if (value) row -= a.HK;
        from = value ? a.v : a.k;
        at = t * (value ? a.v_stride : a.k_stride) + row * a.D;
        out[n] = value ? a.v_out : a.k_out;
        to[n] = a.table ? page_at[token[n]] + row * a.page_head_stride : t * a.k_out_stride + row * a.D;
        if (value) slot[n] |= 1 << 30;       // passes whole
      }
      const int s = slot[n] & ~(1 << 30);
      const int first = s < sh.pair_slots ? s * kSpan : a.R + (s - sh.pair_slots) * VE;
      at += first;
      to[n] += first;
      x[n][0].load(from, at);
      if (s < sh.pair_slots && kVecs == 2) x[n][kVecs - 1].load(from, at + (HALF ? half_r : VE));
    }
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      if (!out[n]) continue;
      const bool turns = slot[n] < sh.pair_slots && a.freq;
      const int s = slot[n] & ~(1 << 30);
      if (turns) {
        const float2* cs = sines + token[n] * half_r + (HALF ? s * VE : s * kSpan / 2);
        if constexpr (HALF) {
          float y0[VE], y1[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float c = cs[e].x, d = cs[e].y, f = x[n][0].f32(e), g = x[n][1].f32(e);
            y0[e] = f * c - g * d;
            y1[e] = g * c + f * d;
          }
          x[n][0].set(y0);
          x[n][1].set(y1);
        } else if constexpr (VE == 1) {
          const float c = cs[0].x, d = cs[0].y, f = x[n][0].f32(0), g = x[n][1].f32(0);
          const float y0[1] = {f * c - g * d}, y1[1] = {g * c + f * d};
          x[n][0].set(y0);
          x[n][1].set(y1);
        } else {
          float y[VE];
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const float c = cs[e / 2].x, d = cs[e / 2].y, f = x[n][0].f32(e), g = x[n][0].f32(e + 1);
            y[e] = f * c - g * d;
            y[e + 1] = g * c + f * d;
          }
          x[n][0].set(y);
        }
      }
      x[n][0].store(out[n], to[n]);
      if (s < sh.pair_slots && kVecs == 2) x[n][kVecs - 1].store(out[n], to[n] + (HALF ? half_r : VE));
    }
  }
}

template <bool BF, int VE, bool HALF>
cudaError_t launch(const RotaryArgs& a, cudaStream_t st) {
  constexpr int kSpan = HALF ? VE : (VE < 2 ? 2 : VE);
  Shape sh;
  sh.pair_slots = (HALF ? a.R / 2 : a.R) / kSpan;
  const int rows = a.H + a.HK + a.HV;
  const int slots = sh.pair_slots + (a.D - a.R) / VE;
  sh.slots = FastDiv(slots);
  sh.rows = FastDiv(rows);
  const int64_t per_token = static_cast<int64_t>(rows) * slots;
  // About two rounds of kUnroll slots for each thread (rows loaded while others are stored), fewer tokens where
  // that would leave SMs without a block, and no more sines than fit.
  int64_t n = std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, 2 * kUnroll * kThreads / per_token));
  n = std::min<int64_t>(n, std::max<int64_t>(1, a.T / (2 * sm_count())));
  if (a.R) n = std::min<int64_t>(n, std::max<int64_t>(1, kTableBytes / (a.R / 2 * static_cast<int64_t>(sizeof(float2)))));
  sh.tokens = static_cast<int32_t>(n);
  const int64_t blocks = (a.T + n - 1) / n;
  // few tokens: their heads are shared out to several blocks, each forming the sines for itself
  const int64_t split = std::max<int64_t>(
      1, std::min<int64_t>((n * per_token + kThreads - 1) / kThreads, 2 * sm_count() / blocks));
  const size_t smem = a.freq ? n * (a.R / 2) * sizeof(float2) : 0;
  rotary_kernel<BF, VE, HALF><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(split)), kThreads, smem, st>>>(a, sh);
  return cudaGetLastError();
}

template <bool BF, int VE>
cudaError_t launch_layout(const RotaryArgs& a, cudaStream_t st) {
  return a.interleaved ? launch<BF, VE, false>(a, st) : launch<BF, VE, true>(a, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t st) {
  // the widest vectors that every row, half row and tail starts on
  const uint64_t esz = bf16 ? 2 : 4;
  uint64_t bits = static_cast<uint64_t>(a.D) | (a.interleaved ? a.R : a.R / 2) | a.q_stride | a.k_stride | a.v_stride |
                  a.q_out_stride | a.k_out_stride;
  if (a.table) bits |= a.page_stride | a.page_row_stride | a.page_head_stride;
  for (const void* p : {a.q, a.k, a.v, static_cast<const void*>(a.q_out), static_cast<const void*>(a.k_out),
                        static_cast<const void*>(a.v_out)})
    bits |= reinterpret_cast<uintptr_t>(p) / esz;
  if (bf16) {
    if (bits % 8 == 0) return launch_layout<true, 8>(a, st);
    if (bits % 2 == 0) return launch_layout<true, 2>(a, st);
    return launch_layout<true, 1>(a, st);
  }
  if (bits % 4 == 0) return launch_layout<false, 4>(a, st);
  if (bits % 2 == 0) return launch_layout<false, 2>(a, st);
  return launch_layout<false, 1>(a, st);
}

}  // namespace kda
