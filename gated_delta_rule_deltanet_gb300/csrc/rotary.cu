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
// 2^64: two integer multiplications, off by no more than p 2^-64 turns.  Before them f_i / 2 pi is rounded in fp64, the
// constant and the product, together by 2^-52.3 of itself: p f_i 2^-55 turns.  The two top bits give the quadrant, the rest
// an argument of at most an eighth of a turn, rounded to 2^-28 of a turn, for sincospif.
//
// Bound by HBM: every value is read and written once, and the sines (R/2 for each token, whatever its heads) are
// formed once into shared memory by the block that turns the token's heads.  One GB300: 16384 tokens x 40 heads x 128
// bf16 57 us (87% of measured HBM, 57% of the issue slots), 14 k tokens of 16 + 16 heads with v into pages 67 us (76%), one
// token of each of 256 sequences 4.7 us.  With every slot's row and place found by division the first took 67 us.
#include <algorithm>

#include "cache_common.cuh"

namespace kda {

namespace {

// two rounds: 56.8 us for the first case above and 66.8 for the second, four 56.4 and 69.0
constexpr int kThreads = 256, kUnroll = 4, kRounds = 2;
constexpr int kMaxTokens = 16;               // of one block
constexpr int kTableBytes = 16384;           // its sines and cosines

struct Shape {                               // of the launch
  FastDiv slots, rows;                       // slots of a row, rows of a token
  int32_t pair_slots;                        // of pairs (i, i + R/2); the rest pass
  int32_t tokens;                            // of a block
};

// Place of pair i's sine: sixteen bytes more every eight pairs, so that lanes with neighbouring slots read other banks.
__host__ __device__ constexpr int sine_at(int i) { return i + (i >> 3) * 2; }
__host__ __device__ constexpr int sine_pitch(int half_r) { return (sine_at(half_r) + 1) & ~1; }

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

// The sequence that holds token t: the last one whose first token is at most t.  A warp looks at 32 at a time.
__device__ __forceinline__ int sequence_of(const uint32_t* offsets, int B, int64_t t) {
  int lo = 0, n = B;                         // it is among n from lo on
  while (n > 1) {
    const int stride = (n + 31) / 32, at = static_cast<int>(threadIdx.x & 31) * stride;
    const bool before = at < n && static_cast<int64_t>(offsets[lo + at]) <= t;
    const int k = max(0, __popc(__ballot_sync(0xffffffffu, before)) - 1) * stride;
    lo += k;
    n = min(stride, n - k);
  }
  return lo;
}

enum { kSkipQ = 1, kSkipKV = 2 };

// A slot is two vectors of VE elements of a row: of pairs (i, i + R/2) (HALF) VE first halves and their partners, otherwise,
// and of the channels that pass, two behind one another.  A thread has one slot of the row and goes through the rows
// (of all heads, of all tokens of the block); a slot is read whole before it is written, and no other thread touches it, so
// the outputs may be the inputs.  Its first slots are loaded before the sines are formed, its next ones before it comes
// to them.  Three blocks an SM at 80 registers: 56.4 us where four at 64 take 61.0.
template <bool BF, int VE, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryArgs a, const Shape sh) {
  extern __shared__ __align__(16) float2 sines[];        // [tokens][sine_pitch]
  __shared__ int64_t position[kMaxTokens], page_at[kMaxTokens];
  __shared__ int32_t skip[kMaxTokens];
  const int half_r = a.R / 2, pitch = sine_pitch(half_r), slots = sh.slots.d, rows = sh.rows.d;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * sh.tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(sh.tokens), a.T - t0));
  // rows that the block's threads take at a time, and this thread's slot and first row
  const int at_once = max(1, kThreads / slots), all_rows = tokens * rows, step = at_once * gridDim.y;
  const int lane_row = sh.slots.div(threadIdx.x);
  int slot = threadIdx.x - lane_row * slots;
  const int row0 = slots > kThreads || lane_row < at_once ? static_cast<int>(blockIdx.y) * at_once + lane_row : all_rows;

  Vec<BF, VE> x[kUnroll][2];
  int token[kUnroll], row[kUnroll];                      // row counts through the heads of q, k and v
  int first, second;                                     // where the slot's vectors begin
  const auto place = [&]() {
    if (HALF && slot < sh.pair_slots) {
      first = slot * VE;
      second = first + half_r;
    } else {
      first = (HALF ? a.R : 0) + (slot - (HALF ? sh.pair_slots : 0)) * 2 * VE;
      second = first + VE;
    }
  };
  const auto load = [&](int r0) {
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const int r = r0 + n * step;
      token[n] = -1;
      if (r >= all_rows) continue;
      token[n] = static_cast<int>(sh.rows.div(r));
      row[n] = r - token[n] * rows;
      const int64_t t = t0 + token[n];
      const void* from = a.q;
      int64_t at = t * a.q_stride + row[n] * a.D;
      if (row[n] >= a.H) {
        from = a.k;
        at = t * a.k_stride + (row[n] - a.H) * a.D;
        if (row[n] >= a.H + a.HK) {
          from = a.v;
          at = t * a.v_stride + (row[n] - a.H - a.HK) * a.D;
        }
      }
      x[n][0].load(from, at + first);
      if (second < a.D) x[n][1].load(from, at + second);
    }
  };
  place();
  int r0 = row0;
  load(r0);

  // a warp takes a token
  for (int j = threadIdx.x >> 5; j < tokens; j += kThreads / 32) {
    const int64_t t = t0 + j;
    int64_t p = 0, at = 0;
    int sk = 0;
    if (a.table) {
      int s = static_cast<int>(t);
      int64_t bos = t, eos = t + 1;
      if (a.offsets) {
        const int64_t zero = a.offsets[0], end = a.offsets[a.B];
        s = sequence_of(a.offsets, a.B, t);
        bos = a.offsets[s];
        eos = a.offsets[s + 1];
        if (bos > t || end > a.T || zero != 0) {
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
    if ((threadIdx.x & 31) == 0) {
      position[j] = p;
      page_at[j] = at;
      skip[j] = sk;
    }
  }
  __syncthreads();
  if (a.freq) {
    // a thread keeps its pair and goes through the tokens
    const int per = kThreads / max(1, min(half_r, kThreads)), share = threadIdx.x / max(1, half_r);
    for (int i = half_r < kThreads ? threadIdx.x - share * half_r : threadIdx.x; i < half_r && share < per; i += kThreads) {
      const double turns = a.freq[i] * 0.15915494309189533577;     // per position: 1 / 2 pi
      const double fraction = turns - floor(turns);
      // fraction < 1, but its product with 2^64 may round up to 2^64, a whole turn
      const uint64_t turn = fraction * 0x1p64 >= 0x1p64 ? 0 : static_cast<uint64_t>(fraction * 0x1p64);
      for (int j = share; j < tokens; j += per) {
        float2 cs = turned(position[j], turn, a.magnitude);
        if (a.transpose) cs.y = -cs.y;
        sines[j * pitch + sine_at(i)] = cs;
      }
    }
    __syncthreads();
  }

  while (true) {
    if (r0 >= all_rows) {                    // rows of more slots than threads: the next slot
      slot += kThreads;
      if (slots <= kThreads || slot >= slots) break;
      place();
      r0 = row0;
      load(r0);
      continue;
    }
    // turn what is loaded
    const bool turns = a.freq && (HALF ? slot < sh.pair_slots : first < a.R);
    if (turns) {
      const float2* at = sines + sine_at(HALF ? first : first / 2);
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        if (token[n] < 0 || row[n] >= a.H + a.HK) continue;
        const float2* cs = at + token[n] * pitch;
        float y0[VE], y1[VE];
        if constexpr (HALF) {
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
          y0[0] = f * c - g * d;
          y1[0] = g * c + f * d;
          x[n][0].set(y0);
          x[n][1].set(y1);
        } else {
          // pairs from R / 2 on pass, and may share a vector with ones that do not
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const float f = x[n][0].f32(e), g = x[n][0].f32(e + 1);
            const bool on = first + e < a.R;
            const float c = on ? cs[e / 2].x : 1.f, d = on ? cs[e / 2].y : 0.f;
            y0[e] = on ? f * c - g * d : f;
            y0[e + 1] = on ? g * c + f * d : g;
          }
          x[n][0].set(y0);
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const float f = x[n][1].f32(e), g = x[n][1].f32(e + 1);
            const bool on = second + e < a.R;
            const float c = on ? cs[(VE + e) / 2].x : 1.f, d = on ? cs[(VE + e) / 2].y : 0.f;
            y1[e] = on ? f * c - g * d : f;
            y1[e + 1] = on ? g * c + f * d : g;
          }
          x[n][1].set(y1);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      if (token[n] < 0) continue;
      const int64_t t = t0 + token[n];
      const bool query = row[n] < a.H, value = row[n] >= a.H + a.HK;
      if (skip[token[n]] & (query ? kSkipQ : kSkipKV)) continue;
      const int head = row[n] - (query ? 0 : a.H) - (value ? a.HK : 0);
      void* out = query ? a.q_out : value ? a.v_out : a.k_out;
      const int64_t to = query     ? t * a.q_out_stride + head * a.D
                         : a.table ? page_at[token[n]] + head * a.page_head_stride
                                   : t * a.k_out_stride + head * a.D;
      x[n][0].store(out, to + first);
      if (second < a.D) x[n][1].store(out, to + second);
    }
    r0 += step * kUnroll;
    if (r0 < all_rows) load(r0);
  }
}

template <bool BF, int VE, bool HALF>
cudaError_t launch(const RotaryArgs& a, cudaStream_t st) {
  Shape sh;
  const auto slots_of = [](int elements) { return (elements + 2 * VE - 1) / (2 * VE); };
  sh.pair_slots = HALF ? a.R / 2 / VE : 0;
  const int rows = a.H + a.HK + a.HV, slots = HALF ? sh.pair_slots + slots_of(a.D - a.R) : slots_of(a.D);
  sh.slots = FastDiv(slots);
  sh.rows = FastDiv(rows);
  const int64_t per_token = static_cast<int64_t>(rows) * slots;
  // About kRounds rounds of kUnroll slots for each thread, fewer tokens where that would leave SMs without a block,
  // and no more sines than fit.
  int64_t n = std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, kRounds * kUnroll * kThreads / per_token));
  n = std::min<int64_t>(n, std::max<int64_t>(1, a.T / (8 * sm_count())));
  if (a.R)
    n = std::min<int64_t>(n, std::max<int64_t>(1, kTableBytes / (sine_pitch(a.R / 2) * int64_t{sizeof(float2)})));
  sh.tokens = static_cast<int32_t>(n);
  const int64_t blocks = (a.T + n - 1) / n;
  // few tokens: their heads are shared out to several blocks, each forming the sines for itself
  const int64_t split = std::max<int64_t>(
      1, std::min<int64_t>((n * per_token + kThreads - 1) / kThreads, 2 * sm_count() / blocks));
  const size_t smem = a.freq ? n * sine_pitch(a.R / 2) * sizeof(float2) : 0;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(split));
  rotary_kernel<BF, VE, HALF><<<grid, kThreads, smem, st>>>(a, sh);
  return cudaGetLastError();
}

template <bool BF, int VE>
cudaError_t launch_layout(const RotaryArgs& a, cudaStream_t st) {
  return a.interleaved ? launch<BF, VE, false>(a, st) : launch<BF, VE, true>(a, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, cudaStream_t st) {
  // the widest vectors that every row and, of pairs (i, i + R/2), each half starts on
  const uint64_t esz = bf16 ? 2 : 4;
  uint64_t bits = static_cast<uint64_t>(a.D) | (a.interleaved ? 0 : a.R / 2) | a.q_stride | a.k_stride | a.v_stride |
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
