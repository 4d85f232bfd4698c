// cache_attention.cu -- attention of one new token, or of a window of draft tokens, per sequence over the
// pages of a key-value cache.
//
// Query w < W of sequence b stands at position p = len_b - W + w; its own key and those before it are in the
// pages.  For query head h of key head h / (H / HK)
//
//     s_j = c(scale q k_j) + slope_h (j - p),   c(x) = cap tanh(x / cap)   max(0, p - span + 1) <= j <= p
//     o = sum_j e^(s_j - m) v_j / l,   m = max_j s_j,   l = sum_j e^(s_j - m),   lse = m + log l
//
// with m and l kept as running values (Milakov and Gimelshein, "Online normalizer calculation for softmax",
// 2018) in base 2.  A row that sees no key has o = 0 and lse = -infinity.
//
// Bound by HBM: each key and value is read once for all rows of its group (queries x heads of one key head).
// The work is cut into tiles of 4 x BK keys of a (sequence, key head) and the row of all tiles into equal stretches,
// one for each CTA, whatever the sequences' lengths: a stretch that begins or ends inside a (sequence, key
// head) leaves (m, l, unnormalised o) of its part in the workspace, and a second kernel joins the parts in the
// order of the stretches, so that repeated calls give the same bits.  The lengths stay on the device: a captured
// graph follows them.
//
// Inside a CTA each of four warps takes every fourth block of BK keys, copies it into its own ring in shared
// memory (cp.async, rows of 16-byte pieces stored at piece ^ (row mod 8)) and keeps its own m, l and o, so that the
// warps wait for one another only where a part ends.
//
//   bf16   BK = 16: scores and o by mma.m16n8k16 with fp32 accumulators, the rows as M.  A window's rows are
//          few: at 16 rows the products take a fifth of the time that the copies take, so the tensor memory path,
//          whose smallest M is 64 and whose accumulators come back through tcgen05.ld, would have nothing to give.
//   fp32   BK = 8: fp32 on CUDA cores (tensor cores would round the operands to tf32).
#include <algorithm>

#include "cache_common.cuh"

namespace kda {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMinTiles = 2;                 // of a stretch: a part costs a write and a read of its rows' sums

// The (m, l, o) of a part: rows of D + 2 floats -- o, then m, l.  Stretch c leaves a part that began
// in an earlier stretch at 2 c, one that goes on in a later stretch at 2 c + 1.
struct Join {                                // where stretch c begins inside an item that began in c - 1
  int32_t seq, item, parts, pad;             // parts == 0: nothing to join here
};

struct Range {                               // a sequence's keys
  int32_t len, first, begin, tiles;          // first visible key; begin: first rounded down to a block
};

template <int BK>
__device__ __forceinline__ Range range_of(const AttentionArgs& a, int b) {
  Range r;
  const int cap = static_cast<int>(min(static_cast<int64_t>(a.max_pages) * a.P, static_cast<int64_t>(0x7fffff00)));
  r.len = a.lens[b];
  if (r.len < 0 || r.len > cap) {
    raise_device_error(a.err, KDA_DEVERR_PAGE);
    r.len = r.len < 0 ? 0 : cap;
  }
  r.first = a.span ? static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(r.len) - a.W - a.span + 1)) : 0;
  r.first = min(r.first, r.len);
  r.begin = r.first & ~(BK - 1);
  r.tiles = max(1, (r.len - r.begin + kWarps * BK - 1) / (kWarps * BK));
  return r;
}

struct Walk {                                // a stretch of tiles, item by item
  int b, item, tile;                         // where it stands
  int64_t left;                              // tiles still to do
  Range r;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Finds this CTA's stretch.  Every CTA adds the tiles of all sequences up (B numbers); stretch c of n begins at
// tile floor(c total / n).  Also notes where the CTA begins inside an item.
template <int BK>
__device__ Walk find_stretch(const AttentionArgs& a, int items, Join* joins) {
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int32_t found;                  // the sequence in which the stretch begins
  __shared__ int64_t before;                 // and the tiles of those before it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += static_cast<int64_t>(range_of<BK>(a, b).tiles) * items;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t total = 0, excl = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) excl += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t n = min(static_cast<int64_t>(gridDim.x), (total + kMinTiles - 1) / kMinTiles);
  const int64_t c = blockIdx.x;
  Walk w;
  w.left = 0;
  if (c >= n) {
    if (tid == 0) joins[c].parts = 0;
    return w;
  }
  // floor(c total / n) without leaving 64 bits: total = k n + rest
  const int64_t k = total / n, rest = total - k * n;
  const int64_t t0 = c * k + c * rest / n, t1 = (c + 1) * k + (c + 1) * rest / n;
  if (excl <= t0 && t0 < excl + mine) {
    for (int b = b0; b < b1; ++b) {
      const int64_t x = static_cast<int64_t>(range_of<BK>(a, b).tiles) * items;
      if (t0 < excl + x) {
        found = b;
        before = excl;
        break;
      }
      excl += x;
    }
  }
  __syncthreads();
  w.b = found;
  w.r = range_of<BK>(a, w.b);
  const int64_t at = t0 - before;
  w.item = static_cast<int>(at / w.r.tiles);
  w.tile = static_cast<int>(at - static_cast<int64_t>(w.item) * w.r.tiles);
  w.left = t1 - t0;
  if (tid == 0) {
    const int64_t begin = t0 - w.tile, end = begin + w.r.tiles;      // the item's tiles
    Join j{w.b, w.item, 0, 0};
    if (w.tile > 0 && (c - 1) * k + (c - 1) * rest / n <= begin) {
      // the first stretch that begins inside the item: it and those after it up to the item's end, and c - 1's part
      int64_t e = c;
      // the last stretch that begins before `end`: stretches are k or k + 1 tiles long
      e = min(n - 1, c + (end - 1 - t0) / k);
      while (e > c && e * k + e * rest / n >= end) --e;
      j.parts = static_cast<int32_t>(e - c + 2);
    }
    joins[c] = j;
  }
  return w;
}

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// DP: the head's channels rounded up (zeros behind D), MT: row tiles of 16, STAGES of the ring
template <int DP, int MT, int STAGES>
struct Mma {
  static constexpr int kBK = 16, kRows = 16 * MT, kRowBytes = DP * 2;
  static constexpr int kStage = 2 * kBK * kRowBytes;           // keys, then values, of one block
  static constexpr int kRing = kWarps * STAGES * kStage;
  static constexpr int kPart = kWarps * kRows * (DP + 2) * 4;  // the warps' sums, over the ring
  static constexpr int kQ = kRows * kRowBytes;
  static constexpr size_t kSmem = (kRing > kPart ? kRing : kPart) + kQ;
};

struct RowPlace {                            // where a row's results go
  int64_t o;                                 // row of o and lse: (b W + w) H + h
  int32_t w, h;
};
__device__ __forceinline__ RowPlace row_place(const AttentionArgs& a, int b, int hk, int r) {
  const int g = a.H / a.HK, w = r / g, h = hk * g + r - w * g;
  return RowPlace{(static_cast<int64_t>(b) * a.W + w) * a.H + h, w, h};
}

template <bool BF_OUT>
__device__ __forceinline__ void store_out(const AttentionArgs& a, int64_t at, float x) {
  if constexpr (BF_OUT) static_cast<uint16_t*>(a.o)[at] = f32_to_bf16_bits(x);
  else static_cast<float*>(a.o)[at] = x;
}

// Adds the warps' sums (in shared memory, rows of DP + 2 floats) up and writes the rows of a part: final
// where the part is the whole item, otherwise to the workspace.  A warp takes a row.
template <int DP, int ROWS, bool BF_OUT>
__device__ void finish_part(const AttentionArgs& a, const float* sums, int b, int hk, int row0, int rows, float* part) {
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < min(ROWS, rows - row0); r += kWarps) {
    float m = -INFINITY, f[kWarps], l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sums[(w * ROWS + r) * (DP + 2) + DP]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* s = sums + (w * ROWS + r) * (DP + 2);
      f[w] = ex2(s[DP] - base);
      l += f[w] * s[DP + 1];
    }
    const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);       // a NaN stays one
    const RowPlace at = row_place(a, b, hk, row0 + r);
    float* out = part + static_cast<int64_t>(r) * (a.D + 2);
    for (int d = lane; d < a.D; d += 32) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += f[w] * sums[(w * ROWS + r) * (DP + 2) + d];
      x = l == 0.f ? 0.f : x * inv;
      if (part) out[d] = x;
      else store_out<BF_OUT>(a, at.o * a.D + d, x);
    }
    if (lane == 0) {
      if (part) {
        out[a.D] = m;
        out[a.D + 1] = l;
      } else if (a.lse) {
        a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

__device__ __forceinline__ bool bf16x2_not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

// SPLIT: where o is stored in fp32, the weights e^(s - m) enter the second product as three bf16 parts (24 bits
// in all); where o is bf16, as one, whose rounding (2^-9) is o's own.
template <int DP, int MT, int STAGES, bool BF_OUT>
__global__ void __launch_bounds__(kThreads) attend_bf16_kernel(const AttentionArgs a, FastDiv page_div, int row_tiles,
                                                               Join* joins, float* parts) {
  using C = Mma<DP, MT, STAGES>;
  constexpr bool SPLIT = !BF_OUT;
  constexpr int BK = C::kBK, CH = DP / 8, KS = DP / 16;        // 16-byte pieces of a row, steps along D
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t block_valid[kWarps][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = a.H / a.HK, rows = a.W * g, pieces = a.D / 8;
  unsigned char* ring = smem + warp * STAGES * C::kStage;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  unsigned char* q_smem = smem + C::kSmem - C::kQ;
  const uint32_t q_u = static_cast<uint32_t>(__cvta_generic_to_shared(q_smem));
  const float scale2 = a.scale * kLog2e, cap2 = a.softcap * kLog2e, inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;

  Walk walk = find_stretch<BK>(a, a.HK * row_tiles, joins);
  while (walk.left > 0 && walk.b < a.B) {
    const int hk = walk.item / row_tiles, row0 = (walk.item - hk * row_tiles) * C::kRows;
    const int n = static_cast<int>(min(walk.left, static_cast<int64_t>(walk.r.tiles - walk.tile)));
    const Range r = walk.r;
    const int b = walk.b;

    // The previous part's sums are read; the ring's pieces behind D become zeros once more (its sums lay over them), and
    // the rows of q land beside the ring.
    __syncthreads();
    for (int i = tid; pieces < CH && i < kWarps * STAGES * 2 * BK * CH; i += kThreads) {
      const int row = i / CH, ch = i - row * CH;
      if (ch >= pieces)
        *reinterpret_cast<uint4*>(smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
    }
    for (int i = tid; i < C::kRows * CH; i += kThreads) {
      const int row = i / CH, ch = i - row * CH;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row0 + row < rows && ch < pieces) {
        const RowPlace at = row_place(a, b, hk, row0 + row);
        x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                            (static_cast<int64_t>(b) * a.W + at.w) * a.q_stride +
                                            static_cast<int64_t>(at.h) * a.D + ch * 8);
      }
      *reinterpret_cast<uint4*>(q_smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = x;
    }
    __syncthreads();

    // block i of this warp begins at key base(i)
    const auto base = [&](int i) { return r.begin + ((walk.tile + i) * kWarps + warp) * BK; };
    const auto page_of = [&](int i) {
      const int key = base(i) + (lane & 15);
      if (i >= n || key < r.first || key >= r.len) return -1;
      return a.table[static_cast<int64_t>(b) * a.max_pages + page_div.div(key)];
    };
    const auto issue = [&](int i, int page) {
      const int key = base(i) + (lane & 15);
      const bool inside = i < n && key >= r.first && key < r.len;
      const bool ok = inside && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages);
      if (inside && !ok) raise_device_error(a.err, KDA_DEVERR_PAGE);
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int in_page = key - static_cast<int>(page_div.div(key)) * a.P;
      const int64_t off = ok ? page * a.page_stride + in_page * a.page_row_stride + hk * a.page_head_stride : 0;
      const int slot = i % STAGES;
      if (lane == 0) block_valid[warp][slot] = valid;
      const uint32_t dst = ring_u + slot * C::kStage;
      if (i < n) {
#pragma unroll
        for (int it = 0; it < BK * CH / 32; ++it) {
          const int row = (it * 32 + lane) / CH, ch = (it * 32 + lane) % CH;
          const int64_t from = __shfl_sync(0xffffffffu, off, row) + ch * 8;
          const bool have = (valid >> row) & 1;
          if (ch < pieces) {
            const uint32_t to = dst + row * C::kRowBytes + ((ch ^ (row & 7)) << 4);
            cp_async16(to, static_cast<const uint16_t*>(a.k) + (have ? from : 0), have);
            cp_async16(to + BK * C::kRowBytes, static_cast<const uint16_t*>(a.v) + (have ? from : 0), have);
          }
        }
      }
      cp_async_commit();
    };

    float m[MT][2], l[MT][2], o[MT][DP / 8][4];
    int pos[MT][2];                          // positions of this thread's rows
    float slope[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[t][i] = -INFINITY;
        l[t][i] = 0.f;
        const int row = min(row0 + t * 16 + i * 8 + (lane >> 2), rows - 1);
        const RowPlace at = row_place(a, b, hk, row);
        pos[t][i] = r.len - a.W + at.w;
        slope[t][i] = a.slopes ? a.slopes[at.h] * kLog2e : 0.f;
      }
#pragma unroll
      for (int d = 0; d < DP / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;
    }
    uint32_t qf[MT == 1 ? KS : 1][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int row = lane & 15, ch = kk * 2 + (lane >> 4);
        ldmatrix4(qf[kk], q_u + row * C::kRowBytes + ((ch ^ (row & 7)) << 4));
      }
    }

#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(i, page_of(i));
    int next_page = page_of(STAGES - 1);
    for (int i = 0; i < n; ++i) {
      issue(i + STAGES - 1, next_page);
      next_page = page_of(i + STAGES);
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const int slot = i % STAGES, key0 = base(i);
      const uint32_t ks = ring_u + slot * C::kStage, vs = ks + BK * C::kRowBytes;
      const uint32_t valid = block_valid[warp][slot];

      float s[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][j][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        if (kk * 16 >= a.D) break;
        uint32_t kf[4];
        {
          const int row = (lane & 7) + ((lane >> 4) << 3), ch = kk * 2 + ((lane >> 3) & 1);
          ldmatrix4(kf, ks + row * C::kRowBytes + ((ch ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t qt[4];
          if constexpr (MT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) qt[e] = qf[kk][e];
          } else {
            const int row = t * 16 + (lane & 15), ch = kk * 2 + (lane >> 4);
            ldmatrix4(qt, q_u + row * C::kRowBytes + ((ch ^ (row & 7)) << 4));
          }
          mma16816(s[t][0], qt, kf[0], kf[1]);
          mma16816(s[t][1], qt, kf[2], kf[3]);
        }
      }

      // Does every row see every key?  (the rows' positions are len - W .. len - 1)
      const bool whole = valid == 0xffffu && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      bool poison = false;
      if (!whole) {
        // A value that is not finite would reach the rows whose mask leaves it out as 0 x infinity.
        bool bad = false;
#pragma unroll
        for (int it = 0; it < BK * CH / 32; ++it) {
          const uint4 x = *reinterpret_cast<const uint4*>(ring + slot * C::kStage + BK * C::kRowBytes + (it * 32 + lane) * 16);
          bad |= bf16x2_not_finite(x.x) | bf16x2_not_finite(x.y) | bf16x2_not_finite(x.z) | bf16x2_not_finite(x.w);
        }
        poison = __any_sync(0xffffffffu, bad);
      }
      uint32_t pa[MT][4], pb[MT][4], pc[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float x[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = s[t][j][e];
            const int key = key0 + j * 8 + (lane & 3) * 2 + (e & 1), p = pos[t][e >> 1];
            y = a.softcap > 0.f ? cap2 * tanhf(y * inv_cap) : y * scale2;
            if (a.slopes) y += slope[t][e >> 1] * static_cast<float>(key - p);
            if (!whole) {
              const bool seen = ((valid >> (key - key0)) & 1) && key <= p && (a.span == 0 || key > p - a.span);
              y = seen ? y : -INFINITY;
            }
            x[j][e] = y;
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float now = fmaxf(m[t][i], top);
          const float from = now == -INFINITY ? 0.f : now;
          if (__any_sync(0xffffffffu, now > m[t][i])) {
            const float f = ex2(m[t][i] - from);
            l[t][i] *= f;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) {
              o[t][d][2 * i] *= f;
              o[t][d][2 * i + 1] *= f;
            }
            m[t][i] = now;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float y0 = ex2(x[j][2 * i] - from), y1 = ex2(x[j][2 * i + 1] - from);
            l[t][i] += y0 + y1;
            x[j][2 * i] = y0;
            x[j][2 * i + 1] = y1;
            const uint32_t hi = pack_bf16(y0, y1);
            pa[t][j * 2 + i] = hi;
            if constexpr (SPLIT) {
              const float r0 = y0 - __uint_as_float(hi << 16), r1 = y1 - __uint_as_float(hi & 0xffff0000u);
              const uint32_t mid = pack_bf16(r0, r1);
              pb[t][j * 2 + i] = mid;
              pc[t][j * 2 + i] = pack_bf16(r0 - __uint_as_float(mid << 16), r1 - __uint_as_float(mid & 0xffff0000u));
            }
          }
        }
        if (poison) {
          // key by key, leaving out what a row does not see
#pragma unroll 1
          for (int key = 0; key < BK; ++key) {
            const int src = (lane & ~3) | ((key & 7) >> 1);
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float u0 = __shfl_sync(0xffffffffu, x[0][2 * i], src), u1 = __shfl_sync(0xffffffffu, x[0][2 * i + 1], src);
              const float u2 = __shfl_sync(0xffffffffu, x[1][2 * i], src), u3 = __shfl_sync(0xffffffffu, x[1][2 * i + 1], src);
              w[i] = key < 8 ? ((key & 1) ? u1 : u0) : ((key & 1) ? u3 : u2);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int p = pos[t][i], at = key0 + key;
              const bool seen = ((valid >> key) & 1) && at <= p && (a.span == 0 || at > p - a.span);
              if (seen) {
#pragma unroll
                for (int d = 0; d < DP / 8; ++d) {
                  const uint32_t v = *reinterpret_cast<const uint32_t*>(ring + slot * C::kStage + (BK + key) * C::kRowBytes +
                                                                        ((d ^ (key & 7)) << 4) + (lane & 3) * 4);
                  o[t][d][2 * i] += w[i] * __uint_as_float(v << 16);
                  o[t][d][2 * i + 1] += w[i] * __uint_as_float(v & 0xffff0000u);
                }
              }
            }
          }
        }
      }
      if (!poison) {
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          if (d * 16 >= a.D) break;
          uint32_t vf[4];
          const int row = lane & 15, ch = d * 2 + (lane >> 4);
          ldmatrix4_trans(vf, vs + row * C::kRowBytes + ((ch ^ (row & 7)) << 4));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            if constexpr (SPLIT) {
              // the tensor cores cut their sums off, which over a long cache would lean one way: those of a block
              // are formed by themselves and added in fp32
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816(x, pc[t], vf[2 * j], vf[2 * j + 1]);
                mma16816(x, pb[t], vf[2 * j], vf[2 * j + 1]);
                mma16816(x, pa[t], vf[2 * j], vf[2 * j + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][2 * d + j][e] += x[e];
              }
            } else {
              mma16816(o[t][2 * d], pa[t], vf[0], vf[1]);
              mma16816(o[t][2 * d + 1], pa[t], vf[2], vf[3]);
            }
          }
        }
      }
      __syncwarp();
    }

    // the warps' sums, over the ring
    cp_async_wait<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[t][i];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        float* to = sums + (warp * C::kRows + t * 16 + i * 8 + (lane >> 2)) * (DP + 2);
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
          *reinterpret_cast<float2*>(to + d * 8 + (lane & 3) * 2) = make_float2(o[t][d][2 * i], o[t][d][2 * i + 1]);
        if ((lane & 3) == 0) *reinterpret_cast<float2*>(to + DP) = make_float2(m[t][i], x);
      }
    __syncthreads();
    float* part = nullptr;
    if (n < r.tiles)
      part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * C::kRows * (a.D + 2);
    finish_part<DP, C::kRows, BF_OUT>(a, sums, b, hk, row0, rows, part);

    walk.left -= n;
    walk.tile = 0;
    if (walk.left > 0 && ++walk.item == a.HK * row_tiles) {
      walk.item = 0;
      ++walk.b;
      if (walk.b < a.B) walk.r = range_of<BK>(a, walk.b);
    }
  }
}

// ------------------------------------------------------------------ fp32

template <int DP, int STAGES>
struct Simt {
  static constexpr int kBK = 8, kRows = 8, kRowBytes = DP * 4;
  static constexpr int kStage = 2 * kBK * kRowBytes;
  static constexpr int kRing = kWarps * STAGES * kStage;
  static constexpr int kPart = kWarps * kRows * (DP + 2) * 4;
  static constexpr int kQStride = DP + 4;                      // two rows apart is eight banks apart
  static constexpr int kQ = kRows * kQStride * 4;
  static constexpr size_t kSmem = (kRing > kPart ? kRing : kPart) + kQ + kWarps * kBK * kRows * 4 + kWarps * kRows * 4;
};

// A lane forms the scores of one key (lane mod 8) and two rows (2 (lane / 8), + 1); for the weighted sum
// it owns DP / 32 channels of all eight rows.
template <int DP, int STAGES, bool BF_OUT>
__global__ void __launch_bounds__(kThreads) attend_f32_kernel(const AttentionArgs a, FastDiv page_div, int row_tiles,
                                                              Join* joins, float* parts) {
  using C = Simt<DP, STAGES>;
  constexpr int BK = C::kBK, CH = DP / 4, OC = DP / 32;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t block_valid[kWarps][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = a.H / a.HK, rows = a.W * g, pieces = a.D / 4;
  unsigned char* ring = smem + warp * STAGES * C::kStage;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  constexpr int kTop = C::kRing > C::kPart ? C::kRing : C::kPart;
  float* q_smem = reinterpret_cast<float*>(smem + kTop);
  float* weights = reinterpret_cast<float*>(smem + kTop + C::kQ) + warp * BK * C::kRows;   // [key][row]
  float* factors = reinterpret_cast<float*>(smem + kTop + C::kQ) + kWarps * BK * C::kRows + warp * C::kRows;
  const float scale2 = a.scale * kLog2e, cap2 = a.softcap * kLog2e, inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const int key_lane = lane & 7, pair = lane >> 3;

  Walk walk = find_stretch<BK>(a, a.HK * row_tiles, joins);
  while (walk.left > 0 && walk.b < a.B) {
    const int hk = walk.item / row_tiles, row0 = (walk.item - hk * row_tiles) * C::kRows;
    const int n = static_cast<int>(min(walk.left, static_cast<int64_t>(walk.r.tiles - walk.tile)));
    const Range r = walk.r;
    const int b = walk.b;

    __syncthreads();                         // the previous part's sums are read
    for (int i = tid; pieces < CH && i < kWarps * STAGES * 2 * BK * CH; i += kThreads) {
      const int row = i / CH, ch = i - row * CH;
      if (ch >= pieces)
        *reinterpret_cast<uint4*>(smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
    }
    for (int i = tid; i < C::kRows * CH; i += kThreads) {
      const int row = i / CH, ch = i - row * CH;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row0 + row < rows && ch < pieces) {
        const RowPlace at = row_place(a, b, hk, row0 + row);
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                             (static_cast<int64_t>(b) * a.W + at.w) * a.q_stride +
                                             static_cast<int64_t>(at.h) * a.D + ch * 4);
      }
      *reinterpret_cast<float4*>(q_smem + row * C::kQStride + ch * 4) = x;
    }
    __syncthreads();

    const auto base = [&](int i) { return r.begin + ((walk.tile + i) * kWarps + warp) * BK; };
    const auto page_of = [&](int i) {
      const int key = base(i) + key_lane;
      if (i >= n || key < r.first || key >= r.len) return -1;
      return a.table[static_cast<int64_t>(b) * a.max_pages + page_div.div(key)];
    };
    const auto issue = [&](int i, int page) {
      const int key = base(i) + key_lane;
      const bool inside = i < n && key >= r.first && key < r.len;
      const bool ok = inside && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages);
      if (inside && !ok) raise_device_error(a.err, KDA_DEVERR_PAGE);
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffu;
      const int in_page = key - static_cast<int>(page_div.div(key)) * a.P;
      const int64_t off = ok ? page * a.page_stride + in_page * a.page_row_stride + hk * a.page_head_stride : 0;
      const int slot = i % STAGES;
      if (lane == 0) block_valid[warp][slot] = valid;
      const uint32_t dst = ring_u + slot * C::kStage;
      if (i < n) {
#pragma unroll
        for (int it = 0; it < BK * CH / 32; ++it) {
          const int row = (it * 32 + lane) / CH, ch = (it * 32 + lane) % CH;
          const int64_t from = __shfl_sync(0xffffffffu, off, row) + ch * 4;
          const bool have = (valid >> row) & 1;
          if (ch < pieces) {
            // keys are read by eight lanes a row each: pieces change places; values by whole rows
            const uint32_t to = dst + row * C::kRowBytes;
            cp_async16(to + ((ch ^ (row & 7)) << 4), static_cast<const float*>(a.k) + (have ? from : 0), have);
            cp_async16(to + BK * C::kRowBytes + ((ch ^ (row & 7)) << 4), static_cast<const float*>(a.v) + (have ? from : 0), have);
          }
        }
      }
      cp_async_commit();
    };

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, slope[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const RowPlace at = row_place(a, b, hk, min(row0 + pair * 2 + i, rows - 1));
      pos[i] = r.len - a.W + at.w;
      slope[i] = a.slopes ? a.slopes[at.h] * kLog2e : 0.f;
    }
    float o[C::kRows][OC];
#pragma unroll
    for (int t = 0; t < C::kRows; ++t)
#pragma unroll
      for (int e = 0; e < OC; ++e) o[t][e] = 0.f;

#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(i, page_of(i));
    int next_page = page_of(STAGES - 1);
    for (int i = 0; i < n; ++i) {
      issue(i + STAGES - 1, next_page);
      next_page = page_of(i + STAGES);
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const int slot = i % STAGES, key0 = base(i);
      const unsigned char* ks = ring + slot * C::kStage;
      const unsigned char* vs = ks + BK * C::kRowBytes;
      const uint32_t valid = block_valid[warp][slot];

      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 8
      for (int ch = 0; ch < pieces; ++ch) {
        const float4 k = *reinterpret_cast<const float4*>(ks + key_lane * C::kRowBytes + ((ch ^ key_lane) << 4));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float4 q = *reinterpret_cast<const float4*>(q_smem + (pair * 2 + t) * C::kQStride + ch * 4);
          acc[t] = fma2(make_float2(k.x, k.y), make_float2(q.x, q.y), acc[t]);
          acc[t] = fma2(make_float2(k.z, k.w), make_float2(q.z, q.w), acc[t]);
        }
      }
      const bool whole = valid == 0xffu && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      const int key = key0 + key_lane;
      bool grew = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float y = acc[t].x + acc[t].y;
        y = a.softcap > 0.f ? cap2 * tanhf(y * inv_cap) : y * scale2;
        if (a.slopes) y += slope[t] * static_cast<float>(key - pos[t]);
        const bool seen = whole || (((valid >> key_lane) & 1) && key <= pos[t] && (a.span == 0 || key > pos[t] - a.span));
        y = seen ? y : -INFINITY;
        float top = y;
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        const float now = fmaxf(m[t], top), from = now == -INFINITY ? 0.f : now;
        const float f = ex2(m[t] - from);
        grew |= now > m[t];
        const float w = ex2(y - from);
        l[t] = l[t] * f + w;
        m[t] = now;
        // a weight of a key that the row does not see is negative zero: its product is left out below
        weights[key_lane * C::kRows + pair * 2 + t] = seen ? w : -0.f;
        if (key_lane == 0) factors[pair * 2 + t] = f;
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int t = 0; t < C::kRows; ++t) {
          const float f = factors[t];
#pragma unroll
          for (int e = 0; e < OC; ++e) o[t][e] *= f;
        }
      }
#pragma unroll
      for (int j = 0; j < BK; ++j) {
        float v[OC];
        const unsigned char* vrow = vs + j * C::kRowBytes;
        if constexpr (OC == 2) {
          const int ch = lane >> 1;
          const float2 x = *reinterpret_cast<const float2*>(vrow + ((ch ^ j) << 4) + (lane & 1) * 8);
          v[0] = x.x; v[1] = x.y;
        } else {
#pragma unroll
          for (int c = 0; c < OC / 4; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(vrow + (((lane + 32 * c) ^ j) << 4));
            v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
          }
        }
        const float4 w0 = *reinterpret_cast<const float4*>(weights + j * C::kRows);
        const float4 w1 = *reinterpret_cast<const float4*>(weights + j * C::kRows + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        if (whole) {
#pragma unroll
          for (int t = 0; t < C::kRows; ++t)
#pragma unroll
            for (int e = 0; e < OC; e += 2) {
              const float2 x = fma2(make_float2(w[t], w[t]), make_float2(v[e], v[e + 1]), make_float2(o[t][e], o[t][e + 1]));
              o[t][e] = x.x;
              o[t][e + 1] = x.y;
            }
        } else {
#pragma unroll
          for (int t = 0; t < C::kRows; ++t)
            if (__float_as_uint(w[t]) != 0x80000000u)
#pragma unroll
              for (int e = 0; e < OC; ++e) o[t][e] += w[t] * v[e];
        }
      }
      __syncwarp();
    }

    cp_async_wait<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float x = l[t];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      if (key_lane == 0) {
        float* to = sums + (warp * C::kRows + pair * 2 + t) * (DP + 2) + DP;
        to[0] = m[t];
        to[1] = x;
      }
    }
#pragma unroll
    for (int t = 0; t < C::kRows; ++t) {
      float* to = sums + (warp * C::kRows + t) * (DP + 2);
      if constexpr (OC == 2) {
        to[2 * lane] = o[t][0];
        to[2 * lane + 1] = o[t][1];
      } else {
#pragma unroll
        for (int c = 0; c < OC / 4; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(lane + 32 * c) * 4 + e] = o[t][4 * c + e];
      }
    }
    __syncthreads();
    float* part = nullptr;
    if (n < r.tiles)
      part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * C::kRows * (a.D + 2);
    finish_part<DP, C::kRows, BF_OUT>(a, sums, b, hk, row0, rows, part);

    walk.left -= n;
    walk.tile = 0;
    if (walk.left > 0 && ++walk.item == a.HK * row_tiles) {
      walk.item = 0;
      ++walk.b;
      if (walk.b < a.B) walk.r = range_of<BK>(a, walk.b);
    }
  }
}

// ------------------------------------------------------------------ joining

// Block (c, r): row r of the item that stretch c begins inside, where c is the first to.  Parts c - 1 (its second
// place) and c, c + 1, .. (their first places) are added in a fixed order.  A warp takes every fourth part, then the
// warps' sums are added.
template <bool BF_OUT>
__global__ void __launch_bounds__(kThreads) join_kernel(const AttentionArgs a, int row_tiles, int tile_rows, const Join* joins,
                                                        const float* parts) {
  __shared__ float warp_l[kWarps], warp_o[kWarps][256];
  const Join j = joins[blockIdx.x];
  if (j.parts == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = j.item / row_tiles, row0 = (j.item - hk * row_tiles) * tile_rows, r = blockIdx.y;
  if (row0 + r >= a.W * (a.H / a.HK)) return;
  const int64_t row_floats = a.D + 2, part_floats = tile_rows * row_floats;
  const auto row_of = [&](int i) {
    const int64_t place = i == 0 ? 2 * (static_cast<int64_t>(blockIdx.x) - 1) + 1 : 2 * (static_cast<int64_t>(blockIdx.x) + i - 1);
    return parts + place * part_floats + r * row_floats;
  };
  float m = -INFINITY, l = 0.f, o[8] = {};
  for (int i = lane; i < j.parts; i += 32) m = fmaxf(m, __ldcg(row_of(i) + a.D));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  const float base = m == -INFINITY ? 0.f : m;
  for (int i = warp; i < j.parts; i += kWarps) {
    const float* p = row_of(i);
    const float f = ex2(__ldcg(p + a.D) - base);
    l += f * __ldcg(p + a.D + 1);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < a.D) o[e] += f * __ldcg(p + lane + 32 * e);
  }
  if (lane == 0) warp_l[warp] = l;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (lane + 32 * e < a.D) warp_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) l += warp_l[w];
  const RowPlace at = row_place(a, j.seq, hk, row0 + r);
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += warp_o[w][d];
    store_out<BF_OUT>(a, at.o * a.D + d, l == 0.f ? 0.f : x / l);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ host

constexpr int kMaxStretches = 152 * 4;       // of any variant on any device of this kind

struct Variant {
  int rows, ctas;                            // rows of a tile, CTAs an SM
};
Variant variant_of(bool bf16, int D, int rows) {
  if (!bf16) return Variant{8, D <= 64 ? 3 : D <= 128 ? 2 : 1};
  if (D > 128) return Variant{16, 1};
  return Variant{rows > 16 ? 32 : 16, D <= 64 ? 3 : 2};
}

int stretches_of(const Variant& v) { return std::min(kMaxStretches, sm_count() * v.ctas); }

template <auto K, typename Config>
cudaError_t run(const AttentionArgs& a, int row_tiles, int stretches, Join* joins, float* parts, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = raise_smem(K, Config::kSmem, done);
  if (e != cudaSuccess) return e;
  K<<<stretches, kThreads, Config::kSmem, st>>>(a, FastDiv(a.P), row_tiles, joins, parts);
  return cudaGetLastError();
}

template <bool BF_OUT>
cudaError_t launch(const AttentionArgs& a, bool bf16, cudaStream_t st) {
  const int rows = a.W * (a.H / a.HK);
  const Variant v = variant_of(bf16, a.D, rows);
  const int n = stretches_of(v), tiles = (rows + v.rows - 1) / v.rows;
  Join* joins = static_cast<Join*>(a.workspace);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kMaxStretches * sizeof(Join));
  cudaError_t e;
  if (bf16) {
    if (a.D <= 64) {
      e = v.rows == 16 ? run<attend_bf16_kernel<64, 1, 4, BF_OUT>, Mma<64, 1, 4>>(a, tiles, n, joins, parts, st)
                       : run<attend_bf16_kernel<64, 2, 4, BF_OUT>, Mma<64, 2, 4>>(a, tiles, n, joins, parts, st);
    } else if (a.D <= 128) {
      e = v.rows == 16 ? run<attend_bf16_kernel<128, 1, 3, BF_OUT>, Mma<128, 1, 3>>(a, tiles, n, joins, parts, st)
                       : run<attend_bf16_kernel<128, 2, 3, BF_OUT>, Mma<128, 2, 3>>(a, tiles, n, joins, parts, st);
    } else {
      e = run<attend_bf16_kernel<256, 1, 3, BF_OUT>, Mma<256, 1, 3>>(a, tiles, n, joins, parts, st);
    }
  } else {
    if (a.D <= 64) e = run<attend_f32_kernel<64, 4, BF_OUT>, Simt<64, 4>>(a, tiles, n, joins, parts, st);
    else if (a.D <= 128) e = run<attend_f32_kernel<128, 3, BF_OUT>, Simt<128, 3>>(a, tiles, n, joins, parts, st);
    else e = run<attend_f32_kernel<256, 3, BF_OUT>, Simt<256, 3>>(a, tiles, n, joins, parts, st);
  }
  if (e != cudaSuccess) return e;
  join_kernel<BF_OUT><<<dim3(n, std::min(v.rows, rows)), kThreads, 0, st>>>(a, tiles, v.rows, joins, parts);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attention_workspace(const kda_cache_params_t& p) {
  const int rows = p.window * (p.num_q_heads / p.num_kv_heads);
  const Variant v = variant_of(p.dtype == KDA_DTYPE_BF16, p.head_dim, rows);
  return kMaxStretches * sizeof(Join) +
         static_cast<size_t>(2) * stretches_of(v) * v.rows * (p.head_dim + 2) * sizeof(float);
}

cudaError_t launch_cache_attention(const AttentionArgs& a, bool bf16, bool bf16_out, cudaStream_t st) {
  return bf16_out ? launch<true>(a, bf16, st) : launch<false>(a, bf16, st);
}

}  // namespace kda
