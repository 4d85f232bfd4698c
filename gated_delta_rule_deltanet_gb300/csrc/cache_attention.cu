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
#include <type_traits>

#include "cache_common.cuh"

namespace kda {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A stretch is counted in tiles and what an item costs beside them: the ring runs empty at its end, and the
// warps' sums are joined.
constexpr int kItemCost = 2, kMinUnits = 4;

// A running maximum follows the scores only when one is this far above it (in powers of two): sums grow by up
// to 2^10 more than they need to, which fp32 holds without loss, and most blocks need no exchange between lanes.
constexpr float kSlack = 10.f;

struct Join {                                // where stretch c begins inside an item that began in an earlier one
  int32_t seq, item, parts, pad;             // parts == 0: nothing to join here
};

struct Range {                               // a sequence's keys
  int32_t len, first, begin, tiles;          // first visible key; begin: first rounded down to 16 keys
};

template <int TILE>
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
  r.begin = r.first & ~15;
  r.tiles = max(1, (r.len - r.begin + TILE - 1) / TILE);
  return r;
}

struct Walk {                                // a stretch, item by item
  int b, item, tile;                         // where it stands
  int64_t left;                              // units still to do
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

// Finds this CTA's stretch.  Every CTA adds the units of all sequences up (B numbers); stretch c of n begins at
// unit floor(c total / n).  Also notes where the CTA begins inside an item.
template <int TILE>
__device__ Walk find_stretch(const AttentionArgs& a, int items, Join* joins) {
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int32_t found;                  // the sequence in which the stretch begins
  __shared__ int64_t before;                 // and the units of those before it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += static_cast<int64_t>(range_of<TILE>(a, b).tiles + kItemCost) * items;
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
  const int c = blockIdx.x;
  const int n = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kMinUnits - 1) / kMinUnits));
  Walk w;
  w.left = 0;
  if (c >= n) {
    if (tid == 0) joins[c].parts = 0;
    return w;
  }
  // floor(c total / n) in parts that fit: total = k n + rest
  const int64_t k = total / n;
  const int rest = static_cast<int>(total - k * n);
  const auto begin_of = [&](int i) { return i * k + i * rest / n; };
  const int64_t t0 = begin_of(c), t1 = begin_of(c + 1);
  if (excl <= t0 && t0 < excl + mine) {
    for (int b = b0; b < b1; ++b) {
      const int64_t x = static_cast<int64_t>(range_of<TILE>(a, b).tiles + kItemCost) * items;
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
  w.r = range_of<TILE>(a, w.b);
  const int64_t at = t0 - before;
  const int units = w.r.tiles + kItemCost;
  w.item = at <= 0x7fffffff ? static_cast<int>(at) / units : static_cast<int>(at / units);
  w.tile = static_cast<int>(at - static_cast<int64_t>(w.item) * units);
  w.left = t1 - t0;
  if (tid == 0) {
    const int64_t begin = t0 - w.tile, end = begin + w.r.tiles;      // the item's tiles
    Join j{w.b, w.item, 0, 0};
    if (w.tile > 0 && w.tile < w.r.tiles && begin_of(c - 1) <= begin) {
      // the first stretch that begins inside the item: it, those after it that do, and the one before it
      int e = static_cast<int>(min(static_cast<int64_t>(n - 1), c + (end - 1 - t0) / k));
      while (e > c && begin_of(e) >= end) --e;
      j.parts = e - c + 2;
    }
    joins[c] = j;
  }
  return w;
}

// The next piece of the stretch: tiles [walk.tile, + n) of walk.item; false at the stretch's end.
template <int TILE>
__device__ __forceinline__ bool next_piece(const AttentionArgs& a, int items, Walk& w, int& n) {
  while (w.left > 0 && w.b < a.B) {
    n = static_cast<int>(min(w.left, static_cast<int64_t>(w.r.tiles - w.tile)));
    if (n > 0) return true;
    w.left -= w.r.tiles + kItemCost - w.tile;            // begins behind the item's tiles
    w.tile = 0;
    if (++w.item == items) {
      w.item = 0;
      if (++w.b < a.B) w.r = range_of<TILE>(a, w.b);
    }
  }
  return false;
}
template <int TILE>
__device__ __forceinline__ void piece_done(const AttentionArgs& a, int items, Walk& w) {
  w.left -= w.r.tiles + kItemCost - w.tile;
  w.tile = 0;
  if (w.left > 0 && ++w.item == items) {
    w.item = 0;
    if (++w.b < a.B) w.r = range_of<TILE>(a, w.b);
  }
}

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

// Parts in the workspace: ROWS rows of D sums, then ROWS pairs (m, l).  Stretch c leaves a part that began in an
// earlier stretch at place 2 c, one that goes on in a later stretch at 2 c + 1.
__device__ __forceinline__ int64_t part_floats(int rows, int D) { return static_cast<int64_t>(rows) * (D + 2); }

// Adds the groups' sums (in shared memory, rows of DP + 2 floats: o, m, l) up and writes the rows of a piece: final
// where the piece is the whole item, otherwise to the workspace.  A warp takes a row.
template <int DP, int ROWS, int GROUPS, bool BF_OUT>
__device__ void finish_piece(const AttentionArgs& a, const float* sums, int b, int hk, int row0, int rows, float* part) {
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < min(ROWS, rows - row0); r += kWarps) {
    float m = -INFINITY, f[GROUPS], l = 0.f;
#pragma unroll
    for (int w = 0; w < GROUPS; ++w) m = fmaxf(m, sums[(w * ROWS + r) * (DP + 2) + DP]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < GROUPS; ++w) {
      const float* s = sums + (w * ROWS + r) * (DP + 2);
      f[w] = ex2(s[DP] - base);
      l += f[w] * s[DP + 1];
    }
    const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);       // a NaN stays one
    const RowPlace at = row_place(a, b, hk, row0 + r);
#pragma unroll
    for (int d = lane; d < DP; d += 32) {
      if (d >= a.D) break;
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < GROUPS; ++w) x += f[w] * sums[(w * ROWS + r) * (DP + 2) + d];
      x = l == 0.f ? 0.f : x * inv;
      if (part) part[static_cast<int64_t>(r) * a.D + d] = x;
      else store_out<BF_OUT>(a, at.o * a.D + d, x);
    }
    if (lane == 0) {
      if (part) {
        float* ml = part + static_cast<int64_t>(ROWS) * a.D + 2 * r;
        ml[0] = m;
        ml[1] = l;
      } else if (a.lse) {
        a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// an 8 x 8 matrix of 16-bit elements, two a lane, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

__device__ __forceinline__ bool bf16x2_not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

// DP: the head's channels rounded up (zeros behind D).  RW warps, each with eight rows, share a ring and with
// it every block of BK keys; the 4 / RW groups take the blocks of a tile in turn.  H halves (the keys or the values of a
// block) make a ring.
template <int DP, int RW>
struct Mma {
  static constexpr int kGroups = kWarps / RW, kRows = 8 * RW, kRowBytes = DP * 2;
  static constexpr int kCopyRows = DP == 64 ? 4 : 2;           // rows that a lane copies a part of
  static constexpr int kBK = 8 * kCopyRows * RW;
  static constexpr int kHalves = DP == 256 ? 3 : 4, kHalf = kBK * kRowBytes;
  static constexpr int kRing = kGroups * kHalves * kHalf;
  static constexpr int kPart = kGroups * kRows * (DP + 2) * 4; // the groups' sums, over the rings
  static constexpr int kTop = kRing > kPart ? kRing : kPart;
  static constexpr int kQ = kRows * kRowBytes;
  static constexpr size_t kSmem = kTop + kQ;
  static constexpr int kCtas = DP == 256 ? 2 : 3;              // an SM, by shared memory and registers
};

// Scores and sums transposed: S^T = K Q^T and O^T += V^T P^T, keys and channels as the M of m16n8k16, rows
// as its N: eight rows fill it.  A lane's scores are those of keys lane / 4 (+ 8, ..) and rows 2 (lane mod 4), + 1, its
// part of O^T belongs to the same two rows, and a pair of packed weights becomes an operand by one transposition.
//
// The weights e^(s - m) enter the second product in two bf16 parts (16 bits), three (24) where o is stored in
// fp32: one part's rounding (2^-9) would be as large as that of a bf16 o.
template <int DP, int RW, bool BF_OUT>
__global__ void __launch_bounds__(kThreads, Mma<DP, RW>::kCtas)
    attend_bf16_kernel(const AttentionArgs a, FastDiv page_div, int row_tiles, Join* joins, float* parts) {
  using C = Mma<DP, RW>;
  constexpr int BK = C::kBK, H = C::kHalves, CR = C::kCopyRows, MB = BK / 16, PARTS = BF_OUT ? 2 : 3;
  constexpr int CH = DP / 8, KS = DP / 16;                     // 16-byte pieces of a row, steps along D
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp / RW, row_warp = warp % RW;
  const int rows = a.W * (a.H / a.HK), pieces = a.D / 8, items = a.HK * row_tiles;
  unsigned char* ring = smem + group * H * C::kHalf;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  unsigned char* q_smem = smem + C::kTop;
  const uint32_t q_u = static_cast<uint32_t>(__cvta_generic_to_shared(q_smem));
  const float scale2 = a.scale * kLog2e, cap2 = a.softcap * kLog2e, inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const auto group_sync = [&]() {
    if constexpr (RW == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * RW) : "memory");
  };

  // copies: this lane takes rows 8 (CR row_warp + x) + lane / 4, x < CR, pieces lane % 4, + 4, ..; piece p of row r
  // lies at p ^ (r mod 8), of which only the bit of 4 depends on the step
  const int row_c = lane >> 2, piece_c = lane & 3, row_first = 8 * CR * row_warp + row_c;
  const uint32_t to_even = row_first * C::kRowBytes + ((piece_c ^ row_c) << 4), to_odd = to_even ^ 64;
  // fragments: the same with the row that this lane names to ldmatrix; a step of 16 channels is two pieces
  const uint32_t k_frag = (lane & 15) * C::kRowBytes + ((((lane >> 4) & 1) ^ (lane & 7)) << 4);
  const uint32_t v_frag = ((lane & 7) + ((lane >> 4) << 3)) * C::kRowBytes + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);

  Walk walk = find_stretch<C::kGroups * BK>(a, items, joins);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n;
  while (next_piece<C::kGroups * BK>(a, items, walk, n)) {
    const int hk = walk.item / row_tiles, row0 = (walk.item - hk * row_tiles) * C::kRows;
    const Range r = walk.r;
    const int b = walk.b;
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
    const int64_t head = static_cast<int64_t>(hk) * a.page_head_stride + piece_c * 8;

    // The previous piece's sums are read; the rings' pieces behind D become zeros once more (its sums lay over
    // them), and the rows of q land beside the rings.
    __syncthreads();
    if (pieces < CH) {
      for (int i = tid; i < C::kGroups * H * BK * CH; i += kThreads) {
        const int row = i / CH, ch = i - row * CH;
        if (ch >= pieces)
          *reinterpret_cast<uint4*>(smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
    }

    // Block i of this group begins at key base(i); half 2 i is its keys, 2 i + 1 its values.
    const auto base = [&](int i) { return r.begin + ((walk.tile + i) * C::kGroups + group) * BK; };
    int page[CR];
    int64_t off[CR];                         // the rows of the newest block in the ring, or -1
    const auto pages_of = [&](int i) {
#pragma unroll
      for (int x = 0; x < CR; ++x) {
        const int key = base(i) + row_first + 8 * x;
        page[x] = i < n && key >= r.first && key < r.len ? table[page_div.div(key)] : -2;
      }
    };
    const auto copy_half = [&](const void* from, int h) {
      const uint32_t dst = ring_u + (h % H) * C::kHalf;
#pragma unroll
      for (int x = 0; x < CR; ++x) {
        const bool ok = off[x] >= 0;
        const uint16_t* src = static_cast<const uint16_t*>(from) + (ok ? off[x] : 0);
#pragma unroll
        for (int c = 0; c < CH / 4; ++c)
          if (c * 4 + piece_c < pieces)
            cp_async16(dst + ((c & 1) ? to_odd : to_even) + (c >> 1) * 128 + x * 8 * C::kRowBytes, src + (ok ? c * 32 : 0), ok);
      }
    };
    const auto issue = [&](int h) {
      const int i = h >> 1;
      if (i < n) {
        if (h & 1) {
          copy_half(a.v, h);
        } else {
#pragma unroll
          for (int x = 0; x < CR; ++x) {
            const int key = base(i) + row_first + 8 * x;
            off[x] = -1;
            if (static_cast<uint32_t>(page[x]) < static_cast<uint32_t>(a.num_pages)) {
              const int in_page = key - static_cast<int>(page_div.div(key)) * a.P;
              off[x] = page[x] * a.page_stride + in_page * a.page_row_stride + head;
            } else if (page[x] != -2) {
              raise_device_error(a.err, KDA_DEVERR_PAGE);
            }
          }
          copy_half(a.k, h);
          pages_of(i + 1);
        }
      }
      cp_async_commit();
    };

    pages_of(0);
#pragma unroll
    for (int h = 0; h < H - 1; ++h) issue(h);

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
    float m[2], l[2], o[KS][4], slope[2];
    int pos[2];                              // positions of this lane's rows
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
      const RowPlace at = row_place(a, b, hk, min(row0 + row_warp * 8 + piece_c * 2 + e, rows - 1));
      pos[e] = r.len - a.W + at.w;
      slope[e] = a.slopes ? a.slopes[at.h] * kLog2e : 0.f;
    }
#pragma unroll
    for (int d = 0; d < KS; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    __syncthreads();
    // q as the second operand: one ldmatrix holds two steps
    uint32_t qf[KS / 2][4];
#pragma unroll
    for (int kk = 0; kk < KS / 2; ++kk)
      ldmatrix4(qf[kk], (q_u + (row_warp * 8 + (lane & 7)) * C::kRowBytes + (((lane >> 3) ^ (lane & 7)) << 4)) ^ (kk << 6));

    for (int i = 0; i < n; ++i) {
      const int key0 = base(i);
      cp_async_wait<H - 2>();
      group_sync();
      issue(2 * i + H - 1);
      const uint32_t ks = ring_u + ((2 * i) % H) * C::kHalf;

      float s[MB][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS / 2; ++kk) {
        if (kk * 32 >= a.D) break;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          uint32_t k0[4], k1[4];
          const uint32_t at = ((ks + k_frag) ^ (kk << 6)) + mb * 16 * C::kRowBytes;
          ldmatrix4(k0, at);
          ldmatrix4(k1, at ^ 32);
          mma16816(s[mb], k0, qf[kk][0], qf[kk][1]);
          mma16816(s[mb], k1, qf[kk][2], qf[kk][3]);
        }
      }

      // Does every row see every key?  (the rows' positions are len - W .. len - 1)
      const bool whole = key0 >= r.first && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      const auto seen = [&](int key, int p) { return key >= r.first && key <= p && (a.span == 0 || key > p - a.span); };
      bool grows = false;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = s[mb][e];
          const int key = key0 + mb * 16 + row_c + (e >> 1) * 8, p = pos[e & 1];
          y = a.softcap > 0.f ? cap2 * tanhf(y * inv_cap) : y * scale2;
          if (a.slopes) y += slope[e & 1] * static_cast<float>(key - p);
          if (!whole) y = seen(key, p) ? y : -INFINITY;
          s[mb][e] = y;
          grows |= y > m[e & 1] + kSlack;
        }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) top = fmaxf(top, fmaxf(s[mb][e], s[mb][e + 2]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float now = fmaxf(m[e], top);
          const float f = ex2(m[e] - (now == -INFINITY ? 0.f : now));
          m[e] = now;
          l[e] *= f;
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[d][e] *= f;
            o[d][e + 2] *= f;
          }
        }
      }
      uint32_t pf[MB][PARTS][2];
      const float from[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mb][e] = ex2(s[mb][e] - from[e & 1]);
          l[e & 1] += s[mb][e];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y0 = s[mb][2 * j], y1 = s[mb][2 * j + 1];
#pragma unroll
          for (int x = 0; x < PARTS; ++x) {
            const uint32_t w = pack_bf16(y0, y1);
            pf[mb][x][j] = transpose8(w);
            y0 -= __uint_as_float(w << 16);
            y1 -= __uint_as_float(w & 0xffff0000u);
          }
        }
      }

      cp_async_wait<H - 2>();
      group_sync();
      issue(2 * i + H);
      const uint32_t vs = ring_u + ((2 * i + 1) % H) * C::kHalf;
      bool poison = false;
      if (!whole) {
        // A value that is not finite would reach the rows whose mask leaves it out as 0 x infinity.
        bool bad = false;
        for (int x = lane; x < BK * CH; x += 32) {
          const uint4 y = *reinterpret_cast<const uint4*>(ring + (vs - ring_u) + x * 16);
          bad |= bf16x2_not_finite(y.x) | bf16x2_not_finite(y.y) | bf16x2_not_finite(y.z) | bf16x2_not_finite(y.w);
        }
        poison = __any_sync(0xffffffffu, bad);
      }
      if (poison) {
        // key by key, leaving out what a row does not see
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
#pragma unroll 1
          for (int j = 0; j < 16; ++j) {
            const int src = ((j & 7) << 2) | (lane & 3), key = key0 + mb * 16 + j;
            const float u0 = __shfl_sync(0xffffffffu, s[mb][0], src), u1 = __shfl_sync(0xffffffffu, s[mb][1], src);
            const float u2 = __shfl_sync(0xffffffffu, s[mb][2], src), u3 = __shfl_sync(0xffffffffu, s[mb][3], src);
            const float w[2] = {j < 8 ? u0 : u2, j < 8 ? u1 : u3};
            const unsigned char* v = ring + (vs - ring_u) + (mb * 16 + j) * C::kRowBytes;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!seen(key, pos[e])) continue;
#pragma unroll
              for (int d = 0; d < KS; ++d)
#pragma unroll
                for (int h = 0; h < 2; ++h) {          // channel 16 d + 8 h + lane / 4
                  const uint16_t x = *reinterpret_cast<const uint16_t*>(v + (((d * 2 + h) ^ (j & 7)) << 4) + row_c * 2);
                  o[d][2 * h + e] += w[e] * bf16_bits_to_f32(x);
                }
            }
          }
        }
      } else {
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          if (d * 16 >= a.D) break;
          float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            uint32_t vf[4];
            ldmatrix4_trans(vf, ((vs + v_frag) ^ (d << 5)) + mb * 16 * C::kRowBytes);
            if constexpr (BF_OUT) {
              mma16816(o[d], vf, pf[mb][0][0], pf[mb][0][1]);
              mma16816(o[d], vf, pf[mb][1][0], pf[mb][1][1]);
            } else {
              // the tensor cores cut their sums off, which over a long cache would lean one way: those of a block
              // are formed by themselves and added in fp32
#pragma unroll
              for (int y = PARTS - 1; y >= 0; --y) mma16816(x, vf, pf[mb][y][0], pf[mb][y][1]);
            }
          }
          if constexpr (!BF_OUT) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] += x[e];
          }
        }
      }
    }

    // the groups' sums, over the rings
    cp_async_wait<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      float* to = sums + (group * C::kRows + row_warp * 8 + piece_c * 2 + e) * (DP + 2);
#pragma unroll
      for (int d = 0; d < KS; ++d) {
        to[d * 16 + row_c] = o[d][e];
        to[d * 16 + 8 + row_c] = o[d][e + 2];
      }
      if (row_c == 0) {
        to[DP] = m[e];
        to[DP + 1] = x;
      }
    }
    __syncthreads();
    float* part = nullptr;
    if (n < r.tiles) part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * part_floats(C::kRows, a.D);
    finish_piece<DP, C::kRows, C::kGroups, BF_OUT>(a, sums, b, hk, row0, rows, part);
    piece_done<C::kGroups * BK>(a, items, walk);
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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = a.H / a.HK, rows = a.W * g, pieces = a.D / 4, items = a.HK * row_tiles;
  unsigned char* ring = smem + warp * STAGES * C::kStage;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  constexpr int kTop = C::kRing > C::kPart ? C::kRing : C::kPart;
  float* q_smem = reinterpret_cast<float*>(smem + kTop);
  float* weights = reinterpret_cast<float*>(smem + kTop + C::kQ) + warp * BK * C::kRows;   // [key][row]
  float* factors = reinterpret_cast<float*>(smem + kTop + C::kQ) + kWarps * BK * C::kRows + warp * C::kRows;
  const float scale2 = a.scale * kLog2e, cap2 = a.softcap * kLog2e, inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const int key_lane = lane & 7, pair = lane >> 3;

  // copies: this lane takes row lane / 4 of a block, pieces lane % 4, + 4, ..; piece x of row r lies at x ^ r
  const int row_c = lane >> 2, piece_c = lane & 3;
  const uint32_t to_even = row_c * C::kRowBytes + ((piece_c ^ row_c) << 4), to_odd = to_even ^ 64;

  Walk walk = find_stretch<kWarps * BK>(a, items, joins);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n;
  while (next_piece<kWarps * BK>(a, items, walk, n)) {
    const int hk = walk.item / row_tiles, row0 = (walk.item - hk * row_tiles) * C::kRows;
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

    // block i of this warp begins at key base(i); this lane copies key base(i) + row_c
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
    const auto base = [&](int i) { return r.begin + ((walk.tile + i) * kWarps + warp) * BK; };
    const auto inside = [&](int i, int key) { return i < n && key >= r.first && key < r.len; };
    const auto page_of = [&](int i) {
      const int key = base(i) + row_c;
      return inside(i, key) ? table[page_div.div(key)] : -1;
    };
    uint32_t flags = 0;                      // a bit a stage, the newest lowest: is this lane's key there?
    const auto issue = [&](int i, int page) {
      const int key = base(i) + row_c;
      const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages);
      if (!ok && inside(i, key)) raise_device_error(a.err, KDA_DEVERR_PAGE);
      flags = (flags << 1) | (ok ? 1u : 0u);
      if (i < n) {
        const int in_page = key - static_cast<int>(page_div.div(key)) * a.P;
        const int64_t off = ok ? page * a.page_stride + in_page * a.page_row_stride +
                                     static_cast<int64_t>(hk) * a.page_head_stride + piece_c * 4 : 0;
        const float *k = static_cast<const float*>(a.k) + off, *v = static_cast<const float*>(a.v) + off;
        const uint32_t dst = ring_u + (i % STAGES) * C::kStage;
#pragma unroll
        for (int c = 0; c < CH / 4; ++c) {
          if (c * 4 + piece_c >= pieces) break;
          const uint32_t at = dst + ((c & 1) ? to_odd : to_even) + (c >> 1) * 128;
          cp_async16(at, ok ? k + c * 16 : k, ok);
          cp_async16(at + BK * C::kRowBytes, ok ? v + c * 16 : v, ok);
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
      const uint32_t there = __ballot_sync(0xffffffffu, (flags >> (STAGES - 1)) & 1u);   // key j's at bit 4 j

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
      const bool whole = there == 0xffffffffu && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      const int key = key0 + key_lane;
      bool grew = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float y = acc[t].x + acc[t].y;
        y = a.softcap > 0.f ? cap2 * tanhf(y * inv_cap) : y * scale2;
        if (a.slopes) y += slope[t] * static_cast<float>(key - pos[t]);
        const bool seen = whole || (((there >> (4 * key_lane)) & 1) && key <= pos[t] && (a.span == 0 || key > pos[t] - a.span));
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
    if (n < r.tiles) part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * part_floats(C::kRows, a.D);
    finish_piece<DP, C::kRows, kWarps, BF_OUT>(a, sums, b, hk, row0, rows, part);
    piece_done<kWarps * BK>(a, items, walk);
  }
}

// ------------------------------------------------------------------ joining

// Block (c, r): row r of the item that stretch c begins inside, where c is the first to.  Parts c - 1 (its second
// place) and c, c + 1, .. (their first places) are added in a fixed order: a warp takes every eighth part, then the
// warps' sums are added.  A chain of loads: the maxima, then the rows, four in flight for each warp.
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;

template <bool BF_OUT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttentionArgs a, int row_tiles, int tile_rows,
                                                            const Join* joins, const float* parts) {
  __shared__ float warp_l[kJoinWarps];
  __shared__ float4 warp_o[kJoinWarps][64];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 raw = __ldcg(reinterpret_cast<const int4*>(joins) + blockIdx.x);
  const Join j{raw.x, raw.y, raw.z, 0};
  if (j.parts == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = j.item / row_tiles, row0 = (j.item - hk * row_tiles) * tile_rows, r = blockIdx.y;
  if (row0 + r >= a.W * (a.H / a.HK)) return;
  const int64_t stride = part_floats(tile_rows, a.D);
  const auto part_of = [&](int i) {
    return parts + stride * (i == 0 ? 2 * (static_cast<int64_t>(blockIdx.x) - 1) + 1 : 2 * (static_cast<int64_t>(blockIdx.x) + i - 1));
  };
  const auto ml_of = [&](int i) {
    return __ldcg(reinterpret_cast<const float2*>(part_of(i) + static_cast<int64_t>(tile_rows) * a.D) + r);
  };
  const int pieces = a.D / 4;
  float m = -INFINITY, l = 0.f;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i = lane; i < j.parts; i += 32) m = fmaxf(m, ml_of(i).x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int i = warp; i < j.parts; i += kJoinWarps) {
    const float2 ml = ml_of(i);
    const float4* p = reinterpret_cast<const float4*>(part_of(i) + static_cast<int64_t>(r) * a.D);
    const float f = ex2(ml.x - base);
    l += f * ml.y;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < pieces) {
        const float4 x = __ldcg(p + lane + 32 * e);
        o[e].x += f * x.x;
        o[e].y += f * x.y;
        o[e].z += f * x.z;
        o[e].w += f * x.w;
      }
  }
  if (lane == 0) warp_l[warp] = l;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < pieces) warp_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += warp_l[w];
  const RowPlace at = row_place(a, j.seq, hk, row0 + r);
  if (threadIdx.x < a.D) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) x += reinterpret_cast<const float*>(warp_o[w])[threadIdx.x];
    store_out<BF_OUT>(a, at.o * a.D + threadIdx.x, l == 0.f ? 0.f : x / l);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ host

constexpr int kMaxStretches = 152 * 4;       // of any variant on any device of this kind

struct Variant {
  int rows, ctas;                            // rows of a tile, CTAs an SM
};
Variant variant_of(bool bf16, int D, int rows) {
  if (!bf16) return Variant{8, D <= 64 ? 4 : D <= 128 ? 3 : 1};
  return Variant{rows > 16 ? 32 : rows > 8 ? 16 : 8, D > 128 ? 2 : 3};
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
  const auto bf16_of = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    if (v.rows == 8) return run<attend_bf16_kernel<DP, 1, BF_OUT>, Mma<DP, 1>>(a, tiles, n, joins, parts, st);
    if (v.rows == 16) return run<attend_bf16_kernel<DP, 2, BF_OUT>, Mma<DP, 2>>(a, tiles, n, joins, parts, st);
    return run<attend_bf16_kernel<DP, 4, BF_OUT>, Mma<DP, 4>>(a, tiles, n, joins, parts, st);
  };
  if (bf16) {
    e = a.D <= 64    ? bf16_of(std::integral_constant<int, 64>{})
        : a.D <= 128 ? bf16_of(std::integral_constant<int, 128>{})
                     : bf16_of(std::integral_constant<int, 256>{});
  } else {
    if (a.D <= 64) e = run<attend_f32_kernel<64, 3, BF_OUT>, Simt<64, 3>>(a, tiles, n, joins, parts, st);
    else if (a.D <= 128) e = run<attend_f32_kernel<128, 2, BF_OUT>, Simt<128, 2>>(a, tiles, n, joins, parts, st);
    else e = run<attend_f32_kernel<256, 3, BF_OUT>, Simt<256, 3>>(a, tiles, n, joins, parts, st);
  }
  if (e != cudaSuccess) return e;
  // launched while the stretches still run: its blocks wait for them on the device
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(n, std::min(v.rows, rows));
  config.blockDim = dim3(kJoinThreads);
  config.stream = st;
  cudaLaunchAttribute attribute;
  attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attribute.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attribute;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, join_kernel<BF_OUT>, a, tiles, v.rows, static_cast<const Join*>(joins),
                            static_cast<const float*>(parts));
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
