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
// Bound by HBM: each key and value is read once for up to 64 rows of its group (queries x heads of one key head), 32 where
// heads are wider than 128 and 8 with fp32 pages; more rows read it once more for each such tile of rows.  The
// work is cut into tiles of keys of an item (a sequence, a key head and one of its tiles of rows), and the row of all
// tiles into equal stretches, one for each CTA, whatever the sequences' lengths: a stretch that begins or ends inside an
// item leaves (m, l, unnormalised o) of its part in the workspace, and a second kernel joins the parts in the order of
// the stretches, so that repeated calls give the same bits.  The lengths stay on the device: a captured graph follows
// them.
//
// Inside a CTA four warps form groups of one, two or four, as the rows of an item ask for.  A group takes every
// so many-th block of keys, copies it into a ring of its own in shared memory (cp.async, rows of 16-byte pieces stored at
// piece ^ (row mod 8)) and keeps m, l and o for itself, so that groups wait for one another only where a piece ends.
//
//   bf16   products by mma.sync with fp32 accumulators: at eight rows the tensor pipe is active for 14% of the time that
//          the copies take, so the tensor memory path, whose smallest M is 64 and whose accumulators come back through
//          tcgen05.ld, would have nothing to give.
//   fp32   CUDA cores throughout.  Products of two tf32 parts on tensor cores took 282 us where these take 194 (64
//          sequences, 1.2 GB) and left 1.2e-6 of the norm where these leave 1.2e-7.
//
// One GB300 (of measured HBM): 256 sequences of 256 to 8192 keys, 8 key heads of 128, 2.2 GB of bf16 pages 345-356 us
// (92-95%); 3 sequences of up to 262144 keys 150-156 us (91-95%); heads of 64 75-81%, of 256 79%; 32 and 64 rows a key
// head 76% and 31%; fp32 pages 87-93% with two rows, 75% with eight.  One sequence of 5000 keys 9.9 us: a chain of some
// 12 k cycles through both kernels.
#include <algorithm>
#include <type_traits>

#include "cache_common.cuh"

namespace kda {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A stretch is counted in units: tiles, and what an item costs beside them (the ring runs empty at its end, and the
// groups' sums are joined).  61 short sequences with costs of 1, 2 and 4: 30.4, 27.5, 31.3 us; one sequence of 5000 keys
// in stretches of 2 units 9.9 us, of 4 12.0.
constexpr int kItemCost = 2, kMinUnits = 2;

// A running maximum follows the scores only when one is this far above it (in powers of two): sums grow by up
// to 2^10 more than they need to, and most blocks need no exchange between lanes.
constexpr float kSlack = 10.f;

// Sums of weighted values from 2^115 (kLarge) on might overflow, if not now then where up to four groups and 608 parts
// are added, although their quotient by l does not.  A piece with such sums is done again with weights times 2^-33
// (`shrink`), so that values up to the end of fp32's range add up over 2^22 keys; l is scaled alike and m raised by 33.
// What this costs every call: 0.3 us of 27 (fp32 drafts), 1 of 111 (64 rows); elsewhere nothing to be seen.
constexpr float kLarge = 0x1p115f, kShrink = 33.f;
__device__ __forceinline__ float shrink(float w) {           // what is above zero stays so: an infinite value remains one
  return w > 0.f ? fmaxf(w * 0x1p-33f, 0x1p-149f) : w;
}
// raises m, from a whole number on, which is exact; returns the factor of l and o that goes with the rounding up
__device__ __forceinline__ float raise(float& m) {
  const float whole = ceilf(m), f = ex2(m == -INFINITY ? 0.f : m - whole);
  m = whole + kShrink;
  return f;
}
__device__ __forceinline__ float max_nan(float x, float y) { // NaN where one of the two is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

struct Join {                                // an item that several stretches share
  int32_t seq, item, parts, stretch;         // stretch: the first that begins inside it; parts == 0: nothing to join
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
    r.len = 0;
  }
  r.first = a.span ? static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(r.len) - a.W - a.span + 1)) : 0;
  r.first = min(r.first, r.len);
  r.begin = r.first & ~15;
  r.tiles = max(1, (r.len - r.begin + TILE - 1) / TILE);
  return r;
}

struct Walk {                                // a stretch, item by item
  int b, item, tile;                         // where it stands
  int left;                                  // units still to do
  int n, k, rest, begin;                     // n stretches; stretch i begins at unit i k + i rest / n
  Range r;
  __device__ __forceinline__ int begin_of(int i) const {
    return i * k + static_cast<uint32_t>(i * rest) / static_cast<uint32_t>(n);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Finds this CTA's stretch.  Every CTA adds the units of all sequences up (B numbers, fewer than 2^31 units in all);
// stretch c of n begins at unit floor(c total / n).
template <int TILE>
__device__ Walk find_stretch(const AttentionArgs& a, int items) {
  __shared__ int warp_sum[kWarps];
  __shared__ Walk found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int mine = 0;
  Range r{};
  for (int b = b0; b < b1; ++b) {
    r = range_of<TILE>(a, b);
    mine += (r.tiles + kItemCost) * items;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int total = 0, excl = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) excl += warp_sum[w];
    total += warp_sum[w];
  }
  const int c = blockIdx.x;
  Walk w;
  w.n = min(static_cast<int>(gridDim.x), (total + kMinUnits - 1) / kMinUnits);
  w.left = 0;
  if (c >= w.n) return w;
  w.k = static_cast<uint32_t>(total) / static_cast<uint32_t>(w.n);           // total = k n + rest
  w.rest = total - w.k * w.n;
  w.begin = w.begin_of(c);
  w.left = w.begin_of(c + 1) - w.begin;
  if (excl <= w.begin && w.begin < excl + mine) {
    for (int b = b0; b < b1; ++b) {
      if (per > 1) r = range_of<TILE>(a, b);
      const int units = r.tiles + kItemCost;
      if (w.begin < excl + units * items) {
        w.b = b;
        w.r = r;
        w.item = static_cast<uint32_t>(w.begin - excl) / static_cast<uint32_t>(units);
        w.tile = w.begin - excl - w.item * units;
        found = w;
        break;
      }
      excl += units * items;
    }
  }
  __syncthreads();
  return found;
}

// Leaves word of the items that have to be joined, for the join kernel's block `at`: with as many blocks as items
// (few items) that of the item, otherwise that of the stretch which is the first to begin inside it.
__device__ __forceinline__ void note_joins(const AttentionArgs& a, const Walk& w, int items, int join_blocks, Join* joins) {
  const int c = blockIdx.x;
  Join j{w.b, w.item, 0, c};                 // of a stretch without work: parts 0
  if (w.left > 0 && w.tile > 0 && w.tile < w.r.tiles) {
    const int first = w.begin - w.tile, end = first + w.r.tiles;             // the item's tiles
    if (w.begin_of(c - 1) <= first) {        // the first stretch to begin here: those after it that do, too
      int e = c + min(w.n - 1 - c, static_cast<int>(static_cast<uint32_t>(end - 1 - w.begin) / static_cast<uint32_t>(w.k)));
      while (e > c && w.begin_of(e) >= end) --e;
      j.parts = e - c + 2;
    }
  }
  if (static_cast<int64_t>(a.B) * items > join_blocks) joins[c] = j;
  else if (j.parts) joins[w.b * items + w.item] = j;
}
__device__ __forceinline__ void note_whole(const AttentionArgs& a, const Walk& w, int items, int join_blocks, Join* joins) {
  if (static_cast<int64_t>(a.B) * items <= join_blocks) joins[w.b * items + w.item].parts = 0;
}

// The next piece of the stretch: tiles [walk.tile, + n) of walk.item; false at the stretch's end.
template <int TILE>
__device__ __forceinline__ bool next_piece(const AttentionArgs& a, int items, Walk& w, int& n) {
  while (w.left > 0 && w.b < a.B) {
    n = min(w.left, w.r.tiles - w.tile);
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

// two channels; o need only be aligned to its elements
template <bool BF_OUT>
__device__ __forceinline__ void store_out2(const AttentionArgs& a, int64_t at, float2 x) {
  if constexpr (BF_OUT) {
    uint16_t* o = static_cast<uint16_t*>(a.o) + at;
    o[0] = f32_to_bf16_bits(x.x);
    o[1] = f32_to_bf16_bits(x.y);
  } else {
    float* o = static_cast<float*>(a.o) + at;
    o[0] = x.x;
    o[1] = x.y;
  }
}

// Parts in the workspace: ROWS rows of D sums, then ROWS pairs (m, l).  Stretch c leaves a part that began in an
// earlier stretch at place 2 c, one that goes on in a later stretch at 2 c + 1.
__device__ __forceinline__ int64_t part_floats(int rows, int D) { return static_cast<int64_t>(rows) * (D + 2); }

// Adds the groups' sums (in shared memory, rows of DP + 2 floats: o, m, l) up and writes the rows of a piece: final
// where the piece is the whole item, otherwise to the workspace.  Sixteen threads take a row. 
template <int DP, int ROWS, int GROUPS, bool BF_OUT>
__device__ void finish_piece(const AttentionArgs& a, const float* sums, int b, int hk, int row0, int rows, float* part) {
  const int x0 = threadIdx.x & 15;
#pragma unroll
  for (int pass = 0; pass < (ROWS + kThreads / 16 - 1) / (kThreads / 16); ++pass) {
    const int r = pass * (kThreads / 16) + (threadIdx.x >> 4);
    if (r >= min(ROWS, rows - row0)) break;
    float m = -INFINITY, f[GROUPS], l = 0.f;
#pragma unroll
    for (int w = 0; w < GROUPS; ++w) m = fmaxf(m, sums[(w * ROWS + r) * (DP + 2) + DP]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < GROUPS; ++w) {
      const float2 ml = *reinterpret_cast<const float2*>(sums + (w * ROWS + r) * (DP + 2) + DP);
      f[w] = ex2(ml.x - base);
      l += f[w] * ml.y;
    }
    const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);       // a NaN stays one
    const RowPlace at = row_place(a, b, hk, row0 + r);
#pragma unroll
    for (int d = 2 * x0; d < DP; d += 32) {
      if (d >= a.D) break;
      float2 x = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < GROUPS; ++w) {
        const float2 y = *reinterpret_cast<const float2*>(sums + (w * ROWS + r) * (DP + 2) + d);
        x = fma2(make_float2(f[w], f[w]), y, x);
      }
      x = l == 0.f ? make_float2(0.f, 0.f) : make_float2(x.x * inv, x.y * inv);
      if (part) *reinterpret_cast<float2*>(part + static_cast<int64_t>(r) * a.D + d) = x;
      else store_out2<BF_OUT>(a, at.o * a.D + d, x);
    }
    if (x0 == 0) {
      if (part) *reinterpret_cast<float2*>(part + static_cast<int64_t>(ROWS) * a.D + 2 * r) = make_float2(m, l);
      else if (a.lse) a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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

// DP: the head's channels rounded up (zeros behind D).  RW warps, each with NT tiles of eight rows, share a ring and
// with it every block of BK keys; the 4 / RW groups take the blocks of a tile in turn.  H halves (the keys or the values of
// a block) make a ring.
template <int DP, int RW, int NT>
struct Mma {
  static constexpr int kGroups = kWarps / RW, kRows = 8 * NT * RW, kRowBytes = DP * 2;
  static constexpr int kCopyRows = DP == 64 ? 4 : 2;           // rows that a lane copies a part of
  static constexpr int kBK = 8 * kCopyRows * RW;
  static constexpr int kHalves = DP == 256 ? 3 : 4, kHalf = kBK * kRowBytes;
  static constexpr int kRing = kGroups * kHalves * kHalf;
  static constexpr int kPart = kGroups * kRows * (DP + 2) * 4; // the groups' sums, over the rings
  static constexpr int kTop = kRing > kPart ? kRing : kPart;
  static constexpr int kQ = kRows * kRowBytes;
  static constexpr size_t kSmem = kTop + kQ;
  // an SM, by shared memory and registers; four with rings of three halves: 352 us where three take 345 (2.2 GB)
  static constexpr int kCtas = DP == 256 || NT == 2 ? 2 : 3;
};

// Scores and sums transposed: S^T = K Q^T and O^T += V^T P^T, keys and channels as the M of m16n8k16, rows
// as its N: eight rows fill it.  A lane's scores are those of keys lane / 4 (+ 8, ..) and rows 2 (lane mod 4), + 1, its
// part of O^T belongs to the same two rows, and a pair of packed weights becomes an operand by one transposition.
//
// The weights e^(s - m) enter the second product in two bf16 parts (16 bits), three (24) where o is stored in
// fp32: one part's rounding (2^-9) would be as large as that of a bf16 o.
//
// Weights and parts of zero turn an infinite value into a NaN, also where a row's mask leaves its key out.  So a piece
// whose sums do not come out finite, or too large, is done again with `exact` set: the weighted sums key by key on CUDA
// cores, of what a row sees alone, scaled as said at kShrink.
template <int DP, int RW, int NT, bool BF_OUT>
__global__ void __launch_bounds__(kThreads, Mma<DP, RW, NT>::kCtas)
    attend_bf16_kernel(const AttentionArgs a, FastDiv page_div, int row_tiles, int join_blocks, Join* joins,
                       float* parts) {
  using C = Mma<DP, RW, NT>;
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

  Walk walk = find_stretch<C::kGroups * BK>(a, items);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool noted = false, exact = false;
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
    int page[CR], page_after[CR];            // of the next block to be copied and the one after it
    int64_t off[CR];                         // the rows of the newest block in the ring, or -1
    const auto pages_of = [&](int i, int (&to)[CR]) {
#pragma unroll
      for (int x = 0; x < CR; ++x) {
        const int key = base(i) + row_first + 8 * x;
        to[x] = i < n && key >= r.first && key < r.len ? table[page_div.div(key)] : -1;
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
            cp_async16(dst + ((c & 1) ? to_odd : to_even) + (c >> 1) * 128 + x * 8 * C::kRowBytes,
                       src + (ok ? c * 32 : 0), ok);
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
            } else if (key >= r.first && key < r.len) {       // any other entry is a bad one; zeros are read
              raise_device_error(a.err, KDA_DEVERR_PAGE);
            }
          }
          copy_half(a.k, h);
#pragma unroll
          for (int x = 0; x < CR; ++x) page[x] = page_after[x];
          pages_of(i + 2, page_after);
        }
      }
      cp_async_commit();
    };

    pages_of(0, page);
    pages_of(1, page_after);
    constexpr int QN = (C::kRows * CH + kThreads - 1) / kThreads;
    uint4 q[QN];
#pragma unroll
    for (int x = 0; x < QN; ++x) {
      const int i = tid + x * kThreads, row = i / CH, ch = i - row * CH;
      q[x] = make_uint4(0, 0, 0, 0);
      if (row < C::kRows && row0 + row < rows && ch < pieces) {
        const RowPlace at = row_place(a, b, hk, row0 + row);
        q[x] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                               (static_cast<int64_t>(b) * a.W + at.w) * a.q_stride +
                                               static_cast<int64_t>(at.h) * a.D + ch * 8);
      }
    }
#pragma unroll 1
    for (int h = 0; h < H - 1; ++h) issue(h);

    if (!noted && tid == 0) note_joins(a, walk, items, join_blocks, joins);  // while the copies are under way
    noted = true;
#pragma unroll
    for (int x = 0; x < QN; ++x) {
      const int i = tid + x * kThreads, row = i / CH, ch = i - row * CH;
      if (row < C::kRows) *reinterpret_cast<uint4*>(q_smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = q[x];
    }
    float m[NT][2], l[NT][2], o[NT][KS][4], slope[NT][2];
    int pos[NT][2];                          // positions of this lane's rows
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = -INFINITY;
        l[t][e] = 0.f;
        const RowPlace at = row_place(a, b, hk, min(row0 + (row_warp * NT + t) * 8 + piece_c * 2 + e, rows - 1));
        pos[t][e] = r.len - a.W + at.w;
        slope[t][e] = a.slopes ? a.slopes[at.h] * kLog2e : 0.f;
      }
#pragma unroll
      for (int d = 0; d < KS; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;
    }
    __syncthreads();
    // q as the second operand: one ldmatrix holds two steps
    uint32_t qf[NT][KS / 2][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int kk = 0; kk < KS / 2; ++kk)
        ldmatrix4(qf[t][kk], (q_u + ((row_warp * NT + t) * 8 + (lane & 7)) * C::kRowBytes +
                              (((lane >> 3) ^ (lane & 7)) << 4)) ^ (kk << 6));

    for (int i = 0; i < n; ++i) {
      const int key0 = base(i);
      cp_async_wait<H - 2>();
      group_sync();
      issue(2 * i + H - 1);
      const uint32_t ks = ring_u + ((2 * i) % H) * C::kHalf;

      float s[NT][MB][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][mb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS / 2; ++kk) {
        if (kk * 32 >= a.D) break;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          uint32_t k0[4], k1[4];
          const uint32_t at = ((ks + k_frag) ^ (kk << 6)) + mb * 16 * C::kRowBytes;
          ldmatrix4(k0, at);
          ldmatrix4(k1, at ^ 32);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816(s[t][mb], k0, qf[t][kk][0], qf[t][kk][1]);
            mma16816(s[t][mb], k1, qf[t][kk][2], qf[t][kk][3]);
          }
        }
      }

      // Does every row see every key?  (the rows' positions are len - W .. len - 1)
      const bool whole = key0 >= r.first && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      const auto seen = [&](int key, int p) { return key >= r.first && key <= p && (a.span == 0 || key > p - a.span); };
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = s[t][mb][e];
            const int key = key0 + mb * 16 + row_c + (e >> 1) * 8, p = pos[t][e & 1];
            y = a.softcap > 0.f ? cap2 * tanhf(y * inv_cap) : y * scale2;
            if (a.slopes) y += slope[t][e & 1] * static_cast<float>(key - p);
            if (!whole) y = seen(key, p) ? y : -INFINITY;
            s[t][mb][e] = y;
            grows |= y > m[t][e & 1] + kSlack;
          }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -INFINITY;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) top = fmaxf(top, fmaxf(s[t][mb][e], s[t][mb][e + 2]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float now = fmaxf(m[t][e], top);
            const float f = ex2(m[t][e] - (now == -INFINITY ? 0.f : now));
            m[t][e] = now;
            l[t][e] *= f;
#pragma unroll
            for (int d = 0; d < KS; ++d) {
              o[t][d][e] *= f;
              o[t][d][e + 2] *= f;
            }
          }
      }
      uint32_t pf[NT][MB][PARTS][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float from[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[t][mb][e] = ex2(s[t][mb][e] - from[e & 1]);
            l[t][e & 1] += s[t][mb][e];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float y0 = s[t][mb][2 * j], y1 = s[t][mb][2 * j + 1];
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              const uint32_t w = pack_bf16(y0, y1);
              pf[t][mb][x][j] = transpose8(w);
              y0 -= __uint_as_float(w << 16);
              y1 -= __uint_as_float(w & 0xffff0000u);
            }
          }
        }
      }

      cp_async_wait<H - 2>();
      group_sync();
      issue(2 * i + H);
      const uint32_t vs = ring_u + ((2 * i + 1) % H) * C::kHalf;
      if (exact) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
              const int src = ((j & 7) << 2) | (lane & 3), key = key0 + mb * 16 + j;
              const float u0 = __shfl_sync(0xffffffffu, s[t][mb][0], src), u1 = __shfl_sync(0xffffffffu, s[t][mb][1], src);
              const float u2 = __shfl_sync(0xffffffffu, s[t][mb][2], src), u3 = __shfl_sync(0xffffffffu, s[t][mb][3], src);
              const float w[2] = {shrink(j < 8 ? u0 : u2), shrink(j < 8 ? u1 : u3)};
              const unsigned char* v = ring + (vs - ring_u) + (mb * 16 + j) * C::kRowBytes;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (!seen(key, pos[t][e])) continue;
#pragma unroll
                for (int d = 0; d < KS; ++d)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {        // channel 16 d + 8 h + lane / 4
                    const uint16_t x = *reinterpret_cast<const uint16_t*>(v + (((d * 2 + h) ^ (j & 7)) << 4) + row_c * 2);
                    o[t][d][2 * h + e] += w[e] * bf16_bits_to_f32(x);
                  }
              }
            }
          }
      } else {
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          if (d * 16 >= a.D) break;
          // For an fp32 o the sums of a block are formed by themselves and added in fp32: the tensor cores cut their sums
          // off, which over a long cache would lean one way.
          float x[NT][4] = {};
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            uint32_t vf[4];
            ldmatrix4_trans(vf, ((vs + v_frag) ^ (d << 5)) + mb * 16 * C::kRowBytes);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int y = PARTS - 1; y >= 0; --y) mma16816(BF_OUT ? o[t][d] : x[t], vf, pf[t][mb][y][0], pf[t][mb][y][1]);
          }
          if constexpr (!BF_OUT) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][d][e] += x[t][e];
          }
        }
      }
    }

    // the groups' sums, over the rings
    cp_async_wait<0>();
    float largest = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      largest = max_nan(largest, l[t][0] + l[t][1]);
#pragma unroll
      for (int d = 0; d < KS; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) largest = max_nan(largest, fabsf(o[t][d][e]));
    }
    const bool fine = !__syncthreads_or(!(largest < kLarge));
    if (!fine && !exact) {
      exact = true;
      continue;
    }
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        float* to = sums + (group * C::kRows + (row_warp * NT + t) * 8 + piece_c * 2 + e) * (DP + 2);
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          to[d * 16 + row_c] = o[t][d][e];
          to[d * 16 + 8 + row_c] = o[t][d][e + 2];
        }
        if (row_c == 0) {
          // m + 33 is rounded to 2^-19: 1.3e-6 of the piece's weight beside others.  Raised from a whole number, as in fp32,
          // 64 rows take 114 us instead of 112.
          to[DP] = exact ? m[t][e] + kShrink : m[t][e];
          to[DP + 1] = exact ? shrink(x) : x;
        }
      }
    exact = false;
    __syncthreads();
    float* part = nullptr;
    if (n < r.tiles)
      part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * part_floats(C::kRows, a.D);
    finish_piece<DP, C::kRows, C::kGroups, BF_OUT>(a, sums, b, hk, row0, rows, part);
    if (!part && tid == 0) note_whole(a, walk, items, join_blocks, joins);
    piece_done<C::kGroups * BK>(a, items, walk);
  }
  if (!noted && tid == 0) note_joins(a, walk, items, join_blocks, joins);      // nothing to do here
}

// ------------------------------------------------------------------ fp32

// R rows (two, four or eight).  A lane forms the scores of KL keys (lane mod 8, + 8, ..) and two rows, where R < 8 of a
// share of the channels; for the weighted sum it owns DP / 32 channels of all rows.
template <int DP, int R>
struct Simt {
  static constexpr int kKeys = DP == 256 ? 1 : 2;              // keys of a lane
  static constexpr int kBK = 8 * kKeys, kRows = R, kRowBytes = DP * 4;
  static constexpr int kHalves = DP == 64 ? 4 : 3, kHalf = kBK * kRowBytes;
  static constexpr int kRing = kWarps * kHalves * kHalf;
  static constexpr int kPart = kWarps * kRows * (DP + 2) * 4;
  static constexpr int kTop = kRing > kPart ? kRing : kPart;
  static constexpr int kQStride = DP + 4;                      // two rows apart is eight banks apart
  static constexpr int kQ = kRows * kQStride * 4;
  static constexpr size_t kSmem = kTop + kQ + kWarps * (kBK + 1) * kRows * 4;
  static constexpr int kCtas = DP == 64 ? 3 : 2;
};

template <int DP, int R, bool BF_OUT>
__global__ void __launch_bounds__(kThreads, Simt<DP, R>::kCtas)
    attend_f32_kernel(const AttentionArgs a, FastDiv page_div, int row_tiles, int join_blocks, Join* joins, float* parts) {
  using C = Simt<DP, R>;
  constexpr int BK = C::kBK, KL = C::kKeys, H = C::kHalves, CH = DP / 4, OC = DP / 32, DS = 8 / R;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = a.W * (a.H / a.HK), pieces = a.D / 4, items = a.HK * row_tiles;
  unsigned char* ring = smem + warp * H * C::kHalf;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  float* q_smem = reinterpret_cast<float*>(smem + C::kTop);
  float* weights = q_smem + C::kRows * C::kQStride + warp * (BK + 1) * R;    // [key][row], then the rows' factors
  float* factors = weights + BK * R;
  const float scale2 = a.scale * kLog2e, cap2 = a.softcap * kLog2e, inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const int key_lane = lane & 7, pair = (lane >> 3) / DS, share = (lane >> 3) % DS;

  // copies: this lane takes rows lane / 4 (+ 8) of a block, pieces lane % 4, + 4, ..; piece x of row r lies at
  // x ^ (r mod 8)
  const int row_c = lane >> 2, piece_c = lane & 3;
  const uint32_t to_even = row_c * C::kRowBytes + ((piece_c ^ row_c) << 4), to_odd = to_even ^ 64;

  Walk walk = find_stretch<kWarps * BK>(a, items);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool noted = false, again = false;         // again: the sums came out too large, see kShrink
  int n;
  while (next_piece<kWarps * BK>(a, items, walk, n)) {
    const int hk = walk.item / row_tiles, row0 = (walk.item - hk * row_tiles) * C::kRows;
    const Range r = walk.r;
    const int b = walk.b;
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
    const int64_t head = static_cast<int64_t>(hk) * a.page_head_stride + piece_c * 4;

    __syncthreads();                         // the previous piece's sums are read
    if (pieces < CH) {
      for (int i = tid; i < kWarps * H * BK * CH; i += kThreads) {
        const int row = i / CH, ch = i - row * CH;
        if (ch >= pieces)
          *reinterpret_cast<uint4*>(smem + row * C::kRowBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
    }

    // block i of this warp begins at key base(i); half 2 i is its keys, 2 i + 1 its values
    const auto base = [&](int i) { return r.begin + ((walk.tile + i) * kWarps + warp) * BK; };
    int page[KL], page_after[KL];            // of the next block to be copied and the one after it
    int64_t off[KL];
    const auto pages_of = [&](int i, int (&to)[KL]) {
#pragma unroll
      for (int x = 0; x < KL; ++x) {
        const int key = base(i) + row_c + 8 * x;
        to[x] = i < n && key >= r.first && key < r.len ? table[page_div.div(key)] : -1;
      }
    };
    const auto copy_half = [&](const void* from, int h) {
      const uint32_t dst = ring_u + (h % H) * C::kHalf;
#pragma unroll
      for (int x = 0; x < KL; ++x) {
        const bool ok = off[x] >= 0;
        const float* src = static_cast<const float*>(from) + (ok ? off[x] : 0);
#pragma unroll
        for (int c = 0; c < CH / 4; ++c)
          if (c * 4 + piece_c < pieces)
            cp_async16(dst + ((c & 1) ? to_odd : to_even) + (c >> 1) * 128 + x * 8 * C::kRowBytes,
                       src + (ok ? c * 16 : 0), ok);
      }
    };
    const auto issue = [&](int h) {
      const int i = h >> 1;
      if (i < n) {
        if (h & 1) {
          copy_half(a.v, h);
        } else {
#pragma unroll
          for (int x = 0; x < KL; ++x) {
            const int key = base(i) + row_c + 8 * x;
            off[x] = -1;
            if (static_cast<uint32_t>(page[x]) < static_cast<uint32_t>(a.num_pages)) {
              const int in_page = key - static_cast<int>(page_div.div(key)) * a.P;
              off[x] = page[x] * a.page_stride + in_page * a.page_row_stride + head;
            } else if (key >= r.first && key < r.len) {       // any other entry is a bad one; zeros are read
              raise_device_error(a.err, KDA_DEVERR_PAGE);
            }
          }
          copy_half(a.k, h);
#pragma unroll
          for (int x = 0; x < KL; ++x) page[x] = page_after[x];
          pages_of(i + 2, page_after);
        }
      }
      cp_async_commit();
    };

    pages_of(0, page);
    pages_of(1, page_after);
    constexpr int QN = (C::kRows * CH + kThreads - 1) / kThreads;
    float4 q[QN];
#pragma unroll
    for (int x = 0; x < QN; ++x) {
      const int i = tid + x * kThreads, row = i / CH, ch = i - row * CH;
      q[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < C::kRows && row0 + row < rows && ch < pieces) {
        const RowPlace at = row_place(a, b, hk, row0 + row);
        q[x] = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                (static_cast<int64_t>(b) * a.W + at.w) * a.q_stride +
                                                static_cast<int64_t>(at.h) * a.D + ch * 4);
      }
    }
#pragma unroll 1
    for (int h = 0; h < H - 1; ++h) issue(h);

    if (!noted && tid == 0) note_joins(a, walk, items, join_blocks, joins);  // while the copies are under way
    noted = true;
#pragma unroll
    for (int x = 0; x < QN; ++x) {
      const int i = tid + x * kThreads, row = i / CH, ch = i - row * CH;
      if (row < C::kRows) *reinterpret_cast<float4*>(q_smem + row * C::kQStride + ch * 4) = q[x];
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, slope[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const RowPlace at = row_place(a, b, hk, min(row0 + pair * 2 + i, rows - 1));
      pos[i] = r.len - a.W + at.w;
      slope[i] = a.slopes ? a.slopes[at.h] * kLog2e : 0.f;
    }
    float2 o[R][OC / 2];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int e = 0; e < OC / 2; ++e) o[t][e] = make_float2(0.f, 0.f);
    __syncthreads();

    for (int i = 0; i < n; ++i) {
      const int key0 = base(i);
      cp_async_wait<H - 2>();
      __syncwarp();
      issue(2 * i + H - 1);
      const unsigned char* ks = ring + ((2 * i) % H) * C::kHalf + key_lane * C::kRowBytes;

      float2 acc[KL][2][2];                  // [key][row][half of a piece]: independent chains
#pragma unroll
      for (int x = 0; x < KL; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) acc[x][t][0] = acc[x][t][1] = make_float2(0.f, 0.f);
#pragma unroll 8
      for (int ch = share; ch < pieces; ch += DS) {
        float4 q[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) q[t] = *reinterpret_cast<const float4*>(q_smem + (pair * 2 + t) * C::kQStride + ch * 4);
#pragma unroll
        for (int x = 0; x < KL; ++x) {
          const float4 k = *reinterpret_cast<const float4*>(ks + x * 8 * C::kRowBytes + ((ch ^ key_lane) << 4));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            acc[x][t][0] = fma2(make_float2(k.x, k.y), make_float2(q[t].x, q[t].y), acc[x][t][0]);
            acc[x][t][1] = fma2(make_float2(k.z, k.w), make_float2(q[t].z, q[t].w), acc[x][t][1]);
          }
        }
      }
      const bool whole = key0 >= r.first && key0 + BK - 1 <= r.len - a.W && (a.span == 0 || key0 > r.len - 1 - a.span);
      float y[KL][2];
      bool grows = false, sees[KL][2];
#pragma unroll
      for (int x = 0; x < KL; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int key = key0 + key_lane + 8 * x, p = pos[t];
          float z = (acc[x][t][0].x + acc[x][t][0].y) + (acc[x][t][1].x + acc[x][t][1].y);
#pragma unroll
          for (int d = 1; d < DS; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, 8 * d);
          z = a.softcap > 0.f ? cap2 * tanhf(z * inv_cap) : z * scale2;
          if (a.slopes) z += slope[t] * static_cast<float>(key - p);
          sees[x][t] = whole || (key >= r.first && key <= p && (a.span == 0 || key > p - a.span));
          y[x][t] = sees[x][t] ? z : -INFINITY;
          grows |= y[x][t] > m[t] + kSlack;
        }
      const bool rescale = __any_sync(0xffffffffu, grows);
      if (rescale) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float top = y[0][t];
#pragma unroll
          for (int x = 1; x < KL; ++x) top = fmaxf(top, y[x][t]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          const float now = fmaxf(m[t], top), f = ex2(m[t] - (now == -INFINITY ? 0.f : now));
          l[t] *= f;
          m[t] = now;
          if (key_lane == 0 && share == 0) factors[pair * 2 + t] = f;
        }
      }
#pragma unroll
      for (int x = 0; x < KL; ++x) {
        float w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          w[t] = ex2(y[x][t] - (m[t] == -INFINITY ? 0.f : m[t]));
          if (again) w[t] = shrink(w[t]);
          l[t] += w[t];
          // a weight of a key that the row does not see is negative zero: its product is left out below
          if (!sees[x][t]) w[t] = -0.f;
        }
        if (share == 0) *reinterpret_cast<float2*>(weights + (key_lane + 8 * x) * R + pair * 2) = make_float2(w[0], w[1]);
      }

      cp_async_wait<H - 2>();
      __syncwarp();
      issue(2 * i + H);
      const unsigned char* vs = ring + ((2 * i + 1) % H) * C::kHalf;
      if (rescale) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const float f = factors[t];
#pragma unroll
          for (int e = 0; e < OC / 2; ++e) o[t][e] = mul2(make_float2(f, f), o[t][e]);
        }
      }
      // key j's values and weights
      const auto fetch = [&](int j, float2 (&v)[OC / 2], float (&w)[R]) {
        const unsigned char* vrow = vs + j * C::kRowBytes;
        if constexpr (OC == 2) {
          v[0] = *reinterpret_cast<const float2*>(vrow + (((lane >> 1) ^ (j & 7)) << 4) + (lane & 1) * 8);
        } else {
#pragma unroll
          for (int c = 0; c < OC / 4; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(vrow + (((lane + 32 * c) ^ (j & 7)) << 4));
            v[2 * c] = make_float2(x.x, x.y);
            v[2 * c + 1] = make_float2(x.z, x.w);
          }
        }
        if constexpr (R == 2) {
          const float2 x = *reinterpret_cast<const float2*>(weights + j * R);
          w[0] = x.x; w[1] = x.y;
        } else {
#pragma unroll
          for (int c = 0; c < R / 4; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(weights + j * R + 4 * c);
            w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
          }
        }
      };
      if (whole) {
#pragma unroll
        for (int j = 0; j < BK; ++j) {
          float2 v[OC / 2];
          float w[R];
          fetch(j, v, w);
#pragma unroll
          for (int t = 0; t < R; ++t)
#pragma unroll
            for (int e = 0; e < OC / 2; ++e) o[t][e] = fma2(make_float2(w[t], w[t]), v[e], o[t][e]);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < BK; ++j) {
          float2 v[OC / 2];
          float w[R];
          fetch(j, v, w);
#pragma unroll
          for (int t = 0; t < R; ++t) {
            const bool left_out = __float_as_uint(w[t]) == 0x80000000u;
#pragma unroll
            for (int e = 0; e < OC / 2; ++e) {
              const float2 x = fma2(make_float2(w[t], w[t]), v[e], o[t][e]);
              o[t][e] = left_out ? o[t][e] : x;
            }
          }
        }
      }
    }

    cp_async_wait<0>();
    float largest = 0.f;
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int e = 0; e < OC / 2; ++e) largest = max_nan(largest, max_nan(fabsf(o[t][e].x), fabsf(o[t][e].y)));
    const bool fine = !__syncthreads_or(!(largest < kLarge));
    if (!fine && !again) {
      again = true;
      continue;
    }
    if (again) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float f = raise(m[t]);
        l[t] *= f;
        if (key_lane == 0 && share == 0) factors[pair * 2 + t] = f;
      }
      __syncwarp();
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float f = factors[t];
#pragma unroll
        for (int e = 0; e < OC / 2; ++e) o[t][e] = mul2(make_float2(f, f), o[t][e]);
      }
      again = false;
    }
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float x = l[t];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      if (key_lane == 0 && share == 0)
        *reinterpret_cast<float2*>(sums + (warp * R + pair * 2 + t) * (DP + 2) + DP) = make_float2(m[t], x);
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float2* to = reinterpret_cast<float2*>(sums + (warp * R + t) * (DP + 2));
      if constexpr (OC == 2) {
        to[lane] = o[t][0];
      } else {
#pragma unroll
        for (int c = 0; c < OC / 4; ++c) {
          to[(lane + 32 * c) * 2] = o[t][2 * c];
          to[(lane + 32 * c) * 2 + 1] = o[t][2 * c + 1];
        }
      }
    }
    __syncthreads();
    float* part = nullptr;
    if (n < r.tiles)
      part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (walk.tile > 0 ? 0 : 1)) * part_floats(C::kRows, a.D);
    finish_piece<DP, R, kWarps, BF_OUT>(a, sums, b, hk, row0, rows, part);
    if (!part && tid == 0) note_whole(a, walk, items, join_blocks, joins);
    piece_done<kWarps * BK>(a, items, walk);
  }
  if (!noted && tid == 0) note_joins(a, walk, items, join_blocks, joins);      // nothing to do here
}

// ------------------------------------------------------------------ joining

// Row r of the item that note_joins left at place x, which stretch c is the first to begin inside: parts c - 1 (its second
// place) and c, c + 1, .. (their first places) are added in a fixed order.  WPR warps take a row, every WPR-th part each,
// kJoinDepth of them in flight, then their sums are added.  Eight warps where an item has many parts (41 of each of 16 rows:
// the call takes 9.9 us, 14.9 with one warp), one where items are many and have few (two or three of each of 64 rows
// of 256 items: 155 us with eight, whose blocks' launches set the pace, 111 with one).
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps, kJoinDepth = 4, kFewParts = 8;

template <int WPR, bool BF_OUT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttentionArgs a, int row_tiles, int tile_rows,
                                                            int rows_of_item, int all_rows, const Join* joins,
                                                            const float* parts) {
  __shared__ float2 warp_ml[kJoinWarps];
  __shared__ float4 warp_o[kJoinWarps][64];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int index = blockIdx.x * (kJoinWarps / WPR) + warp / WPR;
  const int place = index / rows_of_item, r = index - place * rows_of_item;
  Join j{0, 0, 0, 0};
  if (index < all_rows) {
    const int4 raw = __ldcg(reinterpret_cast<const int4*>(joins) + place);
    j = Join{raw.x, raw.y, raw.z, raw.w};
  }
  const int hk = j.item / row_tiles, row0 = (j.item - hk * row_tiles) * tile_rows;
  if (row0 + r >= a.W * (a.H / a.HK)) j.parts = 0;
  if (WPR == kJoinWarps && j.parts == 0) return;          // otherwise warps of a block may have rows while others have none
  const int64_t stride = part_floats(tile_rows, a.D);
  const auto part_of = [&](int i) {
    const int64_t c = j.stretch;
    return parts + stride * (i == 0 ? 2 * (c - 1) + 1 : 2 * (c + i - 1));
  };
  // a lane holds pieces of four channels lane, + 32
  const int pieces = a.D / 4;
  float m = -INFINITY, l = 0.f;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = warp % WPR; i0 < j.parts; i0 += WPR * kJoinDepth) {
    float2 ml[kJoinDepth];
    float4 x[kJoinDepth][2];
#pragma unroll
    for (int y = 0; y < kJoinDepth; ++y) {
      const int i = i0 + y * WPR;
      ml[y] = make_float2(-INFINITY, 0.f);
      x[y][0] = x[y][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < j.parts) {
        const float* part = part_of(i);
        ml[y] = __ldcg(reinterpret_cast<const float2*>(part + static_cast<int64_t>(tile_rows) * a.D) + r);
        const float4* p = reinterpret_cast<const float4*>(part + static_cast<int64_t>(r) * a.D);
        if (lane < pieces) x[y][0] = __ldcg(p + lane);
        if (lane + 32 < pieces) x[y][1] = __ldcg(p + lane + 32);
      }
    }
    float now = m;
#pragma unroll
    for (int y = 0; y < kJoinDepth; ++y) now = fmaxf(now, ml[y].x);
    const float base = now == -INFINITY ? 0.f : now, f = ex2(m - base);
    l *= f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      o[e].x *= f;
      o[e].y *= f;
      o[e].z *= f;
      o[e].w *= f;
    }
#pragma unroll
    for (int y = 0; y < kJoinDepth; ++y) {
      const float g = ex2(ml[y].x - base);
      l += g * ml[y].y;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o[e].x += g * x[y][e].x;
        o[e].y += g * x[y][e].y;
        o[e].z += g * x[y][e].z;
        o[e].w += g * x[y][e].w;
      }
    }
    m = now;
  }
  const RowPlace at = row_place(a, j.seq, hk, row0 + r);
  if constexpr (WPR == 1) {
    if (j.parts == 0) return;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < pieces) {
        const int64_t to = at.o * a.D + 4 * (lane + 32 * e);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store_out2<BF_OUT>(a, to, l == 0.f ? make_float2(0.f, 0.f) : make_float2(o[e].x * inv, o[e].y * inv));
        store_out2<BF_OUT>(a, to + 2, l == 0.f ? make_float2(0.f, 0.f) : make_float2(o[e].z * inv, o[e].w * inv));
      }
  } else {
    if (lane == 0) warp_ml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < pieces) warp_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, warp_ml[w].x);
    const float base = m == -INFINITY ? 0.f : m;
    float f[kJoinWarps];
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      f[w] = ex2(warp_ml[w].x - base);
      l += f[w] * warp_ml[w].y;
    }
    const int d = 2 * threadIdx.x;
    if (d < a.D) {
      float2 x = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w)
        x = fma2(make_float2(f[w], f[w]), reinterpret_cast<const float2*>(warp_o[w])[threadIdx.x], x);
      store_out2<BF_OUT>(a, at.o * a.D + d, l == 0.f ? make_float2(0.f, 0.f) : make_float2(x.x / l, x.y / l));
    }
  }
  if ((WPR == 1 ? lane : static_cast<int>(threadIdx.x)) == 0 && a.lse)
    a.lse[at.o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ host

constexpr int kMaxStretches = 152 * 4;       // of any variant on any device of this kind

struct Variant {
  int rows, ctas;                            // rows of a tile, CTAs an SM
};
Variant variant_of(bool bf16, int D, int rows) {
  if (!bf16) return Variant{rows > 4 ? 8 : rows > 2 ? 4 : 2, D > 64 ? 2 : 3};
  if (D > 128) return Variant{rows > 16 ? 32 : rows > 8 ? 16 : 8, 2};
  return rows > 8 ? Variant{rows > 32 ? 64 : rows > 16 ? 32 : 16, 2} : Variant{8, 3};
}

int stretches_of(const Variant& v) { return std::min(kMaxStretches, sm_count() * v.ctas); }

template <auto K, typename Config>
cudaError_t run(const AttentionArgs& a, int row_tiles, int stretches, int join_blocks, Join* joins, float* parts,
                cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = raise_smem(K, Config::kSmem, done);
  if (e != cudaSuccess) return e;
  K<<<stretches, kThreads, Config::kSmem, st>>>(a, FastDiv(a.P), row_tiles, join_blocks, joins, parts);
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
  const int join_blocks = static_cast<int>(std::min<int64_t>(n, static_cast<int64_t>(a.B) * a.HK * tiles));
  const auto bf16_of = [&](auto dp, auto rw, auto nt) {
    constexpr int DP = decltype(dp)::value, RW = decltype(rw)::value, NT = decltype(nt)::value;
    return run<attend_bf16_kernel<DP, RW, NT, BF_OUT>, Mma<DP, RW, NT>>(a, tiles, n, join_blocks, joins, parts, st);
  };
  const auto f32_of = [&](auto dp, auto rows_of_tile) {
    constexpr int DP = decltype(dp)::value, R = decltype(rows_of_tile)::value;
    return run<attend_f32_kernel<DP, R, BF_OUT>, Simt<DP, R>>(a, tiles, n, join_blocks, joins, parts, st);
  };
  using std::integral_constant;
  const auto of_width = [&](auto dp) {
    if (!bf16) {
      if (v.rows == 2) return f32_of(dp, integral_constant<int, 2>{});
      if (v.rows == 4) return f32_of(dp, integral_constant<int, 4>{});
      return f32_of(dp, integral_constant<int, 8>{});
    }
    if (v.rows == 8) return bf16_of(dp, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    // Two tiles a warp where their sums fit the registers: each key and value is read from the ring for both (64
    // rows: one pass over the keys instead of two).
    constexpr int NT = decltype(dp)::value > 128 ? 1 : 2, RW = 2 / NT;
    constexpr integral_constant<int, NT> nt{};
    if (v.rows == 16) return bf16_of(dp, integral_constant<int, RW>{}, nt);
    if (v.rows == 32) return bf16_of(dp, integral_constant<int, 2 * RW>{}, nt);
    return bf16_of(dp, integral_constant<int, 4>{}, nt);
  };
  e = a.D <= 64    ? of_width(std::integral_constant<int, 64>{})
      : a.D <= 128 ? of_width(std::integral_constant<int, 128>{})
                   : of_width(std::integral_constant<int, 256>{});
  if (e != cudaSuccess) return e;
  // launched while the stretches still run: its blocks wait for them on the device
  const int rows_of_item = std::min(v.rows, rows), all_rows = join_blocks * rows_of_item;
  const bool few = static_cast<int64_t>(a.B) * a.HK * tiles * kFewParts >= n;            // parts of an item, about
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(few ? (all_rows + kJoinWarps - 1) / kJoinWarps : all_rows);
  config.blockDim = dim3(kJoinThreads);
  config.stream = st;
  cudaLaunchAttribute attribute;
  attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attribute.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attribute;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, few ? join_kernel<1, BF_OUT> : join_kernel<kJoinWarps, BF_OUT>, a, tiles, v.rows,
                            rows_of_item, all_rows, static_cast<const Join*>(joins), static_cast<const float*>(parts));
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
