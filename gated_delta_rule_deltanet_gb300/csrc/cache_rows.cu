// cache_rows.cu -- the page tables of a key-value cache from one step to the next, the compaction of its pools
// and the copying of pages (or of any pool's slots).
//
// Row r of a table holds len_r tokens in ceil(len_r / P) pages; refs[q] counts the references to page q, those of
// the table and of anyone else; q is free where refs[q] is zero.
//
// An update makes new rows.  New row i goes on from old row parent[i] (or from nothing) with its first
// kept_i = min(len of the parent, new_len_i) tokens and has pages for new_len_i.  Pages that the kept tokens fill are
// shared.  A page that they end inside is open: tokens will be written behind them, so only one row may
// hold it and no one else read it.  The lowest row that goes on in an open page keeps it if no full row and
// no one outside the table refers to it; every other row gets a fresh page and the open one's contents.  Rows that no new
// row goes on from are thereby freed, rows with several continuations forked, longer rows grown.
// Fresh pages are the free ones from the lowest on, given out row by row.  Nothing is written to the old tables, and
// fresh pages were free in them, so what still reads them (a step in flight) is not disturbed.
//
// A compaction of n used pages moves the k-th used page from n on into the k-th free page before n: as few pages as
// can be, each into a page that is free, so that the old tables stay valid here too.
//
// Both are chains of short passes (count, rank, assign) over at most some million integers, bound by the latency of the
// passes: one thread-block cluster runs them in one launch, with the cluster's hardware barrier between them.
// One GB300: 256 rows of up to 250 pages one step on 14 us, with a list of copies that is empty; 64 rows to 512 of up to
// 960 pages 33 us, 12 of them copies; a compaction that moves 1.15 GB 379 us, 358 of them copies (95% of measured HBM).
#include <algorithm>
#include <limits.h>

#include "cache_common.cuh"

namespace kda {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
// Entries of the new table and references from which sixteen blocks run instead of eight: what an SM moves bounds large
// tables, the barriers small ones.  2.0 M entries 130 us by eight, 74 by sixteen; 520 k (with copies) 37.1 and 33.1; 70 k
// 14.2 and 14.4; a compaction of 2 k 10.5 and 12.3.
constexpr int64_t kManyEntries = 1 << 17;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// inclusive sum over the block; `total` gets the sum.  Two barriers.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  T s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  __syncthreads();
  return incl + (warp ? before : 0);
}

struct Segment {                             // the pages of one CTA; the first has the rows to see to and none
  int begin, end;
};
template <int CL>
__device__ __forceinline__ Segment segment(int n, int rank) {
  const int per = (n + CL - 2) / (CL - 1);
  Segment s;
  s.begin = rank == 0 ? 0 : min(static_cast<int64_t>(rank - 1) * per, static_cast<int64_t>(n));
  s.end = rank == 0 ? 0 : min(s.begin + per, n);
  return s;
}

// Calls f(page, is it one, ones before it) for the pages of the segment, in order, with `before` ones ahead of the
// segment: each thread takes kPages pages behind one another, and `is` says of them at once which are ones.
constexpr int kPages = 8;
template <typename Is, typename F>
__device__ __forceinline__ void rank_pages(const Segment& seg, int before, int* warp_sums, const Is& is, const F& f) {
  for (int q0 = seg.begin; q0 < seg.end; q0 += kThreads * kPages) {
    const int at = q0 + threadIdx.x * kPages;
    bool one[kPages];
    int mine = 0, total;
    is(at, seg.end, one);
#pragma unroll
    for (int x = 0; x < kPages; ++x) mine += one[x];
    int rank = block_scan(mine, warp_sums, total) - mine + before;
#pragma unroll
    for (int x = 0; x < kPages; ++x) {
      if (at + x < seg.end) f(at + x, one[x], rank);
      rank += one[x];
    }
    before += total;
  }
}

// pages of the row, or -1 for a length that its row cannot hold
__device__ __forceinline__ int pages_of(int len, int P, int width) {
  if (len < 0) return -1;
  const int n = len / P + (len % P != 0);
  return n <= width ? n : -1;
}

// One new row: where it goes on from and what it keeps.
struct Row {
  int parent, len, kept, full, want, end;    // full pages kept; pages of the new row and of its parent (-1: too many)
};
__device__ __forceinline__ Row row_of(const RowsArgs& a, int i) {
  Row r;
  r.parent = a.parent ? a.parent[i] : i;
  const int len = r.len = a.new_lens[i];
  const bool from = r.parent >= 0 && r.parent < a.S;
  const int old = from ? a.lens[r.parent] : 0;
  r.kept = max(0, min(old, len));
  r.full = r.kept / a.P;
  r.want = r.parent >= -1 && r.parent < a.S ? pages_of(len, a.P, a.width) : -1;
  r.end = pages_of(old, a.P, a.width);
  return r;
}

constexpr int kCounted = 4096;               // old rows whose children are counted; of more, each page is counted singly
// A free page's count starts at the lowest integer, so that it stays below this whatever rows add to it.
constexpr int kFreeBelow = -(1 << 30);
constexpr int kAhead = 8;                    // entries of a row that a lane loads before it uses the first

// Scratch of an update (int32): [N] counts, [N] first open row, [N] free pages in order, [S_out] pages that a row
// keeps (its open one included), [S_out] its place among the fresh pages, words of the launch: 0 the error,
// 1 copies in all, 8.. the CTAs' free pages.
//
// Each pass is a few dependent loads deep; what a pass needs of the rows and tables is loaded ahead of the barrier
// before it where that barrier does not order it.
template <int CL>
__global__ void __launch_bounds__(kThreads) update_kernel(const RowsArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int64_t warp_sums64[32];
  __shared__ int children[kCounted], shared_pages[kCounted];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  const int all = CL * kThreads, me = rank * kThreads + tid;
  const int my_row = warp * CL + rank, rows_at_once = CL * kWarps;
  int32_t* counts = a.scratch;
  int32_t* first = counts + a.N;
  int32_t* free_list = first + a.N;
  int32_t* have = free_list + a.N;
  int32_t* place = have + a.S_out;
  int32_t* words = place + a.S_out;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Segment seg = segment<CL>(a.N, rank);
  const auto in_pool = [&](int q) { return static_cast<uint32_t>(q) < static_cast<uint32_t>(a.N); };

  // 1. references as they are; free pages of the CTA
  if (rank == 0 && tid == 0) words[0] = 0;
  // The two rows that this warp, and in the first CTA that this thread, comes to first, and how an old row goes on: its
  // children and the full pages that all of them keep, counted by each CTA for itself.
  const Row mine_row = my_row < a.S_out ? row_of(a, my_row) : Row{};
  const Row next_row = my_row + rows_at_once < a.S_out ? row_of(a, my_row + rows_at_once) : Row{};
  const auto row_at = [&](int i) {
    return i == my_row ? mine_row : i == my_row + rows_at_once ? next_row : row_of(a, i);
  };
  const Row thread_row = tid < a.S_out ? row_of(a, tid) : Row{};
  const bool counted = a.S <= kCounted;
  for (int r = tid; counted && r < a.S; r += kThreads) {
    children[r] = 0;
    shared_pages[r] = INT_MAX;
  }
  int mine = 0, total;
#pragma unroll 4
  for (int q = seg.begin + tid; q < seg.end; q += kThreads) {
    const int r = a.refs[q];
    counts[q] = r == 0 ? INT_MIN : r;
    first[q] = INT_MAX;
    if (r == 0) {
      ++mine;
      a.out_refs[q] = 0;
    }
  }
  int thread_open = -1;                      // the page that the thread's row ends inside
  const auto open_of = [&](const Row& r) {
    const bool ok = r.parent >= 0 && r.parent < a.S && r.kept % a.P != 0 && r.full < a.width;
    return ok ? a.table[static_cast<int64_t>(r.parent) * a.width + r.full] : -1;
  };
  if (rank == 0 && tid < a.S_out) thread_open = open_of(thread_row);
  block_scan(mine, warp_sums, total);
  if (tid == 0) words[8 + rank] = total;
  for (int i = tid; counted && i < a.S_out; i += kThreads) {
    const Row r = i == tid ? thread_row : row_of(a, i);
    if (r.parent >= 0 && r.parent < a.S) {
      atomicAdd(children + r.parent, 1);
      atomicMin(shared_pages + r.parent, r.full);
    }
  }
  cluster_sync();

  // 2. References of the old rows taken back, of the new rows' full pages added; a warp takes a row.  The pages that all
  // children of a row keep change by their number less one, which is nothing for a row that only goes on; beyond
  // them each child counts its own.  A row that names a free page is found here where it adds
  // nothing (by refs) or takes back (by the count's start, which the addition returns); what rows only add to a free
  // page is found at its count in pass 3.  All by refs: eight continuations of 64 prompts 38 us instead of 33, 2048 rows
  // one step on 84 instead of 74.
  const auto fault = [&]() { atomicExch(words, 1); };
  const auto pages_shared = [&](int r) { return counted && children[r] > 0 ? shared_pages[r] : 0; };
  for (int r = my_row; r < a.S; r += rows_at_once) {
    const int n = pages_of(a.lens[r], a.P, a.width);
    if (n < 0) {
      if (lane == 0) fault();
      continue;
    }
    const int shared = pages_shared(r), change = counted ? children[r] - 1 : -1;
    const int32_t* row = a.table + static_cast<int64_t>(r) * a.width;
    for (int j0 = lane; j0 < n; j0 += 32 * kAhead) {
      int q[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) q[x] = j0 + 32 * x < n ? row[j0 + 32 * x] : -1;
      const auto add_of = [&](int x) { return j0 + 32 * x < shared ? change : -1; };
      int seen[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        seen[x] = 1;
        if (q[x] == -1) continue;            // a page that the row has given back
        const int add = add_of(x);
        if (!in_pool(q[x])) seen[x] = INT_MIN;
        else if (add > 0) atomicAdd(counts + q[x], add);
        else if (add < 0) seen[x] = atomicAdd(counts + q[x], add);
        else seen[x] = a.refs[q[x]];
      }
      bool bad = false;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) bad |= add_of(x) == 0 ? seen[x] <= 0 : seen[x] < kFreeBelow;
      if (bad) fault();
    }
  }
  for (int i = my_row; i < a.S_out; i += rows_at_once) {
    const Row r = row_at(i);
    if (r.want < 0 || r.end < 0) {
      if (lane == 0) fault();
      continue;
    }
    if (r.parent < 0) continue;
    const int32_t* row = a.table + static_cast<int64_t>(r.parent) * a.width;
    for (int j0 = pages_shared(r.parent) + lane; j0 < r.full; j0 += 32 * kAhead) {
      int q[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) q[x] = j0 + 32 * x < r.full ? row[j0 + 32 * x] : -1;
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (in_pool(q[x])) atomicAdd(counts + q[x], 1);          // one that is not is found with its old row
    }
    if (lane == 0 && r.kept % a.P != 0) {
      const int q = row[r.full];
      if (in_pool(q)) atomicMin(first + q, i);
      else fault();
    }
  }
  cluster_sync();

  // 3. the free pages in order; a page in use whose count went below zero was held more often than refs say, a free one
  // whose count is not what it started with is held by a row
  int before = 0, free_pages = 0;
#pragma unroll
  for (int c = 0; c < CL; ++c) {
    const int n = __ldcg(words + 8 + c);
    if (c < rank) before += n;
    free_pages += n;
  }
  bool wrong = false;
  rank_pages(seg, before, warp_sums,
             [&](int at, int end, bool (&free)[kPages]) {
               int r[kPages], c[kPages];
#pragma unroll
               for (int x = 0; x < kPages; ++x) {
                 r[x] = at + x < end ? a.refs[at + x] : 1;
                 c[x] = at + x < end ? __ldcg(counts + at + x) : 0;
               }
#pragma unroll
               for (int x = 0; x < kPages; ++x) {
                 wrong |= (r[x] < 0) | ((r[x] > 0) & (c[x] < 0)) | ((r[x] == 0) & (c[x] != INT_MIN));
                 free[x] = r[x] == 0;
               }
             },
             [&](int q, bool free, int at) {
               if (free) free_list[at] = q;
             });
  if (wrong) fault();
  // and the rows' needs, by the first CTA
  if (rank == 0) {
    int64_t fresh = 0, sum;                  // in 64 bits: rows may ask for more than there is
    int copies = 0;
    bool bad = false;
    for (int i0 = 0; i0 < a.S_out; i0 += kThreads) {
      const int i = i0 + tid;
      int need = 0, copy = 0, hold = 0, open = -1;
      if (i < a.S_out) {
        const Row r = i0 == 0 ? thread_row : row_of(a, i);
        open = i0 == 0 ? thread_open : open_of(r);
        hold = r.full;
        if (in_pool(open)) {
          const int lowest = __ldcg(first + open), others = __ldcg(counts + open);
          if (lowest == i && others == 0) {
            counts[open] = 1;                // no other row looks at it: each has another first row or finds this one's
            ++hold;
          } else {
            copy = 1;
          }
        }
        need = max(0, r.want - hold);
      }
      const int64_t at = block_scan(static_cast<int64_t>(need), warp_sums64, sum) - need + fresh;
      fresh += sum;
      bad |= fresh > free_pages;
      const int c = block_scan(copy, warp_sums, total) - 1 + copies;
      copies += total;
      if (i < a.S_out) {
        have[i] = hold;
        place[i] = static_cast<int32_t>(at);
        if (copy) {
          a.copy_src[c] = open;
          a.copy_dst[c] = static_cast<int32_t>(at);          // becomes the page itself below
        }
      }
    }
    if (bad && tid == 0) fault();
    if (tid == 0) words[1] = copies;
  }
  cluster_sync();

  // 4. the new rows
  const int copies = __ldcg(words + 1);
  int hold_of[2], place_of[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int i = my_row + x * rows_at_once;
    hold_of[x] = i < a.S_out ? __ldcg(have + i) : 0;
    place_of[x] = i < a.S_out ? __ldcg(place + i) : 0;
  }
  const bool stop = __ldcg(words) != 0;
  if (stop) {
    if (me == 0) raise_device_error(a.err, KDA_DEVERR_PAGE);
    for (int q = seg.begin + tid; q < seg.end; q += kThreads) a.out_refs[q] = a.refs[q];
    for (int64_t i = me; i < static_cast<int64_t>(a.S_out) * a.width; i += all) a.out_table[i] = -1;
    for (int i = me; i < a.S_out; i += all) {
      a.out_lens[i] = 0;
      a.kept[i] = 0;
      a.copy_src[i] = -1;
      a.copy_dst[i] = -1;
    }
    return;
  }
  for (int i = my_row; i < a.S_out; i += rows_at_once) {
    const Row r = row_at(i);
    const int nth = i == my_row ? 0 : i == my_row + rows_at_once ? 1 : 2;
    const int hold = nth == 0 ? hold_of[0] : nth == 1 ? hold_of[1] : __ldcg(have + i);
    const int at = nth == 0 ? place_of[0] : nth == 1 ? place_of[1] : __ldcg(place + i);
    const int32_t* row = a.table + static_cast<int64_t>(max(r.parent, 0)) * a.width;
    int32_t* out = a.out_table + static_cast<int64_t>(i) * a.width;
    for (int j0 = lane; j0 < a.width; j0 += 32 * kAhead) {
      int q[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int j = j0 + 32 * x;
        q[x] = j < hold ? row[j] : j < r.want ? __ldcg(free_list + at + j - hold) : -1;
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int j = j0 + 32 * x;
        if (j >= hold && j < r.want) a.out_refs[q[x]] = 1;
        if (j < a.width) out[j] = q[x];
      }
    }
    if (lane == 0) {
      a.out_lens[i] = r.len;
      a.kept[i] = r.kept;
    }
  }
#pragma unroll 4
  for (int q = seg.begin + tid; q < seg.end; q += kThreads) {
    const int r = a.refs[q], count = __ldcg(counts + q);
    if (r != 0) a.out_refs[q] = count;
  }
  for (int i = me; i < a.S_out; i += all) {
    if (i < copies) {
      a.copy_dst[i] = __ldcg(free_list + __ldcg(a.copy_dst + i));
    } else {
      a.copy_src[i] = -1;
      a.copy_dst[i] = -1;
    }
  }
}

// Scratch of a compaction (int32): [N] the used pages by rank, [N] the free pages by rank, words of the launch:
// 1 used pages among the first n, 8.. the CTAs' used pages, 32.. their errors.  page_map holds the ranks meanwhile.
template <int CL>
__global__ void __launch_bounds__(kThreads) compact_kernel(const RowsArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int stop;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  const int all = CL * kThreads, me = rank * kThreads + tid;
  int32_t* used_list = a.scratch;
  int32_t* free_list = used_list + a.N;
  int32_t* words = free_list + a.N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Segment seg = segment<CL>(a.N, rank);

  int mine = 0, total;
  bool bad = false;
  for (int q = seg.begin + tid; q < seg.end; q += kThreads) {
    const int r = a.refs[q];
    mine += r != 0;
    bad |= r < 0;
  }
  block_scan(mine, warp_sums, total);
  bad = __syncthreads_or(bad);
  if (tid == 0) words[8 + rank] = bad ? -1 : total;
  cluster_sync();

  int before = 0, n = 0;
  bad = false;
  for (int c = 0; c < CL; ++c) {
    const int x = __ldcg(words + 8 + c);
    bad |= x < 0;
    if (c < rank) before += x;
    n += x;
  }
  // A row that names a free page, or a page that is not there, cannot be rewritten; nothing is.
  bool wrong = false;
  for (int r = rank * kWarps + warp; r < a.S; r += CL * kWarps) {
    const int pages = pages_of(a.lens[r], a.P, a.width);
    wrong |= pages < 0;
    for (int j0 = lane; j0 < pages; j0 += 32 * kAhead) {
      int q[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        q[x] = j0 + 32 * x < pages ? a.table[static_cast<int64_t>(r) * a.width + j0 + 32 * x] : -1;
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        wrong |= q[x] != -1 && (static_cast<uint32_t>(q[x]) >= static_cast<uint32_t>(a.N) || a.refs[q[x]] == 0);
    }
  }
  wrong = __syncthreads_or(wrong);
  if (rank == 0 && tid == 0 && n == a.N) words[1] = n;
  if (!bad) {
    rank_pages(seg, before, warp_sums,
               [&](int at, int end, bool (&used)[kPages]) {
                 int r[kPages];
#pragma unroll
                 for (int x = 0; x < kPages; ++x) r[x] = at + x < end ? a.refs[at + x] : 0;
#pragma unroll
                 for (int x = 0; x < kPages; ++x) used[x] = r[x] != 0;
               },
               [&](int q, bool used, int at) {           // `at` used pages before q
                 a.page_map[q] = used ? at : -1;
                 if (used) used_list[at] = q;
                 else free_list[q - at] = q;
                 if (q == n) words[1] = at;
               });
  }
  __syncthreads();
  if (tid == 0) words[32 + rank] = bad || wrong;
  cluster_sync();

  if (tid == 0) {
    int s = 0;
    for (int c = 0; c < CL; ++c) s |= __ldcg(words + 32 + c);
    stop = s;
  }
  __syncthreads();
  const int half = a.N / 2;
  if (stop) {                                // everything stays where it is
    if (me == 0) raise_device_error(a.err, KDA_DEVERR_PAGE);
    for (int q = me; q < a.N; q += all) {
      a.page_map[q] = a.refs[q] != 0 ? q : -1;
      a.out_refs[q] = a.refs[q];
    }
    for (int64_t i = me; i < static_cast<int64_t>(a.S) * a.width; i += all) a.out_table[i] = a.table[i];
    for (int i = me; i < half; i += all) {
      a.copy_src[i] = -1;
      a.copy_dst[i] = -1;
    }
    return;
  }
  // where page q goes: to its rank's place in front, which a used page before n keeps
  const int front = __ldcg(words + 1);       // used pages among the first n: those that stay
  for (int q = me; q < a.N; q += all) {
    const int at = __ldcg(a.page_map + q);
    if (q >= n) a.out_refs[q] = 0;
    if (at < 0) continue;
    const int to = q < n ? q : __ldcg(free_list + at - front);
    a.page_map[q] = to;
    a.out_refs[to] = a.refs[q];
  }
  for (int i = me; i < half; i += all) {
    const bool moves = i < n - front;
    a.copy_src[i] = moves ? __ldcg(used_list + front + i) : -1;
    a.copy_dst[i] = moves ? __ldcg(free_list + i) : -1;
  }
  cluster_sync();
  for (int r = rank * kWarps + warp; r < a.S; r += CL * kWarps) {
    const int pages = pages_of(a.lens[r], a.P, a.width);
    const int64_t at = static_cast<int64_t>(r) * a.width;
    for (int j0 = lane; j0 < a.width; j0 += 32 * kAhead) {
      int q[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) q[x] = j0 + 32 * x < pages ? a.table[at + j0 + 32 * x] : -1;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) q[x] = q[x] < 0 ? -1 : __ldcg(a.page_map + q[x]);
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (j0 + 32 * x < a.width) a.out_table[at + j0 + 32 * x] = q[x];
    }
  }
}

// ------------------------------------------------------------------ copies

constexpr int kMaxPools = 64, kCopyThreads = 256, kCopyUnroll = 4;

struct Pools {
  char* base[kMaxPools];
  int64_t stride[kMaxPools];                 // bytes from page to page
};

// pool[dst[i]] = pool[src[i]] for i up to the list's end, every pool.  VB bytes a thread and move; a
// block takes pieces of kCopyThreads * kCopyUnroll of them, all loaded before the first is stored.  Bound by HBM.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const Pools pools, int num_pools, int64_t bytes, int64_t pieces,
                                                            const int32_t* src, const int32_t* dst, int64_t n, int num_pages,
                                                            int32_t* err) {
  constexpr int64_t kPiece = static_cast<int64_t>(sizeof(V)) * kCopyThreads * kCopyUnroll;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // launched while what makes the list may still run
  const int64_t per_entry = pieces * num_pools;
  for (int64_t at = blockIdx.x; at < n * per_entry; at += gridDim.x) {
    const int64_t i = at / per_entry, rest = at - i * per_entry, pool = rest / pieces, piece = rest - pool * pieces;
    const int32_t s = src[i], d = dst[i];
    if (s < 0) return;                       // the list's end
    if (s >= num_pages || d < 0 || d >= num_pages) {
      if (threadIdx.x == 0) raise_device_error(err, KDA_DEVERR_PAGE);
      continue;
    }
    const char* from = pools.base[pool] + s * pools.stride[pool];
    char* to = pools.base[pool] + d * pools.stride[pool];
    const int64_t b0 = piece * kPiece + threadIdx.x * static_cast<int64_t>(sizeof(V));
    V x[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int64_t b = b0 + u * kCopyThreads * static_cast<int64_t>(sizeof(V));
      if (b < bytes) x[u] = *reinterpret_cast<const V*>(from + b);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int64_t b = b0 + u * kCopyThreads * static_cast<int64_t>(sizeof(V));
      if (b < bytes) *reinterpret_cast<V*>(to + b) = x[u];
    }
  }
}

template <typename V>
cudaError_t copy(const Pools& pools, int num_pools, int64_t bytes, const int32_t* src, const int32_t* dst, int64_t n,
                 int num_pages, int32_t* err, cudaStream_t st) {
  const int64_t pieces = (bytes + static_cast<int64_t>(sizeof(V)) * kCopyThreads * kCopyUnroll - 1) /
                         (static_cast<int64_t>(sizeof(V)) * kCopyThreads * kCopyUnroll);
  const int64_t blocks = std::min<int64_t>(n * pieces * num_pools, static_cast<int64_t>(sm_count()) * 8);
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(blocks));
  config.blockDim = dim3(kCopyThreads);
  config.stream = st;
  cudaLaunchAttribute attribute;
  attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attribute.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attribute;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, copy_kernel<V>, pools, num_pools, bytes, pieces, src, dst, n, num_pages, err);
}

}  // namespace

size_t cache_rows_workspace(const kda_cache_rows_params_t& p) {
  return (static_cast<size_t>(3) * p.num_pages + 2 * static_cast<size_t>(p.rows_out) + 64) * sizeof(int32_t);
}

namespace {

// One cluster of CL blocks.  Sixteen are more than every device has to grant a cluster: `granted` says whether this one does.
template <int CL, auto K>
cudaError_t launch_cluster(const RowsArgs& a, cudaStream_t st, bool* granted = nullptr) {
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(CL);
  config.blockDim = dim3(kThreads);
  config.stream = st;
  cudaLaunchAttribute attribute;
  attribute.id = cudaLaunchAttributeClusterDimension;
  attribute.val.clusterDim = {CL, 1, 1};
  config.attrs = &attribute;
  config.numAttrs = 1;
  if (granted) {
    static std::atomic<uint64_t> yes{0}, no{0};          // by device, asked once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (!((yes.load(std::memory_order_relaxed) | no.load(std::memory_order_relaxed)) & bit)) {
      int n = 0;
      const bool ok = cudaFuncSetAttribute(K, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&n, K, &config) == cudaSuccess && n > 0;
      if (!ok) cudaGetLastError();
      (ok ? yes : no).fetch_or(bit, std::memory_order_relaxed);
    }
    *granted = (yes.load(std::memory_order_relaxed) & bit) != 0;
    if (!*granted) return cudaSuccess;
  }
  return cudaLaunchKernelEx(&config, K, a);
}

template <auto K8, auto K16>
cudaError_t launch_rows(const RowsArgs& a, int64_t entries, cudaStream_t st) {
  if (entries >= kManyEntries) {
    bool granted = false;
    const cudaError_t e = launch_cluster<16, K16>(a, st, &granted);
    if (e != cudaSuccess || granted) return e;
  }
  return launch_cluster<8, K8>(a, st);
}

}  // namespace

cudaError_t launch_cache_update(const RowsArgs& a, cudaStream_t st) {
  return launch_rows<update_kernel<8>, update_kernel<16>>(a, static_cast<int64_t>(a.S_out) * a.width + a.N, st);
}

cudaError_t launch_cache_compact(const RowsArgs& a, cudaStream_t st) {
  return launch_rows<compact_kernel<8>, compact_kernel<16>>(a, static_cast<int64_t>(a.S) * a.width + a.N, st);
}

cudaError_t launch_cache_copy(void* const* pools, const int64_t* bytes, const int64_t* strides, int num_pools,
                              const int32_t* src, const int32_t* dst, int64_t n, int num_pages, int32_t* err,
                              cudaStream_t st) {
  // pools of one page size and alignment go into one launch
  for (int first = 0; first < num_pools;) {
    Pools p;
    int count = 0;
    const int64_t size = bytes[first];
    uint64_t bits = size;
    while (first + count < num_pools && count < kMaxPools && bytes[first + count] == size) {
      p.base[count] = static_cast<char*>(pools[first + count]);
      p.stride[count] = strides[first + count];
      bits |= reinterpret_cast<uintptr_t>(pools[first + count]) | strides[first + count];
      ++count;
    }
    cudaError_t e = cudaSuccess;
    if (size > 0) {
      if (bits % 16 == 0) e = copy<uint4>(p, count, size, src, dst, n, num_pages, err, st);
      else if (bits % 4 == 0) e = copy<uint32_t>(p, count, size, src, dst, n, num_pages, err, st);
      else e = copy<uint8_t>(p, count, size, src, dst, n, num_pages, err, st);
    }
    if (e != cudaSuccess) return e;
    first += count;
  }
  return cudaSuccess;
}

}  // namespace kda
