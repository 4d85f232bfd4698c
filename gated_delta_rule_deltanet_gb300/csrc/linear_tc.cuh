// linear_tc.cuh -- the matrix product of gemm.cuh on tcgen05 tensor cores.
//
//     D[i, j] = sum_c A(i, c) B(j, c)        out[j, i] = residual + scale act(D + bias[i])
//
// i, the contiguous dimension of the output, is the MMA's M (tensor-memory lanes), j its N
// (columns): a warp reads 32 lanes of one column and stores 32 consecutive elements of a row, so
// the epilogue needs no transpose and bias[i] is one value a thread.  An operand is K-major (c
// contiguous) or MN-major (i or j contiguous), both staged by TMA with the 128-byte swizzle, so
// the three products of a training step (x w^T, dz w, dz^T x) read their operands as they lie.
//
// Two kernels.
//
//   gemm_pair_kernel   large products.  A pair of CTAs (cta_group::2) works on a 256 x BN tile (BN
//                      128 to 256, see launch_pair): each stages its own half of the rows of A and
//                      of B, so a 64-wide step of c moves 32 KB into each SM for 512 tensor
//                      cycles, half of what two single CTAs with the same accumulators would
//                      move.  Persistent: the two accumulators alternate, one being multiplied
//                      into while eight warps store the other through shared memory and TMA.
//                      Bound by the tensor pipe and, over seconds, by power: 32768 x 4096 x 4096
//                      539 us, 2.04 PFLOP/s (the vendor library's product: 538 us), in a
//                      long loop 608 us (600 us).
//   gemm_split_kernel  small products, mostly few rows (decode: the weight is the work).  One CTA
//                      holds a 128 x BN tile; a cluster of S CTAs splits the sum over c: each
//                      pushes its part of every other CTA's columns into that CTA's shared
//                      memory and adds what it receives in rank order, so the result does not
//                      depend on timing and needs no workspace.  Bound by HBM and by set-up: 16
//                      rows through 4096 -> 16384 from HBM 25.7 us (5.2 TB/s), 64 through 4096
//                      -> 4096 11.6 us.
//
// fp32 operands are split into three bf16 parts, x = hi + mid + lo with every part rounded to
// nearest, which hold all 24 bits; the six products of parts above 2^-27 relative are summed,
// smallest first.  The tensor cores cut the accumulator's low bits at every step of 16 instead of
// rounding them, always towards zero, so a long sum would lose several times fp32's rounding.
// The split kernel therefore moves the accumulator into registers every 64 steps of c, where it is
// added with rounding (c = 4096: 1.7e-7 of the norm, an fp32 product on CUDA cores 1.1e-6, at 2.6
// times its speed; short sums are no closer than an fp32 product's, 1.2e-7 at c = 517).  Where bf16
// operands have an fp32 result over more than 1024 steps both kernels do the same every 512, the pair
// kernel into a third stretch of tensor memory of 160 columns (c = 4096: 4.8e-7 against 4.4e-6
// without; 4096 x 8192 x 4096 246 us against 150).  A bf16 result rounds by far more than the truncation.
//
// Every wait is bounded; one that gives up raises KDA_DEVERR_TIMEOUT, and the CTAs leave through
// the same barriers as otherwise.
#pragma once

#include <algorithm>

#include "gemm.cuh"
#include "tc_utils.cuh"
#include "tma_maps.cuh"

namespace kda {

namespace {

constexpr uint32_t kWaitLimit = 1u << 30;
constexpr int kBK = 64;                            // c per stage: one 128-byte swizzled row
constexpr uint32_t kOpBytes = 128 * kBK * 2;       // 128 rows of an operand

// ------------------------------------------------------------------ PTX beyond tc_utils.cuh

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// One lane of the (converged) warp.  The role loops below run on whole warps with only the
// asynchronous instructions under this predicate: loop state and descriptors then live in uniform
// registers, where a loop inside a one-lane branch moves them there for every instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the shared::cluster address of `saddr` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Bulk copy of `bytes` (a multiple of 16) from this CTA's shared memory to `dst` in another CTA's,
// completing on that CTA's barrier `bar` (both shared::cluster addresses).  Only that barrier
// tells when the source has been read: such a copy belongs to no bulk group of the issuing thread.
__device__ __forceinline__ void push_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// TMA load whose bytes complete on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_3d_pair(uint32_t sdst, const void* map, int32_t x, int32_t y,
                                                 int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sdst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Tiled TMA store of one box from shared memory (tracked by the issuing thread's bulk groups);
// rows and columns past the map's extents are not written.
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t ssrc, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(ssrc)
               : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n\t"
               "tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// arrives on the barrier at this address in both CTAs of the pair when the MMAs so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// ------------------------------------------------------------------ shared pieces

// Tensor maps of the output side: boxes of 128 columns (i) x `rows` rows (j), not swizzled.
struct OutMaps {
  CUtensorMap y, z, res;
};

// The residual is loaded by the storing threads, or by TMA: into the chunk of y that it is added to
// (y's type), or as a chunk of its own.
enum : int32_t { kResDirect = 0, kResInPlace = 1, kResChunk = 2 };
// The kinds of staged chunks, in the order they follow one another for the same columns.
enum : int { kChunkZ = 0, kChunkRes = 1, kChunkY = 2 };

// The three planes of parts that fp32 operands are split into.
struct PartPlanes {
  const uint16_t *a, *b;
  int64_t lda, ldb, plane_a, plane_b;   // elements between stored rows, and between planes
  int64_t C;
};

struct TcArgs {
  GemmEpilogue epi;
  PartPlanes parts;
  int64_t I, J;
  bool staged;              // y (and z) leave through shared memory and TMA
  int32_t res_mode;         // pair kernel: how the residual comes, kRes*
  int32_t bn;               // pair kernel: columns (j) of a tile, a multiple of 32 from 128 to 256
  int32_t first_half;       // and those of them that the first four epilogue warps store
  int32_t cols;             // pair kernel: columns (j) of a staged chunk
  int32_t kblocks;          // 64-wide steps over c
  int32_t tiles_i, tiles_j;
  int32_t* err;
  unsigned long long wait_ns;   // what a wait may take: far beyond the kernel's run
};

// The products of parts of one step of c, smallest first (0 = hi, 1 = mid, 2 = lo).
__device__ __forceinline__ constexpr int part_a(int q) { return (0x201100 >> (4 * (5 - q))) & 15; }   // lo hi mid mid hi hi
__device__ __forceinline__ constexpr int part_b(int q) { return (0x021010 >> (4 * (5 - q))) & 15; }   // hi lo mid hi mid hi

// Eight steps of c of one row or column, put together again; zeros past the last step.
template <bool MN>
__device__ __forceinline__ void join8(const uint16_t* p, int64_t ld, int64_t plane, int64_t r, int64_t c, int64_t C,
                                      float (&x)[8]) {
  if constexpr (MN) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t* at = p + (c + e) * ld + r;
      x[e] = c + e < C ? bf16_bits_to_f32(at[0]) + bf16_bits_to_f32(at[plane]) + bf16_bits_to_f32(at[2 * plane]) : 0.f;
    }
  } else {                                         // (rows are whole 128-byte lines)
    const Raw8<true> hi = load_chunk<true, true>(p + r * ld + c, 0, 0, 8),
                     mid = load_chunk<true, true>(p + plane + r * ld + c, 0, 0, 8),
                     lo = load_chunk<true, true>(p + 2 * plane + r * ld + c, 0, 0, 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < C ? hi.f32(e) + mid.f32(e) + lo.f32(e) : 0.f;
  }
}
// The sum of element (i, j) as fp32 makes it, from the operands themselves.  The parts of an infinity are
// itself, 0 and 0, and its products with another operand's parts have either sign, so that the sum of
// the six products is NaN where fp32's is infinite.  Only sums that are not finite come here, one thread a
// sum (1024 x 2048 -> 2048 with one infinity in every row: 8.6 ms where finite rows take 57 us).
template <bool AMN, bool BMN>
__device__ __noinline__ float sum_again(const PartPlanes& P, int64_t i, int64_t j) {
  float s = 0.f;
  for (int64_t c = 0; c < P.C && s == s; c += 8) {
    float a[8], b[8];
    join8<AMN>(P.a, P.lda, P.plane_a, i, c, P.C, a);
    join8<BMN>(P.b, P.ldb, P.plane_b, j, c, P.C, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
  }
  return s;
}

// Waits for a phase; gives up after `limit` ns or once another role of the CTA has.
template <typename TryWait>
__device__ __forceinline__ bool wait_bounded(TryWait try_wait, unsigned long long limit, volatile int* abort) {
  unsigned long long start = 0;
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (try_wait()) return true;
    if ((i & 63) == 63) {
      const unsigned long long t = now_ns();
      if (start == 0) start = t;
      if (*abort || t - start > limit) return false;
    }
  }
  return false;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, unsigned long long limit, volatile int* abort) {
  return wait_bounded([&] { return tc::mbar_try_wait(bar, parity); }, limit, abort);
}
// the same for a barrier that the other CTA of the pair arrives on
__device__ __forceinline__ bool wait_phase_cluster(uint64_t* bar, uint32_t parity, unsigned long long limit,
                                                   volatile int* abort) {
  return wait_bounded([&] { return try_wait_cluster(bar, parity); }, limit, abort);
}
// after a timeout: the copies or products in flight
__device__ __forceinline__ void drain_phase(uint64_t* bar, uint32_t parity) {
  int never = 0;
  wait_phase(bar, parity, 100000000ull, &never);
}

// A position in a ring of N stages and the parity of the pass over it.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1;
    }
  }
};

// Descriptor of 128 (or BN) operand rows staged at `saddr`.  K-major: 8-row groups of 1024 bytes.
// MN-major: boxes of 64 rows of i (or j) by 64 steps of c (of every plane), 8192 bytes a plane; 8
// steps of c are 1024 bytes apart.
template <bool MN, int PLANES = 1>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  return MN ? (tc::smem_desc(saddr, PLANES * 8192, 1024) | (static_cast<uint64_t>(2) << 61))
            : tc::smem_desc_sw128(saddr, 1024);
}
// bytes from one MMA's 16 steps of c to the next
template <bool MN>
__device__ __forceinline__ constexpr uint32_t k_advance() { return MN ? 2048 : 32; }

// `ROWS` rows of an operand from row r0 and step c0: one box K-major, ROWS / 64 boxes MN-major
template <bool MN, int ROWS, int PLANES = 1, typename Load>
__device__ __forceinline__ void load_operand(uint32_t sdst, int64_t r0, int c0, Load load) {
  if constexpr (MN) {
#pragma unroll
    for (int b = 0; b < ROWS / 64; ++b) load(sdst + b * PLANES * 8192, static_cast<int32_t>(r0) + 64 * b, c0);
  } else {
    load(sdst, c0, static_cast<int32_t>(r0));
  }
}

// 16 columns (rows j0 .. j0 + n - 1 of the output, n <= 16) of this thread's element i, stored
// directly: any alignment.  Every load is issued before the first is used.
template <bool BF>
__device__ __forceinline__ void gather16(const void* p, int64_t ld, int64_t at, int n, float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = e < n ? load_elem<BF>(p, at + e * ld) : 0.f;
}
template <bool BF>
__device__ __forceinline__ void scatter16(void* p, int64_t ld, int64_t at, int n, const float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < n) {
      if constexpr (BF) static_cast<uint16_t*>(p)[at + e * ld] = f32_to_bf16_bits(x[e]);
      else static_cast<float*>(p)[at + e * ld] = x[e];
    }
}
// scale act(v), the choice of activation outside the loops: with two epilogue warps a scheduler a
// test an element set the pace of the persistent kernel (SiLU with the pre-activation kept on 6731
// x 4096 -> 8192: 323 us, now 293 us).  bf16 results take the faster functions.
template <typename F>
__device__ __forceinline__ void map16(float (&v)[16], float scale, F f) {
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = scale * f(v[e]);
}
__device__ __forceinline__ void activate16(const GemmEpilogue& E, float (&v)[16]) {
  const float s = E.scale;
  switch (E.act) {
    case KDA_ACT_RELU: map16(v, s, [](float z) { return act_f<true>(KDA_ACT_RELU, z); }); break;
    case KDA_ACT_SILU:
      if (E.out_bf) map16(v, s, [](float z) { return act_f<true>(KDA_ACT_SILU, z); });
      else map16(v, s, [](float z) { return act_f<false>(KDA_ACT_SILU, z); });
      break;
    case KDA_ACT_GELU:
      if (E.out_bf) map16(v, s, [](float z) { return act_f<true>(KDA_ACT_GELU, z); });
      else map16(v, s, [](float z) { return act_f<false>(KDA_ACT_GELU, z); });
      break;
    case KDA_ACT_SIGMOID:
      if (E.out_bf) map16(v, s, [](float z) { return act_f<true>(KDA_ACT_SIGMOID, z); });
      else map16(v, s, [](float z) { return act_f<false>(KDA_ACT_SIGMOID, z); });
      break;
    default: map16(v, s, [](float z) { return z; }); break;
  }
}
// FULL: with bias, activation, residual and pre-activation (the forward's K-major products; the
// gradients only scale).
template <bool FULL>
__device__ __forceinline__ void store16(const GemmEpilogue& E, float (&v)[16], int64_t i, int64_t j0, int64_t J) {
  const int n = static_cast<int>(J - j0 < 16 ? J - j0 : 16);
  if constexpr (FULL) {
    float res[16];
    if (E.res) {
      if (E.res_bf) gather16<true>(E.res, E.res_ld, j0 * E.res_ld + i, n, res);
      else gather16<false>(E.res, E.res_ld, j0 * E.res_ld + i, n, res);
    }
    if (E.z) {
      if (E.z_bf) scatter16<true>(E.z, E.z_ld, j0 * E.z_ld + i, n, v);
      else scatter16<false>(E.z, E.z_ld, j0 * E.z_ld + i, n, v);
    }
    activate16(E, v);
    if (E.res) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += res[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] *= E.scale;
  }
  if (E.out_bf) scatter16<true>(E.out, E.out_ld, j0 * E.out_ld + i, n, v);
  else scatter16<false>(E.out, E.out_ld, j0 * E.out_ld + i, n, v);
}
__device__ __forceinline__ void load16(uint32_t src, float bias, float (&v)[16]) {
  uint32_t r[16];
  tc::tmem_ld16(src, r);
  tc::tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]) + bias;
}

// 16 columns of a staged [column][128] tile at `at` (this thread's element of its first column);
// the residual, if it is staged, lies where the result goes
template <bool BF>
__device__ __forceinline__ void put16(unsigned char* at, bool add, const float (&v)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if constexpr (BF) {
      uint16_t* p = reinterpret_cast<uint16_t*>(at + e * 256);
      *p = f32_to_bf16_bits(add ? v[e] + bf16_bits_to_f32(*p) : v[e]);
    } else {
      float* p = reinterpret_cast<float*>(at + e * 512);
      *p = add ? v[e] + *p : v[e];
    }
  }
}
__device__ __forceinline__ void put16(unsigned char* tile, bool bf, int col, int row, bool add, const float (&v)[16]) {
  if (bf) {
    unsigned char* at = tile + col * 256 + row * 2;
    if (add) put16<true>(at, true, v);
    else put16<true>(at, false, v);
  } else {
    unsigned char* at = tile + col * 512 + row * 4;
    if (add) put16<false>(at, true, v);
    else put16<false>(at, false, v);
  }
}

__device__ __forceinline__ void add16(const unsigned char* tile, bool bf, int col, int row, float (&v)[16]) {
  if (bf) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      v[e] += bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(tile + (col + e) * 256 + row * 2));
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] += *reinterpret_cast<const float*>(tile + (col + e) * 512 + row * 4);
  }
}

// ------------------------------------------------------------------ pairs of CTAs

constexpr int kPairStages = 6;
constexpr int kPairStretch = 8;                    // PROMOTE: 64-wide steps in one accumulator
constexpr int kPromoteBN = 160;
constexpr int kPairThreads = 384;                  // TMA, MMA, 2 output warps, 8 epilogue warps
constexpr uint32_t kPairStage = 2 * kOpBytes;
constexpr uint32_t kSlot = 8192;                   // a staged chunk: 128 x 32 bf16 or 128 x 16 fp32
constexpr size_t kPairSmem = kPairStages * kPairStage + 4 * kSlot + 1024;
constexpr int kRaster = 16;                        // i tiles taken together, for reuse in L2

// Tile t of the persistent order: groups of kRaster i tiles, j slowest inside a group, so that a
// group's rows of A stay in L2 while those of B pass by (16384 x 4096 x 4096: 4 tiles 312 us, 8
// 305 us, 16 301 us).
__device__ __forceinline__ void tile_of(int t, int tiles_i, int tiles_j, int& ti, int& tj) {
  const int per = kRaster * tiles_j;
  const int grp = t / per, in = t - grp * per;
  const int width = min(kRaster, tiles_i - grp * kRaster);
  tj = in / width;
  ti = grp * kRaster + in - tj * width;
}

// The chunks of one half (the first columns or the others) of this CTA's tiles, in the order the epilogue forms them:
// per `cols` columns the pre-activation (if it is kept), a residual of another type than y's, then y.
struct Chunk {
  int t, c, width, kind;
  int64_t i0, j0;
  __device__ __forceinline__ static int first_kind(const TcArgs& A) {
    return A.epi.z ? kChunkZ : A.res_mode == kResChunk ? kChunkRes : kChunkY;
  }
  __device__ __forceinline__ void place(const TcArgs& A, uint32_t rank, int half, int tiles, int step) {
    for (; t < tiles; t += step) {
      int ti, tj;
      tile_of(t, A.tiles_i, A.tiles_j, ti, tj);
      i0 = static_cast<int64_t>(ti) * 256 + rank * 128;
      j0 = static_cast<int64_t>(tj) * A.bn + half * A.first_half;
      width = half ? A.bn - A.first_half : A.first_half;
      if (i0 < A.I && j0 < A.J && width > 0) return;
    }
  }
  __device__ __forceinline__ void start(const TcArgs& A, uint32_t rank, int half, int first, int tiles, int step) {
    t = first;
    c = 0;
    kind = first_kind(A);
    place(A, rank, half, tiles, step);
  }
  __device__ __forceinline__ void next(const TcArgs& A, uint32_t rank, int half, int tiles, int step) {
    if (kind != kChunkY) {
      kind = kind == kChunkZ && A.res_mode == kResChunk ? kChunkRes : kChunkY;
      return;
    }
    kind = first_kind(A);
    c += A.cols;
    if (c >= width || j0 + c >= A.J) {
      c = 0;
      t += step;
      place(A, rank, half, tiles, step);
    }
  }
};

template <bool AMN, bool BMN, bool PROMOTE>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ OutMaps maps, const __grid_constant__ TcArgs A) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2], drain;
  __shared__ __align__(8) uint64_t ready[2][2], written[2][2];   // [half][slot] of the staged chunks
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const uint32_t smem = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int tiles = A.tiles_i * A.tiles_j;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  // columns of an accumulator, and the steps of c that one takes
  constexpr int kAcc = PROMOTE ? kPromoteBN : 256;
  constexpr bool FULL = !AMN;
  const int stretch = PROMOTE ? kPairStretch : A.kblocks;

  if (threadIdx.x == 32) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 16);            // 8 epilogue warps of both CTAs
      for (int h = 0; h < 2; ++h) {
        tc::mbar_init(&ready[h][b], 1);
        tc::mbar_init(&written[h][b], 128);
      }
    }
    tc::mbar_init(&drain, 1);
    tc::fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 2) tmem_alloc_pair(&s_tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {                                 // both CTAs: stage this CTA's rows of A and B
    Ring<kPairStages> at;
    int it = 0;                                    // loads issued so far
    bool ok = true;
    const uint32_t full0 = map_rank(tc::smem_u32(&full[0]), 0);
    // both CTAs' rows (an MN-major operand comes in boxes of 64 columns, all 128 of them)
    const uint32_t stage_bytes = 2 * (kOpBytes + (BMN ? kOpBytes : A.bn / 2 * kBK * 2));
    for (int t = first; t < tiles && ok; t += step) {
      int ti, tj;
      tile_of(t, A.tiles_i, A.tiles_j, ti, tj);
      const int64_t i0 = static_cast<int64_t>(ti) * 256 + rank * 128;
      const int64_t j0 = static_cast<int64_t>(tj) * A.bn + rank * (A.bn / 2);
      for (int k = 0; k < A.kblocks; ++k, ++it, at.next()) {
        const int s = at.s;
        if (!__all_sync(0xffffffffu, wait_phase(&empty[s], at.ph ^ 1, A.wait_ns, &s_abort))) {
          ok = false;
          break;
        }
        const uint32_t bar = full0 + s * 8;
        const uint32_t sa = smem + s * kPairStage, sb = sa + kOpBytes;
        if (elect_one()) {
          if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], stage_bytes);
          load_operand<AMN, 128>(sa, i0, k * kBK, [&](uint32_t d, int32_t x, int32_t y) {
            tma_load_3d_pair(d, &map_a, x, y, 0, bar);
          });
          load_operand<BMN, 128>(sb, j0, k * kBK, [&](uint32_t d, int32_t x, int32_t y) {
            tma_load_3d_pair(d, &map_b, x, y, 0, bar);
          });
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
      // the copies still in flight (their bytes count on the leader's barriers)
      if (rank == 0) {
        const int from = it > kPairStages ? it - kPairStages : 0;
        for (int j = from; j < it; ++j)
          drain_phase(&full[j % kPairStages], (j / kPairStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {                               // the leader multiplies for the pair
      const uint32_t idesc = tc::idesc_f16(256, A.bn, tc::kBF16, false, AMN, BMN);
      const uint64_t da0 = operand_desc<AMN>(smem), db0 = operand_desc<BMN>(smem + kOpBytes);
      Ring<kPairStages> at;
      int n = 0;
      int64_t left = static_cast<int64_t>((tiles - first + step - 1) / step) * A.kblocks;   // stages to come
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int base = 0; base < A.kblocks && ok; base += stretch, ++n) {
          const int b = n & 1;
          if (!__all_sync(0xffffffffu, wait_phase_cluster(&acc_empty[b], ((n >> 1) & 1) ^ 1, A.wait_ns, &s_abort))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t d = tmem + b * kAcc;
          const int k1 = min(A.kblocks, base + stretch);
          for (int k = base; k < k1; ++k) {
            const int s = at.s;
            if (!__all_sync(0xffffffffu, wait_phase(&full[s], at.ph, A.wait_ns, &s_abort))) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const uint64_t da = tc::desc_add(da0, s * kPairStage), db = tc::desc_add(db0, s * kPairStage);
            at.next();
            if (elect_one()) {
#pragma unroll
              for (int q = 0; q < kBK / 16; ++q)
                mma_pair(d, tc::desc_add(da, q * k_advance<AMN>()), tc::desc_add(db, q * k_advance<BMN>()), idesc,
                         k > base || q > 0);
              // (A release that no load waits for could arrive when the CTA, or its peer, is gone.)
              if (left > kPairStages) commit_pair(&empty[s]);
            }
            --left;
            __syncwarp();
          }
          if (ok && elect_one()) commit_pair(&acc_full[b]);
          __syncwarp();
        }
      }
      if (!ok && lane == 0) {
        s_abort = 1;
        raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
        commit_pair(&drain);                       // the products still in flight
        drain_phase(&drain, 0);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // One thread a half moves the staged chunks: it hands a slot to the epilogue (with the
    // residual's values loaded into it, or just free), and stores it once it is written.
    if (lane == 0 && A.staged) {
      const int half = warp - 2;
      const uint32_t bytes = 128u * A.cols * (A.epi.res_bf ? 2 : 4);
      Chunk cur, ahead;
      cur.start(A, rank, half, first, tiles, step);
      ahead = cur;
      auto hand_over = [&](int q) {
        if (ahead.t >= tiles) return;
        uint64_t* bar = &ready[half][q & 1];
        if (ahead.kind == kChunkRes || (ahead.kind == kChunkY && A.res_mode == kResInPlace)) {
          tc::mbar_arrive_expect_tx(bar, bytes);
          tc::tma_load_2d(smem + kPairStages * kPairStage + (half * 2 + (q & 1)) * kSlot, &maps.res,
                          static_cast<int32_t>(ahead.i0), static_cast<int32_t>(ahead.j0) + ahead.c, bar);
        } else {
          tc::mbar_arrive(bar);
        }
        ahead.next(A, rank, half, tiles, step);
      };
      hand_over(0);
      hand_over(1);
      int q = 0;
      for (; cur.t < tiles; ++q, cur.next(A, rank, half, tiles, step)) {
        if (!wait_phase(&written[half][q & 1], (q >> 1) & 1, A.wait_ns, &s_abort)) {
          s_abort = 1;
          raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
          if (A.res_mode != kResDirect) {          // loads in flight
            drain_phase(&ready[half][q & 1], (q >> 1) & 1);
            drain_phase(&ready[half][(q + 1) & 1], ((q + 1) >> 1) & 1);
          }
          break;
        }
        if (cur.kind != kChunkRes) {
          tma_store_2d(cur.kind == kChunkZ ? &maps.z : &maps.y,
                       smem + kPairStages * kPairStage + (half * 2 + (q & 1)) * kSlot, static_cast<int32_t>(cur.i0),
                       static_cast<int32_t>(cur.j0) + cur.c);
          tc::bulk_commit();
          tc::bulk_wait_read();
        }
        hand_over(q + 2);
      }
      tc::bulk_wait_read();                        // (the stores themselves end with the kernel)
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lead = map_rank(tc::smem_u32(&acc_empty[0]), 0);
    unsigned char* slots = smem_raw + (smem - tc::smem_u32(smem_raw)) + kPairStages * kPairStage + half * 2 * kSlot;
    // the whole warp takes the same way, as its tensor-memory loads need
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_phase(bar, parity, A.wait_ns, &s_abort)) != 0;
    };
    int n = 0, q = 0;
    for (int t = first; t < tiles; t += step, ++n) {
      int ti, tj;
      tile_of(t, A.tiles_i, A.tiles_j, ti, tj);
      const int64_t ib = static_cast<int64_t>(ti) * 256 + rank * 128;
      const int64_t i = ib + quad * 32 + lane;
      const int64_t j0 = static_cast<int64_t>(tj) * A.bn + half * A.first_half;
      const int width = half ? A.bn - A.first_half : A.first_half;
      const bool in = i < A.I;
      const float bias = FULL && A.epi.bias && in ? __ldg(A.epi.bias + i) : 0.f;
      bool got = wait_warp(&acc_full[n & 1], (n >> 1) & 1);
      tc::fence_after_sync();
      const uint32_t mine = tmem + half * A.first_half + (static_cast<uint32_t>(quad * 32) << 16);
      const uint32_t sum = mine + 2 * kAcc;
      if constexpr (PROMOTE) {                     // all stretches but the last go into the sum
        for (int base = stretch; base < A.kblocks && got; base += stretch) {
#pragma unroll 1
          for (int c = 0; c < width; c += 16) {
            float v[16];
            load16(mine + (n & 1) * kAcc + c, 0.f, v);
            if (base > stretch) {
              float u[16];
              load16(sum + c, 0.f, u);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] += u[e];
            }
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(v[e]);
            tc::tmem_st16(sum + c, r);
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) arrive_remote(lead + (n & 1) * 8);
          ++n;
          got = wait_warp(&acc_full[n & 1], (n >> 1) & 1);
          tc::fence_after_sync();
        }
      }
      const int b = n & 1;
      const uint32_t src = mine + b * kAcc;
      const bool summed = PROMOTE && A.kblocks > stretch;
      auto load_cols = [&](int c, float (&v)[16]) {
        load16(src + c, bias, v);
        if (summed) {
          float u[16];
          load16(sum + c, 0.f, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] += u[e];
        }
      };
      // the columns of this half that exist (none where the CTA's rows are past the end)
      const int ncol = ib < A.I ? static_cast<int>(A.J - j0 < width ? (A.J > j0 ? A.J - j0 : 0) : width) : 0;
      if (!A.staged) {
#pragma unroll 1
        for (int c = 0; c < ncol && got; c += 16) {
          float v[16];
          load_cols(c, v);
          if (in) store16<FULL>(A.epi, v, i, j0 + c, A.J);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < ncol && got; c += A.cols) {
          float v[2][16] = {};
          load_cols(c, v[0]);
          if (A.cols == 32) load_cols(c + 16, v[1]);
          if (FULL && A.epi.z) {
            got = got && wait_warp(&ready[half][q & 1], (q >> 1) & 1);
            unsigned char* tile = slots + (q & 1) * kSlot;
            put16(tile, A.epi.z_bf, 0, quad * 32 + lane, false, v[0]);
            if (A.cols == 32) put16(tile, A.epi.z_bf, 16, quad * 32 + lane, false, v[1]);
            tc::fence_async_smem();
            tc::mbar_arrive(&written[half][q & 1]);
            ++q;
          }
          if constexpr (FULL) {
            activate16(A.epi, v[0]);
            if (A.cols == 32) activate16(A.epi, v[1]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v[0][e] *= A.epi.scale;
              v[1][e] *= A.epi.scale;
            }
          }
          if (FULL && A.res_mode == kResChunk) {
            got = got && wait_warp(&ready[half][q & 1], (q >> 1) & 1);
            const unsigned char* tile = slots + (q & 1) * kSlot;
            add16(tile, A.epi.res_bf, 0, quad * 32 + lane, v[0]);
            if (A.cols == 32) add16(tile, A.epi.res_bf, 16, quad * 32 + lane, v[1]);
            tc::mbar_arrive(&written[half][q & 1]);
            ++q;
          } else if (FULL && A.epi.res && A.res_mode == kResDirect && in) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int m = min(16, ncol - c - 16 * u);
              if (m <= 0 || 16 * u >= A.cols) continue;
              const int64_t at = (j0 + c + 16 * u) * A.epi.res_ld + i;
              float r[16];
              if (A.epi.res_bf) gather16<true>(A.epi.res, A.epi.res_ld, at, m, r);
              else gather16<false>(A.epi.res, A.epi.res_ld, at, m, r);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[u][e] += r[e];
            }
          }
          got = got && wait_warp(&ready[half][q & 1], (q >> 1) & 1);
          unsigned char* tile = slots + (q & 1) * kSlot;
          put16(tile, A.epi.out_bf, 0, quad * 32 + lane, FULL && A.res_mode == kResInPlace, v[0]);
          if (A.cols == 32) put16(tile, A.epi.out_bf, 16, quad * 32 + lane, FULL && A.res_mode == kResInPlace, v[1]);
          tc::fence_async_smem();
          tc::mbar_arrive(&written[half][q & 1]);
          ++q;
        }
      }
      if (!got) {
        raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
        s_abort = 1;
        break;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_remote(lead + b * 8);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();                                  // the peer's copies, products and arrivals are done
  tc::fence_after_sync();
  if (warp == 2) tmem_free_pair(tmem, 512);
}

// ------------------------------------------------------------------ one CTA a tile, split over c

constexpr int kSplitThreads = 320;                 // TMA, MMA, 8 epilogue warps

// PARTS: how the sum over c is kept.  0: in one accumulator.  1: promoted every kPairStretch steps.
// 6: fp32 operands; a stage holds all three parts of both, so that they are read once for
// their six products, and every step of c is promoted.
template <int BN, int PARTS>
struct SplitShape {
  static constexpr int planes = PARTS == 6 ? 3 : 1;
  static constexpr uint32_t a_bytes = planes * kOpBytes;
  static constexpr uint32_t stage = a_bytes + planes * BN * kBK * 2;
  // the ring: some 200 KB, one CTA an SM (with 96 KB and two CTAs the narrow tile's loads waited on
  // the ring: 16 x 4096 -> 16384 from HBM 32.6 us, so 25.2 us)
  static constexpr int stages = PARTS == 6 ? (BN == 64 ? 3 : 2) : BN == 64 ? 8 : 6;
  static constexpr size_t smem = static_cast<size_t>(stage) * stages + 1024;
  // a split's own part and those received (7 shares of up to BN / 8 + 7 columns, or one of BN / 2)
  static_assert(static_cast<size_t>(stage) * stages >= 128 * 4 * (BN + 7 * 8 + BN),
                "the parts reuse the ring");
};

template <bool AMN, bool BMN, int BN, int PARTS>
__global__ void __launch_bounds__(kSplitThreads)
gemm_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ OutMaps maps, const __grid_constant__ TcArgs A, const int splits) {
  using S = SplitShape<BN, PARTS>;
  constexpr bool PROMOTE = PARTS > 0;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[S::stages], empty[S::stages], acc_full[2], acc_empty[2], received;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const uint32_t smem = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  float* part = reinterpret_cast<float*>(smem_raw + (smem - tc::smem_u32(smem_raw)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / splits;
  const int64_t i0 = static_cast<int64_t>(tile % A.tiles_i) * 128, j0 = static_cast<int64_t>(tile / A.tiles_i) * BN;
  const int k0 = static_cast<int>(static_cast<int64_t>(A.kblocks) * rank / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(A.kblocks) * (rank + 1) / splits);
  // the steps of c that one accumulator takes
  const int stretch = PARTS == 6 ? 1 : PARTS == 1 ? kPairStretch : k1 - k0;
  constexpr uint32_t kCols = PROMOTE ? 2 * BN : BN;

  auto load_stage = [&](int s, int k) {
    const uint32_t sa = smem + s * S::stage, sb = sa + S::a_bytes;
    tc::mbar_arrive_expect_tx(&full[s], S::stage);
    load_operand<AMN, 128, S::planes>(sa, i0, k * kBK, [&](uint32_t d, int32_t x, int32_t y) {
      tc::tma_load_3d(d, &map_a, x, y, 0, &full[s]);
    });
    load_operand<BMN, BN, S::planes>(sb, j0, k * kBK, [&](uint32_t d, int32_t x, int32_t y) {
      tc::tma_load_3d(d, &map_b, x, y, 0, &full[s]);
    });
  };
  // The first stages are requested before the block meets: the loads need nothing but their barriers.
  const int early = min(S::stages, k1 - k0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 8);             // the epilogue warps
    }
    tc::mbar_init(&received, 1);
    tc::fence_mbar_init();
    s_abort = 0;
    for (int s = 0; s < early; ++s) load_stage(s, k0 + s);
  }
  if (warp == 1) {
    tc::tmem_alloc(&s_tmem, kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    Ring<S::stages> at;                            // after a first pass over the ring
    at.ph = 1;
    int it = early;
    bool ok = true;
    for (int k = k0 + early; k < k1; ++k, ++it, at.next()) {
      const int s = at.s;
      if (!__all_sync(0xffffffffu, wait_phase(&empty[s], at.ph ^ 1, A.wait_ns, &s_abort))) {
        ok = false;
        break;
      }
      if (elect_one()) load_stage(s, k);
      __syncwarp();
    }
    if (!ok && lane == 0) {                        // wait for the copies in flight
      s_abort = 1;
      raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
      for (int j = max(0, it - S::stages); j < it; ++j)
        drain_phase(&full[j % S::stages], (j / S::stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16(128, BN, tc::kBF16, false, AMN, BMN);
    const uint64_t da0 = operand_desc<AMN, S::planes>(smem), db0 = operand_desc<BMN, S::planes>(smem + S::a_bytes);
    Ring<S::stages> at;
    bool ok = true;
    int n = 0;
    for (int base = k0; base < k1 && ok; base += stretch, ++n) {
      const int b = n & 1;
      const uint32_t d = tmem + (PROMOTE ? b * BN : 0);
      if (PROMOTE && !__all_sync(0xffffffffu, wait_phase(&acc_empty[b], ((n >> 1) & 1) ^ 1, A.wait_ns, &s_abort))) {
        ok = false;
        break;
      }
      const int last = min(base + stretch, k1);
      for (int k = base; k < last; ++k) {
        const int s = at.s;
        if (!__all_sync(0xffffffffu, wait_phase(&full[s], at.ph, A.wait_ns, &s_abort))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint64_t da = tc::desc_add(da0, s * S::stage), db = tc::desc_add(db0, s * S::stage);
        at.next();
        if (elect_one()) {
#pragma unroll
          for (int p = 0; p < (PARTS == 6 ? 6 : 1); ++p) {
            // a part's place in the stage
            const uint32_t pa = PARTS == 6 ? part_a(p) * (AMN ? 8192 : kOpBytes) : 0;
            const uint32_t pb = PARTS == 6 ? part_b(p) * (BMN ? 8192 : BN * kBK * 2) : 0;
#pragma unroll
            for (int q = 0; q < kBK / 16; ++q)
              tc::mma_ss(d, tc::desc_add(da, pa + q * k_advance<AMN>()), tc::desc_add(db, pb + q * k_advance<BMN>()),
                         idesc, k > base || p > 0 || q > 0);
          }
          if (k + S::stages < k1) tc::mma_commit(&empty[s]);   // (only releases that a load waits for)
        }
        __syncwarp();
      }
      if (elect_one()) tc::mma_commit(&acc_full[b]);   // also after a timeout: the products in flight
      __syncwarp();
    }
    if (!ok) {
      s_abort = 1;
      raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
    }
  }
  // Epilogue warps: 32 lanes of the tile (quad), every other 16 columns (half).
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const int64_t i = i0 + quad * 32 + lane;
  const bool in = i < A.I;
  constexpr bool FULL = !AMN;
  const float bias = FULL && warp >= 2 && A.epi.bias && in ? __ldg(A.epi.bias + i) : 0.f;
  const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  if (FULL && warp >= 2 && A.epi.res && i0 + quad * 32 < A.I) {   // the residual, towards L2 meanwhile
    const char* r = static_cast<const char*>(A.epi.res) + (i0 + quad * 32) * (A.epi.res_bf ? 2 : 4);
    for (int c = half * 32 + lane; c < BN && j0 + c < A.J; c += 64)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r + (j0 + c) * A.epi.res_ld * (A.epi.res_bf ? 2 : 4)));
  }
  bool ready = true;
  float sum[PROMOTE ? BN / 2 : 1];                 // PROMOTE: this thread's half row of the tile
  if (warp >= 2) {
    int n = 0;
    if constexpr (PROMOTE) {
#pragma unroll
      for (int c = 0; c < BN / 2; ++c) sum[c] = 0.f;
      for (int base = k0; base < k1 && ready; base += stretch, ++n) {
        ready = __all_sync(0xffffffffu, wait_phase(&acc_full[n & 1], (n >> 1) & 1, A.wait_ns, &s_abort));
        if (!ready) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < BN / 2; c += 16) {
          float v[16];
          load16(src + (n & 1) * BN + 2 * c + half * 16, 0.f, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[c + e] += v[e];
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[n & 1]);
      }
      ready = !tc::named_sync_or(2, 256, !ready);
    } else {
      ready = !tc::named_sync_or(2, 256, !wait_phase(&acc_full[0], 0, A.wait_ns, &s_abort));
    }
    if (!ready) raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
    tc::fence_after_sync();
  }
  // The CTA's columns [c0, c1) of the tile.  Split: every CTA lays its part of the tile out as
  // [column][row]; rank r gets the r-th share of the columns (a multiple of 8) of every other
  // part, one stretch of memory each, behind its own, and adds the parts in rank order.
  const int ncol = static_cast<int>(A.J - j0 < BN ? A.J - j0 : BN);
  const int per = ((ncol + splits - 1) / splits + 7) / 8 * 8;
  int c0 = 0, c1 = ncol;
  if (splits > 1) {
    c0 = min(ncol, rank * per);
    c1 = min(ncol, c0 + per);
    if (warp >= 2) {
      float* at = part + quad * 32 + lane;
      if constexpr (PROMOTE) {
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) {
          const int col = (c / 16) * 32 + half * 16 + c % 16;
          if (col < ncol) at[col * 128] = sum[c];
        }
      } else {
#pragma unroll 1
        for (int c = half * 16; c < ncol; c += 32) {
          float v[16];
          load16(src + c, 0.f, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) at[(c + e) * 128] = v[e];
        }
      }
      tc::fence_async_smem();
    }
    cluster_sync();                                // every ring is free, every part laid out
    if (threadIdx.x == 0) {
      if (c1 > c0) tc::mbar_arrive_expect_tx(&received, static_cast<uint32_t>((splits - 1) * (c1 - c0)) * 512);
      for (int d = 1; d < splits; ++d) {           // the next ranks first, so that no CTA is everyone's target
        const int to = rank + d < splits ? rank + d : rank + d - splits;
        const int p0 = min(ncol, to * per), n = min(ncol, p0 + per) - p0;
        // the sender's place among the receiver's others, in rank order
        const int place = rank < to ? rank : rank - 1;
        if (n > 0)
          push_cluster(map_rank(smem + 128 * BN * 4 + place * per * 512, static_cast<uint32_t>(to)), smem + p0 * 512,
                       static_cast<uint32_t>(n) * 512, map_rank(tc::smem_u32(&received), static_cast<uint32_t>(to)));
      }
    }
    __syncwarp();
    if (warp >= 2 && c1 > c0) {
      ready = !tc::named_sync_or(2, 256, !wait_phase_cluster(&received, 0, A.wait_ns, &s_abort)) && ready;
      if (!ready) raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
    }
    cluster_arrive();                              // this CTA has received what it waits for
  }
  // the finished tile, [column - c0][128], for TMA: behind the parts if there are any
  unsigned char* out = smem_raw + (smem - tc::smem_u32(smem_raw)) +
                       (splits > 1 ? 128 * BN * 4 + (splits - 1) * per * 512 : 0);
  const int cpad = (c1 - c0 + 15) / 16 * 16;
  unsigned char* out_z = out + cpad * 128 * (A.epi.out_bf ? 2 : 4);
  if (warp >= 2 && ready) {
    const float* mine = part + quad * 32 + lane;
    // sums of parts that are not finite: 16 columns of the tile from c
    auto mend = [&](float (&v)[16], int c) {
      if constexpr (PARTS == 6) {
        float zero = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) zero = fmaf(v[e], 0.f, zero);
        if (zero == 0.f) return;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (!(fabsf(v[e]) < INFINITY) && in && c + e < c1) v[e] = sum_again<AMN, BMN>(A.parts, i, j0 + c + e);
      }
    };
    // (unrolled where the tile is in registers, whose places are fixed at compile time)
#pragma unroll (PROMOTE ? BN / 32 : 1)
    for (int cc = 0; cc < BN / 2; cc += 16) {
      const int c = c0 + 2 * cc + half * 16;
      if (c >= c1) break;
      float v[16];
      if (splits == 1) {
        if constexpr (PROMOTE) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = sum[cc + e];
          mend(v, c);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] += bias;
        } else {
          load16(src + c, bias, v);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        const int n = min(16, c1 - c);
#pragma unroll 1
        for (int p = 0; p < splits; ++p) {
          const float* at = p == rank ? mine + c * 128
                                      : mine + 128 * BN + ((p < rank ? p : p - 1) * per + c - c0) * 128;
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] += e < n ? at[e * 128] : 0.f;
        }
        mend(v, c);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] += bias;
      }
      if (!A.staged) {
        if (in) store16<FULL>(A.epi, v, i, j0 + c, j0 + c1);
      } else {
        if constexpr (FULL) {
          const int m = min(16, c1 - c);
          float r[16];
          if (A.epi.res && in) {
            const int64_t at = (j0 + c) * A.epi.res_ld + i;
            if (A.epi.res_bf) gather16<true>(A.epi.res, A.epi.res_ld, at, m, r);
            else gather16<false>(A.epi.res, A.epi.res_ld, at, m, r);
          }
          if (A.epi.z) put16(out_z, A.epi.z_bf, c - c0, quad * 32 + lane, false, v);
          activate16(A.epi, v);
          if (A.epi.res && in) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += r[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] *= A.epi.scale;
        }
        put16(out, A.epi.out_bf, c - c0, quad * 32 + lane, false, v);
      }
    }
    if (A.staged) {
      tc::fence_async_smem();
      tc::named_sync(1, 256);
      if (warp == 2 && lane == 0) {                // boxes of 8 columns
        for (int c = c0; c < c1; c += 8) {
          tma_store_2d(&maps.y, tc::smem_u32(out) + (c - c0) * 128 * (A.epi.out_bf ? 2 : 4),
                       static_cast<int32_t>(i0), static_cast<int32_t>(j0) + c);
          if (A.epi.z)
            tma_store_2d(&maps.z, tc::smem_u32(out_z) + (c - c0) * 128 * (A.epi.z_bf ? 2 : 4),
                         static_cast<int32_t>(i0), static_cast<int32_t>(j0) + c);
        }
        tc::bulk_commit();
        tc::bulk_wait_read();                      // (the stores themselves end with the kernel)
      }
    }
  }
  // Every CTA has received its shares, so this one's pushes have read its shared memory: it may leave.
  // (The arrival comes before the epilogue, which hides the wait.)
  __syncwarp();
  if (splits > 1) cluster_wait();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------------ tensor maps, launches

// boxes of 64 columns (128 bytes, swizzled) x box_rows rows x every plane
bool encode_operand(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t planes,
                    uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc || rows == 0 || (reinterpret_cast<uintptr_t>(base) & 15u) || (ld & 7u)) return false;
  const cuuint64_t dims[3] = {cols, rows, planes};
  const cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  const cuuint32_t box[3] = {64, box_rows, planes};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode(CUtensorMap* m, const GemmOperand& X, int64_t R, int64_t C, int planes, int tile_rows) {
  // stored rows are r (K-major) or c (MN-major)
  return X.mn ? encode_operand(m, X.p, C, R, X.ld, planes, 64) : encode_operand(m, X.p, R, C, X.ld, planes, tile_rows);
}

// a [J, I] array on the output side, in boxes of 128 columns x `rows` rows
bool encode_out(CUtensorMap* m, const void* base, bool bf, int64_t I, int64_t J, int64_t ld, int rows) {
  auto enc = tensor_map_encoder();
  const cuuint64_t es = bf ? 2 : 4;
  if (!enc || (reinterpret_cast<uintptr_t>(base) & 15u) || ld * es % 16) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(I), static_cast<cuuint64_t>(J)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output leaves by TMA where y and z have 16-byte aligned rows; the residual arrives by it
// (pair kernel) where it has such rows too.
void encode_outputs(const Gemm& g, TcArgs* A, OutMaps* m, int rows, bool residual) {
  const GemmEpilogue& E = g.epi;
  A->staged = encode_out(&m->y, E.out, E.out_bf, g.I, g.J, E.out_ld, rows) &&
              (!E.z || encode_out(&m->z, E.z, E.z_bf, g.I, g.J, E.z_ld, rows));
  A->res_mode = kResDirect;
  if (residual && A->staged && E.res && encode_out(&m->res, E.res, E.res_bf, g.I, g.J, E.res_ld, rows))
    A->res_mode = E.res_bf == E.out_bf ? kResInPlace : kResChunk;
}

template <bool AMN, bool BMN, bool PROMOTE>
cudaError_t launch_pair(const Gemm& g, TcArgs A, int planes, int pairs, cudaStream_t st) {
  CUtensorMap ma, mb;
  OutMaps out;
  A.cols = g.epi.out_bf && (!g.epi.z || g.epi.z_bf) && (!g.epi.res || g.epi.res_bf) ? 32 : 16;
  encode_outputs(g, &A, &out, A.cols, true);
  // The width that wastes least in the last wave.  A narrower tile moves more bytes for its
  // products, so it takes longer than its share of a wide one's time (measured on 16384 x 4096 x
  // 4096, in thousandths).  dw of 16384 x 2048 -> 6144, 2.53 waves of 256 columns: 233 us, 2.95
  // waves of 224: 218 us.
  constexpr int kWidth[5] = {256, 224, 192, 160, 128}, kCost[5] = {1000, 885, 820, 760, 730};
  int64_t best = 0;
  for (int c = 0; c < 5; ++c) {
    const int64_t tiles = ((g.I + 255) / 256) * ((g.J + kWidth[c] - 1) / kWidth[c]);
    const int64_t cost = (tiles + pairs - 1) / pairs * kCost[c];
    if (best == 0 || cost < best) {
      best = cost;
      A.bn = kWidth[c];
    }
  }
  if (PROMOTE) A.bn = kPromoteBN;
  A.first_half = PROMOTE ? kPromoteBN / 2 : 128;
  if (!encode(&ma, g.A, g.I, g.C, planes, 128) || !encode(&mb, g.B, g.J, g.C, planes, A.bn / 2)) return cudaErrorInvalidValue;
  A.tiles_i = static_cast<int32_t>((g.I + 255) / 256);
  A.tiles_j = static_cast<int32_t>((g.J + A.bn - 1) / A.bn);
  auto k = gemm_pair_kernel<AMN, BMN, PROMOTE>;
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_smem(k, kPairSmem, raised);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(A.tiles_i) * A.tiles_j;
  if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(tiles, pairs));
  k<<<grid, kPairThreads, kPairSmem, st>>>(ma, mb, out, A);
  return cudaGetLastError();
}

// How many clusters of `size` CTAs of kernel k run at once on the current device (asked once).
template <typename Kernel>
int active_clusters(Kernel k, int size, size_t smem, std::atomic<int> (&known)[16][9]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return 0;
  int n = known[dev][size].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(size);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) n = 0;
    n = std::max(n, 1);
    known[dev][size].store(n, std::memory_order_relaxed);
  }
  return n;
}

// `splits`: the most ways that pay; fewer where their clusters would not all run at once (a cluster
// lies within a group of SMs: 48 clusters of three on 152 SMs took two waves, 14.2 us against 9.9
// for 48 of two).
template <bool AMN, bool BMN, int BN, int PARTS>
cudaError_t launch_split(const Gemm& g, TcArgs A, int planes, int splits, cudaStream_t st) {
  CUtensorMap ma, mb;
  OutMaps out;
  A.tiles_i = static_cast<int32_t>((g.I + 127) / 128);
  A.tiles_j = static_cast<int32_t>((g.J + BN - 1) / BN);
  const int64_t tiles = static_cast<int64_t>(A.tiles_i) * A.tiles_j;
  auto k = gemm_split_kernel<AMN, BMN, BN, PARTS>;
  static std::atomic<uint64_t> raised{0};
  cudaError_t e = raise_smem(k, (SplitShape<BN, PARTS>::smem), raised);
  if (e != cudaSuccess) return e;
  static std::atomic<int> active[16][9];
  while (splits > 1 &&
         (tiles * splits > sm_count() || tiles > active_clusters(k, splits, (SplitShape<BN, PARTS>::smem), active)))
    --splits;
  // what does not fit behind the parts is stored directly
  const size_t cols = splits == 1 ? BN : ((BN + splits - 1) / splits + 15) / 16 * 16;
  const size_t bytes = (splits == 1 ? 0 : 128 * BN * 4 + (splits - 1) * cols * 512) +
                       cols * 128 * ((g.epi.out_bf ? 2 : 4) + (!g.epi.z ? 0 : g.epi.z_bf ? 2 : 4));
  if (bytes <= (SplitShape<BN, PARTS>::smem) - 1024) encode_outputs(g, &A, &out, 8, false);
  else A.staged = false;
  if (!encode(&ma, g.A, g.I, g.C, planes, 128) || !encode(&mb, g.B, g.J, g.C, planes, BN)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = (SplitShape<BN, PARTS>::smem);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(splits);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, k, ma, mb, out, A, splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool AMN, bool BMN>
cudaError_t launch_shape(const Gemm& g, int planes, cudaStream_t st) {
  TcArgs A{};
  A.epi = g.epi;
  A.I = g.I; A.J = g.J;
  A.kblocks = static_cast<int32_t>((g.C + kBK - 1) / kBK);
  A.err = g.err;
  if (planes == 3)
    A.parts = {static_cast<const uint16_t*>(g.A.p), static_cast<const uint16_t*>(g.B.p), g.A.ld, g.B.ld,
               (AMN ? g.C : g.I) * g.A.ld, (BMN ? g.C : g.J) * g.B.ld, g.C};
  A.wait_ns = 2000000000ull + static_cast<unsigned long long>(A.kblocks) * 4000ull;
  const int sms = sm_count();
  const int64_t big = ((g.I + 255) / 256) * ((g.J + 255) / 256);
  const bool promote = planes == 3 || (!g.epi.out_bf && A.kblocks > 16);
  if (planes == 1 && big >= sms / 4 && g.J > 128)
    return promote ? launch_pair<AMN, BMN, true>(g, A, planes, sms / 2, st)
                   : launch_pair<AMN, BMN, false>(g, A, planes, sms / 2, st);
  // Few tiles, or few rows.  128 columns, 64 where there are no more rows or too few tiles to fill the SMs
  // with a split.  An SM takes in some 90 GB/s, so a weight streams at HBM's rate only into most of them:
  // splits as many as run at once (launch_split), with four steps a CTA at least; more than four ways only
  // of long sums (16 x 8192 -> 2048: 4 ways 14.1 us, 8 ways 12.3 us; of half that eight would gain less, 16 x
  // 4096 -> 2048 9.6 and 9.1 us).
  auto tiles_for = [&](int n) { return ((g.I + 127) / 128) * ((g.J + n - 1) / n); };
  const int bn = g.J <= 64 || tiles_for(128) * 8 <= sms ? 64 : 128;
  const int steps = A.kblocks * (planes == 3 ? 6 : 1);
  const int splits = std::max(1, std::min(std::min(steps >= 128 ? 8 : 4, steps / 4), A.kblocks));
  if (tiles_for(bn) * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (planes == 3)
    return bn == 64 ? launch_split<AMN, BMN, 64, 6>(g, A, planes, splits, st)
                    : launch_split<AMN, BMN, 128, 6>(g, A, planes, splits, st);
  if (promote)
    return bn == 64 ? launch_split<AMN, BMN, 64, 1>(g, A, planes, splits, st)
                    : launch_split<AMN, BMN, 128, 1>(g, A, planes, splits, st);
  return bn == 64 ? launch_split<AMN, BMN, 64, 0>(g, A, planes, splits, st)
                  : launch_split<AMN, BMN, 128, 0>(g, A, planes, splits, st);
}

}  // namespace

}  // namespace kda
