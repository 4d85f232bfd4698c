// linear_tc.cu -- the matrix product of gemm.cuh on tcgen05 tensor cores.
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
//   gemm_pair_kernel   large products.  A pair of CTAs (cta_group::2) works on a 256 x 256 tile: each
//                      stages its own 128 rows of A and of B, so a 64-wide step of c moves 32 KB
//                      into each SM for 512 tensor cycles, half of what two single CTAs with
//                      the same accumulators would move.  Persistent: the two 256-column
//                      accumulators alternate, one being multiplied into while eight warps
//                      store the other.  Bound by the tensor pipe and, over seconds, by power.
//   gemm_split_kernel  small products, mostly few rows (decode: the weight is the work).  One CTA
//                      holds a 128 x BN tile; a cluster of S CTAs splits the sum over c and adds
//                      its parts through distributed shared memory in rank order, so the
//                      result does not depend on timing and needs no workspace.  Bound by HBM
//                      for few rows: a deep TMA ring keeps the weight streaming.
//
// fp32 operands are split into three bf16 parts, x = hi + mid + lo with every part rounded to
// nearest, which hold all 24 bits; the six products of parts above 2^-27 relative are summed,
// smallest first (the sum then rounds like an fp32 sum).
//
// Every wait is bounded; one that gives up raises KDA_DEVERR_TIMEOUT, and the CTAs leave through
// the same barriers as otherwise.
#include <algorithm>

#include "gemm.cuh"
#include "tc_utils.cuh"
#include "tma_maps.cuh"

namespace kda {

namespace {

constexpr uint32_t kWaitLimit = 1u << 30;
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr int kBK = 64;                            // c per stage: one 128-byte swizzled row
constexpr uint32_t kOpBytes = 128 * kBK * 2;       // 128 rows of an operand

// ------------------------------------------------------------------ PTX beyond tc_utils.cuh

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the shared::cluster address of `saddr` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
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

struct TcArgs {
  GemmEpilogue epi;
  int64_t I, J;
  int32_t kblocks;          // 64-wide steps over c
  int32_t iters;            // kblocks times the products of parts
  int32_t tiles_i, tiles_j;
  int32_t* err;
};

// Step `it` of the sum: with three parts (0 = hi, 1 = mid, 2 = lo) the products of parts follow one
// another, smallest first; a is the part of A, b of B.
__device__ __forceinline__ void part_of(int iters, int kblocks, int it, int& kb, int& a, int& b) {
  if (iters == kblocks) {
    kb = it; a = b = 0;
    return;
  }
  const int q = it / kblocks;
  kb = it - q * kblocks;
  a = (0x201100 >> (4 * (5 - q))) & 15;          // (lo, hi) (hi, lo) (mid, mid) (mid, hi)
  b = (0x021010 >> (4 * (5 - q))) & 15;          // (hi, mid) (hi, hi)
}

// Waits for a phase; gives up after kWaitNs (far beyond any kernel's run) or once another role of
// the CTA has.
template <typename TryWait>
__device__ __forceinline__ bool wait_bounded(TryWait try_wait, volatile int* abort) {
  if (try_wait()) return true;
  const unsigned long long start = now_ns();
  for (uint32_t i = 1; i < kWaitLimit; ++i) {
    if (try_wait()) return true;
    if ((i & 63) == 0 && (*abort || now_ns() - start > kWaitNs)) return false;
  }
  return false;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return wait_bounded([&] { return tc::mbar_try_wait(bar, parity); }, abort);
}
// the same for a barrier that the other CTA of the pair arrives on
__device__ __forceinline__ bool wait_phase_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return wait_bounded([&] { return try_wait_cluster(bar, parity); }, abort);
}
// after a timeout: the copies or products in flight
__device__ __forceinline__ void drain_phase(uint64_t* bar, uint32_t parity) {
  int never = 0;
  wait_phase(bar, parity, &never);
}

// Descriptor of 128 (or BN) operand rows staged at `saddr`.  K-major: 8-row groups of 1024 bytes.
// MN-major: boxes of 64 rows of i (or j) by 64 steps of c, 8192 bytes apart; 8 steps of c are
// 1024 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  return MN ? (tc::smem_desc(saddr, 8192, 1024) | (static_cast<uint64_t>(2) << 61))
            : tc::smem_desc_sw128(saddr, 1024);
}
// bytes from one MMA's 16 steps of c to the next
template <bool MN>
__device__ __forceinline__ constexpr uint32_t k_advance() { return MN ? 2048 : 32; }

// `ROWS` rows of an operand from row r0 and step c0: one box K-major, ROWS / 64 boxes MN-major
template <bool MN, int ROWS, typename Load>
__device__ __forceinline__ void load_operand(uint32_t sdst, int64_t r0, int c0, Load load) {
  if constexpr (MN) {
#pragma unroll
    for (int b = 0; b < ROWS / 64; ++b) load(sdst + b * 8192, static_cast<int32_t>(r0) + 64 * b, c0);
  } else {
    load(sdst, c0, static_cast<int32_t>(r0));
  }
}

// 16 columns (rows j0 .. j0 + 15 of the output) of this thread's element i
__device__ __forceinline__ void store16(const GemmEpilogue& E, const uint32_t (&r)[16], float bias, int64_t i,
                                        bool in, int64_t j0, int64_t J) {
  if (!in || j0 >= J) return;
  const int n = static_cast<int>(J - j0 < 16 ? J - j0 : 16);
  float v[16], res[16];
  if (E.res) {
#pragma unroll
    for (int e = 0; e < 16; ++e) res[e] = e < n ? ld_any(E.res, E.res_bf, (j0 + e) * E.res_ld + i) : 0.f;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]) + bias;
  if (E.z) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < n) st_any(E.z, E.z_bf, (j0 + e) * E.z_ld + i, v[e]);
  }
  if (E.act != KDA_ACT_NONE) {
    if (E.out_bf) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = act_f<true>(E.act, v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = act_f<false>(E.act, v[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= E.scale;
  if (E.res) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] += res[e];
  }
  if (E.out_bf) {
    uint16_t* o = static_cast<uint16_t*>(E.out) + j0 * E.out_ld + i;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < n) o[e * E.out_ld] = f32_to_bf16_bits(v[e]);
  } else {
    float* o = static_cast<float*>(E.out) + j0 * E.out_ld + i;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < n) o[e * E.out_ld] = v[e];
  }
}

// ------------------------------------------------------------------ pairs of CTAs, 256 x 256 tiles

constexpr int kPairStages = 6;
constexpr int kPairThreads = 384;                  // TMA, MMA, TMEM, idle, 8 epilogue warps
constexpr uint32_t kPairStage = 2 * kOpBytes;
constexpr size_t kPairSmem = kPairStages * kPairStage + 1024;
constexpr int kRaster = 8;                         // i tiles taken together, for reuse in L2

// Tile t of the persistent order: groups of kRaster i tiles, j slowest inside a group, so that
// the tiles in flight at one time are about as many rows of A as of B.
__device__ __forceinline__ void tile_of(int t, int tiles_i, int tiles_j, int& ti, int& tj) {
  const int per = kRaster * tiles_j;
  const int grp = t / per, in = t - grp * per;
  const int width = min(kRaster, tiles_i - grp * kRaster);
  tj = in / width;
  ti = grp * kRaster + in - tj * width;
}

template <bool AMN, bool BMN>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const TcArgs A) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const uint32_t smem = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int tiles = A.tiles_i * A.tiles_j;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 16);            // 8 epilogue warps of both CTAs
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

  if (warp == 0) {
    if (lane == 0) {                               // both CTAs: stage this CTA's rows of A and B
      int it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        int ti, tj;
        tile_of(t, A.tiles_i, A.tiles_j, ti, tj);
        const int64_t i0 = static_cast<int64_t>(ti) * 256 + rank * 128;
        const int64_t j0 = static_cast<int64_t>(tj) * 256 + rank * 128;
        for (int k = 0; k < A.iters; ++k, ++it) {
          const int s = it % kPairStages;
          if (!wait_phase(&empty[s], ((it / kPairStages) & 1) ^ 1, &s_abort)) {
            ok = false;
            break;
          }
          int kb, pa, pb;
          part_of(A.iters, A.kblocks, k, kb, pa, pb);
          if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], 2 * kPairStage);
          const uint32_t bar = map_rank(tc::smem_u32(&full[s]), 0);
          const uint32_t sa = smem + s * kPairStage, sb = sa + kOpBytes;
          load_operand<AMN, 128>(sa, i0, kb * kBK, [&](uint32_t d, int32_t x, int32_t y) {
            tma_load_3d_pair(d, &map_a, x, y, pa, bar);
          });
          load_operand<BMN, 128>(sb, j0, kb * kBK, [&](uint32_t d, int32_t x, int32_t y) {
            tma_load_3d_pair(d, &map_b, x, y, pb, bar);
          });
        }
      }
      if (!ok) {
        s_abort = 1;
        raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
      }
      // after a timeout: the copies still in flight (their bytes count on the leader's barriers)
      if (!ok && rank == 0) {
        const int from = it > kPairStages ? it - kPairStages : 0;
        for (int j = from; j < it; ++j)
          drain_phase(&full[j % kPairStages], (j / kPairStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {                  // the leader multiplies for the pair
      const uint32_t idesc = tc::idesc_f16(256, 256, tc::kBF16, false, AMN, BMN);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++n) {
        const int b = n & 1;
        if (!wait_phase_cluster(&acc_empty[b], ((n >> 1) & 1) ^ 1, &s_abort)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t d = tmem + b * 256;
        for (int k = 0; k < A.iters; ++k, ++it) {
          const int s = it % kPairStages;
          if (!wait_phase(&full[s], (it / kPairStages) & 1, &s_abort)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t da = operand_desc<AMN>(smem + s * kPairStage);
          const uint64_t db = operand_desc<BMN>(smem + s * kPairStage + kOpBytes);
#pragma unroll
          for (int q = 0; q < kBK / 16; ++q)
            mma_pair(d, tc::desc_add(da, q * k_advance<AMN>()), tc::desc_add(db, q * k_advance<BMN>()), idesc,
                     (k | q) != 0);
          commit_pair(&empty[s]);
        }
        if (ok) commit_pair(&acc_full[b]);
      }
      if (!ok) {
        s_abort = 1;
        raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
        commit_pair(&drain);                       // the products still in flight
        drain_phase(&drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lead = map_rank(tc::smem_u32(&acc_empty[0]), 0);
    int n = 0;
    for (int t = first; t < tiles; t += step, ++n) {
      int ti, tj;
      tile_of(t, A.tiles_i, A.tiles_j, ti, tj);
      const int b = n & 1;
      const int64_t i = static_cast<int64_t>(ti) * 256 + rank * 128 + quad * 32 + lane;
      const int64_t j0 = static_cast<int64_t>(tj) * 256 + half * 128;
      const bool in = i < A.I;
      const float bias = A.epi.bias && in ? __ldg(A.epi.bias + i) : 0.f;
      const bool got = wait_phase(&acc_full[b], (n >> 1) & 1, &s_abort);
      if (__any_sync(0xffffffffu, !got)) {
        if (!got) raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
        s_abort = 1;
        break;
      }
      tc::fence_after_sync();
      const uint32_t src = tmem + b * 256 + half * 128 + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        if (j0 + c >= A.J) break;                  // the same for the whole warp
        uint32_t r[16];
        tc::tmem_ld16(src + c, r);
        tc::tmem_wait_ld();
        store16(A.epi, r, bias, i, in, j0 + c, A.J);
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

constexpr int kSplitThreads = 192;                 // TMA, MMA, 4 epilogue warps

template <int BN>
struct SplitShape {
  static constexpr uint32_t stage = kOpBytes + BN * kBK * 2;
  // the ring: as deep as 2 CTAs an SM allow for narrow tiles, 200 KB for the widest
  static constexpr int stages = BN <= 32 ? 5 : BN == 64 ? 4 : BN == 128 ? 6 : 4;
  static constexpr size_t smem = static_cast<size_t>(stage) * stages + 1024;
  static constexpr uint32_t cols = BN < 32 ? 32 : BN;
  static_assert(static_cast<size_t>(stage) * stages >= 128 * BN * 4, "the partial tile reuses the ring");
};

template <bool AMN, bool BMN, int BN>
__global__ void __launch_bounds__(kSplitThreads)
gemm_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const TcArgs A, const int splits) {
  using S = SplitShape<BN>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[S::stages], empty[S::stages], acc_full;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const uint32_t smem = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  float* part = reinterpret_cast<float*>(smem_raw + (smem - tc::smem_u32(smem_raw)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / splits;
  const int64_t i0 = static_cast<int64_t>(tile % A.tiles_i) * 128, j0 = static_cast<int64_t>(tile / A.tiles_i) * BN;
  const int k0 = static_cast<int>(static_cast<int64_t>(A.iters) * rank / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(A.iters) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(&acc_full, 1);
    tc::fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 1) {
    tc::tmem_alloc(&s_tmem, S::cols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % S::stages;
        if (!wait_phase(&empty[s], ((it / S::stages) & 1) ^ 1, &s_abort)) {
          ok = false;
          break;
        }
        int kb, pa, pb;
        part_of(A.iters, A.kblocks, k, kb, pa, pb);
        tc::mbar_arrive_expect_tx(&full[s], S::stage);
        const uint32_t sa = smem + s * S::stage, sb = sa + kOpBytes;
        load_operand<AMN, 128>(sa, i0, kb * kBK, [&](uint32_t d, int32_t x, int32_t y) {
          tc::tma_load_3d(d, &map_a, x, y, pa, &full[s]);
        });
        load_operand<BMN, BN>(sb, j0, kb * kBK, [&](uint32_t d, int32_t x, int32_t y) {
          tc::tma_load_3d(d, &map_b, x, y, pb, &full[s]);
        });
      }
      if (!ok) {                                   // wait for the copies in flight
        s_abort = 1;
        raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
        const int from = it > S::stages ? it - S::stages : 0;
        for (int j = from; j < it; ++j)
          drain_phase(&full[j % S::stages], (j / S::stages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = tc::idesc_f16(128, BN, tc::kBF16, false, AMN, BMN);
      int it = 0;
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % S::stages;
        if (!wait_phase(&full[s], (it / S::stages) & 1, &s_abort)) {
          s_abort = 1;
          raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
          break;
        }
        tc::fence_after_sync();
        const uint64_t da = operand_desc<AMN>(smem + s * S::stage);
        const uint64_t db = operand_desc<BMN>(smem + s * S::stage + kOpBytes);
#pragma unroll
        for (int q = 0; q < kBK / 16; ++q)
          tc::mma_ss(tmem, tc::desc_add(da, q * k_advance<AMN>()), tc::desc_add(db, q * k_advance<BMN>()), idesc,
                     (k > k0 || q > 0) ? 1u : 0u);
        tc::mma_commit(&empty[s]);
      }
      tc::mma_commit(&acc_full);                   // also after a timeout: the products in flight
    }
    __syncwarp();
  }
  const int quad = warp & 3;
  const int64_t i = i0 + quad * 32 + lane;
  const bool in = i < A.I;
  const float bias = warp >= 2 && A.epi.bias && in ? __ldg(A.epi.bias + i) : 0.f;
  const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  bool ready = true;
  if (warp >= 2) {
    ready = __all_sync(0xffffffffu, wait_phase(&acc_full, 0, &s_abort));
    if (!ready) raise_device_error(A.err, KDA_DEVERR_TIMEOUT);
    tc::fence_after_sync();
  }
  if (splits == 1) {
    if (warp >= 2 && ready) {
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        if (j0 + c >= A.J) break;
        uint32_t r[16];
        tc::tmem_ld16(src + c, r);
        tc::tmem_wait_ld();
        store16(A.epi, r, bias, i, in, j0 + c, A.J);
      }
    }
  } else {
    // every CTA publishes its part of the tile as [column][row]; rank r adds and stores the r-th
    // share of the columns, the parts in rank order
    const int ncol = static_cast<int>(A.J - j0 < BN ? A.J - j0 : BN);
    if (warp >= 2) {
#pragma unroll 1
      for (int c = 0; c < ncol; c += 16) {
        uint32_t r[16];
        tc::tmem_ld16(src + c, r);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * 128 + quad * 32 + lane] = __uint_as_float(r[e]);
      }
    }
    cluster_sync();
    if (warp >= 2) {
      const int per = (ncol + splits - 1) / splits;
      const int c1 = min(ncol, (rank + 1) * per);
      uint32_t base[8];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        base[p] = map_rank(smem + (quad * 32 + lane) * 4, static_cast<uint32_t>(p < splits ? p : 0));
      for (int c = rank * per; c < c1; c += 4) {
        float v[4][8];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int p = 0; p < 8; ++p)
            if (p < splits && c + e < c1) v[e][p] = ld_cluster(base[p] + (c + e) * 512);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + e >= c1 || !in) continue;
          float acc = v[e][0];
#pragma unroll
          for (int p = 1; p < 8; ++p)
            if (p < splits) acc += v[e][p];
          epilogue_store(A.epi, j0 + c + e, i, acc);
        }
      }
    }
    cluster_sync();                                // the peers are done reading this CTA's part
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, S::cols);
  }
}

// ------------------------------------------------------------------ aligned copies, fp32 parts

__device__ __forceinline__ void split3(float x, uint16_t (&p)[3]) {
  // rounded to nearest at each step; a finite x whose rounding would overflow is cut instead
  p[0] = f32_to_bf16_bits(x);
  if ((p[0] & 0x7fff) == 0x7f80) p[0] = static_cast<uint16_t>(__float_as_uint(x) >> 16);
  const float hi = bf16_bits_to_f32(p[0]);
  const float r = (p[0] & 0x7f80) == 0x7f80 ? 0.f : x - hi;     // infinities and NaN have no rest
  p[1] = f32_to_bf16_bits(r);
  p[2] = f32_to_bf16_bits(r - bf16_bits_to_f32(p[1]));
}

// rows of `cols` elements copied into rows of ld (a multiple of 8) elements: bf16 as they are,
// fp32 as three planes of parts
template <bool BF>
__global__ void __launch_bounds__(256) repack_kernel(const void* src, int64_t src_ld, int64_t rows, int64_t cols,
                                                     int64_t ld, uint16_t* dst) {
  const int64_t plane = rows * ld;
  const int64_t cb = (cols + 1023) / 1024;
  for (int64_t u = blockIdx.x; u < rows * cb; u += gridDim.x) {
    const int64_t r = u / cb;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = (u - r * cb) * 1024 + e * 256 + threadIdx.x;
      if (c >= cols) continue;
      if constexpr (BF) {
        dst[r * ld + c] = static_cast<const uint16_t*>(src)[r * src_ld + c];
      } else {
        uint16_t p[3];
        split3(static_cast<const float*>(src)[r * src_ld + c], p);
#pragma unroll
        for (int q = 0; q < 3; ++q) dst[q * plane + r * ld + c] = p[q];
      }
    }
  }
}

// ------------------------------------------------------------------ tensor maps, launches

// boxes of 64 columns (128 bytes, swizzled) x box_rows rows of one plane
bool encode_operand(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t planes,
                    uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc || rows == 0 || (reinterpret_cast<uintptr_t>(base) & 15u) || (ld & 7u)) return false;
  const cuuint64_t dims[3] = {cols, rows, planes};
  const cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode(CUtensorMap* m, const GemmOperand& X, int64_t R, int64_t C, int planes, int tile_rows) {
  // stored rows are r (K-major) or c (MN-major)
  return X.mn ? encode_operand(m, X.p, C, R, X.ld, planes, 64) : encode_operand(m, X.p, R, C, X.ld, planes, tile_rows);
}

template <bool AMN, bool BMN>
cudaError_t launch_pair(const Gemm& g, TcArgs A, int planes, int pairs, cudaStream_t st) {
  CUtensorMap ma, mb;
  if (!encode(&ma, g.A, g.I, g.C, planes, 128) || !encode(&mb, g.B, g.J, g.C, planes, 128)) return cudaErrorInvalidValue;
  A.tiles_i = static_cast<int32_t>((g.I + 255) / 256);
  A.tiles_j = static_cast<int32_t>((g.J + 255) / 256);
  auto k = gemm_pair_kernel<AMN, BMN>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPairSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(A.tiles_i) * A.tiles_j;
  if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(tiles, pairs));
  k<<<grid, kPairThreads, kPairSmem, st>>>(ma, mb, A);
  return cudaGetLastError();
}

template <bool AMN, bool BMN, int BN>
cudaError_t launch_split(const Gemm& g, TcArgs A, int planes, int splits, cudaStream_t st) {
  CUtensorMap ma, mb;
  if (!encode(&ma, g.A, g.I, g.C, planes, 128) || !encode(&mb, g.B, g.J, g.C, planes, BN)) return cudaErrorInvalidValue;
  A.tiles_i = static_cast<int32_t>((g.I + 127) / 128);
  A.tiles_j = static_cast<int32_t>((g.J + BN - 1) / BN);
  auto k = gemm_split_kernel<AMN, BMN, BN>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(SplitShape<BN>::smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(A.tiles_i) * A.tiles_j * splits));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = SplitShape<BN>::smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(splits);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, k, ma, mb, A, splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool AMN, bool BMN>
cudaError_t launch_shape(const Gemm& g, const TcArgs& A, int planes, cudaStream_t st) {
  const int sms = sm_count();
  const int64_t big = ((g.I + 255) / 256) * ((g.J + 255) / 256);
  if (big >= sms / 4) return launch_pair<AMN, BMN>(g, A, planes, sms / 2, st);
  // Few tiles: the narrowest tile that holds the rows (MN-major boxes are 64 wide), and enough
  // CTAs along c to fill the SMs, each with at least four steps.
  int bn = 16;
  while (bn < 256 && bn < g.J) bn *= 2;
  if (BMN) bn = std::max(bn, 64);
  auto tiles_for = [&](int n) { return ((g.I + 127) / 128) * ((g.J + n - 1) / n); };
  while (bn > 64 && tiles_for(bn) * 8 < sms) bn /= 2;
  const int64_t tiles = tiles_for(bn);
  int splits = static_cast<int>(std::min<int64_t>(8, std::max<int64_t>(1, sms / tiles)));
  splits = std::max(1, std::min(splits, A.iters / 4));
  if (tiles * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  switch (bn) {
    case 16: if constexpr (!BMN) return launch_split<AMN, BMN, 16>(g, A, planes, splits, st);
    case 32: if constexpr (!BMN) return launch_split<AMN, BMN, 32>(g, A, planes, splits, st);
    case 64: return launch_split<AMN, BMN, 64>(g, A, planes, splits, st);
    case 128: return launch_split<AMN, BMN, 128>(g, A, planes, splits, st);
    default: return launch_split<AMN, BMN, 256>(g, A, planes, splits, st);
  }
}

}  // namespace

size_t repacked_bytes(int64_t rows, int64_t cols, bool bf16) {
  return static_cast<size_t>(rows) * ((cols + 7) / 8 * 8) * 2 * (bf16 ? 1 : 3);
}

cudaError_t launch_repack(const void* src, int64_t src_ld, int64_t rows, int64_t cols, bool bf16, void* dst,
                          cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t ld = (cols + 7) / 8 * 8, units = rows * ((cols + 1023) / 1024);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, static_cast<int64_t>(sm_count()) * 16));
  if (bf16) repack_kernel<true><<<grid, 256, 0, st>>>(src, src_ld, rows, cols, ld, static_cast<uint16_t*>(dst));
  else repack_kernel<false><<<grid, 256, 0, st>>>(src, src_ld, rows, cols, ld, static_cast<uint16_t*>(dst));
  return cudaGetLastError();
}

// g.A and g.B: 16-byte aligned bf16 rows, `planes` (1 or 3) planes of them one after another
cudaError_t launch_gemm_tc(const Gemm& g, int planes, cudaStream_t st) {
  if (g.I == 0 || g.J == 0) return cudaSuccess;
  TcArgs A{};
  A.epi = g.epi;
  A.I = g.I; A.J = g.J;
  A.kblocks = static_cast<int32_t>((g.C + kBK - 1) / kBK);
  A.iters = A.kblocks * (planes == 3 ? 6 : 1);
  A.err = g.err;
  if (g.A.mn) return g.B.mn ? launch_shape<true, true>(g, A, planes, st) : launch_shape<true, false>(g, A, planes, st);
  return launch_shape<false, false>(g, A, planes, st);
}

}  // namespace kda
