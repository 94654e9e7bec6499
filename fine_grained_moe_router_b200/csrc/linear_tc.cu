// The linear layer's products on the 5th-generation tensor cores (sm_100a):
// C [M, N] = A B^T over a reduction of length K, bf16 operands, fp32 sums, with
// bias, activation and residual applied before C is rounded and stored.
// "MoE architecture in production" §3.1 (Linear, GeLU, Linear).
//
// Three products use it, with no copy of any operand:
//   y  = x W^T     A = x  [T, in]   B = W [out, in]   both along their rows
//   dx = dz W      A = dz [T, out]  B = W, reduced along its columns
//   dW = dz^T x    A = dz, B = x, both reduced along their columns
// An operand reduced along its rows is a K-major shared-memory tile (box of 64
// reduction elements by rows); one reduced along its columns is an M/N-major
// tile (box of 64 columns by 128 reduction rows). The MMA reads either.
//
// Tile: 128 rows of A by `bn` of B on one CTA, or 256 by `bn` on a CTA pair
// (cta_group::2: each CTA loads 128 rows of A and half of B). A ring stage holds
// 128 reduction elements of both operands. The units (CTAs or pairs) take whole
// tiles in turn. The tiles of a last round that would leave most units idle can
// be shared: each by `parts` units, which take equal shares of its reduction. The
// host picks bn and the sharing from the shape (linear_plan).
//
// Per CTA (persistent, 352 threads): warps 0-7 epilogue, warp 8 loads A, warp 9
// loads B, warp 10 allocates TMEM and issues the MMAs. Two 256-column
// accumulators let the epilogue of one tile overlap the next tile's MMAs. Every
// mbarrier wait is bounded (tc_ptx.cuh); on expiry the kernel records
// kStatusTimeout, drains and returns.
//
// A part of a tile is stored as fp32 partial sums: blocks of 32 columns by 32 rows,
// one bulk copy from shared memory each. The last part to arrive adds them up in
// reduction order (the result does not depend on who arrives when) and finishes
// the tile.
//
// Bound by the tensor cores at many tokens, by the stream of W at few. Measured
// on B200, in short bursts: 4096 x 4096 -> 14336 forward 311 us (1.55 PFLOP/s; 365 for
// seconds on end, at the power cap), input gradient 327, weight gradient 322; 512 x 4096
// -> 4096 18.6 us; 16 x 4096 -> 4096 11.6 us from L2 and 15.3 from memory (5.2 the floor).
#include <atomic>

#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace linear_tc {
namespace {

constexpr int kTM = 128;                      // rows of A per CTA
constexpr int kSub = 64;                      // elements of a 128-byte swizzled line
constexpr int kStageK = 128;                  // reduction elements per ring stage
constexpr int kMnBlock = kStageK * 128;       // one M/N-major box: 128 lines of 128 bytes
constexpr int kLinMaxStages = 12;
constexpr int kRing = 192 * 1024;
constexpr int kAcc = 256;                     // columns of one accumulator
constexpr int kLinEpiWarps = 8;
constexpr int kLoadA = kLinEpiWarps, kLoadB = kLinEpiWarps + 1, kIssue = kLinEpiWarps + 2;
constexpr int kLinThreads = (kLinEpiWarps + 3) * 32;
constexpr int kChunk32 = 32;                  // columns of C that a warp finishes at a time
constexpr int kStageOut = 32 * kChunk32 * 2;  // one chunk of 32 rows in bf16
constexpr int kOutArea = kLinEpiWarps * 2 * kStageOut;   // two buffers per epilogue warp
constexpr size_t kLinSmem = 2048 + kRing + kOutArea;

struct LinearArgs {
  LinearEpilogue epi;
  float* partials;        // [units, CTAs of a unit, bn / 32, 4, 32 columns, 32 rows]
  int* arrivals;          // one counter per shared tile and CTA of a unit, zero between launches
  uint32_t* status;
  int M, N, K;
  int bn, m_tiles, n_tiles;
  int k_stages;           // ring stages of a tile
  int whole;              // tiles taken as a whole, in turn; the others are shared
  int parts;              // units that share such a tile
  int units;
  int a_rows;             // rows of the A box (K-major A), a multiple of 8
  int a_bytes, stage_bytes, n_stages;
  int group_m;            // row tiles walked before the next column tile: 16 of them, 4096
                          // rows, stay in L2 while B streams past
};

// 128-byte swizzled M/N-major tile of boxes of 64 columns by kStageK lines:
// 8-line groups (1024 bytes) follow one another along the reduction, blocks of
// 64 columns are kMnBlock apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kMnBlock >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// wait_bounded by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t* status) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, status));
}

// A piece of a unit's work: stages [k0, k1) of a tile.
struct Piece {
  int tile, k0, k1;
};

// The pieces of one unit in order (its whole tiles, then at most one share of
// another); every role of a CTA walks its own copy.
struct Pieces {
  int unit, next;
  bool shared;

  __device__ __forceinline__ Pieces(const LinearArgs& a, int u) : unit(u), next(u) {
    shared = u < (a.m_tiles * a.n_tiles - a.whole) * a.parts;
  }
  __device__ __forceinline__ bool take(const LinearArgs& a, Piece& p) {
    if (next < a.whole) {
      p.tile = next;
      p.k0 = 0;
      p.k1 = a.k_stages;
      next += a.units;
      return true;
    }
    if (!shared) return false;
    shared = false;
    const int i = unit % a.parts;
    p.tile = a.whole + unit / a.parts;
    p.k0 = i * a.k_stages / a.parts;
    p.k1 = (i + 1) * a.k_stages / a.parts;
    return true;
  }
};

// Row and column tile: the row tiles of a group first, then column tiles.
__device__ __forceinline__ int2 tile_at(const LinearArgs& a, int t) {
  const int per_group = a.group_m * a.n_tiles;
  const int g = t / per_group, r = t % per_group;
  const int rows = min(a.group_m, a.m_tiles - g * a.group_m);
  return make_int2(g * a.group_m + r % rows, r / rows);
}

__device__ __forceinline__ void epi_sync() {
  asm volatile("bar.sync 1, %0;" ::"r"(kLinEpiWarps * 32) : "memory");
}

// A warp's two output buffers: 32 rows of 64 bytes, 16-byte pieces swizzled as a
// 64-byte-swizzle TMA box has them. Stores are asynchronous; a buffer is taken
// again once the store before the last has read it.
struct OutBuffers {
  uint8_t* base;
  int turn;

  __device__ __forceinline__ uint4* piece(int row, int i) const {
    return reinterpret_cast<uint4*>(base + turn * kStageOut + row * 64 +
                                    ((i ^ ((row >> 1) & 3)) << 4));
  }
  __device__ __forceinline__ void take() {
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void put(const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) *piece(lane, i) = RowVec<__nv_bfloat16>::pack(v + 8 * i);
  }
  // Stores the buffer at (column x, row y) of the map's matrix; what lies past
  // its edges is left out.
  __device__ __forceinline__ void send(const CUtensorMap* map, int x, int y) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      asm volatile(
          "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
              reinterpret_cast<uint64_t>(map)),
          "r"(x), "r"(y), "r"(smem_u32(base + turn * kStageOut))
          : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  __device__ __forceinline__ void finish() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
};

// The residual of one chunk, four lanes per row: on its way while the chunk
// before is finished, then turned to one row per lane in the output buffer.
__device__ __forceinline__ void load_residual(const LinearArgs& a, uint4 (&r)[4], int row0,
                                              int col0) {
  const int lane = threadIdx.x & 31, col = col0 + (lane & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + i * 8 + (lane >> 2);
    r[i] = row < a.M && col < a.N
               ? *reinterpret_cast<const uint4*>(
                     static_cast<const __nv_bfloat16*>(a.epi.residual) + (size_t)row * a.N + col)
               : make_uint4(0, 0, 0, 0);
  }
}

// Finishes the sums v (a row per lane) of the 32 rows from row0 on and the columns
// n0 + c0 on of a tile with `cols` columns. `residual`: this chunk's; on return
// that of the chunk at column n0 + after, if there is one.
template <int kAct>
__device__ __forceinline__ void finish_chunk(const LinearArgs& a, const CUtensorMap* tm_out,
                                             const CUtensorMap* tm_pre, OutBuffers& buf,
                                             float (&v)[32], int row0, int n0, int c0, int after,
                                             int cols, uint4 (&residual)[4]) {
  using V = RowVec<__nv_bfloat16>;
  const int lane = threadIdx.x & 31;
  if (a.epi.bias) {
    const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(a.epi.bias) + n0 + c0;
#pragma unroll
    for (int q = 0; q < 32; q += 8) {
      float f[8];
      V::unpack(c0 + q < cols ? __ldg(reinterpret_cast<const uint4*>(bias + q))
                              : make_uint4(0, 0, 0, 0),
                f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[q + i] += f[i];
    }
  }
  if (a.epi.pre) {
    buf.take();
    buf.put(v);
    buf.send(tm_pre, n0 + c0, row0);
  }
  linear_act<__nv_bfloat16, kAct>(v);
  buf.take();
  if (a.epi.residual) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *buf.piece(i * 8 + (lane >> 2), lane & 3) = residual[i];
    __syncwarp();
    if (after < cols) load_residual(a, residual, row0, n0 + after);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
      V::unpack(*buf.piece(lane, i), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * i + j] += f[j];
    }
  }
  buf.put(v);   // its own row: no other lane reads it
  buf.send(tm_out, n0 + c0, row0);
}

// A warp's 32 rows (from row0) and every other chunk of a tile's columns.
template <int kAct>
__device__ __forceinline__ void finish_columns(const LinearArgs& a, const CUtensorMap* tm_out,
                                               const CUtensorMap* tm_pre, OutBuffers& buf,
                                               uint32_t taddr, int half, int cols, int row0,
                                               int n0, uint4 (&residual)[4]) {
  for (int c0 = half * kChunk32; c0 < cols; c0 += 2 * kChunk32) {
    uint32_t u[32];
    __syncwarp();
    tmem_ld32(taddr + (uint32_t)c0, u);
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
    finish_chunk<kAct>(a, tm_out, tm_pre, buf, v, row0, n0, c0, c0 + 2 * kChunk32, cols, residual);
  }
}

__device__ __forceinline__ float* partial_at(const LinearArgs& a, int unit, int ctas, int rank) {
  return a.partials + (size_t)(unit * ctas + rank) * a.bn * kTM;
}

// Offset of (column, row) in a CTA's partial sums.
__device__ __forceinline__ int partial_offset(int col, int row) {
  return (col >> 5) * (32 * kTM) + (row >> 5) * 1024 + (col & 31) * 32 + (row & 31);
}

// Both output buffers of the warp hold one block.
__device__ __forceinline__ void store_partial(float* p, OutBuffers& buf, uint32_t taddr, int half,
                                              int cols, int quarter) {
  const int lane = threadIdx.x & 31;
  float* block = reinterpret_cast<float*>(buf.base);
  for (int c0 = half * 32; c0 < cols; c0 += 64) {
    uint32_t r[32];
    __syncwarp();
    tmem_ld32(taddr + (uint32_t)c0, r);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) block[i * 32 + lane] = __uint_as_float(r[i]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                       p + partial_offset(c0, quarter * 32)),
                   "r"(smem_u32(block)), "r"(4096)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  // written, not only read: the arrival that follows says so to the other CTAs
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
}

// The CTA's rows of a tile whose parts have all arrived: sums in the order of the
// reduction. The warps take the 32 x 32 blocks in turn; the loads of several parts
// are on their way together: each is a trip to L2.
constexpr int kPartsAtOnce = 2;

template <int kAct>
__device__ __forceinline__ void finish_shared(const LinearArgs& a, const CUtensorMap* tm_out,
                                              const CUtensorMap* tm_pre, OutBuffers& buf, int tile,
                                              int ctas, int rank, int cols, int m0, int n0) {
  const int quarters = (min(kTM, a.M - m0) + 31) / 32, lane = threadIdx.x & 31;
  const float* p = partial_at(a, (tile - a.whole) * a.parts, ctas, rank);
  const size_t step = (size_t)ctas * a.bn * kTM;
  const int blocks = quarters * ((cols + 31) / 32);
  for (int i = threadIdx.x >> 5; i < blocks; i += kLinEpiWarps) {
    const int q = i % quarters, c0 = i / quarters * kChunk32, row0 = m0 + q * 32;
    uint4 residual[4];
    if (a.epi.residual) load_residual(a, residual, row0, n0 + c0);
    const int o = partial_offset(c0, q * 32) + lane;
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __ldcg(p + o + j * 32);
    for (int u = 1; u < a.parts; u += kPartsAtOnce) {
      float w[kPartsAtOnce][32];
#pragma unroll
      for (int t = 0; t < kPartsAtOnce; ++t)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          w[t][j] = u + t < a.parts ? __ldcg(p + (u + t) * step + o + j * 32) : 0.f;
#pragma unroll
      for (int t = 0; t < kPartsAtOnce; ++t)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (u + t < a.parts) v[j] += w[t][j];
    }
    finish_chunk<kAct>(a, tm_out, tm_pre, buf, v, row0, n0, c0, cols, cols, residual);
  }
}

template <bool kPair, bool kAMn, bool kBMn>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_out,
                     const __grid_constant__ CUtensorMap tm_pre, const LinearArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base);
  uint64_t* full = bars;
  uint64_t* empty = bars + kLinMaxStages;
  uint64_t* tfull = bars + 2 * kLinMaxStages;
  uint64_t* tempty = bars + 2 * kLinMaxStages + 2;
  uint64_t* drain = bars + 2 * kLinMaxStages + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kLinMaxStages + 5);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile int* epi_flags = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [4]
  uint8_t* ring = base + 1024;
  const int n_stages = args.n_stages;
  const uint32_t rank = kPair ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  constexpr int kTileM = kPair ? 2 * kTM : kTM;
  const int nb = kPair ? args.bn / 2 : args.bn;   // rows (columns) of B this CTA loads

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), (kPair ? 2 : 1) * kLinEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kIssue) {
    if (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(2 * kAcc));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(2 * kAcc));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  // The loading and issuing warps run their loops as whole warps, and one lane
  // issues: addresses and descriptors are then the same in every lane, and the
  // compiler keeps them in uniform registers, where TMA and MMA take them from.
  if (warp == kLoadA || warp == kLoadB) {
    // -------------------------------------------------------- producers
    const bool is_a = warp == kLoadA;
    const uint32_t one = elect_one();
    // bytes of one stage over both operands (and both CTAs of a pair)
    const uint32_t bytes =
        (kPair ? 2u : 1u) *
        (uint32_t)((kAMn ? 2 * kMnBlock : 2 * args.a_rows * 128) +
                   (kBMn ? (nb + kSub - 1) / kSub * kMnBlock : 2 * nb * 128));
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0, issued_parity = 0;   // bit s: stage s
    bool ok = true;
    Pieces pieces(args, unit);
    for (Piece p; ok && pieces.take(args, p);) {
      const int2 at = tile_at(args, p.tile);
      const int m0 = at.x * kTileM + (int)rank * kTM;
      const int n0 = at.y * args.bn + (int)rank * nb;
      for (int k = p.k0 * kStageK; k < p.k1 * kStageK; k += kStageK) {
        if (!wait_warp(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        const uint32_t sa = smem_u32(ring) + (uint32_t)(stage * args.stage_bytes);
        const uint32_t sb = sa + args.a_bytes;
        const uint32_t fb0 = kPair ? map_to_rank(fb, 0) : fb;
        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
          tma_load_2d_one<kPair>(dst, map, x, y, fb0, one);
        };
        if (is_a) {
          if (leader) mbar_expect_tx_one(fb, bytes, one);
          if (kAMn) {
            load(sa, &tm_a, m0, k);
            load(sa + kMnBlock, &tm_a, m0 + kSub, k);
          } else {
            load(sa, &tm_a, k, m0);
            load(sa + args.a_rows * 128, &tm_a, k + kSub, m0);
          }
        } else if (kBMn) {
          for (int c = 0; c < nb; c += kSub)
            load(sb + c / kSub * kMnBlock, &tm_b, n0 + c, k);
        } else {
          load(sb, &tm_b, k, n0);
          load(sb + nb * 128, &tm_b, k + kSub, n0);
        }
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy has landed before the CTAs tear down (the leader's barriers
    // count the copies of both operands and both CTAs)
    if (leader)
      for (int s = 0; s < n_stages; ++s)
        if ((issued >> s) & 1u)
          wait_warp(smem_u32(&full[s]), (issued_parity >> s) & 1u, nullptr, args.status);
  } else if (warp == kIssue) {
    // ------------------------------------------------------- MMA issuer
    const uint32_t one = elect_one();
    if (leader) {
      const uint32_t idesc = idesc_bf16(args.bn, kTileM) | (kAMn ? 1u << 15 : 0u) |
                             (kBMn ? 1u << 16 : 0u);
      // descriptor steps (16-byte units) to the second half of a K-major stage
      const uint32_t a_sub = kAMn ? 0u : (uint32_t)(args.a_rows * 128 / 16);
      const uint32_t b_sub = kBMn ? 0u : (uint32_t)(nb * 128 / 16);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      Pieces pieces(args, unit);
      for (Piece p; ok && pieces.take(args, p);) {
        if (!wait_warp(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, args.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kAcc);
        const int k0 = p.k0 * kStageK;
        const int k_end = min(args.K, p.k1 * kStageK);
        for (int k = k0; k < k_end; k += kStageK) {
          if (!wait_warp(smem_u32(&full[stage]), phase, abort_flag, args.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring) + (uint32_t)(stage * args.stage_bytes);
          const uint32_t sb = sa + args.a_bytes;
          const uint64_t ad = kAMn ? mn_desc(sa) : sw128_desc(sa);
          const uint64_t bd = kBMn ? mn_desc(sb) : sw128_desc(sb);
          const int steps = min(kStageK / 16, (k_end - k + 15) / 16);
          auto issue = [&](int s) {
            const uint64_t da = ad + (kAMn ? (uint32_t)(s * 128)
                                           : (uint32_t)(s % 4 * 2) + (s >= 4 ? a_sub : 0u));
            const uint64_t db = bd + (kBMn ? (uint32_t)(s * 128)
                                           : (uint32_t)(s % 4 * 2) + (s >= 4 ? b_sub : 0u));
            const uint32_t accum = (k != k0 || s != 0) ? 1u : 0u;
            mma_bf16_one<kPair>(d_tmem, da, db, idesc, accum, one);
          };
          if (steps == kStageK / 16) {
#pragma unroll
            for (int s = 0; s < kStageK / 16; ++s) issue(s);
          } else {
            for (int s = 0; s < steps; ++s) issue(s);
          }
          mma_commit_one<kPair>(smem_u32(&empty[stage]), one);
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_one<kPair>(smem_u32(&tfull[acc]), one);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // retire every MMA issued before TMEM is released (in both CTAs)
      mma_commit_one<kPair>(smem_u32(drain), one);
      wait_warp(smem_u32(drain), 0, nullptr, args.status);
    } else if (kPair) {
      wait_warp(smem_u32(drain), 0, nullptr, args.status);
    }
  } else {
    // --------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes 32 (w % 4) .. +31 (thread = row of C) and every
    // other chunk of 32 columns. With shared tiles the warps go in lockstep (one
    // thread waits, the others follow through a named barrier), since their
    // ends hold barriers that all of them have to reach.
    constexpr int kCtas = kPair ? 2 : 1;
    int acc = 0;
    uint32_t acc_phase = 0;
    const int quarter = warp & 3, half = warp >> 2;
    const bool lockstep = args.whole < args.m_tiles * args.n_tiles;
    int it = 0;
    OutBuffers out{ring + kRing + warp * 2 * kStageOut, 0};
    Pieces pieces(args, unit);
    for (Piece p; pieces.take(args, p); ++it) {
      const int2 at = tile_at(args, p.tile);
      const bool partial = p.k1 - p.k0 < args.k_stages;
      const int n0 = at.y * args.bn;
      const int cols = min(args.bn, args.N - n0);
      const int in_tile = quarter * 32 + lane;
      const int row = at.x * kTileM + (int)rank * kTM + in_tile;
      uint4 residual[4];   // of the first chunk, ahead of the accumulator
      if (args.epi.residual && !partial) load_residual(args, residual, row - lane, n0 + half * 32);
      int ok = 1;
      if (lockstep) {
        if (threadIdx.x == 0)
          epi_flags[it & 1] =
              wait_bounded(smem_u32(&tfull[acc]), acc_phase, abort_flag, args.status) ? 1 : 0;
        epi_sync();
        ok = epi_flags[it & 1];
      } else {
        if (lane == 0)
          ok = wait_bounded(smem_u32(&tfull[acc]), acc_phase, abort_flag, args.status) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kAcc);
      if (row - lane < args.M) {
        if (partial)
          store_partial(partial_at(args, unit, kCtas, (int)rank), out, taddr, half, cols,
                        quarter);
        else if (args.epi.act == MOE_ACT_GELU)
          finish_columns<MOE_ACT_GELU>(args, &tm_out, &tm_pre, out, taddr, half, cols, row - lane,
                                       n0, residual);
        else if (args.epi.act == MOE_ACT_SILU)
          finish_columns<MOE_ACT_SILU>(args, &tm_out, &tm_pre, out, taddr, half, cols, row - lane,
                                       n0, residual);
        else
          finish_columns<MOE_ACT_NONE>(args, &tm_out, &tm_pre, out, taddr, half, cols, row - lane,
                                       n0, residual);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t te = smem_u32(&tempty[acc]);
        if (kPair)
          mbar_arrive_cluster(map_to_rank(te, 0));
        else
          mbar_arrive(te);
      }
      if (partial) {
        asm volatile("fence.proxy.async;" ::: "memory");
        __threadfence();   // this warp's partial sums are visible to the other CTAs
        epi_sync();
        volatile int* owner = epi_flags + 2 + (it & 1);
        if (threadIdx.x == 0) {
          int* count = args.arrivals + (p.tile - args.whole) * kCtas + (int)rank;
          const bool last = atomicAdd(count, 1) == args.parts - 1;
          // every part has arrived: the counter is zero again for the next launch
          if (last) *count = 0;
          *owner = last ? 1 : 0;
        }
        epi_sync();
        if (*owner) {
          __threadfence();
          const int m0 = at.x * kTileM + (int)rank * kTM;
          if (m0 < args.M) {
            if (args.epi.act == MOE_ACT_GELU)
              finish_shared<MOE_ACT_GELU>(args, &tm_out, &tm_pre, out, p.tile, kCtas, (int)rank, cols,
                                          m0, n0);
            else if (args.epi.act == MOE_ACT_SILU)
              finish_shared<MOE_ACT_SILU>(args, &tm_out, &tm_pre, out, p.tile, kCtas, (int)rank, cols,
                                          m0, n0);
            else
              finish_shared<MOE_ACT_NONE>(args, &tm_out, &tm_pre, out, p.tile, kCtas, (int)rank, cols,
                                          m0, n0);
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    out.finish();
  }

  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // no CTA of the pair leaves while the other may signal it
  if (warp == kIssue) {
    tc_fence_after();
    if (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                   "r"(2 * kAcc));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                   "r"(2 * kAcc));
  }
}

// Row-major [rows, cols] bf16 matrix, boxes of box_cols columns (64: 128-byte
// swizzle, 32: 64-byte) by box_rows rows, zeros outside the matrix.
bool linear_map(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint32_t box_rows,
                uint32_t box_cols = kSub) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_cols == (uint32_t)kSub ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace linear_tc

// Tile width, sharing and ring of one product, from its shape alone (so that the
// workspace size depends on the shape alone, too): the choice of least estimated
// cycles. The constants were measured on B200:
//   - a CTA pair's stage takes the MMAs' bn / 2 cycles per 16 elements, or the
//     time of its operands at 53 bytes per cycle and SM from L2, whichever is
//     more (wide tiles read less per MMA);
//   - one CTA (M <= 128) streams B at 23 bytes per cycle (its share of the
//     memory rate) next to A from L2, and issues a stage in 700 cycles at least;
//   - sharing a tile costs its parts' stores and the last one's loads and
//     stores, at 28 bytes per cycle, and 2000 cycles of waiting. (16 tokens,
//     4096 x 4096: 18.1 us whole, 11.6 in four parts per tile; 4096 tokens, 14336
//     -> 4096: 335 us whole, 323 with the last round in two parts. Dealing the
//     reduction of all tiles out evenly, so that every unit gets the same and
//     works at a place of its own in it, was slower than an idle round: units
//     that walk the reduction together ask L2 for the same lines at the same
//     time.)
// An M/N-major B is read in lines of 64 columns: its tiles start at multiples of
// 64 per CTA, so that no line of a box straddles two of memory. Others go by 32,
// the step of a pair's MMA and the epilogue's chunk.
LinearPlan linear_plan(int M, int N, int K, bool a_mn, bool b_mn, int sms) {
  using namespace linear_tc;
  LinearPlan best{};
  const bool pair = M > kTM;
  const int all = pair ? sms / 2 : sms;
  const int m_tiles = (M + (pair ? 2 * kTM : kTM) - 1) / (pair ? 2 * kTM : kTM);
  const int a_rows = pair ? kTM : std::min(kTM, (M + 7) / 8 * 8);
  const int step = b_mn ? (pair ? 128 : 64) : 32;
  const int k_stages = (K + kStageK - 1) / kStageK;
  double best_cost = -1;
  auto consider = [&](int bn, long long tiles, long long whole, int parts, double cost) {
    if (best_cost >= 0 && cost >= best_cost) return;
    best_cost = cost;
    best.bn = bn;
    best.n_tiles = (N + bn - 1) / bn;
    best.whole = (int)whole;
    best.parts = parts;
    best.units = (int)(whole > 0 ? std::min<long long>(tiles, all) : tiles * parts);
  };
  const int narrowest = std::min(std::max(step, pair ? 64 : 32), (N + step - 1) / step * step);
  for (int bn = narrowest; bn <= (pair ? 256 : 128); bn += step) {
    const long long tiles = (long long)m_tiles * ((N + bn - 1) / bn);
    const double stage = pair ? std::max(8 * bn / 2.0, (kTM + bn / 2.0) * kStageK * 2 / 53)
                              : std::max(11.0 * bn + 5.0 * a_rows + 200, 700.0);
    const double turn = 3000;   // a tile's start and end
    const double part_bytes = 4.0 * bn * (pair ? kTM : (a_rows + 31) / 32 * 32);
    const long long rounds = tiles / all, left = tiles % all;
    consider(bn, tiles, tiles, 1, (rounds + (left > 0)) * (k_stages * stage + turn));
    for (int j = 2; left > 0 && j <= k_stages && j * left <= all; ++j)
      consider(bn, tiles, rounds * all, j,
               rounds * (k_stages * stage + turn) + (k_stages + j - 1) / j * stage + turn + 2000 +
                   part_bytes * (1 + j) / 28);
  }
  best.pair = pair;
  best.m_tiles = m_tiles;
  best.a_rows = a_rows;
  best.k_stages = k_stages;
  const int nb = pair ? best.bn / 2 : best.bn;
  best.a_bytes = a_mn ? 2 * kMnBlock : 2 * a_rows * 128;
  const int b_bytes = b_mn ? (nb + kSub - 1) / kSub * kMnBlock : 2 * nb * 128;
  best.stage_bytes = best.a_bytes + b_bytes;
  // The MMA reads 128 rows of A whatever the box holds (the rows past it feed
  // outputs that are not stored): those of the last stage stay inside the ring.
  const int past = a_mn ? 0 : std::max(0, a_rows * 128 + kTM * 128 - best.stage_bytes);
  best.n_stages = std::min(kLinMaxStages, (kRing - past) / best.stage_bytes);
  best.partial_bytes = sizeof(float) * (m_tiles * best.n_tiles - best.whole) * best.parts *
                       (pair ? 2 : 1) * best.bn * kTM;
  return best;
}

cudaError_t launch_linear_tc(const LinearPlan& p, int M, int N, int K, const void* A, bool a_mn,
                             const void* B, bool b_mn, const LinearEpilogue& epi,
                             float* partials, int* arrivals, uint32_t* status,
                             cudaStream_t st) {
  using namespace linear_tc;
  LinearArgs a{};
  a.epi = epi;
  a.partials = partials;
  a.arrivals = arrivals;
  a.status = status;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bn = p.bn;
  a.m_tiles = p.m_tiles;
  a.n_tiles = p.n_tiles;
  a.k_stages = p.k_stages;
  a.whole = p.whole;
  a.parts = p.parts;
  a.units = p.units;
  a.a_rows = p.a_rows;
  a.a_bytes = p.a_bytes;
  a.stage_bytes = p.stage_bytes;
  a.n_stages = p.n_stages;
  a.group_m = 16;
  const int nb = p.pair ? p.bn / 2 : p.bn;
  CUtensorMap ma, mb, mo, mp;
  if (!(a_mn ? linear_map(&ma, A, K, M, kStageK) : linear_map(&ma, A, M, K, p.a_rows)) ||
      !(b_mn ? linear_map(&mb, B, K, N, kStageK) : linear_map(&mb, B, N, K, nb)) ||
      !linear_map(&mo, epi.out, M, N, 32, kChunk32) ||
      !linear_map(&mp, epi.pre ? epi.pre : epi.out, M, N, 32, kChunk32))
    return cudaErrorInvalidValue;
  auto go = [&](auto kernel, std::atomic<bool>* set) -> cudaError_t {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kLinSmem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_release);
    }
    if (p.pair)
      return launch_pdl_cluster2(kernel, dim3(2 * p.units), dim3(kLinThreads),
                                 kLinSmem, st, ma, mb, mo, mp, a);
    return launch_pdl(kernel, dim3(p.units), dim3(kLinThreads), kLinSmem, st, ma, mb, mo, mp, a);
  };
#define MOE_LINEAR_CASE(P, AM, BM)                           \
  if (p.pair == P && a_mn == AM && b_mn == BM) {             \
    static std::atomic<bool> set[64];                        \
    return go(linear_tc_kernel<P, AM, BM>, set);             \
  }
  MOE_LINEAR_CASE(false, false, false)
  MOE_LINEAR_CASE(true, false, false)
  MOE_LINEAR_CASE(false, false, true)
  MOE_LINEAR_CASE(true, false, true)
  MOE_LINEAR_CASE(false, true, true)
  MOE_LINEAR_CASE(true, true, true)
#undef MOE_LINEAR_CASE
  return cudaErrorInvalidValue;
}

}  // namespace moe
