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
// (cta_group::2: each CTA loads 128 rows of A and half of B). The host picks
// bn and the number of reduction splits from the shape (linear_plan). A ring
// stage holds 128 reduction elements of both operands.
//
// Per CTA (persistent, 352 threads): warps 0-7 epilogue, warp 8 loads A, warp 9
// loads B, warp 10 allocates TMEM and issues the MMAs. Two 256-column
// accumulators let the epilogue of one tile overlap the next tile's MMAs. Every
// mbarrier wait is bounded (tc_ptx.cuh); on expiry the kernel records
// kStatusTimeout, drains and returns.
//
// A split tile stores fp32 partial sums; the last of its splits to arrive adds
// them in split order (the result does not depend on who arrives when) and
// finishes the tile.
#include <atomic>

#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace tc {
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
constexpr size_t kLinSmem = 2048 + kRing;

struct LinearArgs {
  LinearEpilogue epi;
  float* partials;        // [splits, M, N] when splits > 1
  int* arrivals;          // one counter per tile and CTA of a pair, zero between launches
  uint32_t* status;
  int M, N, K;
  int bn, m_tiles, n_tiles, splits, k_per;   // k_per: reduction elements per split
  int a_rows;             // rows of the A box (K-major A), a multiple of 8
  int a_bytes, stage_bytes, n_stages;
  int group_m;            // row tiles walked before the next column tile
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

struct Work {
  int m, n, split;
};
// Work item i: split fastest, then the row tiles of a group, then column tiles.
__device__ __forceinline__ Work work_at(const LinearArgs& a, int i) {
  Work w;
  w.split = i % a.splits;
  i /= a.splits;
  const int per_group = a.group_m * a.n_tiles;
  const int g = i / per_group, r = i % per_group;
  const int rows = min(a.group_m, a.m_tiles - g * a.group_m);
  w.m = g * a.group_m + r % rows;
  w.n = r / rows;
  return w;
}

__device__ __forceinline__ void epi_sync() {
  asm volatile("bar.sync 1, %0;" ::"r"(kLinEpiWarps * 32) : "memory");
}

template <int kAct>
__device__ __forceinline__ void finish_columns(const LinearArgs& a, uint32_t taddr, int half,
                                               int cols, int row, int n0) {
  for (int c0 = half * 32; c0 < cols; c0 += 64) {
    uint32_t r[32];
    __syncwarp();
    tmem_ld32(taddr + (uint32_t)c0, r);
    if (row >= a.M) continue;
#pragma unroll
    for (int q = 0; q < 32; q += 8) {
      if (c0 + q < cols) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[q + i]);
        const int col = n0 + c0 + q;
        linear_finish<__nv_bfloat16, kAct>(a.epi, (size_t)row * a.N + col, col, v);
      }
    }
  }
}

__device__ __forceinline__ void store_partial(const LinearArgs& a, uint32_t taddr, int half,
                                              int cols, int row, int n0, int split) {
  for (int c0 = half * 32; c0 < cols; c0 += 64) {
    uint32_t r[32];
    __syncwarp();
    tmem_ld32(taddr + (uint32_t)c0, r);
    if (row >= a.M) continue;
    float* p = a.partials + ((size_t)split * a.M + row) * a.N + n0 + c0;
#pragma unroll
    for (int q = 0; q < 32; q += 4)
      if (c0 + q < cols)
        *reinterpret_cast<uint4*>(p + q) = make_uint4(r[q], r[q + 1], r[q + 2], r[q + 3]);
  }
}

// The CTA's rows of a tile whose splits have all arrived: sums in split order.
template <int kAct>
__device__ __forceinline__ void finish_split(const LinearArgs& a, int m0, int rows, int n0,
                                             int cols) {
  const int groups = cols / 8;
  for (int i = threadIdx.x; i < rows * groups; i += kLinEpiWarps * 32) {
    const int row = m0 + i / groups, col = n0 + i % groups * 8;
    const float* p = a.partials + (size_t)row * a.N + col;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(p + (size_t)s * a.M * a.N));
      const float4 w = __ldcg(reinterpret_cast<const float4*>(p + (size_t)s * a.M * a.N) + 1);
      v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
      v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
    }
    linear_finish<__nv_bfloat16, kAct>(a.epi, (size_t)row * a.N + col, col, v);
  }
}

template <bool kPair, bool kAMn, bool kBMn>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b, const LinearArgs args) {
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
  const int n_units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  constexpr int kTileM = kPair ? 2 * kTM : kTM;
  const int nb = kPair ? args.bn / 2 : args.bn;   // rows (columns) of B this CTA loads
  const int n_work = args.m_tiles * args.n_tiles * args.splits;

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

  if (warp == kLoadA || warp == kLoadB) {
    // -------------------------------------------------------- producers
    if (lane == 0) {
      const bool is_a = warp == kLoadA;
      // bytes of one stage over both operands (and both CTAs of a pair)
      const uint32_t bytes =
          (kPair ? 2u : 1u) *
          (uint32_t)((kAMn ? 2 * kMnBlock : 2 * args.a_rows * 128) +
                     (kBMn ? (nb + kSub - 1) / kSub * kMnBlock : 2 * nb * 128));
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;   // bit s: stage s
      bool ok = true;
      for (int i = unit; ok && i < n_work; i += n_units) {
        const Work w = work_at(args, i);
        const int m0 = w.m * kTileM + (int)rank * kTM;
        const int n0 = w.n * args.bn + (int)rank * nb;
        const int k_end = min(args.K, (w.split + 1) * args.k_per);
        for (int k = w.split * args.k_per; k < k_end; k += kStageK) {
          if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.status)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t sa = smem_u32(ring + (size_t)stage * args.stage_bytes);
          const uint32_t fb0 = kPair ? map_to_rank(fb, 0) : fb;
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
            if (kPair)
              tma_load_2d_pair(dst, map, x, y, fb0);
            else
              tma_load_2d(dst, map, x, y, fb);
          };
          if (is_a) {
            if (leader) mbar_expect_tx(fb, bytes);
            if (kAMn) {
              load(sa, &tm_a, m0, k);
              load(sa + kMnBlock, &tm_a, m0 + kSub, k);
            } else {
              load(sa, &tm_a, k, m0);
              load(sa + args.a_rows * 128, &tm_a, k + kSub, m0);
            }
          } else {
            const uint32_t sb = sa + args.a_bytes;
            if (kBMn) {
              for (int c = 0; c < nb; c += kSub)
                load(sb + c / kSub * kMnBlock, &tm_b, n0 + c, k);
            } else {
              load(sb, &tm_b, k, n0);
              load(sb + nb * 128, &tm_b, k + kSub, n0);
            }
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
            wait_bounded(smem_u32(&full[s]), (issued_parity >> s) & 1u, nullptr, args.status);
    }
  } else if (warp == kIssue) {
    // ------------------------------------------------------- MMA issuer
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_bf16(args.bn, kTileM) | (kAMn ? 1u << 15 : 0u) |
                             (kBMn ? 1u << 16 : 0u);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = unit; ok && i < n_work; i += n_units) {
        const Work w = work_at(args, i);
        if (!wait_bounded(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, args.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kAcc);
        const int k0 = w.split * args.k_per;
        const int k_end = min(args.K, k0 + args.k_per);
        for (int k = k0; k < k_end; k += kStageK) {
          if (!wait_bounded(smem_u32(&full[stage]), phase, abort_flag, args.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + (size_t)stage * args.stage_bytes);
          const uint32_t sb = sa + args.a_bytes;
          const uint64_t ad = kAMn ? mn_desc(sa) : sw128_desc(sa);
          const uint64_t bd = kBMn ? mn_desc(sb) : sw128_desc(sb);
          // descriptor steps (16-byte units) to the second half of a K-major stage
          const uint64_t a_sub = (uint64_t)(args.a_rows * 128 / 16);
          const uint64_t b_sub = (uint64_t)(nb * 128 / 16);
          const int steps = min(kStageK / 16, (k_end - k + 15) / 16);
#pragma unroll
          for (int s = 0; s < kStageK / 16; ++s) {
            if (s >= steps) break;
            const uint64_t da = ad + (kAMn ? (uint64_t)(s * 16 * 128 / 16)
                                           : (uint64_t)(s % 4 * 2) + (s >= 4 ? a_sub : 0));
            const uint64_t db = bd + (kBMn ? (uint64_t)(s * 16 * 128 / 16)
                                           : (uint64_t)(s % 4 * 2) + (s >= 4 ? b_sub : 0));
            const uint32_t accum = (k != k0 || s != 0) ? 1u : 0u;
            if (kPair)
              mma_bf16_pair(d_tmem, da, db, idesc, accum);
            else
              mma_bf16(d_tmem, da, db, idesc, accum);
          }
          if (kPair)
            mma_commit_pair(smem_u32(&empty[stage]));
          else
            mma_commit(smem_u32(&empty[stage]));
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (kPair)
          mma_commit_pair(smem_u32(&tfull[acc]));
        else
          mma_commit(smem_u32(&tfull[acc]));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // retire every MMA issued before TMEM is released (in both CTAs)
      if (kPair)
        mma_commit_pair(smem_u32(drain));
      else
        mma_commit(smem_u32(drain));
      wait_bounded(smem_u32(drain), 0, nullptr, args.status);
    } else if (kPair && lane == 0) {
      wait_bounded(smem_u32(drain), 0, nullptr, args.status);
    }
  } else {
    // --------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes 32 (w % 4) .. +31 (thread = row of C) and every
    // other chunk of 32 columns. With splits the warps go in lockstep (one
    // thread waits, the others follow through a named barrier), since the
    // fixup holds barriers that all of them have to reach.
    int acc = 0;
    uint32_t acc_phase = 0;
    const int quarter = warp & 3, half = warp >> 2;
    int it = 0;
    for (int i = unit; i < n_work; i += n_units, ++it) {
      const Work w = work_at(args, i);
      int ok = 1;
      if (args.splits > 1) {
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
      const int m0 = w.m * kTileM + (int)rank * kTM;
      const int n0 = w.n * args.bn;
      const int cols = min(args.bn, args.N - n0);
      const int row = m0 + quarter * 32 + lane;
      if (m0 + quarter * 32 < args.M) {
        if (args.splits > 1)
          store_partial(args, taddr, half, cols, row, n0, w.split);
        else if (args.epi.act == MOE_ACT_GELU)
          finish_columns<MOE_ACT_GELU>(args, taddr, half, cols, row, n0);
        else if (args.epi.act == MOE_ACT_SILU)
          finish_columns<MOE_ACT_SILU>(args, taddr, half, cols, row, n0);
        else
          finish_columns<MOE_ACT_NONE>(args, taddr, half, cols, row, n0);
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
      if (args.splits > 1) {
        __threadfence();   // this thread's partial sums are visible to the other CTAs
        epi_sync();
        volatile int* owner = epi_flags + 2 + (it & 1);
        if (threadIdx.x == 0) {
          int* count = args.arrivals + (w.n * args.m_tiles + w.m) * 2 + (int)rank;
          const bool last = atomicAdd(count, 1) == args.splits - 1;
          // every split has arrived: the counter is zero again for the next launch
          if (last) *count = 0;
          *owner = last ? 1 : 0;
        }
        epi_sync();
        if (*owner) {
          __threadfence();
          const int rows = min(kTM, args.M - m0);
          if (rows > 0) {
            if (args.epi.act == MOE_ACT_GELU)
              finish_split<MOE_ACT_GELU>(args, m0, rows, n0, cols);
            else if (args.epi.act == MOE_ACT_SILU)
              finish_split<MOE_ACT_SILU>(args, m0, rows, n0, cols);
            else
              finish_split<MOE_ACT_NONE>(args, m0, rows, n0, cols);
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
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

// Row-major [rows, cols] bf16 matrix, boxes of 64 columns by box_rows rows,
// 128-byte swizzle, zeros outside the matrix.
bool linear_map(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {(cuuint32_t)kSub, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace tc

// Tile width, reduction splits and ring of one product. Depends on the shape
// alone, so the workspace size does too.
//   M <= 128: one CTA per tile. The weights stream past a few rows, so every SM
//     should carry an equal share of B: the cost of a choice is its rounds of
//     CTAs times the bytes of a tile, plus a fixed charge for adding splits up.
//   M > 128: CTA pairs; the cost is rounds of pairs times tile width (MMA time
//     goes with the width), plus a fixed width for the tile's turnaround.
LinearPlan linear_plan(int M, int N, int K, bool a_mn, bool b_mn, int sms) {
  using namespace tc;
  LinearPlan best{};
  best.pair = M > kTM;
  const int units = best.pair ? sms / 2 : sms;
  const int tile_m = best.pair ? 2 * kTM : kTM;
  best.m_tiles = (M + tile_m - 1) / tile_m;
  best.a_rows = best.pair ? kTM : std::min(kTM, (M + 7) / 8 * 8);
  const int step = b_mn && !best.pair ? 64 : 16;
  const int widest = best.pair ? 256 : 128;
  const int k_stages = (K + kStageK - 1) / kStageK;
  double best_cost = 0;
  for (int bn = best.pair ? 64 : std::max(32, step); bn <= widest; bn += step) {
    const int n_tiles = (N + bn - 1) / bn;
    const long long tiles = (long long)best.m_tiles * n_tiles;
    const int most = tiles >= units ? 1 : std::min(16, std::max(1, k_stages / 2));
    for (int sp = 1; sp <= most; ++sp) {
      const int per = (k_stages + sp - 1) / sp;
      const int splits = (k_stages + per - 1) / per;
      if (splits != sp) continue;
      const double rounds = (double)((tiles * splits + units - 1) / units);
      const double width = best.pair ? bn + 16 : bn + 0.25 * best.a_rows;
      const double fix = splits > 1 ? (best.pair ? 8.0 : 2.0) * 128 + 0.5 * splits : 0.0;
      const double cost = rounds * per * width + fix;
      if (best_cost == 0 || cost < best_cost) {
        best_cost = cost;
        best.bn = bn;
        best.n_tiles = n_tiles;
        best.splits = splits;
        best.k_per = per * kStageK;
      }
    }
  }
  const int nb = best.pair ? best.bn / 2 : best.bn;
  best.a_bytes = a_mn ? 2 * kMnBlock : 2 * best.a_rows * 128;
  const int b_bytes = b_mn ? (nb + kSub - 1) / kSub * kMnBlock : 2 * nb * 128;
  best.stage_bytes = best.a_bytes + b_bytes;
  // The MMA reads 128 rows of A whatever the box holds (the rows past it feed
  // outputs that are not stored): those of the last stage stay inside the ring.
  const int past = a_mn ? 0
                        : std::max(0, best.a_rows * 128 + kTM * 128 - best.stage_bytes);
  best.n_stages = std::min(kLinMaxStages, (kRing - past) / best.stage_bytes);
  return best;
}

cudaError_t launch_linear_tc(const LinearPlan& p, int M, int N, int K, const void* A, bool a_mn,
                             const void* B, bool b_mn, const LinearEpilogue& epi,
                             float* partials, int* arrivals, uint32_t* status, int sms,
                             cudaStream_t st) {
  using namespace tc;
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
  a.splits = p.splits;
  a.k_per = p.k_per;
  a.a_rows = p.a_rows;
  a.a_bytes = p.a_bytes;
  a.stage_bytes = p.stage_bytes;
  a.n_stages = p.n_stages;
  a.group_m = 16;
  const int nb = p.pair ? p.bn / 2 : p.bn;
  CUtensorMap ma, mb;
  if (!(a_mn ? linear_map(&ma, A, K, M, kStageK) : linear_map(&ma, A, M, K, p.a_rows)) ||
      !(b_mn ? linear_map(&mb, B, K, N, kStageK) : linear_map(&mb, B, N, K, nb)))
    return cudaErrorInvalidValue;
  const int work = p.m_tiles * p.n_tiles * p.splits;
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
      return launch_pdl_cluster2(kernel, dim3(2 * std::min(sms / 2, work)), dim3(kLinThreads),
                                 kLinSmem, st, ma, mb, a);
    return launch_pdl(kernel, dim3(std::min(sms, work)), dim3(kLinThreads), kLinSmem, st, ma, mb,
                      a);
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
