// moe_linear.cu -- the experts' products on the cast's bytes, block-scaled MXFP8 on the
// 5th-generation tensor cores, and the gradients around them.
//
//   forward  z[m, n] = sum_k x[m, k] w[e(m), n, k] + bias[e(m), n],  y = act(z) + residual
//            for rows m in groups that end at offs (multiples of 128), e(m) the row's
//            group; rows behind the last group are 0.  The gradient of the rows is the
//            same product with the weights cast along their other axis.
//   weights  dw[e, n, k] = sum over the rows m of group e of dz[m, n] x[m, k] (+ addend),
//            both operands and their scales as the cast stores them by columns.
//   epilogue dz = dy act'(z), dbias[e, n] = sum over the rows of group e of dz[m, n].
//
// The product kernel: a pair of CTAs (cta_group::2) owns a tile of 256 columns of the
// output x 256 or 128 of its rows.  The columns are the MMA's M axis, 128 a CTA, so that
// the lanes of tensor memory are neighbours in memory and the epilogue writes whole
// sectors from registers at any pitch; the rows are its N axis, so that a group with an
// odd number of 128-row blocks ends in a tile of half the work and not in an idle half.
// Stages of 128 along K: two operands by TMA with the 128-byte swizzle, and their scale
// atoms (512 bytes for 128 rows x 128 K) by TMA as they are stored, copied to tensor
// memory by the thread that issues the MMAs (tcgen05.cp, in order with them).
//
// Tensor memory: an accumulator takes 256 of the 512 columns and the scales need 24, so
// two accumulators would not fit side by side.  They overlap by 32 columns (0..255 and
// 224..479): the epilogue of a tile reads those first, and from then on runs under the
// next tile's products.  (An overlap of 48 columns, two chunks of the epilogue, costs 30 us
// of the 652 below.)
//
// Bound, for large products, by the tensor pipe with what shares it.  57344 rows x 7168 x
// 2048 in 64 groups, 1.80 TFLOP: 652 us, 2.77 PFLOP/s.  Parts left out: the products alone
// 428 us (4.2 PFLOP/s); with the scales' copies 537 (53 clocks a copy whatever its shape,
// three a stage, in line with the products); the operands' loads alone 361; the output's
// stores are worth 58.  What was tried against the copies: scales written to tensor memory
// by warps of their own (699 us: four stages of scales fit, too few for the way there and
// back), two atoms a copy from shared memory where warps lay them out four times (685),
// copies ahead of the products before them (865), copies and loads for two stages at a
// time (no difference).  Every look at a barrier takes shared memory's bandwidth from the
// operands: waits that are suspended, by one lane of a warp, are worth 31 us of 683.
//
// 128 routed rows to 64 experts of 7168 x 2048: 165 us for the weights of the 51 experts
// that have rows there, a block of 128 each, 854 MB in all, 5.2 TB/s.  The rows' gradient, 61440
// rows of width 2048 to 7168 with the weights' column-wise cast: 693 us, 2.60 PFLOP/s,
// where the forward product takes 611.
//
// Weights' gradient, 24 x [1408, 2176] fp32 onto what is there from 40009 rows: 148 us, 5.0
// TB/s, bound by its epilogue of single additions in L2: a kernel of nothing but these does
// 4.95 TB/s of reads and writes.  (Additions of 16 bytes and bulk ones are 10 to 15% faster
// by themselves; here, where rows had to be brought together for them, nothing was gained.)
// With the addend loaded into registers 174, loaded a chunk ahead no less.  Without an
// addend 120 to 128, where the products' 13 stages a tile are as long as the tile's stores; bf16
// 126, and 142 onto what is there.  64 x [2048, 7168] from 57344 rows: 1508, 790 without the
// addend; from 61440 to bf16 1148 and 760.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mma_pair.cuh"
#include "pair_drain.h"
#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_linear_status = 0;

constexpr int kBlock = 128;                     // rows of a scale atom, and what every size is a multiple of
constexpr int kCols = 256;                      // output columns of a tile
constexpr int kRows = 256;                      // output rows of a tile, at most
constexpr int kStepK = 128;                     // bytes of K per stage: one swizzle row
constexpr int kOperandBytes = kBlock * kStepK;  // of one CTA's half
constexpr int kAtomBytes = 512;
constexpr int kStageBytes = 2 * kOperandBytes + 2048;  // two operands, three atoms and room
constexpr int kStages = 6;
constexpr int kThreads = 384;                   // producer, MMA, allocation, zeros; eight epilogue warps
constexpr int kEpilogueWarps = 8;               // two for each 32 columns, each half of the rows
constexpr int kSmem = 1024 + kStages * kStageBytes;
constexpr uint32_t kAccAt = 224;                // tensor memory columns of the second accumulator
constexpr uint32_t kOverlap = 256 - kAccAt;
constexpr uint32_t kScalesAt = 480, kScalesCols = 16;  // two sets: 4 columns of A, 8 of B
constexpr int kBand = 8;                        // row tiles that share a turn through the columns
static_assert(kOverlap == 32, "one chunk of the epilogue");

enum Activation { kNone = MXQ_ACT_NONE, kRelu = MXQ_ACT_RELU, kSilu = MXQ_ACT_SILU, kGelu = MXQ_ACT_GELU };

struct Maps {
  CUtensorMap a, b;    // operands: [batch, rows, K] bytes, boxes of 128 and of 64 rows
  CUtensorMap sa, sb;  // scale atoms, one after another
};

struct Linear {
  const int32_t* offs;   // ends of the groups, or NULL: one group of all rows
  int32_t groups;
  int32_t grouped;       // rows that the groups divide
  int32_t cols;          // output columns
  int32_t out_rows;      // weights: rows of each group's output
  int32_t ksteps;        // forward: stages along K
  int32_t bias_bf16;
  const void* bias;      // [groups, cols], or NULL
  const void* addend;    // of the output's type, or NULL; may be the output itself
  void *y, *z;           // z: before the activation, or NULL
  int64_t ld_add, ld_y, ld_z;          // elements between rows
  int64_t stride_add, stride_y;        // weights: between the groups' matrices
  uint64_t add_bytes, y_bytes, z_bytes;
};

// The groups of a launch, in shared memory.
struct Groups {
  int32_t ends[MXQ_MAX_GROUPS];
  int32_t tiles[MXQ_MAX_GROUPS];  // forward: row tiles of this group and all before it
};

struct Tile {
  int32_t rows;               // of the output: 256 or 128
  int32_t count;              // stages along K
  int32_t group, row, col;    // of the output
  int32_t a_k, a_row, a_batch, b_k, b_row;   // where the operands begin
  int32_t a_atom, a_next, b_atom, b_next;    // first scale atom, and from one 128-row block to the next
};

template <bool kWeights>
__device__ __forceinline__ Tile tile_at(const Linear& p, const Groups& g, int32_t t) {
  const int32_t across = (p.cols + kCols - 1) / kCols;
  Tile at;
  if (kWeights) {
    const int32_t down = (p.out_rows + kRows - 1) / kRows, per = across * down;
    const int32_t e = t / per, i = t - e * per, f = i / down, r = i - f * down;
    const int32_t lo = e > 0 ? g.ends[e - 1] : 0, count = (g.ends[e] - lo) / kStepK;
    at.rows = p.out_rows - r * kRows >= kRows ? kRows : kBlock;
    at.count = count;
    at.group = e, at.row = r * kRows, at.col = f * kCols;
    at.a_k = at.b_k = lo;
    at.a_row = at.col, at.a_batch = 0, at.b_row = at.row;
    at.a_atom = p.cols / kBlock * (lo / kStepK) + at.col / kBlock * count;
    at.b_atom = p.out_rows / kBlock * (lo / kStepK) + at.row / kBlock * count;
    at.a_next = at.b_next = count;
  } else {
    int32_t e = 0, most = p.groups - 1;  // the first group whose tiles end behind t
    while (e < most) {
      const int32_t mid = (e + most) / 2;
      if (g.tiles[mid] * across > t) most = mid;
      else e = mid + 1;
    }
    const int32_t before = e > 0 ? g.tiles[e - 1] : 0, down = g.tiles[e] - before, i = t - before * across;
    // bands of row tiles, each through all columns: neighbours in time share operands in L2
    const int32_t band = i / (kBand * across), high = min(kBand, down - band * kBand), j = i - band * kBand * across;
    const int32_t f = j / high, r = band * kBand + j - f * high;
    const int32_t lo = e > 0 ? g.ends[e - 1] : 0;
    at.rows = g.ends[e] - lo - r * kRows >= kRows ? kRows : kBlock;
    at.count = p.ksteps;
    at.group = e, at.row = lo + r * kRows, at.col = f * kCols;
    at.a_k = at.b_k = 0;
    at.a_row = at.col, at.a_batch = e, at.b_row = at.row;
    at.a_atom = (e * (p.cols / kBlock) + at.col / kBlock) * p.ksteps;
    at.b_atom = at.row / kBlock * p.ksteps;
    at.a_next = at.b_next = p.ksteps;
  }
  return at;
}

__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// D (+)= A B^T with the E8M0 scales of A and B in tensor memory.
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc;\n\tsetp.ne.b32 acc, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], acc;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// A scale atom of each CTA's shared memory to 4 columns of its tensor memory, for all four
// quarters of the lanes: row r of 128 finds its 4 scales in lane r % 32, column r / 32.
__device__ __forceinline__ void copy_atom_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// K-major operand with the 128-byte swizzle: 1024 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// A scale atom: 32 rows of 16 bytes, no swizzle, 128 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t atom_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
// E4M3 operands, E8M0 scales, M = 256, N = rows; K block k of a stage takes scale byte k.
__device__ __forceinline__ uint32_t instruction_desc(uint32_t rows, uint32_t k) {
  return (k << 4) | ((rows / 8u) << 17) | (1u << 23) | ((kCols / 16u) << 24) | (k << 29);
}

// act(z) and act'(z), NaN kept.  The logistic function is a few units in the last place of
// fp32 off.  gelu is the tanh form, written with 0.5 (1 + tanh u) = logistic(2u).
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;  // 2 sqrt(2 / pi)
template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if (kAct == kRelu) return z < 0.0f ? 0.0f : z;
  if (kAct == kSilu) return z * logistic(z);
  if (kAct == kGelu) return z * logistic(kGeluA * z * fmaf(kGeluB, z * z, 1.0f));
  return z;
}
// The rest 1 - logistic is taken by its own formula: a factor of up to z^3 brings back the
// digits that the difference would lose.  Beyond 128 (gelu 64) it is 0 and the slope 1 or
// 0 in fp32; z is cut there, as its powers would overflow.
template <int kAct>
__device__ __forceinline__ float slope(float z) {
  if (kAct == kRelu) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
  constexpr float kEnd = kAct == kGelu ? 64.0f : 128.0f;
  asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(z) : "f"(kEnd), "f"(-kEnd));  // a NaN stays
  float s, rest;
  if (kAct == kSilu) {
    logistic_pair(z, s, rest);
    return s * fmaf(z, rest, 1.0f);
  }
  if (kAct == kGelu) {
    logistic_pair(kGeluA * z * fmaf(kGeluB, z * z, 1.0f), s, rest);
    return s * fmaf(kGeluA * z * fmaf(3.0f * kGeluB, z * z, 1.0f), rest, 1.0f);
  }
  return 1.0f;
}

// The ends of the groups into shared memory, checked as the cast checks them; false, and
// MXQ_DEV_BADOFFS, where they are not ends of groups of whole 128 rows.
__device__ __forceinline__ bool read_groups(const int32_t* offs, int32_t groups, int32_t rows, int32_t* ends) {
  bool fine = true;
  for (int32_t e = threadIdx.x; e < groups; e += blockDim.x) {
    const int32_t end = offs == nullptr ? rows : read_at(offs, e, groups, 0, &g_linear_status);
    const int32_t before = offs == nullptr || e == 0 ? 0 : read_at(offs, e - 1, groups, 0, &g_linear_status);
    fine = fine && end >= before && end % kBlock == 0 && end >= 0 && end <= rows;
    ends[e] = end;
  }
  fine = __syncthreads_and(fine);
  if (!fine && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_linear_status, MXQ_DEV_BADOFFS);
  return fine;
}

struct alignas(8) Barriers {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_free;
  uint64_t drained;        // the leader's: its MMAs are done, after a wait that ran out
  uint32_t tmem, abort_flag;
  uint32_t leader_gave_up, issued[2];     // by the leader; to the leader: stages each CTA has issued
  uint32_t half[kStages], peer_half[kStages];  // bytes of a slot's last stage, of this CTA and (to the leader) of its peer
};

template <bool kWeights, typename T, int kAct>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Linear p) {
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bars;
  __shared__ Groups groups;
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  volatile uint32_t* abort_flag = &bars.abort_flag;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bars.full[s]), 1);
      mbar_init(smem_u32(&bars.empty[s]), 1);
      bars.half[s] = bars.peer_half[s] = 0u;
    }
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&bars.acc_full[s]), 1);
    mbar_init(smem_u32(&bars.acc_free), 2 * kEpilogueWarps);  // of both CTAs
    mbar_init(smem_u32(&bars.drained), 1);
    bars.abort_flag = bars.leader_gave_up = bars.issued[0] = bars.issued[1] = 0u;
    mbar_init_fence();
    if (p.grouped > 0) {  // else there are no operands
      tma_prefetch_desc(&maps.a);
      tma_prefetch_desc(&maps.b);
      tma_prefetch_desc(&maps.sa);
      tma_prefetch_desc(&maps.sb);
    }
  }
  __syncthreads();
  cluster_sync_all();  // both CTAs of the pair run, with their barriers set up
  if (warp == 2) tmem_alloc_pair(smem_u32(&bars.tmem));
  fence_before();
  __syncthreads();
  cluster_sync_all();
  fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_launch_dependents();

  const bool fine = read_groups(p.offs, p.groups, p.grouped, groups.ends);
  int32_t tiles = 0;
  if (fine && kWeights) tiles = p.groups * ((p.out_rows + kRows - 1) / kRows) * ((p.cols + kCols - 1) / kCols);
  if (fine && !kWeights) {
    if (warp == 0) {  // row tiles of the groups, added up
      int32_t before = 0;
      for (int32_t e0 = 0; e0 < p.groups; e0 += 32) {
        const int32_t e = e0 + lane;
        int32_t n = 0;
        if (e < p.groups) n = (groups.ends[e] - (e > 0 ? groups.ends[e - 1] : 0) + kRows - 1) / kRows;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int32_t other = __shfl_up_sync(0xFFFFFFFFu, n, d);
          if (lane >= d) n += other;
        }
        if (e < p.groups) groups.tiles[e] = before + n;
        before += __shfl_sync(0xFFFFFFFFu, n, 31);
      }
    }
    __syncthreads();
    tiles = groups.tiles[p.groups - 1] * ((p.cols + kCols - 1) / kCols);
  }

  if (warp == 0 && lane == 0) {
    // ---- producer: this CTA's half of A and of B, its atoms of A and all of B ----
    int issued = 0;  // stages loaded so far
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      const Tile at = tile_at<kWeights>(p, groups, t);
      const int32_t half = at.rows / 2, blocks = at.rows / kBlock;
      const uint32_t bytes = kOperandBytes + half * kStepK + (1 + blocks) * kAtomBytes;
      const int32_t row_a = at.a_row + static_cast<int32_t>(rank) * kBlock, row_b = at.b_row + static_cast<int32_t>(rank) * half;
      const int32_t atom_a = at.a_atom + static_cast<int32_t>(rank) * at.a_next;
      for (int k = 0; k < at.count; ++k, ++issued) {
        const int s = issued % kStages;
        if (!wait_suspended(smem_u32(&bars.empty[s]), ((issued / kStages) & 1) ^ 1, abort_flag, &g_linear_status)) {
          ok = false;
          break;
        }
        const uint32_t bar = at_leader(smem_u32(&bars.full[s]));
        bars.half[s] = bytes;
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.full[s]), 2 * bytes);
        const uint32_t da = smem + s * kStageBytes, db = da + kOperandBytes, ds = db + kOperandBytes;
        load_3d_pair(da, &maps.a, at.a_k + k * kStepK, row_a, at.a_batch, bar);
        load_3d_pair(db, &maps.b, at.b_k + k * kStepK, row_b, 0, bar);
        if (half == kBlock) load_3d_pair(db + kOperandBytes / 2, &maps.b, at.b_k + k * kStepK, row_b + kBlock / 2, 0, bar);
        load_2d_pair(ds, &maps.sa, 0, atom_a + k, bar);
        load_2d_pair(ds + kAtomBytes, &maps.sb, 0, at.b_atom + k, bar);
        if (blocks == 2) load_2d_pair(ds + 2 * kAtomBytes, &maps.sb, 0, at.b_atom + at.b_next + k, bar);
      }
    }
    if (rank != 0)
      for (int s = 0; s < kStages; ++s) store_cluster(at_leader(smem_u32(&bars.peer_half[s])), bars.half[s]);
    store_cluster(at_leader(smem_u32(&bars.issued[rank])), static_cast<uint32_t>(issued));
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issue for the pair -------------------------------------------
    int n = 0, done = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      const Tile at = tile_at<kWeights>(p, groups, t);
      if (at.count == 0) continue;
      const int acc = done & 1;
      const uint32_t d = tmem + (acc ? kAccAt : 0u), blocks = at.rows / kBlock;
      ok = wait_suspended(smem_u32(&bars.acc_free), (done & 1) ^ 1, abort_flag, &g_linear_status);
      fence_after();
      for (int k = 0; ok && k < at.count; ++k, ++n) {
        const int s = n % kStages;
        ok = wait_suspended(smem_u32(&bars.full[s]), (n / kStages) & 1, abort_flag, &g_linear_status);
        if (!ok) break;
        fence_after();
        const uint32_t da = smem + s * kStageBytes, ds = da + 2 * kOperandBytes;
        const uint32_t sfa = tmem + kScalesAt + (n & 1) * kScalesCols, sfb = sfa + 4;
        copy_atom_pair(sfa, atom_desc(ds));
        copy_atom_pair(sfb, atom_desc(ds + kAtomBytes));
        if (blocks == 2) copy_atom_pair(sfb + 4, atom_desc(ds + 2 * kAtomBytes));
        const uint64_t a = operand_desc(da), b = operand_desc(da + kOperandBytes);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
          mma_scaled_pair(d, a + 2 * q, b + 2 * q, instruction_desc(at.rows, q), sfa, sfb, (k | q) != 0);
        commit_pair(smem_u32(&bars.empty[s]));
      }
      if (ok) commit_pair(smem_u32(&bars.acc_full[acc]));
      ++done;
    }
    if (!ok) {  // products under way read both CTAs' stages and write their tensor memory
      commit_here(smem_u32(&bars.drained));
      mbar_wait_drain(smem_u32(&bars.drained), 0);
    }
  } else if (warp == 3 && !kWeights) {
    // ---- rows behind the last group ------------------------------------------
    const int32_t from = fine ? groups.ends[p.groups - 1] : p.grouped;
    for (int32_t r = from + static_cast<int32_t>(blockIdx.x); r < p.grouped; r += gridDim.x) {
      T* y = static_cast<T*>(p.y) + r * p.ld_y;
      T* z = static_cast<T*>(p.z) + r * p.ld_z;
      for (int32_t c = lane; c < p.cols; c += 32) {
        if (in_buf(y + c, sizeof(T), p.y, p.y_bytes, &g_linear_status)) y[c] = narrow<T>(0.0f);
        if (p.z != nullptr && in_buf(z + c, sizeof(T), p.z, p.z_bytes, &g_linear_status)) z[c] = narrow<T>(0.0f);
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: 32 of this CTA's 128 columns, half of the rows ------------
    // A sum onto fp32 weights is the memory's own: each element takes one addition, so the
    // order is not open, and no load is waited for.
    constexpr bool kAddInL2 = kWeights && sizeof(T) == 4;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int done = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      const Tile at = tile_at<kWeights>(p, groups, t);
      if (at.count == 0 && p.addend == p.y) continue;  // nothing to add
      const int acc = done & 1, span = at.rows / 2, chunks = span / 32;
      const int32_t col = at.col + static_cast<int32_t>(rank) * kBlock + quarter * 32 + lane;
      const bool mine = at.col + static_cast<int32_t>(rank) * kBlock < p.cols;
      const bool overlapped = at.count != 0 && (acc ? half == 0 : half == 1 && at.rows == kRows);
      float bias = 0.0f;
      if (p.bias != nullptr && mine) {
        const int64_t i = static_cast<int64_t>(at.group) * p.cols + col, all = static_cast<int64_t>(p.groups) * p.cols;
        bias = p.bias_bf16 ? widen(read_at(static_cast<const bf16_t*>(p.bias), i, all, bf16_t{0}, &g_linear_status))
                           : read_at(static_cast<const float*>(p.bias), i, all, 0.0f, &g_linear_status);
      }
      const auto let_go = [&] {  // the next tile's products may begin, as far as this warp goes
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(at_leader(smem_u32(&bars.acc_free)));
      };
      if (at.count != 0) {
        ok = warp_wait(smem_u32(&bars.acc_full[acc]), (done >> 1) & 1, abort_flag, &g_linear_status);
        if (!ok) break;
        fence_after();
        if (!overlapped) let_go();
        ++done;
      }
#pragma unroll 1
      for (int i = 0; i < chunks; ++i) {
        const int c = half * span + 32 * (overlapped && !acc ? chunks - 1 - i : i);
        uint32_t v[32];
        T add[32];
        const int64_t row = at.row + c;
        const T* from = static_cast<const T*>(p.addend) + at.group * p.stride_add + row * p.ld_add + col;
        if (!kAddInL2 && p.addend != nullptr && mine) {
#pragma unroll
          for (int r = 0; r < 32; ++r)
            add[r] = in_buf(from + r * p.ld_add, sizeof(T), p.addend, p.add_bytes, &g_linear_status) ? from[r * p.ld_add]
                                                                                                    : narrow<T>(0.0f);
        }
        if (at.count != 0) {
          tmem_load_32(lanes + (acc ? kAccAt : 0u) + c, v);
          tmem_wait_load();
        } else {
#pragma unroll
          for (int r = 0; r < 32; ++r) v[r] = 0u;
        }
        if (overlapped && i == 0) let_go();
        if (!mine) continue;
        T* y = static_cast<T*>(p.y) + at.group * p.stride_y + row * p.ld_y + col;
        if (kAddInL2 && p.addend != nullptr) {
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (in_buf(y + r * p.ld_y, sizeof(T), p.y, p.y_bytes, &g_linear_status))
              asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(y + r * p.ld_y), "f"(__uint_as_float(v[r])) : "memory");
          continue;
        }
        if (p.z != nullptr) {
          T* z = static_cast<T*>(p.z) + row * p.ld_z + col;
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (in_buf(z + r * p.ld_z, sizeof(T), p.z, p.z_bytes, &g_linear_status))
              z[r * p.ld_z] = narrow<T>(__uint_as_float(v[r]) + bias);
        }
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          float o = activate<kAct>(__uint_as_float(v[r]) + bias);
          if (!kAddInL2 && p.addend != nullptr) o += widen(add[r]);
          if (in_buf(y + r * p.ld_y, sizeof(T), p.y, p.y_bytes, &g_linear_status)) y[r * p.ld_y] = narrow<T>(o);
        }
      }
    }
  }
  // Neither CTA leaves while the other may still signal it or read its memory.  After a
  // wait that ran out the leader, whose barriers count both CTAs' loads, waits for
  // those still in flight (again with a limit) before either lets go of its memory.
  // A leader whose waits all ended has seen every load and product of the pair.
  __syncthreads();
  if (rank == 0 && tid == 0 && bars.abort_flag) store_cluster(at_rank(smem_u32(&bars.leader_gave_up), 1), 1u);
  __syncwarp();
  cluster_sync_all();
  if (rank == 0 ? bars.abort_flag : bars.leader_gave_up) {
    if (rank == 0 && tid == 0) {
      const int own = static_cast<int>(bars.issued[0]), peer = static_cast<int>(bars.issued[1]);
      const PairDrain range = pair_drain(own, peer, kStages);
      for (int n = range.first; n < range.end; ++n) {
        const int s = n % kStages;
        const uint32_t bar = smem_u32(&bars.full[s]);
        if (pair_unannounced(n, own)) mbar_arrive_expect_tx(bar, bars.peer_half[s]);
        if (pair_half_missing(n, peer)) mbar_complete_tx(bar, bars.half[s]);
        mbar_wait_drain(bar, (n / kStages) & 1);
      }
    }
    __syncthreads();
    cluster_sync_all();
  }
  __syncthreads();
  fence_after();
  if (warp == 2) tmem_free_pair(tmem);
}

// ---------------------------------------------------------------------------
// gradient of activation and bias
// ---------------------------------------------------------------------------
// A block takes 128 rows, which lie in one group, and columns of one vector a thread: the
// rows' sums of dz are its part of dbias, added up over the group's blocks in order by the
// second kernel.  57344 x 4096 silu in bf16: 250 us with them, 6.05 TB/s, bound by DRAM.
// Rows that do not all begin at 16 bytes go by single elements: 431 us at a pitch of 4097,
// fp32 of half the width 269 in place of 220.
constexpr int kBackThreads = 256;

struct Epilogue {
  const void *dy, *z;
  void* dz;            // or NULL
  const int32_t* offs;
  float* parts;        // [rows / 128, cols], or NULL
  int32_t rows, cols, groups;
  int64_t ld_dy, ld_z, ld_dz;
  uint64_t dy_bytes, z_bytes, dz_bytes;
};

// The end of the last group where offs are valid; read by every block.
__device__ __forceinline__ bool groups_valid(const int32_t* offs, int32_t groups, int32_t rows, int32_t* end) {
  bool fine = true;
  if (offs != nullptr)
    for (int32_t e = threadIdx.x; e < groups; e += blockDim.x) {
      const int32_t at = read_at(offs, e, groups, 0, &g_linear_status), before = e > 0 ? read_at(offs, e - 1, groups, 0, &g_linear_status) : 0;
      fine = fine && at >= before && at % kBlock == 0 && at <= rows;
    }
  *end = offs == nullptr ? rows : read_at(offs, groups - 1, groups, 0, &g_linear_status);
  fine = __syncthreads_and(fine);
  if (!fine && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_linear_status, MXQ_DEV_BADOFFS);
  return fine;
}

template <typename T, int kV, int kAct>
__global__ void __launch_bounds__(kBackThreads) epilogue_backward_kernel(const Epilogue a, int32_t blocks_across, int32_t tx) {
  extern __shared__ float sums[];  // [kBackThreads, kV]
  pdl_wait();
  int32_t end;
  if (!groups_valid(a.offs, a.groups, a.rows, &end)) return;
  const int32_t block = blockIdx.x / blocks_across, ty = kBackThreads / tx, own = threadIdx.x % tx, down = threadIdx.x / tx;
  const int32_t col = (static_cast<int32_t>(blockIdx.x) % blocks_across * tx + own) * kV;
  const bool live = block * kBlock < end;
  float sum[kV] = {};
  if (col < a.cols) {
    constexpr int kAhead = 4;
    for (int32_t r0 = down; r0 < kBlock; r0 += kAhead * ty) {
      Vec<T, kV> dy[kAhead], z[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int64_t row = static_cast<int64_t>(block) * kBlock + r0 + q * ty;
        const bool in = live && r0 + q * ty < kBlock;
        const T* from = static_cast<const T*>(a.dy) + row * a.ld_dy + col;
        dy[q] = load_if_written<T, kV>(from, in && in_buf(from, sizeof dy[q], a.dy, a.dy_bytes, &g_linear_status));
        if (kAct != kNone) {
          const T* at = static_cast<const T*>(a.z) + row * a.ld_z + col;
          z[q] = load_if<T, kV>(at, in && in_buf(at, sizeof z[q], a.z, a.z_bytes, &g_linear_status));
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (r0 + q * ty >= kBlock) break;
        Vec<T, kV> out;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float d = kAct == kNone ? widen(dy[q].v[j]) : widen(dy[q].v[j]) * slope<kAct>(widen(z[q].v[j]));
          sum[j] += live ? d : 0.0f;
          out.v[j] = narrow<T>(live ? d : 0.0f);
        }
        if (a.dz == nullptr) continue;
        T* to = static_cast<T*>(a.dz) + (static_cast<int64_t>(block) * kBlock + r0 + q * ty) * a.ld_dz + col;
        if (in_buf(to, sizeof out, a.dz, a.dz_bytes, &g_linear_status)) *reinterpret_cast<Vec<T, kV>*>(to) = out;
      }
    }
  }
  if (a.parts == nullptr) return;
#pragma unroll
  for (int j = 0; j < kV; ++j) sums[threadIdx.x * kV + j] = sum[j];
  __syncthreads();
  const int64_t count = static_cast<int64_t>(a.rows / kBlock) * a.cols;
  const int32_t first = static_cast<int32_t>(blockIdx.x) % blocks_across * tx * kV;
  for (int32_t i = threadIdx.x; i < tx * kV && first + i < a.cols; i += kBackThreads) {
    float all = 0.0f;
    for (int32_t y = 0; y < ty; ++y) all += sums[y * tx * kV + i];
    write_at(a.parts, static_cast<int64_t>(block) * a.cols + first + i, count, all, &g_linear_status);
  }
}

// dbias of one group and 128 columns, four a lane: eight warps take every eighth block of
// rows.  (With one column a lane, and four times the blocks, 14 us; now 7.)
__global__ void __launch_bounds__(256) bias_join_kernel(const float* parts, const int32_t* offs, int32_t groups, int32_t rows,
                                                         int32_t cols, float* dbias) {
  __shared__ __align__(16) float by_warp[8][kBlock];
  pdl_wait();
  int32_t end;
  if (!groups_valid(offs, groups, rows, &end)) return;
  const int32_t across = cols / kBlock, e = blockIdx.x / across, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t first = (static_cast<int32_t>(blockIdx.x) - e * across) * kBlock;
  const int32_t lo = offs == nullptr || e == 0 ? 0 : read_at(offs, e - 1, groups, 0, &g_linear_status);
  const int32_t hi = offs == nullptr ? rows : read_at(offs, e, groups, 0, &g_linear_status);
  const uint64_t bytes = static_cast<uint64_t>(rows / kBlock) * cols * 4;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int32_t b = lo / kBlock + warp; b < hi / kBlock; b += 8) {
    const float* at = parts + static_cast<int64_t>(b) * cols + first + 4 * lane;
    if (!in_buf(at, 16, parts, bytes, &g_linear_status)) continue;
    const float4 v = *reinterpret_cast<const float4*>(at);
    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
  }
  *reinterpret_cast<float4*>(&by_warp[warp][4 * lane]) = sum;
  __syncthreads();
  if (threadIdx.x >= kBlock) return;
  float all = by_warp[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < 8; ++w) all += by_warp[w][threadIdx.x];
  write_at(dbias, static_cast<int64_t>(e) * cols + first + threadIdx.x, static_cast<int64_t>(groups) * cols, all, &g_linear_status);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// [batch, rows, K] bytes, rows ld and matrices `stride` bytes apart; boxes of box_rows x 128.
bool encode_operand(CUtensorMap* map, const uint8_t* base, int64_t k, int64_t rows, int64_t batch, int64_t ld, int64_t stride,
                    uint32_t box_rows) {
  const auto fn = driver_tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(batch > 1 ? stride : ld)};
  const cuuint32_t box[3] = {kStepK, box_rows, 1}, ones[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_atoms(CUtensorMap* map, const uint8_t* base, int64_t atoms) {
  const auto fn = driver_tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {kAtomBytes / 4, static_cast<cuuint64_t>(atoms)}, strides[1] = {kAtomBytes};
  const cuuint32_t box[2] = {kAtomBytes / 4, 1}, ones[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kWeights, typename T, int kAct>
int launch_linear(const Maps& maps, const Linear& p, int64_t tiles, int sms, cudaStream_t stream) {
  const auto kernel = linear_kernel<kWeights, T, kAct>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  const int64_t pairs = sms / 2 < tiles ? sms / 2 : tiles;
  return launch_pdl(kernel, static_cast<unsigned>(2 * pairs), kThreads, kSmem, stream, maps, p);
}
template <typename T>
int launch_forward(int act, const Maps& maps, const Linear& p, int64_t tiles, int sms, cudaStream_t stream) {
  switch (act) {
    case kRelu: return launch_linear<false, T, kRelu>(maps, p, tiles, sms, stream);
    case kSilu: return launch_linear<false, T, kSilu>(maps, p, tiles, sms, stream);
    case kGelu: return launch_linear<false, T, kGelu>(maps, p, tiles, sms, stream);
    default: return launch_linear<false, T, kNone>(maps, p, tiles, sms, stream);
  }
}

constexpr int64_t kMostSize = int64_t{1} << 24;   // of rows, columns and K
constexpr int64_t kMostPitch = int64_t{1} << 39;  // elements

bool size_ok(int64_t n) { return n >= 0 && n <= kMostSize && n % kBlock == 0; }
bool type_ok(int t) { return t == MXQ_F32 || t == MXQ_BF16; }
bool operand_ok(int64_t ld, int64_t k) { return ld >= k && ld % 16 == 0 && ld <= kMostPitch; }

// An addend that is the output itself, element for element, may share its memory.
bool same_place(const void* a, int64_t ld_a, const void* b, int64_t ld_b) { return a == b && ld_a == ld_b; }

template <typename T, int kV, int kAct>
int launch_epilogue(const Epilogue& a, cudaStream_t stream) {
  int32_t tx = 8;
  while (tx < kBackThreads && tx * kV < a.cols) tx *= 2;
  if (tx > 64) tx = 64;
  const int32_t across = static_cast<int32_t>(ceil_div(a.cols, tx * kV));
  return launch_pdl(epilogue_backward_kernel<T, kV, kAct>, static_cast<unsigned>(a.rows / kBlock * across), kBackThreads,
                    kBackThreads * kV * 4, stream, a, across, tx);
}
template <typename T, int kV>
int launch_epilogue_act(int act, const Epilogue& a, cudaStream_t stream) {
  switch (act) {
    case kRelu: return launch_epilogue<T, kV, kRelu>(a, stream);
    case kSilu: return launch_epilogue<T, kV, kSilu>(a, stream);
    case kGelu: return launch_epilogue<T, kV, kGelu>(a, stream);
    default: return launch_epilogue<T, kV, kNone>(a, stream);
  }
}
template <typename T>
int launch_epilogue_typed(int act, const Epilogue& a, cudaStream_t stream) {
  const uint64_t es = sizeof(T);
  const int align = common_alignment({address_of(a.dy), a.ld_dy * es, address_of(a.z), a.ld_z * es, address_of(a.dz), a.ld_dz * es});
  return align >= 16 ? launch_epilogue_act<T, 16 / sizeof(T)>(act, a, stream) : launch_epilogue_act<T, 1>(act, a, stream);
}

}  // namespace

namespace mxq {
int linear_status_read(unsigned int* out, bool clear) { return read_status_word(g_linear_status, out, clear); }
int linear_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int mxq_moe_linear(const uint8_t* x, int64_t ldx, const uint8_t* sx, const uint8_t* w, int64_t ldw, int64_t stride_w,
                              const uint8_t* sw, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                              const void* bias, int bias_dtype, int activation, const void* residual, int64_t ldr, int dtype,
                              void* y, int64_t ldy, void* z, int64_t ldz, cudaStream_t stream) {
  if (!type_ok(dtype) || (bias && !type_ok(bias_dtype))) return MXQ_EBADDTYPE;
  if ((offs == nullptr && G != 0) || (offs != nullptr && (G < 1 || G > MXQ_MAX_GROUPS))) return MXQ_EBADOFFS;
  const int64_t groups = offs ? G : 1;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || activation < MXQ_ACT_NONE || activation > MXQ_ACT_GELU) return MXQ_EBADSHAPE;
  if (M == 0 || N == 0) return MXQ_OK;
  if (K == 0 || !operand_ok(ldx, K) || !operand_ok(ldw, K) || ldy < N || ldy > INT32_MAX || (residual && (ldr < N || ldr > INT32_MAX)) ||
      (z && (ldz < N || ldz > INT32_MAX)) || (groups > 1 && (stride_w <= 0 || stride_w % 16 != 0 || stride_w > kMostPitch)))
    return MXQ_EBADSHAPE;
  const int64_t x_atoms = M / kBlock * (K / kStepK), w_atoms = groups * (N / kBlock) * (K / kStepK);
  // a tile for every 128 rows at most, but for those of the groups' ends
  const int64_t tiles = (M / kRows + groups) * ceil_div(N, kCols);
  if (x_atoms > INT32_MAX || w_atoms > INT32_MAX || tiles > INT32_MAX / 2) return MXQ_EBADSHAPE;
  if (!x || !sx || !w || !sw || !y) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(x, 16) || !aligned_to(sx, 16) || !aligned_to(w, 16) || !aligned_to(sw, 16) || !aligned_to(offs, 4) ||
      !aligned_to(y, es) || !aligned_to(z, es) || !aligned_to(residual, es) || (bias && !aligned_to(bias, element_bytes(bias_dtype))))
    return MXQ_EALIGN;
  const bool in_place = residual && same_place(residual, ldr, y, ldy);
  const ByteRange out[2] = {range_of(y, pitched_bytes(M, N, ldy, es)), range_of(z, pitched_bytes(M, N, ldz, es))};
  const ByteRange in[7] = {range_of(x, pitched_bytes(M, K, ldx, 1)),
                           range_of(sx, static_cast<uint64_t>(x_atoms) * kAtomBytes),
                           range_of(w, static_cast<uint64_t>(groups - 1) * stride_w + pitched_bytes(N, K, ldw, 1)),
                           range_of(sw, static_cast<uint64_t>(w_atoms) * kAtomBytes),
                           range_of(offs, 4ull * G),
                           range_of(bias, static_cast<uint64_t>(groups) * N * (bias ? element_bytes(bias_dtype) : 0)),
                           in_place ? ByteRange{0, 0} : range_of(residual, pitched_bytes(M, N, ldr, es))};
  if (outputs_overlap(out, 2, in, 7)) return MXQ_EOVERLAP;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 1) return MXQ_ECUDA;
  Maps maps;
  if (!encode_operand(&maps.a, w, K, N, groups, ldw, stride_w, kBlock) || !encode_operand(&maps.b, x, K, M, 1, ldx, 0, kBlock / 2) ||
      !encode_atoms(&maps.sa, sw, w_atoms) || !encode_atoms(&maps.sb, sx, x_atoms))
    return MXQ_ECUDA;
  Linear p = {};
  p.offs = offs;
  p.groups = static_cast<int32_t>(groups);
  p.grouped = static_cast<int32_t>(M);
  p.cols = static_cast<int32_t>(N);
  p.ksteps = static_cast<int32_t>(K / kStepK);
  p.bias = bias;
  p.bias_bf16 = bias_dtype == MXQ_BF16;
  p.addend = residual;
  p.y = y;
  p.z = z;
  p.ld_add = ldr, p.ld_y = ldy, p.ld_z = ldz;
  p.add_bytes = pitched_bytes(M, N, ldr, es), p.y_bytes = out[0].bytes, p.z_bytes = out[1].bytes;
  return dtype == MXQ_F32 ? launch_forward<float>(activation, maps, p, tiles, sms, stream)
                          : launch_forward<bf16_t>(activation, maps, p, tiles, sms, stream);
}

extern "C" int mxq_moe_weight_gradient(const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b, int64_t ldb,
                                       const uint8_t* sb, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                       int accumulate, int dtype, void* dw, int64_t ldd, int64_t stride_d, cudaStream_t stream) {
  if (!type_ok(dtype)) return MXQ_EBADDTYPE;
  if ((offs == nullptr && G != 0) || (offs != nullptr && (G < 1 || G > MXQ_MAX_GROUPS))) return MXQ_EBADOFFS;
  const int64_t groups = offs ? G : 1;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return MXQ_EBADSHAPE;
  if (N == 0 || K == 0) return MXQ_OK;
  const int es = element_bytes(dtype);
  if (ldd < K || ldd > INT32_MAX || (M > 0 && (!operand_ok(lda, M) || !operand_ok(ldb, M))) || stride_d < 0 || stride_d > kMostPitch ||
      (groups > 1 && stride_d < (N - 1) * ldd + K))
    return MXQ_EBADSHAPE;
  const int64_t a_atoms = N / kBlock * (M / kStepK), b_atoms = K / kBlock * (M / kStepK);
  const int64_t tiles = groups * ceil_div(N, kRows) * ceil_div(K, kCols);
  if (a_atoms > INT32_MAX || b_atoms > INT32_MAX || tiles > INT32_MAX / 2) return MXQ_EBADSHAPE;
  if (!dw || (M > 0 && (!a || !sa || !b || !sb))) return MXQ_ENULL;
  if (!aligned_to(a, 16) || !aligned_to(sa, 16) || !aligned_to(b, 16) || !aligned_to(sb, 16) || !aligned_to(offs, 4) || !aligned_to(dw, es))
    return MXQ_EALIGN;
  const ByteRange out[1] = {range_of(dw, (static_cast<uint64_t>(groups - 1) * stride_d + (N - 1) * ldd + K) * es)};
  const ByteRange in[5] = {range_of(a, pitched_bytes(M > 0 ? N : 0, M, lda, 1)), range_of(sa, static_cast<uint64_t>(a_atoms) * kAtomBytes),
                           range_of(b, pitched_bytes(M > 0 ? K : 0, M, ldb, 1)), range_of(sb, static_cast<uint64_t>(b_atoms) * kAtomBytes),
                           range_of(offs, 4ull * G)};
  if (outputs_overlap(out, 1, in, 5)) return MXQ_EOVERLAP;
  if (M == 0 && accumulate) return MXQ_OK;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 1) return MXQ_ECUDA;
  Maps maps = {};
  // without rows no tile has a stage, and nothing is loaded
  if (M > 0 && (!encode_operand(&maps.a, b, M, K, 1, ldb, 0, kBlock) || !encode_operand(&maps.b, a, M, N, 1, lda, 0, kBlock / 2) ||
                !encode_atoms(&maps.sa, sb, b_atoms) || !encode_atoms(&maps.sb, sa, a_atoms)))
    return MXQ_ECUDA;
  Linear p = {};
  p.offs = offs;
  p.groups = static_cast<int32_t>(groups);
  p.grouped = static_cast<int32_t>(M);
  p.cols = static_cast<int32_t>(K);
  p.out_rows = static_cast<int32_t>(N);
  p.addend = accumulate ? dw : nullptr;
  p.y = dw;
  p.ld_add = p.ld_y = ldd;
  p.stride_add = p.stride_y = groups > 1 ? stride_d : 0;
  p.add_bytes = p.y_bytes = out[0].bytes;
  return dtype == MXQ_F32 ? launch_linear<true, float, kNone>(maps, p, tiles, sms, stream)
                          : launch_linear<true, bf16_t, kNone>(maps, p, tiles, sms, stream);
}

extern "C" int64_t mxq_moe_linear_backward_workspace(int64_t M, int64_t N) {
  if (!size_ok(M) || !size_ok(N) || M / kBlock * N > (int64_t{1} << 40)) return MXQ_EBADSHAPE;
  return M / kBlock * N * 4;
}

extern "C" int mxq_moe_linear_backward(const void* dy, int dtype, int64_t ld_dy, const void* z, int64_t ldz, int activation,
                                       const int32_t* offs, int32_t G, int64_t M, int64_t N, void* dz, int64_t ld_dz, float* dbias,
                                       uint8_t* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (!type_ok(dtype)) return MXQ_EBADDTYPE;
  if ((offs == nullptr && G != 0) || (offs != nullptr && (G < 1 || G > MXQ_MAX_GROUPS))) return MXQ_EBADOFFS;
  const int64_t groups = offs ? G : 1;
  if (!size_ok(M) || !size_ok(N) || activation < MXQ_ACT_NONE || activation > MXQ_ACT_GELU) return MXQ_EBADSHAPE;
  if (N == 0 || (M == 0 && !dbias)) return MXQ_OK;
  const bool slope = activation != MXQ_ACT_NONE;
  if (M > 0 && (ld_dy < N || ld_dy > INT32_MAX || (slope && (ldz < N || ldz > INT32_MAX)) || (dz && (ld_dz < N || ld_dz > INT32_MAX))))
    return MXQ_EBADSHAPE;
  const int64_t need = dbias ? mxq_moe_linear_backward_workspace(M, N) : 0;
  if (need < 0 || M / kBlock * ceil_div(N, 8) > INT32_MAX || groups * (N / kBlock) > INT32_MAX || workspace_bytes < need) return MXQ_EBADSHAPE;
  if ((M > 0 && (!dy || (slope && !z))) || (need > 0 && !workspace)) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(dy, es) || !aligned_to(z, es) || !aligned_to(dz, es) || !aligned_to(offs, 4) || !aligned_to(dbias, 4) ||
      !aligned_to(workspace, 16))
    return MXQ_EALIGN;
  const ByteRange out[3] = {range_of(dz, pitched_bytes(M, N, ld_dz, es)), range_of(dbias, static_cast<uint64_t>(groups) * N * 4),
                            range_of(need > 0 ? workspace : nullptr, need)};
  const ByteRange in[3] = {dz && same_place(dy, ld_dy, dz, ld_dz) ? ByteRange{0, 0} : range_of(dy, pitched_bytes(M, N, ld_dy, es)),
                           range_of(slope ? z : nullptr, pitched_bytes(M, N, ldz, es)), range_of(offs, 4ull * G)};
  if (outputs_overlap(out, 3, in, 3)) return MXQ_EOVERLAP;
  if (!dz && !dbias) return MXQ_OK;
  Epilogue a = {};
  a.dy = dy;
  a.z = slope ? z : nullptr;
  a.dz = dz;
  a.offs = offs;
  a.parts = dbias ? reinterpret_cast<float*>(workspace) : nullptr;
  a.rows = static_cast<int32_t>(M), a.cols = static_cast<int32_t>(N), a.groups = static_cast<int32_t>(groups);
  a.ld_dy = ld_dy, a.ld_z = slope ? ldz : 0, a.ld_dz = dz ? ld_dz : 0;
  a.dy_bytes = pitched_bytes(M, N, ld_dy, es), a.z_bytes = in[1].bytes, a.dz_bytes = out[0].bytes;
  if (M > 0) {
    const int rc = dtype == MXQ_F32 ? launch_epilogue_typed<float>(activation, a, stream) : launch_epilogue_typed<bf16_t>(activation, a, stream);
    if (rc != MXQ_OK || !dbias) return rc;
  }
  return launch_pdl(bias_join_kernel, static_cast<unsigned>(groups * (N / kBlock)), 256, 0, stream, a.parts, offs, a.groups, a.rows, a.cols,
                    dbias);
}
