// orthogonalize.cu -- Newton-Schulz orthogonalisation of a momentum matrix (or
// of a stack of them) on the 5th-generation tensor cores.
//
//   X = g / (|g|_F + eps);  then `steps` times  X <- (aI + bA + cA^2) X  with
//   A = X X^T (X^T X on the other side for a matrix that is taller than wide)
//
// which drives the singular values towards 1.  A step is three products:
//   gram     A = X X^T, symmetric: the tiles of one triangle are computed and
//            stored twice, the second time transposed;
//   square   P = aI + bA + cA A, symmetric again; and
//   update   X <- P X (X P for a tall X).
// All operands are fp16 with fp32 accumulation in tensor memory.  fp16 and not
// bf16: both run at the same rate, the values are bounded (a spectral norm of
// about 1.2 for the usual coefficients, so no element is larger), and the three
// more mantissa bits make the rounding of an operand 2^-12 instead of 2^-9.
// Powers of two keep small elements out of fp16's subnormal range: X is stored
// times 2^13 (and more where |g| is far below eps, see Lift), A and P times powers
// taken from the coefficients' bounds.
//
// The square is completed: with S = A + (b/2c) I, which the gram product's
// epilogue stores in A's place, P = c S S + (a - b^2/4c) I, and the square reads no
// second matrix in its epilogue (64 fp32 matrices of 1024x512: 482 us, 501 with b A added
// from memory).  Where b/2c is large or c is zero (kCompletedSquare) it does.
//
// The rounding that matters is that of the diagonals of S (or A) and P, which hold
// most of their weight once the singular values draw together.  What fp16 leaves of
// them is kept in fp32 vectors and put back: of S as the remainder of its squares,
// onto the square's diagonal; of P as d X in the epilogue of P X = P'X + d X (and of
// A, where it is added, as A'A' + d A' + A'd + d d).  The result's error before its
// own rounding to bf16 (1.7e-3) is then 0.6e-3 to 1.1e-3, over square and long
// matrices alike; without S's part up to 1.8e-3, without either up to 2.5e-3.
// Putting back P's costs 2% with 1024x512 and 13% with 128x512.
// The iteration's map of a singular value has slopes of up to 1.6 around 1, and
// the value of a small matrix hangs on few roundings, so its error can reach 1%
// (sides up to 16 in a simulation; 0.14% from a side of 48 on).  Sides of at
// most kSplitSide therefore carry every matrix as a pair, its rounding to fp16
// and the rounding of what that leaves (22 bits in all), and every product is
// the sum of three: high times high, high times low and low times high.
//
// The product kernel: a pair of CTAs (cta_group::2) owns a 256x256 tile, each
// CTA 128 of its rows.  Stages of 64 along K are loaded by TMA with the 128-byte
// swizzle, operands that lie along the wrong axis (X in the wide update, X in the
// tall gram matrix) as MN-major boxes, so nothing is ever transposed in memory.
// One thread of the pair issues the MMAs; two accumulators of 256 tensor memory
// columns let the epilogue of a tile run under the next tile's products.  The
// grid is persistent, one CTA pair per two SMs.  Ragged edges are the tensor
// maps': loads fill with zero, stores are clipped.
//
// Bound, for large matrices: by the way of the operands from L2, 64 KB a stage and pair
// at about 55 bytes a clock and SM, where a stage's MMAs take 512 clocks and its loads
// 590 or more.  4096x8192 fp32 in five steps: 1.70 to 1.73 ms, 1.4 PFLOP/s of the
// products' one triangle, the tensor pipe active 69 to 75% (of 1.63 ms on the fastest
// GPU met, 1.19 with the loads left out, 1.39 with the MMAs left out).  64 matrices of
// 1024x512 bf16: 452 us, 0.66 PFLOP/s.  Their tiles of the update and of the square have
// 8 stages of K, 2.5 us of operands, but take 5.8 and 7 us: the rest is the epilogue
// (two chunks of a warp one after the other, each after the store before it), and 192
// and 512 tiles on 76 pairs leave part of the last round idle.  One small matrix: 17
// launches of 4 to 6 us, 0.1 of each for the exit that waits for the pair.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pair_drain.h"
#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_ortho_status = 0;

// ---------------------------------------------------------------------------
// norm and conversion
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kAhead = 4;        // loads a thread has in flight
constexpr int kMaxParts = 2048;  // partial sums of squares per matrix
constexpr float kXScale = 8192.0f;

struct Matrix {
  int64_t batch, m, n, ld, stride;  // rows ld, matrices stride elements apart
  int64_t last;                     // elements of the last row
};

// The norm of values anywhere in fp32's range.  A square of a value below 2^-75 is 0 in
// fp32 and one above 2^64 infinite, so the sum is held in three parts: of pieces whose
// largest value is below 2^-43, times 2^85 before they are squared; of those up to
// 2^43; and of larger ones, times 2^-86.  (What a piece loses of its smaller values is
// below 2^-63 of its largest square.)  Every part of up to 2^40 squares stays within
// 2^-128 and 2^126.  A piece is what a thread loads at once, so ordinary values cost one
// comparison each.
constexpr float kSmall = 0x1p-43f, kLarge = 0x1p43f, kSmallUp = 0x1p85f, kLargeDown = 0x1p-86f;
struct Squares {
  float small, plain, large;
};
// The norm as r / unit, unit a power of two.
struct Norm {
  float r, unit;
  __device__ __forceinline__ explicit Norm(const Squares& s) {
    const float lower = s.plain + s.small / kSmallUp / kSmallUp;
    // compared so that a NaN in any part reaches r
    if (!(s.large == 0.0f))
      r = sqrtf(s.large + lower * kLargeDown * kLargeDown), unit = kLargeDown;
    else if (!(s.plain == 0.0f))
      r = sqrtf(lower), unit = 1.0f;
    else
      r = sqrtf(s.small), unit = kSmallUp;
  }
};

// Where |g| is far below eps, X starts far below 1, and fp16 at a fixed scale would have
// no bits for it (|g| = 1e-14 with an eps of 1e-7: two steps of a subnormal).  Such a
// matrix's X is stored 2^h times larger, h = max(0, lift - drop): `lift`, by how many
// whole powers of two |g| + eps exceeds |g|, is the matrix's own, and `drop` grows with
// the steps by what a step can magnify at most.  So |X| 2^h stays at most 1, and X leaves
// the lift behind before it reaches the size of other matrices' X.  At most kMaxLift,
// with which the last product's factor is still a normal number.
constexpr int kMaxLift = 96;
struct Lift {
  const int32_t* of;            // [batch], or NULL: none
  int32_t drop_from, drop_to;   // of the X read and of the X written
  int32_t out_from, in_to;      // powers of 2^-h and 2^h in the product's factor
  int32_t batches;
  __device__ __forceinline__ float factor(int64_t batch) const {
    if (of == nullptr) return 1.0f;
    const int lift = read_at(of, batch, batches, 0, &g_ortho_status), from = max(0, lift - drop_from), to = max(0, lift - drop_to);
    const int e = in_to * to - out_from * from;  // at most 0: what is stored never grows in a product
    return __int_as_float(max(0, e + 127) << 23);
  }
};

// Blocks of a matrix take rows in turn; tx threads (a power of two) share a row.
// Where the matrix and X have no gaps between their rows, the rows are pieces of
// kThreads * kAhead loads instead (launch_scale).  Both kernels are bound by DRAM;
// what they need is loads in flight: with rows of 512 floats a thread had one.
template <typename T, int kV>
__global__ void __launch_bounds__(kThreads)
    norm_kernel(const T* __restrict__ g, const Matrix a, int parts, int tx, Squares* __restrict__ sums) {
  __shared__ float red[kThreads / 32][3];
  pdl_wait();
  const int64_t b = blockIdx.x / parts, part = blockIdx.x % parts;
  const int ty = kThreads / tx;
  const uint64_t bytes = ((a.batch - 1) * a.stride + (a.m - 1) * a.ld + a.last) * sizeof(T);
  Squares sum = {};
  for (int64_t r = part * ty + threadIdx.x / tx; r < a.m; r += static_cast<int64_t>(parts) * ty) {
    const T* row = g + b * a.stride + r * a.ld;
    const int64_t nv = (r == a.m - 1 ? a.last : a.n) / kV;
    if (!in_buf(row, nv * kV * sizeof(T), g, bytes, &g_ortho_status)) continue;
    for (int64_t c = threadIdx.x % tx; c < nv; c += kAhead * tx) {
      Vec<T, kV> v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        v[q] = c + q * tx < nv ? *reinterpret_cast<const Vec<T, kV>*>(row + (c + q * tx) * kV) : Vec<T, kV>{};
      float most = 0.0f;
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int j = 0; j < kV; ++j) most = fmaxf(most, fabsf(widen(v[q].v[j])));
      const auto squares = [&](float unit, float& to) {
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
#pragma unroll
          for (int j = 0; j < kV; ++j) to = fmaf(widen(v[q].v[j]) * unit, widen(v[q].v[j]) * unit, to);
      };
      if (most >= kSmall && most <= kLarge)
        squares(1.0f, sum.plain);
      else if (most > kLarge)
        squares(kLargeDown, sum.large);
      else
        squares(kSmallUp, sum.small);
    }
  }
  sum = {warp_sum(sum.small), warp_sum(sum.plain), warp_sum(sum.large)};
  if ((threadIdx.x & 31) == 0) {
    float* own = red[threadIdx.x >> 5];
    own[0] = sum.small, own[1] = sum.plain, own[2] = sum.large;
  }
  __syncthreads();
  if (threadIdx.x < 3) {  // a thread for each part
    float all = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) all += red[w][threadIdx.x];
    write_at(reinterpret_cast<float*>(sums), 3 * static_cast<int64_t>(blockIdx.x) + threadIdx.x, 3 * static_cast<int64_t>(gridDim.x),
             all, &g_ortho_status);
  }
}

template <typename T, int kV>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const T* __restrict__ g, const Matrix a, int parts, int tx, const Squares* __restrict__ sums, float eps,
                 int32_t* __restrict__ lifts, __half* __restrict__ x, __half* __restrict__ x_low, int64_t ldx, int64_t stride_x) {
  __shared__ float shared_unit, shared_factor;
  pdl_wait();
  const int64_t b = blockIdx.x / parts, part = blockIdx.x % parts;
  const int ty = kThreads / tx;
  if (threadIdx.x < 32) {
    Squares s = {};
    for (int i = threadIdx.x; i < parts; i += 32) {
      const Squares part_sums = read_at(sums, b * parts + i, gridDim.x, Squares{}, &g_ortho_status);
      s.small += part_sums.small, s.plain += part_sums.plain, s.large += part_sums.large;
    }
    s = {warp_sum(s.small), warp_sum(s.plain), warp_sum(s.large)};
    if (threadIdx.x == 0) {
      const Norm norm(s);
      shared_unit = norm.unit;
      // (|g| + eps) / |g|, without the overflow of eps in units of a small norm
      const float over = 1.0f + eps / norm.r * norm.unit;
      const bool lifted = norm.r > 0.0f && over >= 2.0f;
      const int lift = lifted ? min((__float_as_int(over) >> 23) - 127, kMaxLift) : 0;  // its exponent; infinity: the most
      const float less = __int_as_float((127 - lift) << 23);
      shared_factor = kXScale / (lifted ? norm.r * (over * less) : norm.r + eps * norm.unit);
      if (part == 0) write_at(lifts, b, a.batch, lift, &g_ortho_status);
    }
  }
  __syncthreads();
  const float unit = shared_unit, f = shared_factor;
  const uint64_t in_bytes = ((a.batch - 1) * a.stride + (a.m - 1) * a.ld + a.last) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>((a.batch - 1) * stride_x + (a.m - 1) * ldx + a.last) * 2;
  for (int64_t r = part * ty + threadIdx.x / tx; r < a.m; r += static_cast<int64_t>(parts) * ty) {
    const T* row = g + b * a.stride + r * a.ld;
    __half* to = x + b * stride_x + r * ldx;
    const int64_t nv = (r == a.m - 1 ? a.last : a.n) / kV;
    if (!in_buf(row, nv * kV * sizeof(T), g, in_bytes, &g_ortho_status) ||
        !in_buf(to, nv * kV * 2, x, out_bytes, &g_ortho_status))
      continue;
    for (int64_t c = threadIdx.x % tx; c < nv; c += kAhead * tx) {
      Vec<T, kV> v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        v[q] = c + q * tx < nv ? *reinterpret_cast<const Vec<T, kV>*>(row + (c + q * tx) * kV) : Vec<T, kV>{};
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (c + q * tx >= nv) continue;
        __half* at = to + (c + q * tx) * kV;
        Vec<uint16_t, kV> o;
#pragma unroll
        for (int j = 0; j < kV; ++j) o.v[j] = __half_as_ushort(__float2half_rn(widen(v[q].v[j]) * unit * f));
        *reinterpret_cast<Vec<uint16_t, kV>*>(at) = o;
        if (x_low == nullptr) continue;
#pragma unroll
        for (int j = 0; j < kV; ++j)
          o.v[j] = __half_as_ushort(__float2half_rn(widen(v[q].v[j]) * unit * f - __half2float(__ushort_as_half(o.v[j]))));
        if (in_buf(x_low + (at - x), sizeof o, x_low, out_bytes, &g_ortho_status))
          *reinterpret_cast<Vec<uint16_t, kV>*>(x_low + (at - x)) = o;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the product kernel
// ---------------------------------------------------------------------------
constexpr int kTile = 256;                      // rows and columns of a CTA pair's tile
constexpr int kHalf = 128;                      // rows of A and of B that one CTA loads
constexpr int kStepK = 64;                      // elements of K per stage: one 128-byte swizzle row
constexpr int kOperandBytes = kHalf * kStepK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 5;
constexpr int kAccCols = 256;                   // tensor memory columns of one accumulator
constexpr int kChunkCols = 64;                  // columns an epilogue warp stages at a time
constexpr int kStagingBytes = 32 * kChunkCols * 2;
constexpr int kEpilogueWarps = 8;               // two for each 32 rows, each half of the columns
constexpr int kWarpChunks = kTile / kChunkCols / 2;  // and as many staging buffers per warp
constexpr int kGemmThreads = 128 + 32 * kEpilogueWarps;  // producer, MMA, allocation, idle; epilogue
constexpr int kGemmSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kWarpChunks * kStagingBytes;
static_assert(kWarpChunks == 2, "the epilogue pairs its two buffers");

struct Maps {
  CUtensorMap a[2], b[2];  // operands, high and low parts
  CUtensorMap d[2];        // output, high and low parts: boxes of 64 columns x 32 rows
  CUtensorMap add[2];      // addend, the same
  CUtensorMap dt;          // the high part's transpose: boxes of 32 columns x 64 rows
};

struct Product {
  int64_t rows, cols;      // of the output
  int32_t ksteps;          // stages along K of one product
  int32_t tiles_m, tiles_n, tiles;  // tiles: all of the batch and of the slices
  int32_t slices, per_slice;        // K in slices of that many stages, each summed by itself
  float* partial;                   // [slices, batch, rows, d_ld] sums of the slices, or NULL
  int64_t partial_stride;           // elements between the slices
  int32_t a_mn, b_mn;      // operand lies with K along its rows
  // output = scale * acc + (add_scale + scale * (d[row] + d[column])) * addend
  //          and where row == column, + diagonal + add_scale * d + scale * d * d
  float scale, add_scale, diagonal;
  int64_t d_count;                  // batch * d_ld
  const float *d_row, *d_col;       // [batch, d_ld]: what the rounding left of a diagonal; NULL: zero
  float* d_out;                     // the same of this output's diagonal, or NULL;
  int32_t d_squares;                // of the squares of its diagonal instead
  const float* square_rest;         // [batch, d_ld] such squares' remainders: times scale, onto the diagonal; or NULL
  int64_t d_ld;
  // the last update writes bf16 to the caller's matrix
  bf16_t* out;             // NULL: fp16 through map d
  int64_t ldo, stride_o;
  int32_t out_map;         // bf16 through map d
  Lift lift;               // in `scale`
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) { return at_rank(addr, 0); }
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  // relaxed: what it orders are tensor memory reads, by their own fence; a release
  // at cluster scope would wait for the stores before it (2 us a tile, measured)
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Load of a box whose bytes are counted by a barrier of the pair's leader.
__device__ __forceinline__ void load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on the barrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b16 both;\n\tmov.b16 both, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(bar)
      : "memory");
}
// The same in this CTA alone.
__device__ __forceinline__ void commit_here(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc;\n\tsetp.ne.b32 acc, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, acc;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load_32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}

// Shared-memory descriptor of a swizzled operand (128-byte swizzle, version 1).
// K-major: rows of 128 bytes, 1024 bytes between groups of 8 rows.  MN-major:
// boxes of 64 K-rows of 128 bytes; 8192 bytes between boxes along M or N, 1024
// between groups of 8 K-rows.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
  const uint64_t lead = mn ? (64 * 128) >> 4 : 1;
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (lead << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, fp16 operands, 256 rows, n columns.
__device__ __forceinline__ uint32_t instruction_desc(bool a_mn, bool b_mn, uint32_t n) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((n / 8u) << 17) | ((kTile / 16u) << 24);
}
// Columns that a tile's MMAs compute, half of them from each CTA's B: a multiple of
// 128 (64 a CTA, the width of an MN-major box), as few as the matrix has left.
__device__ __forceinline__ int32_t tile_width(const Product& p, int32_t j) {
  const int64_t left = p.cols - static_cast<int64_t>(j) * kTile;
  return left > kTile / 2 ? kTile : kTile / 2;
}

struct TileAt {
  int32_t batch, i, j;  // matrix, tile row, tile column
  int32_t slice;
};
template <bool kSymmetric>
__device__ __forceinline__ TileAt tile_at(const Product& p, int t) {
  const int all = p.tiles / p.slices, slice = t / all;
  t -= slice * all;
  if (!kSymmetric) {
    const int per = p.tiles_m * p.tiles_n;
    const int r = t % per;
    return {t / per, r % p.tiles_m, r / p.tiles_m, slice};
  }
  const int per = p.tiles_m * (p.tiles_m + 1) / 2;
  const int r = t % per;
  int i = static_cast<int>((sqrtf(8.0f * r + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > r) --i;
  while ((i + 1) * (i + 2) / 2 <= r) ++i;
  return {t / per, i, r - i * (i + 1) / 2, slice};
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_values(uint32_t bits) {
  return __half22float2(*reinterpret_cast<const __half2*>(&bits));
}
__device__ __forceinline__ uint32_t bf162_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct alignas(8) Barriers {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint64_t addend[kEpilogueWarps][kWarpChunks];
  uint64_t drained;        // the leader's: its MMAs are done, after a wait that ran out
  uint32_t tmem, abort_flag;
  uint32_t leader_gave_up, issued[2];  // by the leader; to the leader: stages each CTA has issued
};

__device__ __forceinline__ float half_rounded(float v) { return __half2float(__float2half_rn(v)); }
// What rounding to fp16 leaves of v, or of its square.
__device__ __forceinline__ float diagonal_rest(float v, bool square) {
  const float h = half_rounded(v);
  return square ? (v - h) * (v + h) : v - h;
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&v)[8]) {
  const float2 a = half2_values(w.x), b = half2_values(w.y), c = half2_values(w.z), d = half2_values(w.w);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

// kSymmetric: one triangle of tiles, stored twice.  kAddends: parts of the
// addend.  kColumns: the columns' d_col multiplies it (d_row, where given, always
// does).  kBf16: the last update, to the caller's matrix.  kSplit: operands and
// results are pairs, three products.  kPartial: the sums of a slice of K, in fp32.
template <bool kSymmetric, int kAddends, bool kColumns, bool kBf16, bool kSplit, bool kPartial>
__global__ void __launch_bounds__(kGemmThreads, 1) __cluster_dims__(2, 1, 1)
    product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Product p) {
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bars;
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t staging = smem + kStages * kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  volatile uint32_t* abort_flag = &bars.abort_flag;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bars.full[s]), 1);
      mbar_init(smem_u32(&bars.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars.acc_full[s]), 1);
      mbar_init(smem_u32(&bars.acc_empty[s]), 2 * kEpilogueWarps);  // of both CTAs
    }
    for (int w = 0; w < kEpilogueWarps; ++w)
      for (int c = 0; c < kWarpChunks; ++c) mbar_init(smem_u32(&bars.addend[w][c]), 1);
    mbar_init(smem_u32(&bars.drained), 1);
    bars.abort_flag = bars.leader_gave_up = 0u;
    mbar_init_fence();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  __syncthreads();
  cluster_sync_all();  // both CTAs of the pair run, with their barriers set up
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync_all();
  fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int ksteps = kSplit ? 3 * p.ksteps : p.ksteps;
  if (warp == 0 && lane == 0) {
    // ---- producer: this CTA's half of A and of B -------------------------
    int issued = 0;  // stages loaded so far
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += step) {
      const TileAt at = tile_at<kSymmetric>(p, t);
      const int32_t ra = at.i * kTile + static_cast<int32_t>(rank) * kHalf;
      const int32_t rb = at.j * kTile + static_cast<int32_t>(rank) * (tile_width(p, at.j) / 2);
      const int k_end = min(ksteps, (at.slice + 1) * p.per_slice);
      for (int kk = at.slice * p.per_slice; kk < k_end; ++kk, ++issued) {
        const int part = kk / p.ksteps, k = (kk - part * p.ksteps) * kStepK;  // high*high, high*low, low*high
        const CUtensorMap* map_a = &maps.a[part == 2];
        const CUtensorMap* map_b = &maps.b[part == 1];
        const int s = issued % kStages;
        const uint32_t round = issued / kStages;
        if (!mbar_wait_bounded(smem_u32(&bars.empty[s]), (round & 1) ^ 1, abort_flag, &g_ortho_status, MXQ_DEV_TIMEOUT)) {
          ok = false;
          break;
        }
        const uint32_t bar = at_leader(smem_u32(&bars.full[s]));
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.full[s]), 2 * kStageBytes);
        const uint32_t da = smem + s * kStageBytes, db = da + kOperandBytes;
        if (p.a_mn) {
          load_3d_pair(da, map_a, ra, k, at.batch, bar);
          load_3d_pair(da + kOperandBytes / 2, map_a, ra + 64, k, at.batch, bar);
        } else {
          load_3d_pair(da, map_a, k, ra, at.batch, bar);
        }
        if (p.b_mn) {
          load_3d_pair(db, map_b, rb, k, at.batch, bar);
          load_3d_pair(db + kOperandBytes / 2, map_b, rb + 64, k, at.batch, bar);
        } else {
          load_3d_pair(db, map_b, k, rb, at.batch, bar);
        }
      }
    }
    store_cluster(at_leader(smem_u32(&bars.issued[rank])), static_cast<uint32_t>(issued));
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issue for the pair -------------------------------------------
    const uint64_t step_a = (p.a_mn ? 16 * 128 : 32) >> 4, step_b = (p.b_mn ? 16 * 128 : 32) >> 4;  // 16 of K
    int n = 0, done = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += step, ++done) {
      const int acc = done & 1;
      const TileAt at = tile_at<kSymmetric>(p, t);
      const uint32_t idesc = instruction_desc(p.a_mn, p.b_mn, static_cast<uint32_t>(tile_width(p, at.j)));
      const int count = min(ksteps, (at.slice + 1) * p.per_slice) - at.slice * p.per_slice;
      ok = mbar_wait_bounded(smem_u32(&bars.acc_empty[acc]), ((done >> 1) & 1) ^ 1, abort_flag, &g_ortho_status, MXQ_DEV_TIMEOUT);
      fence_after();
      for (int k = 0; ok && k < count; ++k, ++n) {
        const int s = n % kStages;
        ok = mbar_wait_bounded(smem_u32(&bars.full[s]), (n / kStages) & 1, abort_flag, &g_ortho_status, MXQ_DEV_TIMEOUT);
        if (!ok) break;
        fence_after();
        const uint64_t da = operand_desc(smem + s * kStageBytes, p.a_mn);
        const uint64_t db = operand_desc(smem + s * kStageBytes + kOperandBytes, p.b_mn);
#pragma unroll
        for (int q = 0; q < kStepK / 16; ++q)
          mma_pair(tmem + acc * kAccCols, da + q * step_a, db + q * step_b, idesc, (k | q) != 0);
        commit_pair(smem_u32(&bars.empty[s]));
      }
      if (ok) commit_pair(smem_u32(&bars.acc_full[acc]));
    }
    if (!ok) {  // products under way read both CTAs' stages and write their tensor memory
      commit_here(smem_u32(&bars.drained));
      mbar_wait_drain(smem_u32(&bars.drained), 0);
    }
  } else if (warp >= 4) {
    // ---- epilogue: 32 of this CTA's 128 rows and half of the columns per warp --
    // The addend is loaded into the buffers that the results are staged in and
    // replaced piece by piece; the next tile's is loaded while this one's results
    // leave.  Without a second result the two chunks of a warp have a buffer each;
    // with one (the transposed block or the low parts) a chunk takes both.
    const int e = warp - 4, quarter = e & 3;
    const uint32_t buf0 = staging + (2 * e) * kStagingBytes, buf1 = buf0 + kStagingBytes;
    const uint32_t bar0 = smem_u32(&bars.addend[e][0]);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    constexpr bool low = kSplit && !kBf16 && !kPartial;  // a split side has one tile: never mirrored
    // a tile of the diagonal has no transposed block to store, and uses both
    // buffers like one of an ordinary product
    const auto needs_both = [&](const TileAt& at) { return low || (kSymmetric && at.i != at.j); };
    uint32_t phases = 0u, flying = 0u;             // a bit per buffer: parity to wait for, addend in flight
    const auto load_addend = [&](int b, int part, const TileAt& at, int c) {  // lane 0 issues; all lanes keep count
      const int32_t row0 = at.i * kTile + static_cast<int32_t>(rank) * kHalf + quarter * 32;
      const int32_t col0 = at.j * kTile + (2 * (e >> 2) + c) * kChunkCols;
      if (row0 >= p.rows || col0 >= p.cols) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar0 + 8 * b, kStagingBytes);
        load_3d(buf0 + b * kStagingBytes, &maps.add[part], col0, row0, at.batch, bar0 + 8 * b);
      }
      flying |= 1u << b;
    };
    const auto wait_addend = [&](int b) {
      const bool got = mbar_wait_bounded(bar0 + 8 * b, (phases >> b) & 1, abort_flag, &g_ortho_status, MXQ_DEV_TIMEOUT);
      if (!__all_sync(0xFFFFFFFFu, got)) return false;
      flying &= ~(1u << b);
      phases ^= 1u << b;
      return true;
    };
    int done = 0;
    bool ok = true;
    // a tile's addend, as far as there are buffers for it
    const auto load_addends = [&](const TileAt& at) {
      if (kAddends == 1) {
        load_addend(0, 0, at, 0);
        if (!needs_both(at)) load_addend(1, 0, at, 1);
      }
      if (kAddends == 2) {
        load_addend(0, 0, at, 0);
        load_addend(1, 1, at, 0);
      }
    };
    if (first < p.tiles) load_addends(tile_at<kSymmetric>(p, first));
    for (int t = first; ok && t < p.tiles; t += step, ++done) {
      const TileAt at = tile_at<kSymmetric>(p, t);
      const int acc = done & 1;
      const int64_t row0 = static_cast<int64_t>(at.i) * kTile + rank * kHalf + quarter * 32;
      const int64_t row = row0 + lane;
      const bool mirror = kSymmetric && at.i != at.j, both = needs_both(at) || kAddends == 2;
      const float scale = p.scale * p.lift.factor(at.batch);
      const float dr = p.d_row != nullptr && row < p.rows
                           ? read_at(p.d_row, at.batch * p.d_ld + row, p.d_count, 0.0f, &g_ortho_status) : 0.0f;
      if (kColumns && lane < 4) {  // this warp's 128 columns, four lines
        const int64_t col = static_cast<int64_t>(at.j) * kTile + 2 * (e >> 2) * kChunkCols + 32 * lane;
        if (col < p.cols) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.d_col + at.batch * p.d_ld + col));
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(&bars.acc_full[acc]), (done >> 1) & 1, abort_flag,
                                                     &g_ortho_status, MXQ_DEV_TIMEOUT));
      if (!ok) break;
      fence_after();
#pragma unroll 1
      for (int c = 0; c < kWarpChunks; ++c) {
        const int tile_col = (2 * (e >> 2) + c) * kChunkCols;
        const int64_t col0 = static_cast<int64_t>(at.j) * kTile + tile_col;
        const bool inside = row0 < p.rows && col0 < p.cols;
        const uint32_t buf = both || c == 0 ? buf0 : buf1;
        if (inside) {
          if (both && kAddends > 0) {
            if (c > 0) {
              if (lane == 0) bulk_wait_read<0>();
              __syncwarp();
              for (int q = 0; q < kAddends; ++q) load_addend(q, q, at, c);
            }
          } else if (kAddends == 0 && !kPartial) {
            if (lane == 0) {
              if (both || c == 0)
                bulk_wait_read<0>();
              else
                bulk_wait_read<1>();  // the first chunk's store may still read the other buffer
            }
            __syncwarp();
          }
          for (int q = 0; ok && q < kAddends; ++q) ok = wait_addend(kAddends == 2 ? q : both ? 0 : c);
          if (!ok) break;
        }
        if (!inside && c < kWarpChunks - 1) continue;
        // everything of the chunk is read before anything is written: the
        // accesses are volatile and keep their order
        uint32_t raw[2][32];
        tmem_load_32(lanes + acc * kAccCols + tile_col, raw[0]);
        tmem_load_32(lanes + acc * kAccCols + tile_col + 32, raw[1]);
        uint4 a4[8], l4[8];
        const auto piece = [&](int q) { return lane * 128 + ((q ^ (lane & 7)) << 4); };  // the 128-byte swizzle
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (kAddends > 0) a4[q] = lds128(buf + piece(q));
          if (kAddends == 2) l4[q] = lds128(buf1 + piece(q));
        }
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (c == kWarpChunks - 1) {  // this warp is done with the accumulator
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(at_leader(smem_u32(&bars.acc_empty[acc])));
        }
        if (!inside) continue;
        const auto store_partial = [&] {
          if (!kPartial) return false;
          float* to = p.partial + at.slice * p.partial_stride + (static_cast<int64_t>(at.batch) * p.rows + row) * p.d_ld + col0;
          const uint64_t bytes = static_cast<uint64_t>(p.slices) * p.partial_stride * 4;
          if (row < p.rows)
#pragma unroll
            for (int i = 0; i < 64; i += 4)
              if (col0 + i < p.d_ld && in_buf(to + i, 16, p.partial, bytes, &g_ortho_status))  // d_ld: a multiple of 8
                *reinterpret_cast<uint4*>(to + i) =
                    make_uint4(raw[i / 32][i % 32], raw[i / 32][i % 32 + 1], raw[i / 32][i % 32 + 2], raw[i / 32][i % 32 + 3]);
          return true;
        };
        if (store_partial()) continue;
        const float k0 = fmaf(scale, dr, p.add_scale);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 32 columns at a time
          const int64_t col = col0 + 32 * h;
          float4 dc[8];
          if (kColumns) {
            const float4* d = reinterpret_cast<const float4*>(p.d_col + at.batch * p.d_ld + col);
#pragma unroll
            for (int q = 0; q < 8; ++q)  // d_ld is a multiple of 8
              dc[q] = col + 4 * q < p.cols && in_buf(d + q, 16, p.d_col, static_cast<uint64_t>(p.d_count) * 4, &g_ortho_status)
                          ? d[q] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[h][i]) * scale;
          if (kAddends > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float a[8];
              unpack8(a4[4 * h + q], a);
              if (kAddends == 2) {
                float l[8];
                unpack8(l4[4 * h + q], l);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] += l[i];
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 d = dc[2 * q + i / 4];
                const float k = kColumns ? fmaf(scale, i % 4 == 0 ? d.x : i % 4 == 1 ? d.y : i % 4 == 2 ? d.z : d.w, k0) : k0;
                v[8 * q + i] = fmaf(k, a[i], v[8 * q + i]);
              }
            }
          }
          if (kSymmetric && row0 < col + 32 && col < row0 + 32) {  // the warp's rows meet these columns
            const int own_column = static_cast<int>(row - col);
            float on = p.diagonal + p.add_scale * dr + scale * dr * dr;
            if (p.square_rest != nullptr && row < p.rows)
              on = fmaf(scale, read_at(p.square_rest, at.batch * p.d_ld + row, p.d_count, 0.0f, &g_ortho_status), on);
            float own = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] += i == own_column ? on : 0.0f;
              own = i == own_column ? v[i] : own;
            }
            if (!kSplit && p.d_out != nullptr && own_column >= 0 && own_column < 32 && row < p.rows)
              write_at(p.d_out, at.batch * p.d_ld + row, p.d_count, diagonal_rest(own, p.d_squares), &g_ortho_status);
          }
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = kBf16 ? bf162_bits(v[2 * i], v[2 * i + 1]) : half2_bits(v[2 * i], v[2 * i + 1]);
#pragma unroll
          for (int q = 0; q < 4; ++q) sts128(buf + piece(4 * h + q), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          if (mirror) {  // transposed: 64 rows of this warp's 32 rows
#pragma unroll
            for (int i = 0; i < 32; ++i)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(buf1 + (32 * h + i) * 64 + lane * 2),
                           "h"(static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu))
                           : "memory");
          }
          if (low) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = half2_bits(v[2 * i] - half_rounded(v[2 * i]), v[2 * i + 1] - half_rounded(v[2 * i + 1]));
#pragma unroll
            for (int q = 0; q < 4; ++q) sts128(buf1 + piece(4 * h + q), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          }
        }
        if (kBf16 && !p.out_map) {
          // a matrix whose pitch or address no tensor map takes, or rows of part of a
          // 16-byte piece
          __syncwarp();
          bf16_t* out = p.out + at.batch * p.stride_o;
          const uint64_t bytes = ((p.rows - 1) * p.ldo + p.cols) * 2;
          for (int r = 0; r < 32 && row0 + r < p.rows; ++r)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int i = 32 * half + lane;
              uint16_t value;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(value) : "r"(buf + r * 128 + ((((i >> 3) ^ (r & 7)) << 4) | ((i & 7) * 2))));
              bf16_t* to = out + (row0 + r) * p.ldo + col0 + i;
              if (col0 + i < p.cols && in_buf(to, 2, out, bytes, &g_ortho_status)) *to = value;
            }
          fence_proxy_async_smem();  // read before the next addend comes in
          __syncwarp();
          continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int32_t r0 = static_cast<int32_t>(row0), c0 = static_cast<int32_t>(col0);
          store_3d(&maps.d[0], c0, r0, at.batch, buf);
          if (mirror) store_3d(&maps.dt, r0, c0, at.batch, buf1);
          if (low) store_3d(&maps.d[1], c0, r0, at.batch, buf1);
          bulk_commit();
        }
      }
      if (ok && kAddends > 0 && t + step < p.tiles) {
        const TileAt next = tile_at<kSymmetric>(p, t + step);
        // the first chunk's store has been read once at most the second's is left
        const bool second = (static_cast<int64_t>(at.j) * kTile + (2 * (e >> 2) + 1) * kChunkCols) < p.cols;
        if (kSymmetric || kAddends == 2 || !second) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          load_addends(next);
        } else {
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          load_addend(0, 0, next, 0);
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          load_addend(1, 0, next, 1);
        }
      }
    }
    for (int b = 0; b < 2; ++b)  // after a wait that ran out
      if (flying >> b & 1u) mbar_wait_drain(bar0 + 8 * b, (phases >> b) & 1);
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
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
        const uint32_t bar = smem_u32(&bars.full[n % kStages]);
        if (pair_unannounced(n, own)) mbar_arrive_expect_tx(bar, kStageBytes);
        if (pair_half_missing(n, peer)) mbar_complete_tx(bar, kStageBytes);
        mbar_wait_drain(bar, (n / kStages) & 1);
      }
    }
    __syncthreads();
    cluster_sync_all();
  }
  __syncthreads();
  fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The slices' sums added up in order: A (fp16, its low part or its diagonal's
// remainder) from the lower triangle of tiles.
struct Join {
  const float* partial;
  int64_t batch, side, ld, stride;
  int slices;
  float scale, diagonal;
  Lift lift;
  __half *high, *low;
  float* d_out;  // or NULL
  int32_t d_squares;
};
__global__ void __launch_bounds__(kThreads) join_kernel(const Join a) {
  pdl_wait();
  const int64_t n = a.batch * a.side * a.ld;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= n) return;
  const int64_t j = at % a.ld, row = at / a.ld, i = row % a.side;
  if (j >= a.side) return;
  const float* p = a.partial + (i / kTile >= j / kTile ? at : (row - i + j) * a.ld + i);
  float sum = 0.0f;
#pragma unroll 8
  for (int s = 0; s < a.slices; ++s) sum += read_at(a.partial, p - a.partial + s * a.stride, a.slices * a.stride, 0.0f, &g_ortho_status);
  const float v = sum * (a.scale * a.lift.factor(row / a.side)) + (i == j ? a.diagonal : 0.0f), h = half_rounded(v);
  write_at(a.high, at, n, __float2half_rn(v), &g_ortho_status);
  if (a.low != nullptr)
    write_at(a.low, at, n, __float2half_rn(v - h), &g_ortho_status);
  else if (i == j && a.d_out != nullptr)
    write_at(a.d_out, row / a.side * a.ld + i, a.batch * a.ld, diagonal_rest(v, a.d_squares), &g_ortho_status);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// The square is completed where |b| is at most this many |c|, so that |b/2c| stays
// within the bound of A: beyond it the rounding of S would be that of the shift.
// (Completed and not, fp32: 16x16 74 and 80 us, 200 matrices of 128x512 237 and 258, 64
// of 1024x512 482 and 501, 4096x8192 1632 and 1644.)
constexpr float kCompletedSquare = 4.0f;
// Sides up to this carry pairs of fp16 (see the head of the file).
constexpr int64_t kSplitSide = 64;

// Slices of K for the gram matrix: where its tiles are few and K is long, the CTA
// pairs left over take slices of K, and a further launch adds the slices up.
// A stage takes a pair 0.3 us, a slice's sums pass through L2 twice at 4 TB/s, and
// the further launch costs 5 us (64x8192: 661 us with one slice, 128 with 64, the
// choice here; 512x8192: 321 and 212; 300x5000: 236 and 154; 1000x2000: 209 us with
// one, the choice, and 234 with two).  Returns 0 for one slice.  Sized for the pairs of the whole GPU, whatever it has.
// K is sliced in any case after kMostStages: the tensor cores' additions to an fp32
// accumulator cut off what does not fit, a third of a unit in the last place on
// average, and the diagonal's sum of squares loses that with every 16 of K (0.8% of the
// result for 1 x 2^20 in one slice).  512 stages lose 9e-5 of it.  (4096x65536 pays 7%
// for its two slices' way through memory: 11.7 ms, 10.9 in one; others nothing.)
constexpr int64_t kPairs = 76, kSliceStages = 6, kMostStages = 512;
int64_t gram_slices(int64_t batch, int64_t side, int64_t length) {
  const int64_t tiles_m = ceil_div(side, kTile), tiles = batch * tiles_m * (tiles_m + 1) / 2;
  if (tiles == 0) return 0;
  const int64_t stages = ceil_div(length, kStepK) * (side <= kSplitSide ? 3 : 1);
  const double product_us = 0.3 * static_cast<double>(stages);
  const double slice_us = 8.0 * static_cast<double>(batch * side * side) / 4.0e6;
  int64_t most = kPairs / tiles;
  if (most > stages / kSliceStages) most = stages / kSliceStages;
  const int64_t least = ceil_div(stages, kMostStages);
  int64_t best = least > 1 ? least : 0;
  const auto us_of = [&](int64_t n) {
    return product_us / static_cast<double>(n) + slice_us * static_cast<double>(n) + 5.0;
  };
  double best_us = best > 0 ? us_of(best) : product_us;
  for (int64_t n = least > 2 ? least : 2; n <= most; ++n) {
    const double us = us_of(n);
    if (us < best_us) best = n, best_us = us;
  }
  return best;
}

struct Layout {
  int64_t side, ldx, lds;            // pitches of X and of the square matrices
  int parts;                         // 2 with low parts
  int64_t x[2][2];                   // X of the even and of the odd steps: high, low
  int64_t gram[2], poly[2];
  int64_t d_gram, d_poly, sums, lifts, partial, bytes;
};
Layout layout_of(int64_t batch, int64_t m, int64_t n) {
  Layout l;
  const auto up = [](int64_t v, int64_t to) { return ceil_div(v, to) * to; };
  l.side = m < n ? m : n;
  l.ldx = up(n, 8);
  l.lds = up(l.side, 8);
  l.parts = l.side <= kSplitSide ? 2 : 1;
  const int64_t xb = up(batch * m * l.ldx * 2, 256), sb = up(batch * l.side * l.lds * 2, 256);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) { return (at += bytes) - bytes; };
  for (int q = 0; q < 2; ++q) {
    const bool there = q < l.parts;
    l.x[0][q] = take(there ? xb : 0);
    l.x[1][q] = take(there ? xb : 0);
    l.gram[q] = take(there ? sb : 0);
    l.poly[q] = take(there ? sb : 0);
  }
  l.d_gram = take(up(batch * l.lds * 4, 256));
  l.d_poly = take(up(batch * l.lds * 4, 256));
  l.sums = take(up(batch * kMaxParts * static_cast<int64_t>(sizeof(Squares)), 256));
  l.lifts = take(up(batch * 4, 256));
  l.partial = take(up(gram_slices(batch, l.side, l.side == m ? n : m) * batch * l.side * l.lds * 4, 256));
  l.bytes = at;
  return l;
}

struct Stack {  // [batch, rows, cols] with pitch ld
  void* base;
  int64_t batch, rows, cols, ld, stride;
};

bool encode(CUtensorMap* map, const Stack& t, CUtensorMapDataType type, uint32_t box_cols, uint32_t box_rows, bool swizzle) {
  const auto fn = driver_tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows), static_cast<cuuint64_t>(t.batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(t.ld) * 2, static_cast<cuuint64_t>(t.stride) * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1}, ones[3] = {1, 1, 1};
  return fn(map, type, 3, t.base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_half(CUtensorMap* map, const Stack& t, uint32_t box_cols, uint32_t box_rows, bool swizzle) {
  return encode(map, t, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, box_cols, box_rows, swizzle);
}

template <bool kSymmetric, int kAddends, bool kColumns, bool kBf16, bool kSplit, bool kPartial>
int launch_product(const Maps& maps, Product p, int64_t batch, int sms, cudaStream_t stream) {
  p.tiles_m = static_cast<int32_t>(ceil_div(p.rows, kTile));
  p.tiles_n = static_cast<int32_t>(ceil_div(p.cols, kTile));
  const int64_t per = kSymmetric ? static_cast<int64_t>(p.tiles_m) * (p.tiles_m + 1) / 2
                                 : static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (p.slices == 0) {
    p.slices = 1;
    p.per_slice = INT32_MAX / 2;
  }
  p.tiles = static_cast<int32_t>(per * batch * p.slices);
  const auto kernel = product_kernel<kSymmetric, kAddends, kColumns, kBf16, kSplit, kPartial>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem) != cudaSuccess)
      return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  const int pairs = sms / 2 < p.tiles ? sms / 2 : p.tiles;
  return launch_pdl(kernel, 2 * pairs, kGemmThreads, kGemmSmem, stream, maps, p);
}

// The largest power of two that keeps values up to `bound` within half of fp16's range.
float scale_for(double bound) {
  int e = static_cast<int>(floor(log2(32768.0 / (bound > 1e-30 ? bound : 1e-30))));
  if (e > 13) e = 13;
  if (e < -60) e = -60;
  return static_cast<float>(ldexp(1.0, e));
}

template <typename T, int kV>
int launch_scale(const void* g, Matrix a, float eps, uint8_t* ws, const Layout& l, int sms, cudaStream_t stream) {
  int64_t ldx = l.ldx;
  const int64_t stride_x = a.m * ldx;
  if (a.ld == a.n && ldx == a.n) {  // one run of elements, in pieces
    const int64_t total = a.m * a.n;
    a.n = a.ld = ldx = kThreads * kAhead * kV;
    a.m = ceil_div(total, a.n);
    a.last = total - (a.m - 1) * a.n;
  }
  const int64_t nv = (a.m > 1 ? a.n : a.last) / kV;
  int tx = 8;
  while (tx < kThreads && tx < nv) tx *= 2;
  int64_t parts = ceil_div(a.m, kThreads / tx);
  const int64_t most = ceil_div(static_cast<int64_t>(sms) * (2048 / kThreads), a.batch);
  if (parts > most) parts = most;
  if (parts > kMaxParts) parts = kMaxParts;
  const unsigned blocks = static_cast<unsigned>(a.batch * parts);
  Squares* sums = reinterpret_cast<Squares*>(ws + l.sums);
  const int rc = launch_pdl(norm_kernel<T, kV>, blocks, kThreads, 0, stream, static_cast<const T*>(g), a,
                            static_cast<int>(parts), tx, sums);
  if (rc != MXQ_OK) return rc;
  return launch_pdl(scale_kernel<T, kV>, blocks, kThreads, 0, stream, static_cast<const T*>(g), a,
                    static_cast<int>(parts), tx, sums, eps, reinterpret_cast<int32_t*>(ws + l.lifts),
                    reinterpret_cast<__half*>(ws + l.x[0][0]),
                    l.parts == 2 ? reinterpret_cast<__half*>(ws + l.x[0][1]) : nullptr, ldx, stride_x);
}
template <typename T>
int scale_vector(const void* g, const Matrix& a, float eps, uint8_t* ws, const Layout& l, int sms, cudaStream_t stream) {
  const uint64_t es = sizeof(T);
  const int v = common_alignment({address_of(g), a.n * es, a.ld * es, a.stride * es}) / static_cast<int>(es);
  if constexpr (sizeof(T) == 2)
    if (v >= 8) return launch_scale<T, 8>(g, a, eps, ws, l, sms, stream);
  return v >= 4   ? launch_scale<T, 4>(g, a, eps, ws, l, sms, stream)
         : v >= 2 ? launch_scale<T, 2>(g, a, eps, ws, l, sms, stream)
                  : launch_scale<T, 1>(g, a, eps, ws, l, sms, stream);
}

constexpr int64_t kMaxSide = int64_t{1} << 20;

int check_ortho_shape(int64_t batch, int64_t m, int64_t n) {
  if (batch < 0 || m < 0 || n < 0 || batch > 65535 || m > kMaxSide || n > kMaxSide) return MXQ_EBADSHAPE;
  // tiles of a launch within the kernels' counters: the square matrices', with K in slices
  // those of all slices, and X's; and the blocks that add slices up
  const int64_t side = m < n ? m : n, length = m < n ? n : m, slices = gram_slices(batch, side, length);
  const int64_t tiles = ceil_div(side, kTile);
  if (batch * tiles * tiles * (slices > 0 ? slices : 1) > INT32_MAX / 2 || batch * tiles * ceil_div(length, kTile) > INT32_MAX / 2 ||
      (slices > 0 && batch * side * (side + 7) / kThreads >= INT32_MAX))
    return MXQ_EBADSHAPE;
  return MXQ_OK;
}

}  // namespace

namespace mxq {
int ortho_status_read(unsigned int* out, bool clear) { return read_status_word(g_ortho_status, out, clear); }
int ortho_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int64_t mxq_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n) {
  if (check_ortho_shape(batch, m, n) != MXQ_OK) return MXQ_EBADSHAPE;
  return layout_of(batch, m, n).bytes;
}

extern "C" int mxq_orthogonalize(const void* g, int dtype, int64_t batch, int64_t m, int64_t n, int64_t ld,
                                 int64_t stride, int32_t steps, float ca, float cb, float cc, float eps, float scale,
                                 void* out, int64_t ldo, int64_t stride_o, uint8_t* workspace, int64_t workspace_bytes,
                                 cudaStream_t stream) {
  if (dtype != MXQ_F32 && dtype != MXQ_BF16) return MXQ_EBADDTYPE;
  if (check_ortho_shape(batch, m, n) != MXQ_OK || steps < 1 || steps > 64) return MXQ_EBADSHAPE;
  if (batch == 0 || m == 0 || n == 0) return MXQ_OK;
  const int64_t most = int64_t{1} << 40;
  if (ld < n || ldo < n || ld > INT32_MAX || ldo > INT32_MAX || stride < 0 || stride_o < 0 || stride > most ||
      stride_o > most || (batch > 1 && (stride < (m - 1) * ld + n || stride_o < (m - 1) * ldo + n)))
    return MXQ_EBADSHAPE;
  if (!isfinite(ca) || !isfinite(cb) || !isfinite(cc) || !isfinite(eps) || eps < 0 || !isfinite(scale)) return MXQ_EBADSHAPE;
  const Layout l = layout_of(batch, m, n);
  if (workspace_bytes < l.bytes) return MXQ_EBADSHAPE;
  if (!g || !out || !workspace) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(g, es) || !aligned_to(out, 2) || !aligned_to(workspace, 16)) return MXQ_EALIGN;
  const ByteRange o[2] = {range_of(out, static_cast<uint64_t>((batch - 1) * stride_o + (m - 1) * ldo + n) * 2),
                          range_of(workspace, l.bytes)};
  const ByteRange in[1] = {range_of(g, static_cast<uint64_t>((batch - 1) * stride + (m - 1) * ld + n) * es)};
  if (outputs_overlap(o, 2, in, 1)) return MXQ_EOVERLAP;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;

  const Matrix a = {batch, m, n, ld, batch > 1 ? stride : 0, n};
  int rc = dtype == MXQ_F32 ? scale_vector<float>(g, a, eps, workspace, l, sms, stream)
                            : scale_vector<bf16_t>(g, a, eps, workspace, l, sms, stream);
  if (rc != MXQ_OK) return rc;

  const bool wide = m <= n;
  const int64_t side = l.side, length = wide ? n : m;
  const auto matrix = [&](int64_t at) { return Stack{workspace + at, batch, m, n, l.ldx, m * l.ldx}; };
  const auto square = [&](int64_t at) { return Stack{workspace + at, batch, side, side, l.lds, side * l.lds}; };
  // boxes: K-major operand 64 x 128, MN-major operand 64 x 64, stores 64 x 32 and 32 x 64
  struct Set {
    CUtensorMap k, mn, rows, columns;
  } x[2][2], gram[2], poly[2];
  CUtensorMap final_rows;
  bool ok = true;
  const auto set = [&](Set* to, const Stack& t) {
    ok = ok && encode_half(&to->k, t, 64, kHalf, true) && encode_half(&to->mn, t, 64, 64, true) &&
         encode_half(&to->rows, t, 64, 32, true) && encode_half(&to->columns, t, 32, 64, false);
  };
  for (int q = 0; q < l.parts; ++q) {
    for (int i = 0; i < 2; ++i) set(&x[i][q], matrix(l.x[i][q]));
    set(&gram[q], square(l.gram[q]));
    set(&poly[q], square(l.poly[q]));
  }
  if (!ok) return MXQ_ECUDA;
  const int64_t so = batch > 1 ? stride_o : (m * ldo + 7) / 8 * 8;
  // a tensor store clips rows to whole 16-byte pieces: one of another length would write
  // up to 14 bytes behind every row
  const bool out_map =
      n % 8 == 0 && aligned_to(out, 16) && ldo % 8 == 0 && so % 8 == 0 &&
      encode(&final_rows, Stack{out, batch, m, n, ldo, so}, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 64, 32, true);

  // |X| <= 1.5 and so |A| <= 2 are taken as bounds of the iterates
  // P = c (A + b/2c I)^2 + (a - b^2/4c) I where b/2c is no larger than those bounds
  const bool completed = cc != 0.0f && fabsf(cb) <= kCompletedSquare * fabsf(cc);
  const double shift = completed ? 0.5 * cb / cc : 0.0;
  const float sa = scale_for(2.0 + fabs(shift)), sp = scale_for(fabs(ca) + 2 * fabs(cb) + 4 * fabs(cc));
  const int parts = l.parts;
  const bool split = parts == 2;
  float* d_gram = reinterpret_cast<float*>(workspace + l.d_gram);
  float* d_poly = reinterpret_cast<float*>(workspace + l.d_poly);
  // what a step can magnify X by at most while |X| <= 1/2, in powers of two
  const double growth = log2(fmax(1.0, fabs(ca) + fabs(cb) / 4 + fabs(cc) / 16));
  const auto lift = [&](int s, int32_t out_from, int32_t in_to) {
    return Lift{reinterpret_cast<const int32_t*>(workspace + l.lifts), static_cast<int32_t>(ceil(s * growth)),
                static_cast<int32_t>(ceil((s + 1) * growth)), out_from, in_to, static_cast<int32_t>(batch)};
  };
  for (int s = 0; s < steps; ++s) {
    const int from = s & 1, to = from ^ 1;
    Maps maps = {};
    Product p = {};
    // A
    for (int q = 0; q < parts; ++q) {
      maps.a[q] = maps.b[q] = wide ? x[from][q].k : x[from][q].mn;
      maps.d[q] = gram[q].rows;
    }
    maps.dt = gram[0].columns;
    p.rows = p.cols = side;
    p.ksteps = static_cast<int32_t>(ceil_div(length, kStepK));
    p.a_mn = p.b_mn = !wide;
    p.scale = sa / (kXScale * kXScale);
    p.lift = lift(s, 2, 0);
    p.diagonal = static_cast<float>(shift * sa);
    p.d_ld = l.lds;
    p.d_count = batch * l.lds;
    if (!split) {
      p.d_out = d_gram;
      p.d_squares = completed;
    }
    if (const int64_t slices = gram_slices(batch, side, length); slices > 0) {
      p.partial = reinterpret_cast<float*>(workspace + l.partial);
      p.partial_stride = batch * side * l.lds;
      const int64_t stages = p.ksteps * (split ? 3 : 1);
      p.per_slice = static_cast<int32_t>(ceil_div(stages, slices));
      p.slices = static_cast<int32_t>(ceil_div(stages, p.per_slice));
      rc = split ? launch_product<true, 0, false, false, true, true>(maps, p, batch, sms, stream)
                 : launch_product<true, 0, false, false, false, true>(maps, p, batch, sms, stream);
      if (rc != MXQ_OK) return rc;
      const Join join = {p.partial, batch, side, l.lds, p.partial_stride, p.slices, p.scale, p.diagonal, p.lift,
                         reinterpret_cast<__half*>(workspace + l.gram[0]),
                         split ? reinterpret_cast<__half*>(workspace + l.gram[1]) : nullptr, p.d_out, p.d_squares};
      rc = launch_pdl(join_kernel, static_cast<unsigned>(ceil_div(p.partial_stride, kThreads)), kThreads, 0, stream, join);
    } else {
      rc = split ? launch_product<true, 0, false, false, true, false>(maps, p, batch, sms, stream)
                 : launch_product<true, 0, false, false, false, false>(maps, p, batch, sms, stream);
    }
    if (rc != MXQ_OK) return rc;
    // P = aI + bA + cAA
    p = {};
    for (int q = 0; q < parts; ++q) {
      maps.a[q] = maps.b[q] = gram[q].k;
      maps.add[q] = gram[q].rows;
      maps.d[q] = poly[q].rows;
    }
    maps.dt = poly[0].columns;
    p.rows = p.cols = side;
    p.ksteps = static_cast<int32_t>(ceil_div(side, kStepK));
    p.scale = cc * sp / (sa * sa);
    p.diagonal = static_cast<float>((ca - 0.5 * shift * cb) * sp);
    p.d_ld = l.lds;
    p.d_count = batch * l.lds;
    if (!split) p.d_out = d_poly;
    if (completed) {
      if (!split) p.square_rest = d_gram;
      rc = split ? launch_product<true, 0, false, false, true, false>(maps, p, batch, sms, stream)
                 : launch_product<true, 0, false, false, false, false>(maps, p, batch, sms, stream);
    } else {
      p.add_scale = cb * sp / sa;
      if (!split) p.d_row = p.d_col = d_gram;
      rc = split ? launch_product<true, 2, false, false, true, false>(maps, p, batch, sms, stream)
                 : launch_product<true, 1, true, false, false, false>(maps, p, batch, sms, stream);
    }
    if (rc != MXQ_OK) return rc;
    // X <- P X, or X P
    p = {};
    for (int q = 0; q < parts; ++q) {
      maps.a[q] = wide ? poly[q].k : x[from][q].k;
      maps.b[q] = wide ? x[from][q].mn : poly[q].k;
      maps.d[q] = x[to][q].rows;
    }
    p.b_mn = wide;
    p.rows = m;
    p.cols = n;
    p.ksteps = static_cast<int32_t>(ceil_div(side, kStepK));
    p.scale = 1.0f / sp;
    if (!split) {
      maps.add[0] = x[from][0].rows;
      p.d_ld = l.lds;
      p.d_count = batch * l.lds;
      (wide ? p.d_row : p.d_col) = d_poly;
    }
    const bool last = s + 1 == steps;
    if (last) {
      if (out_map) maps.d[0] = final_rows;
      p.out = static_cast<bf16_t*>(out);
      p.ldo = ldo;
      p.stride_o = so;
      p.out_map = out_map;
      p.scale = scale / (sp * kXScale);
    }
    p.lift = lift(s, 1, last ? 0 : 1);
    if (split)
      rc = last ? launch_product<false, 0, false, true, true, false>(maps, p, batch, sms, stream)
                : launch_product<false, 0, false, false, true, false>(maps, p, batch, sms, stream);
    else if (wide)
      rc = last ? launch_product<false, 1, false, true, false, false>(maps, p, batch, sms, stream)
                : launch_product<false, 1, false, false, false, false>(maps, p, batch, sms, stream);
    else
      rc = last ? launch_product<false, 1, true, true, false, false>(maps, p, batch, sms, stream)
                : launch_product<false, 1, true, false, false, false>(maps, p, batch, sms, stream);
    if (rc != MXQ_OK) return rc;
  }
  return MXQ_OK;
}
