// moe_exchange.cu -- the rows that tokens and experts exchange: the plan of the
// expert groups, dispatch, combine, and their gradients.
//
// Assignment i = token*k + j sends a token to its j-th expert.  The plan puts
// the assignments of each expert one after another in token order (a stable
// counting sort), each group starting at a multiple of 128 rows, which is what
// the grouped MXFP8 cast takes: offs[e] is the cumulative end of group e,
// slots[i] the row of assignment i, source[m] the assignment of row m or -1 for
// the rows that only fill a group up or lie past the last one.
//   dispatch           rows[slots[i]] = x[i / k], the other rows zero
//   combine            y[t] = sum_j w_tj rows[slots[tk + j]]   (w = 1 without weights:
//                      the gradient of dispatch)
//   combine_backward   drows[slots[i]] = w_i dy[i / k], the other rows zero;
//                      dweights[i] = <dy[i / k], rows[slots[i]]>
// All of it is bound by HBM: a token's row is read once and its k rows written
// or read by the same threads, with sums over j in ascending order in fp32.  Only
// combine_backward reads dy again, for every four choices, out of L2 as a rule (7168
// tokens of 7168 bf16: k 4 160 us where the bytes take 153, k 8 301 and 274; 2048 of
// 4096, k 32: 199 and 170).
#include <cuda_runtime.h>
#include <stdint.h>

#include "rank_tile.cuh"
#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_exchange_status = 0;

constexpr int kGroupRows = 128;
constexpr int kMaxK = 32;
constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct ExpertKey {
  const int32_t* ids;
  int E;
  int64_t n;
  __device__ int operator()(int64_t i) const {
    const int32_t e = read_at(ids, i, n, -1, &g_exchange_status);
    if (e >= 0 && e < E) return e;
    if (e != -1) atomicOr(&g_exchange_status, MXQ_DEV_BADINDEX);
    return -1;
  }
};

__global__ void __launch_bounds__(kRankThreads)
    plan_count_kernel(const int32_t* __restrict__ ids, RankSplit s, int E, int32_t* chunk_counts) {
  extern __shared__ int32_t counts[];
  pdl_wait();
  pdl_launch_dependents();  // as few blocks follow
  rank_count(s, E, ExpertKey{ids, E, s.n}, counts);
  rank_keep_counts(s, E, counts, chunk_counts, &g_exchange_status);
}

__global__ void __launch_bounds__(kRankThreads)
    plan_kernel(const int32_t* __restrict__ ids, RankSplit s, int E, const int32_t* __restrict__ chunk_counts,
                int32_t* __restrict__ offs, int32_t* __restrict__ slots, int32_t* __restrict__ source, int64_t M) {
  extern __shared__ int32_t smem[];
  int32_t* next = smem;         // [E]
  int32_t* counts = smem + E;   // [warps, E]
  __shared__ int32_t total[kRankMaxBins], begin[kRankMaxBins], work[kRankWarps];
  pdl_wait();
  const ExpertKey key{ids, E, s.n};
  if (s.chunks == 1) {
    rank_count(s, E, key, total);
    for (int e = threadIdx.x; e < E; e += kRankThreads) next[e] = 0;
  } else {
    rank_totals(s, E, chunk_counts, total, next, &g_exchange_status);
  }
  const int32_t end = rank_begins<kGroupRows>(E, total, begin, work);
  const uint64_t m_bytes = static_cast<uint64_t>(M) * 4;
  // rows that fill a group up: a warp per expert
  for (int e = blockIdx.x * kRankWarps + (threadIdx.x >> 5); e < E; e += gridDim.x * kRankWarps) {
    const int64_t lo = begin[e] + total[e];
    const int64_t hi = begin[e] + (total[e] + kGroupRows - 1) / kGroupRows * kGroupRows;
    for (int64_t m = lo + (threadIdx.x & 31); m < hi; m += 32)
      if (in_buf(source + m, 4, source, m_bytes, &g_exchange_status)) source[m] = -1;
    if ((threadIdx.x & 31) == 0) write_at(offs, e, E, static_cast<int32_t>(hi), &g_exchange_status);
  }
  for (int64_t m = end + static_cast<int64_t>(blockIdx.x) * kRankThreads + threadIdx.x; m < M;
       m += static_cast<int64_t>(gridDim.x) * kRankThreads)
    write_at(source, m, M, -1, &g_exchange_status);
  for (int e = threadIdx.x; e < E; e += kRankThreads) next[e] += begin[e];
  __syncthreads();
  const uint64_t s_bytes = static_cast<uint64_t>(s.n) * 4;
  rank_chunk(
      s, E, key,
      [&](int64_t i, int, int32_t place) {
        if (in_buf(slots + i, 4, slots, s_bytes, &g_exchange_status)) slots[i] = place;
        if (place >= 0 && in_buf(source + place, 4, source, m_bytes, &g_exchange_status))
          source[place] = static_cast<int32_t>(i);
      },
      next, counts);
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
struct ExchangeShape {
  int64_t tokens, M, D;
  int64_t ldt, ldm;  // elements between the rows of the token matrix and of the group matrix
  int k, tx;         // tx: threads per token (a power of two)
  int fill;          // rows that a block looks at to zero unused ones
};

// Rows looked at by a block that zeroes unused rows: 8, whose columns its threads
// share, or 256 where rows are narrow and many, 32 for each warp (800000 rows of 64
// bf16: 26 us for the dispatch, 96 with 8; 36000 of 1001: 29, and 33 with 32; 2000
// of 7: 3.2, and 5.7 with 256).
constexpr int kFewRows = 8, kManyRows = kThreads;
inline int fill_rows(const ExchangeShape& s, int esize) {
  return s.D * esize <= 1024 && s.M >= 128 * kManyRows ? kManyRows : kFewRows;
}

// Zeroes those of a block's rows that no assignment fills.  The rows' assignments
// are read at once, a row a lane.
template <typename T, int kV>
__device__ void zero_unused(const ExchangeShape& s, const int32_t* source, T* rows, int64_t block) {
  const int64_t nv = s.D / kV;
  const uint64_t bytes = (static_cast<uint64_t>(s.M - 1) * s.ldm + s.D) * sizeof(T);
  const bool narrow = s.fill == kManyRows;
  const int lane = threadIdx.x & 31, first = narrow ? lane : threadIdx.x, step = narrow ? 32 : kThreads;
  const int64_t m0 = block * s.fill + (narrow ? threadIdx.x & ~31u : 0u);
  uint32_t unused = __ballot_sync(0xFFFFFFFFu, (narrow || lane < kFewRows) && m0 + lane < s.M &&
                                                       read_at(source, m0 + lane, s.M, 0, &g_exchange_status) < 0);
  for (; unused != 0u; unused &= unused - 1) {
    T* row = rows + (m0 + __ffs(unused) - 1) * s.ldm;
    for (int64_t c = first; c < nv; c += step)
      if (in_buf(row + c * kV, kV * sizeof(T), rows, bytes, &g_exchange_status))
        *reinterpret_cast<Vec<T, kV>*>(row + c * kV) = Vec<T, kV>{};
  }
}

// kJ slots are read at once, before the columns: one by one each would wait for
// the one before.  kMore: there may be more of them.  7168 tokens of 7168 bf16, k 8:
// 160 us, 6.5 TB/s.
template <typename T, int kV, int kJ, bool kMore>
__global__ void __launch_bounds__(kThreads)
    dispatch_kernel(const T* __restrict__ x, const ExchangeShape s, const int32_t* __restrict__ slots,
                    const int32_t* __restrict__ source, T* __restrict__ rows, int64_t token_blocks) {
  pdl_wait();
  if (static_cast<int64_t>(blockIdx.x) >= token_blocks) {
    zero_unused<T, kV>(s, source, rows, blockIdx.x - token_blocks);
    return;
  }
  const int ty = kThreads / s.tx;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * ty + threadIdx.x / s.tx;
  if (t >= s.tokens) return;
  const int64_t nv = s.D / kV;
  const uint64_t bytes = (static_cast<uint64_t>(s.M - 1) * s.ldm + s.D) * sizeof(T);
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldt + s.D) * sizeof(T);
  bool bad = false;
  int32_t first[kJ];
  const auto read = [&](int j0, int32_t (&m)[kJ]) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) m[j] = j0 + j < s.k ? read_at(slots, t * s.k + j0 + j, s.tokens * s.k, -1, &g_exchange_status) : -1;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (m[j] >= s.M || m[j] < -1) bad = true;
      if (m[j] >= s.M) m[j] = -1;
    }
  };
  const auto write = [&](const int32_t (&m)[kJ], const Vec<T, kV>& v, int64_t c) {
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (m[j] >= 0 && in_buf(rows + m[j] * s.ldm + c * kV, kV * sizeof(T), rows, bytes, &g_exchange_status))
        *reinterpret_cast<Vec<T, kV>*>(rows + m[j] * s.ldm + c * kV) = v;
  };
  read(0, first);
  for (int64_t c = threadIdx.x % s.tx; c < nv; c += s.tx) {
    const T* p = x + t * s.ldt + c * kV;
    const Vec<T, kV> v = load_if<T, kV>(p, in_buf(p, sizeof v, x, in_bytes, &g_exchange_status));
    write(first, v, c);
    for (int j0 = kJ; kMore && j0 < s.k; j0 += kJ) {
      int32_t m[kJ];
      read(j0, m);
      write(m, v, c);
    }
  }
  if (bad) atomicOr(&g_exchange_status, MXQ_DEV_BADINDEX);
}

// Rows whose lengths, pitches or addresses allow narrow accesses only, kIn elements
// of x at a time.  A token's elements are staged in shared memory and written from
// there in whole 16-byte units of each row, wherever it begins (36000 rows of 1001
// bf16: 32 us, 62 with 2-byte stores; 40000 rows of 1001 fp32: 57 and 83; 32768 of
// 4098 bf16: 65 and 93).  Where rows can begin at any 2 bytes a second copy, 2 bytes
// further on, makes every unit begin at a word of the one or the other.
template <typename T, int kIn>
__global__ void __launch_bounds__(kThreads)
    dispatch_narrow_kernel(const T* __restrict__ x, const ExchangeShape s, const int32_t* __restrict__ slots,
                           const int32_t* __restrict__ source, T* __restrict__ rows, int64_t token_blocks, int tiles, int tile) {
  constexpr bool kTwo = sizeof(T) * kIn == 2;
  constexpr int kLoads = kUnits * 16 / (sizeof(T) * kIn);
  __shared__ uint32_t stage[kTwo ? 2 : 1][kThreads * kUnits * 4 + kThreads / 8];
  pdl_wait();
  if (static_cast<int64_t>(blockIdx.x) >= token_blocks) {
    zero_unused<T, kIn>(s, source, rows, blockIdx.x - token_blocks);
    return;
  }
  const int group = threadIdx.x / s.tx, own = threadIdx.x % s.tx;
  const int64_t t = static_cast<int64_t>(blockIdx.x / tiles) * (kThreads / s.tx) + group;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x % tiles) * tile;
  const int n = t < s.tokens ? static_cast<int>(min(static_cast<int64_t>(tile), s.D - c0)) : 0;
  T* even = reinterpret_cast<T*>(stage[0] + group * (4 * kUnits * s.tx + 1));
  T* odd = reinterpret_cast<T*>(stage[kTwo ? 1 : 0] + group * (4 * kUnits * s.tx + 1)) + 1;  // one element further on
  Vec<T, kIn> v[kLoads];
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldt + s.D) * sizeof(T);
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int i = (q * s.tx + own) * kIn;
    const T* p = x + t * s.ldt + c0 + i;
    v[q] = load_if<T, kIn>(p, i < n && in_buf(p, sizeof v[q], x, in_bytes, &g_exchange_status));
  }
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int i = (q * s.tx + own) * kIn;
    if (i >= n) continue;
#pragma unroll
    for (int e = 0; e < kIn; ++e) even[i + e] = v[q].v[e];
    if (kTwo) odd[i] = v[q].v[0];
  }
  __syncthreads();
  const uint64_t out_bytes = (static_cast<uint64_t>(s.M - 1) * s.ldm + s.D) * sizeof(T);
  bool bad = false;
  for (int j = 0; n > 0 && j < s.k; ++j) {
    const int64_t m = read_at(slots, t * s.k + j, s.tokens * s.k, -1, &g_exchange_status);
    if (m < 0 || m >= s.M) {
      bad |= m != -1;
      continue;
    }
    T* row = rows + m * s.ldm + c0;
    write_staged<T, kTwo>(even, odd, row, n, own, s.tx, [&](const void* at, int size) {
      return in_buf(at, size, rows, out_bytes, &g_exchange_status);
    });
  }
  if (bad && own == 0) atomicOr(&g_exchange_status, MXQ_DEV_BADINDEX);
}

// The rows and weights of kJ choices of a token, from choice j0 on: loaded once,
// before the columns, so that the rows' loads depend on nothing but registers.
template <int kJ>
struct Choices {
  int64_t row[kJ];  // -1: none
  float w[kJ];
  __device__ __forceinline__ Choices(const int32_t* slots, const float* weights, const ExchangeShape& s, int64_t t,
                                     int j0, int64_t ld) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int32_t m = j0 + j < s.k ? read_at(slots, t * s.k + j0 + j, s.tokens * s.k, -1, &g_exchange_status) : -1;
      const bool live = m >= 0 && m < s.M;
      bad |= !live && m != -1;
      row[j] = live ? m * ld : -1;
      w[j] = live ? (weights != nullptr ? read_at(weights, t * s.k + j0 + j, s.tokens * s.k, 0.0f, &g_exchange_status) : 1.0f) : 0.0f;
    }
    if (bad) atomicOr(&g_exchange_status, MXQ_DEV_BADINDEX);
  }
};

// kJ choices and kU columns (kJ * kU = combine_at_once row pieces) are loaded before
// the first is used: enough in flight for HBM with few choices as with many, and
// more of narrow pieces (30021 rows of 2050 fp32, 16 against 8: 54 us and 59; 36000
// rows of 1001 bf16: 26 and 29; 8 choices of 7164 bf16 lack the registers: 173 and
// 158).  Four
// blocks of 256 threads on a multiprocessor (64 registers) and 64 threads a token
// read fastest: 57344 rows of 7168 bf16 in 140 us (6.6 TB/s); 157 with six blocks,
// 234 with 32 threads a token, and 52 us against 28 with 256 threads a token at
// 32768 rows of 2048.  With the choices read inside the column loop the loads
// went one by one (462 us).
template <typename T, int kV, int kJ>
__host__ __device__ constexpr int combine_at_once() {
  return sizeof(T) * kV == 16 || (sizeof(T) * kV == 8 && kJ == 8) ? 8 : 16;
}
constexpr int kCombineBlocks = 4;

// kMore: there may be more than kJ choices.
template <typename T, int kV, int kJ, bool kMore>
__global__ void __launch_bounds__(kThreads, kCombineBlocks)
    combine_kernel(const T* __restrict__ rows, const ExchangeShape s, const int32_t* __restrict__ slots,
                   const float* __restrict__ weights, T* __restrict__ y) {
  pdl_wait();
  constexpr int kU = combine_at_once<T, kV, kJ>() / kJ;
  const int ty = kThreads / s.tx;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * ty + threadIdx.x / s.tx;
  if (t >= s.tokens) return;
  const int64_t nv = s.D / kV;
  const uint64_t in_bytes = (static_cast<uint64_t>(s.M - 1) * s.ldm + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldt + s.D) * sizeof(T);
  const Choices<kJ> first(slots, weights, s, t, 0, s.ldm);
  for (int64_t c = threadIdx.x % s.tx; c < nv; c += kU * s.tx) {
    float acc[kU][kV];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < kV; ++i) acc[u][i] = 0.0f;
    const auto add = [&](const Choices<kJ>& from) {
      Vec<T, kV> v[kJ][kU];
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const T* p = rows + from.row[j] + (c + u * s.tx) * kV;
          v[j][u] = load_if<T, kV>(p, from.row[j] >= 0 && c + u * s.tx < nv &&
                                          in_buf(p, sizeof v[j][u], rows, in_bytes, &g_exchange_status));
        }
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < kV; ++i) acc[u][i] = fmaf(from.w[j], widen(v[j][u].v[i]), acc[u][i]);
    };
    add(first);
    if (kMore)
      for (int j0 = kJ; j0 < s.k; j0 += kJ) add(Choices<kJ>(slots, weights, s, t, j0, s.ldm));
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      Vec<T, kV> out;
#pragma unroll
      for (int i = 0; i < kV; ++i) out.v[i] = narrow<T>(acc[u][i]);
      T* to = y + t * s.ldt + (c + u * s.tx) * kV;
      if (c + u * s.tx < nv && in_buf(to, sizeof out, y, out_bytes, &g_exchange_status)) *reinterpret_cast<Vec<T, kV>*>(to) = out;
    }
  }
}

// Row pieces a thread of the gradient holds at once.  It also keeps the token's
// own piece and writes as much as it reads, so with 16-byte pieces four are
// faster than eight (64 groups, 57344 rows of 7168 bf16: 299 us against 322;
// 32768 rows of 2048: 62 against 72); with narrower ones eight (30021 rows of 2050
// fp32: 121 against 134; 36000 rows of 1001 bf16: 55 against 65).
template <typename T, int kV>
__host__ __device__ constexpr int back_at_once() {
  return sizeof(T) * kV == 16 ? 4 : 8;
}
constexpr int kBackBlocks = 4;

// kGroup threads per token: 8 lanes, a warp, two, or all of the block's.
template <typename T, int kV, int kJ, int kGroup>
__global__ void __launch_bounds__(kThreads, kBackBlocks)
    combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ rows, const ExchangeShape s, int64_t ldr,
                            const int32_t* __restrict__ slots, const int32_t* __restrict__ source,
                            const float* __restrict__ weights, T* __restrict__ drows, float* __restrict__ dweights,
                            int64_t token_blocks) {
  __shared__ float red[kThreads / 32][kJ];
  pdl_wait();
  if (static_cast<int64_t>(blockIdx.x) >= token_blocks) {
    zero_unused<T, kV>(s, source, drows, blockIdx.x - token_blocks);
    return;
  }
  constexpr int kU = back_at_once<T, kV>() / kJ;
  constexpr int kWarps = kGroup > 32 ? kGroup / 32 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / kGroup) + threadIdx.x / kGroup;
  const bool live = t < s.tokens;
  if (kGroup == 32 && !live) return;  // others stay for the warp's sums and the block's barriers
  const int64_t nv = s.D / kV;
  const uint64_t in_bytes = (static_cast<uint64_t>(s.M - 1) * ldr + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.M - 1) * s.ldm + s.D) * sizeof(T);
  const uint64_t dy_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldt + s.D) * sizeof(T);
  for (int j0 = 0; j0 < s.k; j0 += kJ) {
    const Choices<kJ> from(slots, weights, s, live ? t : 0, j0, ldr);
    int64_t to[kJ];
    float dot[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      to[j] = from.row[j] >= 0 && live ? static_cast<int64_t>(read_at(slots, t * s.k + j0 + j, s.tokens * s.k, -1, &g_exchange_status)) * s.ldm : -1;
      dot[j] = 0.0f;
    }
    for (int64_t c = threadIdx.x % kGroup; live && c < nv; c += kU * kGroup) {
      Vec<T, kV> g[kU], v[kJ][kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t col = (c + u * kGroup) * kV;
        const T* d = dy + t * s.ldt + col;
        g[u] = load_if<T, kV>(d, c + u * kGroup < nv && in_buf(d, sizeof g[u], dy, dy_bytes, &g_exchange_status));
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const T* p = rows + from.row[j] + col;
          v[j][u] = load_if<T, kV>(p, from.row[j] >= 0 && c + u * kGroup < nv &&
                                          in_buf(p, sizeof v[j][u], rows, in_bytes, &g_exchange_status));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          Vec<T, kV> out;
#pragma unroll
          for (int i = 0; i < kV; ++i) {
            const float d = widen(g[u].v[i]);
            dot[j] = fmaf(d, widen(v[j][u].v[i]), dot[j]);
            out.v[i] = narrow<T>(from.w[j] * d);
          }
          T* p = drows + to[j] + (c + u * kGroup) * kV;
          if (to[j] >= 0 && c + u * kGroup < nv && in_buf(p, sizeof out, drows, out_bytes, &g_exchange_status))
            *reinterpret_cast<Vec<T, kV>*>(p) = out;
        }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int d = (kGroup < 32 ? kGroup : 32) / 2; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
    if (kWarps > 1) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < kJ; ++j) red[warp][j] = dot[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        dot[j] = 0.0f;
        for (int q = 0; q < kWarps; ++q) dot[j] += red[warp / kWarps * kWarps + q][j];
      }
      __syncthreads();
    }
    if (live && threadIdx.x % kGroup == 0)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (j0 + j < s.k)
          write_at(dweights, t * s.k + j0 + j, s.tokens * s.k, from.row[j] >= 0 ? dot[j] : 0.0f, &g_exchange_status);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
struct RowsCall {
  int dtype;
  const void* in;        // x, or the group rows
  const void* in2;       // dy of combine_backward
  ExchangeShape s;
  int64_t ldr;
  const int32_t *slots, *source;
  const float* weights;
  void* out;
  float* dweights;
  int sms;
  cudaStream_t stream;
};

// 8-byte accesses are staged for long rows with many copies only (60000 rows of
// 2050 fp32, direct and staged: 216 and 240 us with one choice, 117 and 108 with
// eight; of 514 fp32, 200000 rows: 113 and 122 with eight).
template <typename T, int kV>
int launch_dispatch(RowsCall a) {
  const int64_t fill_blocks = ceil_div(a.s.M, a.s.fill);
  const int64_t bytes = a.s.D * sizeof(T);
  if constexpr (sizeof(T) * kV >= 8) {
    if (sizeof(T) * kV == 16 || a.s.k < 8 || bytes < 4096) {
      const int64_t token_blocks = ceil_div(a.s.tokens, kThreads / a.s.tx);
      const auto kernel = a.s.k <= 2   ? dispatch_kernel<T, kV, 2, false>
                          : a.s.k <= 4 ? dispatch_kernel<T, kV, 4, false>
                          : a.s.k <= 8 ? dispatch_kernel<T, kV, 8, false>
                                       : dispatch_kernel<T, kV, 8, true>;
      return launch_pdl(kernel, static_cast<unsigned>(token_blocks + fill_blocks), kThreads, 0, a.stream,
                        static_cast<const T*>(a.in), a.s, a.slots, a.source, static_cast<T*>(a.out), token_blocks);
    }
  }
  if constexpr (sizeof(T) * kV < 16) {
    const StagedTiles split = staged_tiles(a.s.D, sizeof(T), kV, kThreads);
    a.s.tx = split.tx;
    const int64_t token_blocks = ceil_div(a.s.tokens, kThreads / a.s.tx) * split.tiles;
    return launch_pdl(dispatch_narrow_kernel<T, kV>, static_cast<unsigned>(token_blocks + fill_blocks), kThreads, 0, a.stream,
                      static_cast<const T*>(a.in), a.s, a.slots, a.source, static_cast<T*>(a.out), token_blocks,
                      split.tiles, split.tile);
  }
}
// Choices handled at once: 2, 4 or 8, the smallest that holds k.
template <typename T, int kV, int kJ, bool kMore>
int launch_combine(RowsCall a) {
  // 64 threads a token, fewer for rows that have no columns for them (50000 tokens
  // of 35 fp32: 26 us with 64, 10 with 16), more where the tokens are too few to
  // fill the GPU
  constexpr int kU = combine_at_once<T, kV, kJ>() / kJ;
  const int64_t nv = a.s.D / kV;
  const int64_t fill = static_cast<int64_t>(a.sms) * kCombineBlocks * kThreads;
  int tx = 8;
  while (tx < a.s.tx && ((tx < 64 && tx * kU < nv) || tx * a.s.tokens < fill)) tx *= 2;
  a.s.tx = tx;
  return launch_pdl(combine_kernel<T, kV, kJ, kMore>, static_cast<unsigned>(ceil_div(a.s.tokens, kThreads / tx)), kThreads,
                    0, a.stream, static_cast<const T*>(a.in), a.s, a.slots, a.weights, static_cast<T*>(a.out));
}
template <typename T, int kV>
int launch_combine(const RowsCall& a) {
  return a.s.k <= 2   ? launch_combine<T, kV, 2, false>(a)
         : a.s.k <= 4 ? launch_combine<T, kV, 4, false>(a)
         : a.s.k <= 8 ? launch_combine<T, kV, 8, false>(a)
                      : launch_combine<T, kV, 8, true>(a);
}
template <typename T, int kV, int kJ, int kGroup>
int launch_combine_backward(const RowsCall& a) {
  const int64_t token_blocks = ceil_div(a.s.tokens, kThreads / kGroup);
  const int64_t blocks = token_blocks + ceil_div(a.s.M, a.s.fill);
  return launch_pdl(combine_backward_kernel<T, kV, kJ, kGroup>, static_cast<unsigned>(blocks), kThreads, 0, a.stream,
                    static_cast<const T*>(a.in2), static_cast<const T*>(a.in), a.s, a.ldr, a.slots, a.source, a.weights,
                    static_cast<T*>(a.out), a.dweights, token_blocks);
}
// 8 lanes a token for the narrowest rows (100000 tokens of 64 bf16, k 8: 48 us, 109
// with a warp), a warp for narrow ones; for wide ones two, or all of a block's
// where the tokens are too few to fill the GPU.
template <typename T, int kV, int kJ>
int launch_combine_backward(const RowsCall& a) {
  const int64_t nv = a.s.D / kV, fill = static_cast<int64_t>(a.sms) * kBackBlocks * kThreads;
  if (nv <= 16) return launch_combine_backward<T, kV, kJ, 8>(a);
  if (nv < 64) return launch_combine_backward<T, kV, kJ, 32>(a);
  return nv >= kThreads && a.s.tokens * 64 < fill ? launch_combine_backward<T, kV, kJ, kThreads>(a)
                                                  : launch_combine_backward<T, kV, kJ, 64>(a);
}
template <typename T, int kV>
int launch_combine_backward(const RowsCall& a) {
  return a.s.k <= 2 ? launch_combine_backward<T, kV, 2>(a) : launch_combine_backward<T, kV, 4>(a);
}

enum class Rows { kDispatch, kCombine, kCombineBackward };
template <Rows kWhat, typename T, int kV>
int launch_rows(RowsCall a) {
  const int64_t nv = a.s.D / kV;
  int tx = 8;
  while (tx < kThreads && tx < nv) tx *= 2;
  a.s.tx = tx;
  a.s.fill = fill_rows(a.s, sizeof(T));
  if constexpr (kWhat == Rows::kDispatch) return launch_dispatch<T, kV>(a);
  if constexpr (kWhat == Rows::kCombine) return launch_combine<T, kV>(a);
  return launch_combine_backward<T, kV>(a);
}

// The widest access, up to 16 bytes, that divides the row length, every row
// pitch and every base address.
template <Rows kWhat>
int launch_by_alignment(const RowsCall& a) {
  const uint64_t es = element_bytes(a.dtype);
  const int align = common_alignment({a.s.D * es, a.s.ldt * es, a.s.ldm * es, a.ldr * es, address_of(a.in),
                                      address_of(a.in2), address_of(a.out)});
  if (a.dtype == MXQ_F32)
    return align >= 16  ? launch_rows<kWhat, float, 4>(a)
           : align >= 8 ? launch_rows<kWhat, float, 2>(a)
                        : launch_rows<kWhat, float, 1>(a);
  return align >= 16  ? launch_rows<kWhat, bf16_t, 8>(a)
         : align >= 8 ? launch_rows<kWhat, bf16_t, 4>(a)
         : align >= 4 ? launch_rows<kWhat, bf16_t, 2>(a)
                      : launch_rows<kWhat, bf16_t, 1>(a);
}

constexpr int64_t kMaxLd = INT32_MAX;  // no byte range below can wrap

int check_rows_shape(int dtype, int64_t tokens, int64_t D, int64_t ldt, int64_t ldm, int32_t k, int64_t M) {
  if (dtype != MXQ_F32 && dtype != MXQ_BF16) return MXQ_EBADDTYPE;
  if (tokens < 0 || D < 0 || M < 0 || k < 1 || k > kMaxK || M > INT32_MAX || tokens > INT32_MAX ||
      tokens * k > INT32_MAX || D > INT32_MAX || ldt < D || ldm < D || ldt > kMaxLd || ldm > kMaxLd)
    return MXQ_EBADSHAPE;
  return MXQ_OK;
}

}  // namespace

namespace mxq {
int exchange_status_read(unsigned int* out, bool clear) { return read_status_word(g_exchange_status, out, clear); }
int exchange_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int64_t mxq_moe_rows(int64_t tokens, int32_t k, int32_t experts) {
  if (tokens < 0 || tokens > INT32_MAX || k < 1 || k > kMaxK || experts < 1 || experts > MXQ_MAX_GROUPS)
    return MXQ_EBADSHAPE;
  const int64_t n = tokens * k;
  const int64_t m = (n + (kGroupRows - 1) * (n < experts ? n : experts)) / kGroupRows * kGroupRows;
  return m > INT32_MAX ? MXQ_EBADSHAPE : m;
}

extern "C" int64_t mxq_moe_plan_workspace(int64_t tokens, int32_t k, int32_t experts) {
  if (mxq_moe_rows(tokens, k, experts) < 0) return MXQ_EBADSHAPE;
  const RankSplit s = rank_split(tokens * k);
  return s.chunks == 1 ? 0 : static_cast<int64_t>(s.chunks) * experts * 4;
}

extern "C" int mxq_moe_plan(const int32_t* ids, int64_t tokens, int32_t k, int32_t experts, int64_t M, int32_t* offs,
                            int32_t* slots, int32_t* source, uint8_t* workspace, int64_t workspace_bytes,
                            cudaStream_t stream) {
  const int64_t need_m = mxq_moe_rows(tokens, k, experts);
  if (need_m < 0 || M < need_m || M > INT32_MAX || M % kGroupRows != 0) return MXQ_EBADSHAPE;
  const int64_t need = mxq_moe_plan_workspace(tokens, k, experts);
  if (workspace_bytes < need) return MXQ_EBADSHAPE;
  if (!offs || (tokens > 0 && (!ids || !slots)) || (M > 0 && !source) || (need > 0 && !workspace)) return MXQ_ENULL;
  if (!aligned_to(ids, 4) || !aligned_to(offs, 4) || !aligned_to(slots, 4) || !aligned_to(source, 4) ||
      !aligned_to(workspace, 4))
    return MXQ_EALIGN;
  const uint64_t n4 = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[4] = {range_of(offs, 4ull * experts), range_of(slots, n4), range_of(source, 4ull * M),
                            range_of(workspace, need)};
  const ByteRange in[1] = {range_of(ids, n4)};
  if (outputs_overlap(out, 4, in, 1)) return MXQ_EOVERLAP;
  const RankSplit s = rank_split(tokens * k);
  int32_t* counts = reinterpret_cast<int32_t*>(workspace);
  if (s.chunks > 1) {
    const int rc = launch_pdl(plan_count_kernel, s.chunks, kRankThreads, experts * 4, stream, ids, s, experts, counts);
    if (rc != MXQ_OK) return rc;
  }
  return launch_pdl(plan_kernel, s.chunks, kRankThreads, rank_smem(experts), stream, ids, s, experts, counts, offs,
                    slots, source, M);
}

extern "C" int mxq_moe_dispatch(const void* x, int dtype, int64_t tokens, int64_t D, int64_t ldx, int32_t k,
                                const int32_t* slots, const int32_t* source, int64_t M, void* rows, int64_t ldr,
                                cudaStream_t stream) {
  const int rc = check_rows_shape(dtype, tokens, D, ldx, ldr, k, M);
  if (rc != MXQ_OK) return rc;
  if (M == 0 || D == 0) return MXQ_OK;
  if ((tokens > 0 && (!x || !slots)) || !source || !rows) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(x, es) || !aligned_to(rows, es) || !aligned_to(slots, 4) || !aligned_to(source, 4)) return MXQ_EALIGN;
  const ByteRange out[1] = {range_of(rows, pitched_bytes(M, D, ldr, es))};
  const ByteRange in[3] = {range_of(x, pitched_bytes(tokens, D, ldx, es)),
                           range_of(slots, static_cast<uint64_t>(tokens) * k * 4), range_of(source, 4ull * M)};
  if (outputs_overlap(out, 1, in, 3)) return MXQ_EOVERLAP;
  RowsCall a = {};
  a.dtype = dtype;
  a.in = x;
  a.s = {tokens, M, D, ldx, ldr, k, 0, 0};
  a.slots = slots;
  a.source = source;
  a.out = rows;
  a.stream = stream;
  return launch_by_alignment<Rows::kDispatch>(a);
}

extern "C" int mxq_moe_combine(const void* rows, int dtype, int64_t M, int64_t D, int64_t ldr, int64_t tokens,
                               int32_t k, const int32_t* slots, const float* weights, void* y, int64_t ldy,
                               cudaStream_t stream) {
  const int rc = check_rows_shape(dtype, tokens, D, ldy, ldr, k, M);
  if (rc != MXQ_OK) return rc;
  if (tokens == 0 || D == 0) return MXQ_OK;
  if ((M > 0 && !rows) || !slots || !y) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(rows, es) || !aligned_to(y, es) || !aligned_to(slots, 4) || !aligned_to(weights, 4)) return MXQ_EALIGN;
  const uint64_t n4 = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[1] = {range_of(y, pitched_bytes(tokens, D, ldy, es))};
  const ByteRange in[3] = {range_of(rows, pitched_bytes(M, D, ldr, es)), range_of(slots, n4), range_of(weights, n4)};
  if (outputs_overlap(out, 1, in, 3)) return MXQ_EOVERLAP;
  RowsCall a = {};
  a.dtype = dtype;
  a.in = rows;
  a.s = {tokens, M, D, ldy, ldr, k, 0, 0};
  a.slots = slots;
  a.weights = weights;
  a.out = y;
  a.sms = sm_count_current_device(nullptr);
  if (a.sms <= 0) return MXQ_ECUDA;
  a.stream = stream;
  return launch_by_alignment<Rows::kCombine>(a);
}

extern "C" int mxq_moe_combine_backward(const void* dy, int dtype, int64_t tokens, int64_t D, int64_t ldy,
                                        const void* rows, int64_t ldr, int64_t M, int32_t k, const int32_t* slots,
                                        const int32_t* source, const float* weights, void* drows, int64_t ldd,
                                        float* dweights, cudaStream_t stream) {
  const int rc = check_rows_shape(dtype, tokens, D, ldy, ldd, k, M);
  if (rc != MXQ_OK) return rc;
  if (ldr < D || ldr > kMaxLd) return MXQ_EBADSHAPE;
  if (tokens == 0 && (M == 0 || D == 0)) return MXQ_OK;
  const bool has_rows = M > 0 && D > 0;
  if ((tokens > 0 && ((D > 0 && !dy) || !slots || !weights || !dweights)) || (M > 0 && !source) || (has_rows && (!rows || !drows)))
    return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(dy, es) || !aligned_to(rows, es) || !aligned_to(drows, es) || !aligned_to(slots, 4) ||
      !aligned_to(source, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return MXQ_EALIGN;
  const uint64_t n4 = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[2] = {range_of(drows, pitched_bytes(M, D, ldd, es)), range_of(dweights, n4)};
  const ByteRange in[5] = {range_of(dy, pitched_bytes(tokens, D, ldy, es)), range_of(rows, pitched_bytes(M, D, ldr, es)),
                           range_of(slots, n4), range_of(source, 4ull * M), range_of(weights, n4)};
  if (outputs_overlap(out, 2, in, 5)) return MXQ_EOVERLAP;
  RowsCall a = {};
  a.dtype = dtype;
  a.in = rows;
  a.in2 = dy;
  a.s = {tokens, M, D, ldy, ldd, k, 0, 0};
  a.ldr = ldr;
  a.slots = slots;
  a.source = source;
  a.weights = weights;
  a.out = drows;
  a.dweights = dweights;
  a.sms = sm_count_current_device(nullptr);
  if (a.sms <= 0) return MXQ_ECUDA;
  a.stream = stream;
  return launch_by_alignment<Rows::kCombineBackward>(a);
}
