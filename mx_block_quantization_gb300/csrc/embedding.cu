// embedding.cu -- scaled lookup of table rows, and the table's gradient.
//
//   lookup     y[t] = scale * table[ids[t]]
//   gradient   dtable[v] = scale * sum over the tokens t with ids[t] = v of dy[t]
//
// The gradient sorts the tokens by id, stably, so that the tokens of a row lie side
// by side.  Most of its time is writing the table, most rows of which no token has:
// the launches of the sort, which keep few blocks busy, zero the whole table with
// the others (6.2 TB/s), and the last launch writes the rows that have tokens, found
// from the places where a run of equal ids begins.  (Writing every row once, by its
// number, needs the runs before any of it and a search for each block of rows: 259
// us at 131072x4096 bf16 with 16384 tokens, now 213.)  With many tokens and no more
// rows than tokens the last launch zeroes the rows without any (zeroed_late).
// A frequent id would keep one block busy for long, so a run of more than kChunk
// tokens is first summed in pieces, one per chunk of kChunk sorted places, by a
// launch of its own; the row then adds the pieces in order.  That takes the tokens off
// one block, but the pieces of a row are still added by one: 65536 tokens of 4096 bf16
// on 32768 rows take 160 us drawn evenly, 176 with a tenth of them on one id, 524 with
// half and 944 with all.  Sums are in fp32 and their order depends on the ids alone.
#include <cuda_runtime.h>
#include <stdint.h>

#include "rank_tile.cuh"
#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_embedding_status = 0;

constexpr int kThreads = 256;
constexpr int kStarts = 8;         // sorted places whose runs a block of the last launch writes
constexpr int kChunk = 32;         // sorted places per piece of a long run
constexpr int kDigitBits = 10;     // at most kRankMaxBins bins

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
constexpr int64_t kFullGpu = 262144;  // threads that the GPU has at work, or nearly
struct LookupShape {
  int64_t tokens, rows, D, ldw, ldy;
  int tx;
};

// Bound by DRAM where tokens are many: both the ids and the rows are waited for, so
// a group of threads reads the ids of kTokens tokens and then has a column vector of
// each row in flight.  Four tokens a group of at most 64 threads, and one token with
// as many threads as it has columns for: 65536 tokens of 2048 fp32 to bf16 119 us and
// 140, 16384 of 7168 bf16 74 and 86, 10^6 of 16 fp32 14 and 41, 65536 of 4096 bf16
// 161 and 158 (6.7 TB/s); with eight tokens 125, 72, 17 and 233.
template <typename I, typename T, typename U, int kV, int kTokens>
__global__ void __launch_bounds__(kThreads)
    lookup_kernel(const I* __restrict__ ids, const T* __restrict__ table, const LookupShape s, float scale,
                  U* __restrict__ y) {
  pdl_wait();
  const int groups = kThreads / s.tx;
  // the groups' tokens take turns, so that a block's stores lie side by side
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * groups * kTokens + threadIdx.x / s.tx;
  const T* row[kTokens];
  bool live[kTokens];
  int64_t id[kTokens];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) id[k] = t0 + k * groups < s.tokens ? static_cast<int64_t>(read_at(ids, t0 + k * groups, s.tokens, I{0}, &g_embedding_status)) : 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    live[k] = t0 + k * groups < s.tokens && id[k] >= 0 && id[k] < s.rows;
    bad |= t0 + k * groups < s.tokens && !live[k];
    row[k] = table + (live[k] ? id[k] * s.ldw : 0);
  }
  if (bad) atomicOr(&g_embedding_status, MXQ_DEV_BADINDEX);
  const int64_t nv = s.D / kV;
  const uint64_t in_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldy + s.D) * sizeof(U);
  for (int64_t c = threadIdx.x % s.tx; c < nv; c += s.tx) {
    Vec<T, kV> v[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k)
      v[k] = load_if<T, kV>(row[k] + c * kV, live[k] && in_buf(row[k] + c * kV, sizeof v[k], table, in_bytes, &g_embedding_status));
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      Vec<U, kV> out;
#pragma unroll
      for (int i = 0; i < kV; ++i) out.v[i] = live[k] ? narrow<U>(scale * widen(v[k].v[i])) : U{};
      U* to = y + (t0 + k * groups) * s.ldy + c * kV;
      if (t0 + k * groups < s.tokens && in_buf(to, sizeof out, y, out_bytes, &g_embedding_status)) *reinterpret_cast<Vec<U, kV>*>(to) = out;
    }
  }
}

// Rows whose lengths, pitches or addresses allow accesses of 4 bytes or less of y,
// kIn elements at a time: staged as y's, and written in 16-byte units (65536 tokens
// of 1001 bf16 76 us, 136 with 2-byte stores; of 1001 fp32 to bf16 79 and 146; of 33
// fp32 10 and 15).  Not for rows of few bytes: most of a group would have nothing to do.
template <typename I, typename T, typename U, int kIn>
__global__ void __launch_bounds__(kThreads)
    lookup_narrow_kernel(const I* __restrict__ ids, const T* __restrict__ table, const LookupShape s, float scale,
                         U* __restrict__ y, int tiles, int tile) {
  constexpr bool kTwo = sizeof(U) * kIn == 2;
  constexpr int kLoads = kUnits * 16 / (sizeof(U) * kIn);
  __shared__ uint32_t stage[kTwo ? 2 : 1][kThreads * kUnits * 4 + kThreads / 8];
  pdl_wait();
  const int group = threadIdx.x / s.tx, own = threadIdx.x % s.tx;
  const int64_t t = static_cast<int64_t>(blockIdx.x / tiles) * (kThreads / s.tx) + group;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x % tiles) * tile;
  const int n = t < s.tokens ? static_cast<int>(min(static_cast<int64_t>(tile), s.D - c0)) : 0;
  const int64_t id = n > 0 ? static_cast<int64_t>(read_at(ids, t, s.tokens, I{0}, &g_embedding_status)) : -1;
  const bool live = id >= 0 && id < s.rows;
  if (n > 0 && !live && own == 0) atomicOr(&g_embedding_status, MXQ_DEV_BADINDEX);
  const T* row = table + (live ? id * s.ldw + c0 : 0);
  const uint64_t in_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldy + s.D) * sizeof(U);
  U* even = reinterpret_cast<U*>(stage[0] + group * (4 * kUnits * s.tx + 1));
  U* odd = reinterpret_cast<U*>(stage[kTwo ? 1 : 0] + group * (4 * kUnits * s.tx + 1)) + 1;  // one element further on
  Vec<T, kIn> v[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const T* p = row + (q * s.tx + own) * kIn;
    v[q] = load_if<T, kIn>(p, live && (q * s.tx + own) * kIn < n && in_buf(p, sizeof v[q], table, in_bytes, &g_embedding_status));
  }
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int i = (q * s.tx + own) * kIn;
    if (i >= n) continue;
#pragma unroll
    for (int e = 0; e < kIn; ++e) even[i + e] = live ? narrow<U>(scale * widen(v[q].v[e])) : U{};
    if (kTwo) odd[i] = even[i];
  }
  __syncthreads();
  if (n > 0)
    write_staged<U, kTwo>(even, odd, y + t * s.ldy + c0, n, own, s.tx, [&](const void* at, int size) {
      return in_buf(at, size, y, out_bytes, &g_embedding_status);
    });
}

// ---------------------------------------------------------------------------
// gradient: zeroing the table
// ---------------------------------------------------------------------------
// A launch's share of the table: `rows` rows of row_bytes, pitch bytes apart.
struct Fill {
  uint8_t* base;
  int64_t rows, row_bytes, pitch;
  const uint8_t* table;  // the whole table and its bytes, for the checked build
  uint64_t table_bytes;
};

__device__ __forceinline__ void zero_bytes(uint8_t* p, int64_t n, int64_t first, int64_t step, const Fill& f) {
  // 2-byte pieces up to the first 16-byte boundary and after the last one
  int64_t head = static_cast<int64_t>(-reinterpret_cast<intptr_t>(p) & 15);
  if (head > n) head = n;
  const int64_t body = (n - head) / 16, tail = (n - head) % 16;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = first; i < body; i += step)
    if (in_buf(q + i, 16, f.table, f.table_bytes, &g_embedding_status)) q[i] = make_uint4(0u, 0u, 0u, 0u);
  const auto zero_two = [&](uint8_t* at) {
    if (in_buf(at, 2, f.table, f.table_bytes, &g_embedding_status)) *reinterpret_cast<uint16_t*>(at) = 0;
  };
  if (first < head / 2) zero_two(p + 2 * first);
  if (first < tail / 2) zero_two(p + head + 16 * body + 2 * first);
}

// Blocks past the launch's own zero the fill; true for those.
template <int kBlockThreads>
__device__ __forceinline__ bool fill_block(const Fill& f, int own_blocks) {
  const int64_t block = static_cast<int64_t>(blockIdx.x) - own_blocks, blocks = gridDim.x - own_blocks;
  if (block < 0) return false;
  if (f.rows == 1) {
    zero_bytes(f.base, f.row_bytes, block * kBlockThreads + threadIdx.x, blocks * kBlockThreads, f);
  } else {
    for (int64_t r = block; r < f.rows; r += blocks)
      zero_bytes(f.base + r * f.pitch, f.row_bytes, threadIdx.x, kBlockThreads, f);
  }
  return true;
}

// ---------------------------------------------------------------------------
// gradient: sort
// ---------------------------------------------------------------------------
// Ids as keys: an id out of range, or the padding id, takes the key `rows`,
// behind every row of the table.
template <typename I>
struct IdKey {
  const I* ids;
  int64_t rows, padding, n;
  __device__ int full(int64_t i) const {
    const int64_t id = read_at(ids, i, n, I{0}, &g_embedding_status);
    if (id < 0 || id >= rows) {
      atomicOr(&g_embedding_status, MXQ_DEV_BADINDEX);
      return static_cast<int>(rows);
    }
    return static_cast<int>(id == padding ? rows : id);
  }
  __device__ int token(int64_t i) const { return static_cast<int>(i); }
};
struct SortedKey {
  const int32_t *keys, *tokens;
  int64_t n;
  __device__ int full(int64_t i) const { return read_at(keys, i, n, 0, &g_embedding_status); }
  __device__ int token(int64_t i) const { return read_at(tokens, i, n, 0, &g_embedding_status); }
};

template <typename Source>
__global__ void __launch_bounds__(kRankThreads)
    digit_count_kernel(const Source src, const RankSplit s, int shift, int bins, int32_t* chunk_counts, const Fill fill) {
  extern __shared__ int32_t counts[];
  pdl_wait();
  pdl_launch_dependents();  // the sort's blocks wait beside the zeroing ones
  if (fill_block<kRankThreads>(fill, s.chunks)) return;
  rank_count(s, bins, [&](int64_t i) { return (src.full(i) >> shift) & (bins - 1); }, counts);
  rank_keep_counts(s, bins, counts, chunk_counts, &g_embedding_status);
}

template <typename Source>
__global__ void __launch_bounds__(kRankThreads)
    digit_sort_kernel(const Source src, const RankSplit s, int shift, int bins,
                      const int32_t* __restrict__ chunk_counts, int32_t* __restrict__ keys,
                      int32_t* __restrict__ tokens, const Fill fill) {
  extern __shared__ int32_t smem[];
  int32_t* next = smem;
  int32_t* counts = smem + bins;
  __shared__ int32_t total[kRankMaxBins], begin[kRankMaxBins], work[kRankWarps];
  pdl_wait();
  pdl_launch_dependents();
  if (fill_block<kRankThreads>(fill, s.chunks)) return;
  const auto key = [&](int64_t i) { return (src.full(i) >> shift) & (bins - 1); };
  rank_totals(s, bins, chunk_counts, total, next, &g_embedding_status);
  rank_begins<1>(bins, total, begin, work);
  for (int b = threadIdx.x; b < bins; b += kRankThreads) next[b] += begin[b];
  __syncthreads();
  rank_chunk(
      s, bins, key,
      [&](int64_t i, int, int32_t place) {
        write_at(keys, place, s.n, src.full(i), &g_embedding_status);
        write_at(tokens, place, s.n, src.token(i), &g_embedding_status);
      },
      next, counts);
}

// Up to kSmallTokens tokens: all digits in one launch by one block, the items in
// its registers and, between the digits, in its shared memory.  A warp holds
// 32 * rounds consecutive items, so the order stays that of the tokens.
// Against the launches above: 16384 tokens 33 us, about as long, but 4096 13 us instead of 27.
constexpr int kSmallThreads = 1024;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallRounds = 16;
constexpr int64_t kSmallTokens = kSmallThreads * kSmallRounds;

inline size_t small_sort_smem(int64_t n, int bins) {
  return static_cast<size_t>(n) * 8 + static_cast<size_t>(kSmallWarps) * bins * 2 + static_cast<size_t>(bins) * 4;
}

template <int kRounds, typename Source>
__global__ void __launch_bounds__(kSmallThreads)
    small_sort_kernel(const Source src, int n, int passes, int bits, int32_t* __restrict__ keys,
                      int32_t* __restrict__ tokens, const Fill fill) {
  extern __shared__ int32_t smem[];
  __shared__ int32_t warp_sums[kSmallWarps];
  const int holders = (n + 32 * kRounds - 1) / (32 * kRounds);  // warps with items
  pdl_wait();
  pdl_launch_dependents();
  if (fill_block<kSmallThreads>(fill, 1)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bins = 1 << bits;
  int32_t* sorted_keys = smem;                                      // [n]
  int32_t* sorted_tokens = smem + n;                                // [n]
  int32_t* begin = smem + 2 * n;                                    // [bins]
  uint16_t* counts = reinterpret_cast<uint16_t*>(begin + bins);     // [warps, bins]
  uint16_t* mine = counts + warp * bins;
  const int first = warp * (32 * kRounds) + lane;
  int32_t key[kRounds], token[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int i = first + 32 * r;
    key[r] = i < n ? src.full(i) : -1;
    token[r] = i;
  }
  for (int q = 0; q < passes; ++q) {
    for (int i = tid; i < holders * bins / 2; i += kSmallThreads) reinterpret_cast<uint32_t*>(counts)[i] = 0u;
    __syncthreads();
    const int shift = q * bits;
    uint16_t at[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int d = key[r] >= 0 ? (key[r] >> shift) & (bins - 1) : -1;
      const uint32_t same = same_key(d, bits);
      const int before = d >= 0 ? mine[d] : 0;
      at[r] = static_cast<uint16_t>(before + __popc(same & ((1u << lane) - 1u)));
      __syncwarp();
      if (d >= 0 && lane == 31 - __clz(same)) mine[d] = static_cast<uint16_t>(at[r] + 1);
      __syncwarp();
    }
    __syncthreads();
    // per digit: the items of the warps before, and of the digits before
    int32_t total = 0;
    if (tid < bins) {
#pragma unroll 8
      for (int w = 0; w < holders; ++w) {
        const int c = counts[w * bins + tid];
        counts[w * bins + tid] = static_cast<uint16_t>(total);
        total += c;
      }
    }
    int32_t sum = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += y;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    int32_t before = lane < warp ? warp_sums[lane] : 0;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (tid < bins) begin[tid] = before + sum - total;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (key[r] >= 0) {
        const int d = (key[r] >> shift) & (bins - 1);
        const int place = begin[d] + mine[d] + at[r];
        sorted_keys[place] = key[r];
        sorted_tokens[place] = token[r];
      }
    __syncthreads();
    if (q + 1 < passes) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int i = first + 32 * r;
        if (i < n) {
          key[r] = sorted_keys[i];
          token[r] = sorted_tokens[i];
        }
      }
      __syncthreads();
    }
  }
  for (int i = tid; i < n; i += kSmallThreads) {
    write_at(keys, i, n, sorted_keys[i], &g_embedding_status);
    write_at(tokens, i, n, sorted_tokens[i], &g_embedding_status);
  }
}

// ---------------------------------------------------------------------------
// gradient: sums
// ---------------------------------------------------------------------------
struct GradShape {
  int64_t tokens, rows, D, ldd, ldw;
};
__host__ __device__ inline int64_t piece_floats(const GradShape& s) { return ceil_div(s.tokens, kChunk) * 2 * s.D; }

// First place whose key is >= v, by a whole warp: each step splits the range in
// 33 with 32 probes at once (3 dependent loads for 32768 keys, where a binary
// search has 15).
__device__ __forceinline__ int64_t warp_lower_bound(const int32_t* __restrict__ keys, int64_t n, int64_t v) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo) / 33 + 1;
    const int64_t at = lo + step * (lane + 1) - 1;  // probes lo + step - 1, lo + 2 step - 1, ...
    const bool below = at < hi && read_at(keys, at, n, 0, &g_embedding_status) < v;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));  // the first k probes lie below v
    const int64_t next = lo + step * k;
    hi = min(hi, next + step - 1);
    lo = next;
  }
  return lo;
}

// Column vectors and tokens that a thread holds at once: 64 bytes of wide pieces,
// more of narrow ones.
template <typename T, int kV>
__host__ __device__ constexpr int columns_at_once() {
  return sizeof(T) * kV >= 16 ? 1 : 4;
}
template <typename T, int kV>
__host__ __device__ constexpr int tokens_at_once() {
  return sizeof(T) * kV >= 16 ? 8 : sizeof(T) * kV >= 8 ? 2 : 4;
}

// acc[u] += dy[tokens[p]] over the places [lo, hi), in order, for the kU column
// vectors c, c + tx, ...: kU * kAhead loads before the first is used.
template <typename T, int kV, int kU>
__device__ __forceinline__ void add_tokens(const T* __restrict__ dy, const GradShape& s,
                                           const int32_t* tokens, int64_t lo, int64_t hi, int64_t c,
                                           int tx, int64_t nv, float (&acc)[kU][kV]) {
  const uint64_t bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldd + s.D) * sizeof(T);
  constexpr int kAhead = tokens_at_once<T, kV>();
  for (int64_t p = lo; p < hi; p += kAhead) {
    Vec<T, kV> v[kAhead][kU];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const T* row = dy + (p + a < hi ? static_cast<int64_t>(read_at(tokens, p + a, s.tokens, 0, &g_embedding_status)) * s.ldd : 0);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const T* src = row + (c + u * tx) * kV;
        const bool in = p + a < hi && c + u * tx < nv;
        v[a][u] = load_if<T, kV>(src, in && in_buf(src, sizeof v[a][u], dy, bytes, &g_embedding_status));
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[u][i] += widen(v[a][u].v[i]);
  }
}

// Pieces of the runs longer than kChunk places: pieces[2c] is the part of the
// run that holds the first place of chunk c, pieces[2c + 1] that of the run
// that holds its last place where this is another one.  Blocks of a chunk share
// its columns.
constexpr int kPieceThreads = 128;
template <typename T, int kV>
__global__ void __launch_bounds__(kPieceThreads)
    pieces_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ tokens, const T* __restrict__ dy,
                  const GradShape s, int column_blocks, float* __restrict__ pieces) {
  __shared__ int part_lo[2], part_hi[2];  // from the chunk's first place
  pdl_wait();
  static_assert(kChunk == 32, "a lane per place");
  constexpr int kU = columns_at_once<T, kV>();
  const int64_t chunk = blockIdx.x / column_blocks;
  const int64_t lo = chunk * kChunk, hi = min(lo + kChunk, s.tokens);
  if (threadIdx.x < 64) {
    // warp 0: the run of the chunk's first place; warp 1: that of its last one
    const int q = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t at = q == 0 ? lo : hi - 1;
    const auto key_at = [&](int64_t i) { return read_at(keys, i, s.tokens, 0, &g_embedding_status); };
    const int32_t key = key_at(at), first = key_at(lo);
    // equal keys side by side, up to kChunk of them before the place and from it on
    const bool before = at - 1 - lane >= 0 && key_at(at - 1 - lane) == key;
    const bool after = at + lane < s.tokens && key_at(at + lane) == key;
    const int left = __ffs(~__ballot_sync(0xFFFFFFFFu, before)) - 1, right = __ffs(~__ballot_sync(0xFFFFFFFFu, after)) - 1;
    const bool next = at + kChunk < s.tokens && key_at(at + kChunk) == key;  // one more than a whole chunk
    const int n_left = left < 0 ? 32 : left, n_right = right < 0 ? 32 + next : right;
    if (lane == 0) {
      const bool used = key < s.rows && n_left + n_right > kChunk && (q == 0 || key != first);
      const int n = static_cast<int>(hi - lo), place = static_cast<int>(at - lo);
      part_lo[q] = used ? max(0, place - n_left) : 0;
      part_hi[q] = used ? min(n, place + n_right) : 0;
    }
  }
  __syncthreads();
  const int64_t nv = s.D / kV;
  const int tx = column_blocks * kPieceThreads;
  for (int q = 0; q < 2; ++q) {
    if (part_lo[q] == part_hi[q]) continue;
    for (int64_t c = (blockIdx.x % column_blocks) * kPieceThreads + threadIdx.x; c < nv; c += kU * tx) {
      float acc[kU][kV] = {};
      add_tokens<T, kV, kU>(dy, s, tokens, lo + part_lo[q], lo + part_hi[q], c, tx, nv, acc);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c + u * tx < nv)
#pragma unroll
          for (int i = 0; i < kV; ++i)
            write_at(pieces, (2 * chunk + q) * s.D + (c + u * tx) * kV + i, piece_floats(s), acc[u][i], &g_embedding_status);
    }
  }
}

// acc[u] += the pieces of the run [lo, hi) in order, several loaded at once.
template <int kV, int kU>
__device__ __forceinline__ void add_pieces(const float* __restrict__ pieces, const GradShape& s, int64_t lo, int64_t hi,
                                           int64_t c, int tx, int64_t nv, float (&acc)[kU][kV]) {
  constexpr int kF = kV < 4 ? kV : 4, kAhead = kV * kU >= 16 ? 2 : 4;
  const int64_t last = (hi - 1) / kChunk;
  for (int64_t q = lo / kChunk; q <= last; q += kAhead) {
    Vec<float, kF> v[kAhead][kU][kV / kF];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const float* piece = pieces + (2 * (q + a) + ((q + a) * kChunk < lo ? 1 : 0)) * s.D;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int f = 0; f < kV / kF; ++f) {
          v[a][u][f] = Vec<float, kF>{};
          const float* p = piece + (c + u * tx) * kV + f * kF;
          if (q + a <= last && c + u * tx < nv && in_buf(p, sizeof(float) * kF, pieces, piece_floats(s) * 4, &g_embedding_status))
            v[a][u][f] = *reinterpret_cast<const Vec<float, kF>*>(p);
        }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[u][k] += v[a][u][k / kF].v[k % kF];
  }
}

template <typename T, int kV>
__host__ __device__ constexpr int row_columns() {
  return sizeof(T) * kV >= 16 ? 1 : sizeof(T) * kV >= 8 ? 2 : 4;
}

// Zeroes those of kAbsentRows rows of the table that no token has, each found by a
// search among the sorted ids.
constexpr int kAbsentRows = 64;
template <typename U>
__device__ __forceinline__ void zero_absent(const int32_t* __restrict__ keys, const GradShape& s, int64_t block,
                                            U* __restrict__ dtable) {
  __shared__ uint32_t absent[kAbsentRows / 32];
  const int64_t r0 = block * kAbsentRows;
  if (threadIdx.x < kAbsentRows) {
    const int64_t r = r0 + threadIdx.x;
    int64_t lo = 0, hi = s.tokens;
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (read_at(keys, mid, s.tokens, 0, &g_embedding_status) < r)
        lo = mid + 1;
      else
        hi = mid;
    }
    const uint32_t gone = __ballot_sync(0xFFFFFFFFu, r < s.rows && (lo == s.tokens || read_at(keys, lo, s.tokens, 0, &g_embedding_status) != r));
    if ((threadIdx.x & 31) == 0) absent[threadIdx.x / 32] = gone;
  }
  __syncthreads();
  Fill table = {};
  table.table = reinterpret_cast<const uint8_t*>(dtable);
  table.table_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(U);
  for (int w = 0; w < kAbsentRows / 32; ++w)
    for (uint32_t left = absent[w]; left != 0u; left &= left - 1)
      zero_bytes(reinterpret_cast<uint8_t*>(dtable + (r0 + 32 * w + __ffs(left) - 1) * s.ldw), s.D * sizeof(U), threadIdx.x,
                 blockDim.x, table);
}

// The rows of the runs that begin at one of the block's kStarts places.  A thread
// loads its columns of all those places' tokens before it adds any up: which run
// a place belongs to only decides where the sums are cut.  The last run is
// followed past the block's places; the first places may belong to a run that
// began before and are left out.
template <typename T, typename U, int kV>
__global__ void __launch_bounds__(kThreads, 4)
    rows_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ tokens, const T* __restrict__ dy,
                const GradShape s, const float* __restrict__ pieces, float scale, U* __restrict__ dtable, int64_t run_blocks) {
  __shared__ int32_t near_key[64], near_token[64];
  __shared__ uint64_t starts_of;
  pdl_wait();
  if (static_cast<int64_t>(blockIdx.x) >= run_blocks) {
    zero_absent<U>(keys, s, blockIdx.x - run_blocks, dtable);
    return;
  }
  static_assert(kStarts + kChunk < 64, "the ends of short runs lie within the places looked at");
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kStarts;
  if (threadIdx.x < 64) {
    const int64_t at = first + threadIdx.x;
    near_key[threadIdx.x] = at < s.tokens ? read_at(keys, at, s.tokens, -1, &g_embedding_status) : -1;
    near_token[threadIdx.x] = at < s.tokens ? read_at(tokens, at, s.tokens, 0, &g_embedding_status) : 0;
  }
  const int32_t before = first > 0 ? read_at(keys, first - 1, s.tokens, -1, &g_embedding_status) : -1;
  __syncthreads();
  if (threadIdx.x < 32) {  // a bit for each place where another id than before begins, or past the end
    const int i = threadIdx.x;
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, near_key[i] < 0 || near_key[i] != (i > 0 ? near_key[i - 1] : before));
    const uint32_t hi = __ballot_sync(0xFFFFFFFFu, near_key[32 + i] < 0 || near_key[32 + i] != near_key[31 + i]);
    if (i == 0) starts_of = static_cast<uint64_t>(hi) << 32 | lo;
  }
  __syncthreads();
  const uint64_t starts = starts_of;
  // places to add up, and those after which a row is written
  uint32_t live = 0, ends = 0;
  int last = -1, last_end = 0;  // a run that goes on past the block's places: its beginning and end
  bool long_run = false;
#pragma unroll
  for (int p = 0; p < kStarts; ++p) {
    if ((starts >> p & 1u) == 0u || near_key[p] < 0 || near_key[p] >= s.rows) continue;
    const int length = __ffsll(static_cast<long long>(starts >> (p + 1)));  // 0: past the places looked at
    if (length > 0 && p + length <= kStarts) {
      live |= ((1u << length) - 1u) << p;
      ends |= 1u << (p + length - 1);
    } else {
      last = p;
      long_run = length == 0 || length > kChunk;
      last_end = p + length;
      if (!long_run) live |= ((1u << kStarts) - 1u) & ~((1u << p) - 1u);
    }
  }
  if (live == 0u && last < 0) return;
  int64_t long_end = 0;
  if (long_run) long_end = warp_lower_bound(keys, s.tokens, static_cast<int64_t>(near_key[last]) + 1);
  const int64_t nv = s.D / kV;
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldd + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(U);
  constexpr int kU = row_columns<T, kV>();
  const int tx = blockDim.x;
  for (int64_t c = threadIdx.x; c < nv; c += kU * tx) {
    Vec<T, kV> v[kStarts][kU];
    float acc[kU][kV] = {};
    const auto load = [&](int place, bool wanted, Vec<T, kV> (&to)[kU]) {
      const T* src = dy + static_cast<int64_t>(near_token[place]) * s.ldd + c * kV;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        to[u] = load_if<T, kV>(src + u * tx * kV, wanted && c + u * tx < nv &&
                                                      in_buf(src + u * tx * kV, sizeof to[u], dy, in_bytes, &g_embedding_status));
    };
    const auto add = [&](const Vec<T, kV> (&from)[kU]) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[u][k] += widen(from[u].v[k]);
    };
    const auto write = [&](int32_t key) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        Vec<U, kV> out;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          out.v[k] = narrow<U>(scale * acc[u][k]);
          acc[u][k] = 0.0f;
        }
        U* to = dtable + key * s.ldw + (c + u * tx) * kV;
        if (c + u * tx < nv && in_buf(to, sizeof out, dtable, out_bytes, &g_embedding_status))
          *reinterpret_cast<Vec<U, kV>*>(to) = out;
      }
    };
#pragma unroll
    for (int p = 0; p < kStarts; ++p)
      load(p, (live >> p & 1u) != 0u, v[p]);
#pragma unroll
    for (int p = 0; p < kStarts; ++p)
      {
        add(v[p]);  // zero where not wanted
        if (ends >> p & 1u) write(near_key[p]);
      }
    if (last >= 0) {
      if (long_run) {
        add_pieces<kV, kU>(pieces, s, first + last, long_end, c, tx, nv, acc);
      } else {
        for (int p = kStarts; p < last_end; p += kStarts) {
#pragma unroll
          for (int q = 0; q < kStarts; ++q)
            load(p + q < last_end ? p + q : 0, p + q < last_end, v[q]);
#pragma unroll
          for (int q = 0; q < kStarts; ++q)
            add(v[q]);
        }
      }
      write(near_key[last]);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Elements per access: as many as every pitch and base address allow, at most
// 16 bytes of the wider type.
int vector_of(int in_size, int out_size, const void* in, const void* out, int64_t D, int64_t ld_in, int64_t ld_out) {
  const int a = common_alignment({address_of(in), static_cast<uint64_t>(D) * in_size, static_cast<uint64_t>(ld_in) * in_size});
  const int b = common_alignment({address_of(out), static_cast<uint64_t>(D) * out_size, static_cast<uint64_t>(ld_out) * out_size});
  const int va = a / in_size, vb = b / out_size;
  return va < vb ? va : vb;
}

int threads_per_row(int64_t nv) {
  int tx = 8;
  while (tx < kThreads && tx < nv) tx *= 2;
  return tx;
}

struct LookupCall {
  const void *ids, *table;
  LookupShape s;
  float scale;
  void* y;
  cudaStream_t stream;
};
template <typename I, typename T, typename U, int kV>
int launch_lookup(LookupCall a) {
  const I* ids = static_cast<const I*>(a.ids);
  const T* table = static_cast<const T*>(a.table);
  U* y = static_cast<U*>(a.y);
  if constexpr (sizeof(U) * kV <= 4) {
    if (a.s.D * sizeof(U) >= 64) {
      const StagedTiles split = staged_tiles(a.s.D, sizeof(U), kV, kThreads);
      a.s.tx = split.tx;
      return launch_pdl(lookup_narrow_kernel<I, T, U, kV>,
                        static_cast<unsigned>(ceil_div(a.s.tokens, kThreads / a.s.tx) * split.tiles), kThreads, 0, a.stream, ids,
                        table, a.s, a.scale, y, split.tiles, split.tile);
    }
  }
  const int64_t nv = a.s.D / kV;
  a.s.tx = 1;
  while (a.s.tx < 64 && a.s.tx < nv) a.s.tx *= 2;
  const int64_t groups = kThreads / a.s.tx;
  constexpr int kTokens = 4;
  if (a.s.tokens * a.s.tx >= kTokens * kFullGpu)
    return launch_pdl(lookup_kernel<I, T, U, kV, kTokens>, static_cast<unsigned>(ceil_div(a.s.tokens, groups * kTokens)), kThreads,
                      0, a.stream, ids, table, a.s, a.scale, y);
  a.s.tx = threads_per_row(nv);
  return launch_pdl(lookup_kernel<I, T, U, kV, 1>, static_cast<unsigned>(ceil_div(a.s.tokens, kThreads / a.s.tx)), kThreads, 0,
                    a.stream, ids, table, a.s, a.scale, y);
}
template <typename I, typename T, typename U>
int lookup_vector(const LookupCall& a) {
  const int v = vector_of(sizeof(T), sizeof(U), a.table, a.y, a.s.D, a.s.ldw, a.s.ldy);
  if constexpr (sizeof(T) == 2 && sizeof(U) == 2)
    if (v >= 8) return launch_lookup<I, T, U, 8>(a);
  return v >= 4 ? launch_lookup<I, T, U, 4>(a) : v >= 2 ? launch_lookup<I, T, U, 2>(a) : launch_lookup<I, T, U, 1>(a);
}
template <typename I>
int lookup_typed(const LookupCall& a, int dtype, int out_dtype) {
  if (dtype == MXQ_F32)
    return out_dtype == MXQ_F32 ? lookup_vector<I, float, float>(a) : lookup_vector<I, float, bf16_t>(a);
  return out_dtype == MXQ_F32 ? lookup_vector<I, bf16_t, float>(a) : lookup_vector<I, bf16_t, bf16_t>(a);
}

struct GradCall {
  const int32_t *keys, *tokens;
  const void* dy;
  GradShape s;
  float* pieces;
  float scale;
  void* dtable;
  cudaStream_t stream;
};

// The table in `parts` shares for zeroing; share q.  A table without gaps is one
// row, cut at 16-byte pieces.
Fill fill_share(void* dtable, const GradShape& s, int esize, int q, int parts) {
  Fill f = {};
  f.table = static_cast<const uint8_t*>(dtable);
  f.table_bytes = pitched_bytes(s.rows, s.D, s.ldw, esize);
  if (s.ldw == s.D) {
    const int64_t bytes = s.rows * s.D * esize, share = ceil_div(ceil_div(bytes, parts), 16) * 16;
    const int64_t lo = share * q < bytes ? share * q : bytes, hi = share * (q + 1) < bytes ? share * (q + 1) : bytes;
    f.base = static_cast<uint8_t*>(dtable) + lo;
    f.rows = 1;
    f.row_bytes = hi - lo;
  } else {
    const int64_t lo = s.rows * q / parts, hi = s.rows * (q + 1) / parts;
    f.base = static_cast<uint8_t*>(dtable) + lo * s.ldw * esize;
    f.rows = hi - lo;
    f.row_bytes = s.D * esize;
  }
  f.pitch = s.ldw * esize;
  return f;
}

// Where most rows may have a token, those that have none are zeroed by the last
// launch instead of all of them by the sort's, and none is written twice: 65536
// tokens of 4096 bf16, 32768 rows, 155 us instead of 182 (ids drawn evenly; 173 and
// 189 with frequent ones), 65536 rows of 2048 127 and 140 (141 and 140).  Not with
// more rows than tokens (131072 rows, frequent ids: 185 and 182), nor with few
// tokens, whose sort is one block beside which the zeroing costs nothing (16384
// tokens, 32768 rows of 4096: 113 and 94).
inline bool zeroed_late(const GradShape& s) { return s.tokens > kSmallTokens && s.rows <= s.tokens; }

template <typename T, typename U, int kV>
int launch_table(GradCall a) {
  const int64_t nv = a.s.D / kV;
  if (a.s.tokens > kChunk) {
    const int64_t blocks = ceil_div(nv, kPieceThreads * columns_at_once<T, kV>());
    const int column_blocks = static_cast<int>(blocks < 8 ? blocks : 8);
    const int64_t own = ceil_div(a.s.tokens, kChunk) * column_blocks;
    const int rc = launch_pdl(pieces_kernel<T, kV>, static_cast<unsigned>(own), kPieceThreads, 0, a.stream, a.keys,
                              a.tokens, static_cast<const T*>(a.dy), a.s, column_blocks, a.pieces);
    if (rc != MXQ_OK) return rc;
  }
  if (a.s.tokens == 0) return MXQ_OK;
  // as many threads as a row has columns for them, 64 to 256
  int threads = 64;
  while (threads < kThreads && threads * row_columns<T, kV>() < nv) threads *= 2;
  const int64_t run_blocks = ceil_div(a.s.tokens, kStarts);
  const int64_t absent_blocks = zeroed_late(a.s) ? ceil_div(a.s.rows, kAbsentRows) : 0;
  return launch_pdl(rows_kernel<T, U, kV>, static_cast<unsigned>(run_blocks + absent_blocks), threads, 0, a.stream, a.keys,
                    a.tokens, static_cast<const T*>(a.dy), a.s, a.pieces, a.scale, static_cast<U*>(a.dtable), run_blocks);
}
template <typename T, typename U>
int table_vector(const GradCall& a) {
  const int v = vector_of(sizeof(T), sizeof(U), a.dy, a.dtable, a.s.D, a.s.ldd, a.s.ldw);
  if constexpr (sizeof(T) == 2 && sizeof(U) == 2)
    if (v >= 8) return launch_table<T, U, 8>(a);
  return v >= 4 ? launch_table<T, U, 4>(a) : v >= 2 ? launch_table<T, U, 2>(a) : launch_table<T, U, 1>(a);
}

// Digits of the keys 0 .. rows (rows: no row of the table).
struct Digits {
  int passes, bits;
};
Digits digits_of(int64_t rows) {
  int bits = 1;
  while ((rows >> bits) != 0) ++bits;
  const int passes = (bits + kDigitBits - 1) / kDigitBits;
  return {passes, (bits + passes - 1) / passes};
}

struct GradPlan {
  RankSplit s;
  Digits d;
  int64_t counts, keys, pieces, bytes;  // byte offsets of the parts, and their sum
};
GradPlan grad_plan(int64_t tokens, int64_t rows, int64_t D) {
  GradPlan p;
  p.s = rank_split(tokens);
  p.d = digits_of(rows);
  const auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  p.counts = 0;
  p.keys = up(static_cast<int64_t>(p.s.chunks) * (int64_t{4} << p.d.bits));
  p.pieces = p.keys + up(16 * tokens);  // two buffers of keys and tokens
  p.bytes = p.pieces + (tokens > kChunk ? ceil_div(tokens, kChunk) * 2 * D * 4 : 0);
  return p;
}

template <typename Source>
int launch_digit(const Source& src, const GradPlan& p, int shift, int32_t* counts, int32_t* keys, int32_t* tokens,
                 const Fill* fills, int fill_blocks, cudaStream_t stream) {
  const int bins = 1 << p.d.bits;
  const int rc = launch_pdl(digit_count_kernel<Source>, p.s.chunks + fill_blocks, kRankThreads, bins * 4, stream, src, p.s,
                            shift, bins, counts, fills[0]);
  if (rc != MXQ_OK) return rc;
  return launch_pdl(digit_sort_kernel<Source>, p.s.chunks + fill_blocks, kRankThreads, rank_smem(bins), stream, src, p.s,
                    shift, bins, counts, keys, tokens, fills[1]);
}

template <int kRounds, typename Source>
int launch_small_sort(const Source& src, const GradPlan& p, int32_t* keys, int32_t* tokens, const Fill& fill,
                      int fill_blocks, cudaStream_t stream) {
  const auto kernel = small_sort_kernel<kRounds, Source>;
  const size_t most = small_sort_smem(static_cast<int64_t>(kRounds) * kSmallThreads, kRankMaxBins);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)) != cudaSuccess)
      return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  return launch_pdl(kernel, 1 + fill_blocks, kSmallThreads, small_sort_smem(p.s.n, 1 << p.d.bits), stream, src,
                    static_cast<int>(p.s.n), p.d.passes, p.d.bits, keys, tokens, fill);
}

constexpr int kMaxLaunches = 2 * 4;  // four digits of 8 bits at most

template <typename I>
int launch_gradient(const void* ids, const GradPlan& p, int64_t padding, uint8_t* workspace, GradCall a, int dtype,
                    int out_dtype, int sms) {
  int32_t* counts = reinterpret_cast<int32_t*>(workspace + p.counts);
  int32_t* buf = reinterpret_cast<int32_t*>(workspace + p.keys);
  const int64_t n = p.s.n;
  int32_t* keys[2] = {buf, buf + 2 * n};
  int32_t* tokens[2] = {buf + n, buf + 3 * n};
  // every launch of the sort zeroes an equal share of the table
  const bool small = n <= kSmallTokens;
  const int launches = small ? 1 : p.d.passes * 2;  // a digit's counting and its sort
  Fill fills[kMaxLaunches];
  for (int q = 0; q < launches; ++q) fills[q] = fill_share(a.dtable, a.s, element_bytes(out_dtype), q, launches);
  const int64_t want = zeroed_late(a.s) ? 0 : ceil_div(fills[0].rows * fills[0].row_bytes, 16 * kThreads * 4);
  const int fill_blocks = static_cast<int>(want < 8 * sms ? want : 8 * sms);
  const IdKey<I> source{static_cast<const I*>(ids), a.s.rows, padding, n};
  if (small) {
    const int blocks = static_cast<int>(ceil_div(fill_blocks, kSmallThreads / kThreads));
    const int rc = n <= kSmallThreads
                       ? launch_small_sort<1>(source, p, keys[0], tokens[0], fills[0], blocks, a.stream)
                   : n <= 4 * kSmallThreads
                       ? launch_small_sort<4>(source, p, keys[0], tokens[0], fills[0], blocks, a.stream)
                       : launch_small_sort<kSmallRounds>(source, p, keys[0], tokens[0], fills[0], blocks, a.stream);
    if (rc != MXQ_OK) return rc;
    a.keys = keys[0];
    a.tokens = tokens[0];
  } else {
    for (int q = 0; q < p.d.passes; ++q) {
      const int shift = q * p.d.bits, to = q & 1;
      const Fill* f = fills + 2 * q;
      const int rc = q == 0 ? launch_digit(source, p, shift, counts, keys[to], tokens[to], f, fill_blocks, a.stream)
                            : launch_digit(SortedKey{keys[to ^ 1], tokens[to ^ 1], n}, p, shift, counts, keys[to],
                                           tokens[to], f, fill_blocks, a.stream);
      if (rc != MXQ_OK) return rc;
    }
    const int last = (p.d.passes - 1) & 1;
    a.keys = keys[last];
    a.tokens = tokens[last];
  }
  a.pieces = reinterpret_cast<float*>(workspace + p.pieces);
  if (dtype == MXQ_F32) return out_dtype == MXQ_F32 ? table_vector<float, float>(a) : table_vector<float, bf16_t>(a);
  return out_dtype == MXQ_F32 ? table_vector<bf16_t, float>(a) : table_vector<bf16_t, bf16_t>(a);
}

bool good_dtype(int d) { return d == MXQ_F32 || d == MXQ_BF16; }

int check_table_shape(int64_t tokens, int ids_bytes, int64_t rows, int64_t D, int64_t lda, int64_t ldb) {
  if (ids_bytes != 4 && ids_bytes != 8) return MXQ_EBADDTYPE;
  if (tokens < 0 || tokens > INT32_MAX / 4 || rows < 0 || rows >= INT32_MAX || D < 0 || D > INT32_MAX || lda < D ||
      ldb < D || lda > INT32_MAX || ldb > INT32_MAX)
    return MXQ_EBADSHAPE;
  return MXQ_OK;
}

}  // namespace

namespace mxq {
int embedding_status_read(unsigned int* out, bool clear) { return read_status_word(g_embedding_status, out, clear); }
int embedding_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int mxq_embedding(const void* ids, int ids_bytes, int64_t tokens, const void* table, int dtype,
                             int64_t rows, int64_t D, int64_t ldw, float scale, void* y, int out_dtype, int64_t ldy,
                             cudaStream_t stream) {
  if (!good_dtype(dtype) || !good_dtype(out_dtype)) return MXQ_EBADDTYPE;
  const int rc = check_table_shape(tokens, ids_bytes, rows, D, ldw, ldy);
  if (rc != MXQ_OK) return rc;
  if (tokens == 0 || D == 0) return MXQ_OK;
  if (!ids || (rows > 0 && !table) || !y) return MXQ_ENULL;
  const int es = element_bytes(dtype), eo = element_bytes(out_dtype);
  if (!aligned_to(ids, ids_bytes) || !aligned_to(table, es) || !aligned_to(y, eo)) return MXQ_EALIGN;
  const ByteRange out[1] = {range_of(y, pitched_bytes(tokens, D, ldy, eo))};
  const ByteRange in[2] = {range_of(ids, static_cast<uint64_t>(tokens) * ids_bytes),
                           range_of(table, pitched_bytes(rows, D, ldw, es))};
  if (outputs_overlap(out, 1, in, 2)) return MXQ_EOVERLAP;
  const LookupCall a = {ids, table, {tokens, rows, D, ldw, ldy, 0}, scale, y, stream};
  return ids_bytes == 4 ? lookup_typed<int32_t>(a, dtype, out_dtype) : lookup_typed<int64_t>(a, dtype, out_dtype);
}

extern "C" int64_t mxq_embedding_backward_workspace(int64_t tokens, int64_t rows, int64_t D) {
  if (check_table_shape(tokens, 4, rows, D, D, D) != MXQ_OK) return MXQ_EBADSHAPE;
  return grad_plan(tokens, rows, D).bytes;
}

extern "C" int mxq_embedding_backward(const void* ids, int ids_bytes, int64_t tokens, const void* dy, int dtype,
                                      int64_t D, int64_t ldd, int64_t rows, int64_t padding, float scale, void* dtable,
                                      int out_dtype, int64_t ldw, uint8_t* workspace, int64_t workspace_bytes,
                                      cudaStream_t stream) {
  if (!good_dtype(dtype) || !good_dtype(out_dtype)) return MXQ_EBADDTYPE;
  const int rc = check_table_shape(tokens, ids_bytes, rows, D, ldd, ldw);
  if (rc != MXQ_OK) return rc;
  if (rows == 0 || D == 0) return MXQ_OK;
  const GradPlan p = grad_plan(tokens, rows, D);
  if (workspace_bytes < p.bytes) return MXQ_EBADSHAPE;
  if ((tokens > 0 && (!ids || !dy)) || !dtable || !workspace) return MXQ_ENULL;
  const int es = element_bytes(dtype), eo = element_bytes(out_dtype);
  if (!aligned_to(ids, ids_bytes) || !aligned_to(dy, es) || !aligned_to(dtable, eo) || !aligned_to(workspace, 16))
    return MXQ_EALIGN;
  const ByteRange out[2] = {range_of(dtable, pitched_bytes(rows, D, ldw, eo)), range_of(workspace, p.bytes)};
  const ByteRange in[2] = {range_of(ids, static_cast<uint64_t>(tokens) * ids_bytes),
                           range_of(dy, pitched_bytes(tokens, D, ldd, es))};
  if (outputs_overlap(out, 2, in, 2)) return MXQ_EOVERLAP;
  GradCall a = {};
  a.dy = dy;
  a.s = {tokens, rows, D, ldd, ldw};
  a.scale = scale;
  a.dtable = dtable;
  a.stream = stream;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;
  return ids_bytes == 4 ? launch_gradient<int32_t>(ids, p, padding, workspace, a, dtype, out_dtype, sms)
                        : launch_gradient<int64_t>(ids, p, padding, workspace, a, dtype, out_dtype, sms);
}
