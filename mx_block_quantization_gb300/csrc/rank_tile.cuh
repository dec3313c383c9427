// rank_tile.cuh -- stable counting sort by small integer keys, in two launches:
// the keys of each chunk of the input are counted, then every block ranks its
// own chunk behind what the chunks before it hold.  Used with the expert as key
// (the groups of routed tokens) and with digits of an id as key (the tokens of
// each table row).
//
// Ranks within a tile come from matching lanes of a warp: a warp takes 32
// consecutive items at a time, lanes with equal keys find one another with a
// vote for each bit of the key (match.any takes some 370 cycles for 32 different
// keys, a dozen times as long), and the lane's rank is the warp's count so far
// plus the matching lanes below it.
// The order is that of the items, so the result is the same in every run.
#pragma once

#include "train_common.cuh"

namespace mxq {

constexpr int kRankThreads = 256;
constexpr int kRankWarps = kRankThreads / 32;
constexpr int kRankRounds = 4;                             // items per lane and tile
constexpr int kRankTile = kRankThreads * kRankRounds;      // items per tile
constexpr int kRankMaxBins = 1024;
// At most this many chunks: every block of the second launch reads the counts
// of all of them.
constexpr int kRankMaxChunks = 128;

// The lanes of the warp with this lane's key, of the lanes with a key >= 0.
__device__ __forceinline__ uint32_t same_key(int key, int bits) {
  uint32_t same = __ballot_sync(0xFFFFFFFFu, key >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b & 1) != 0;
    const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// How n items are split: `chunks` blocks of `per` items (a multiple of a tile).
struct RankSplit {
  int64_t n, per;
  int chunks;
};
inline RankSplit rank_split(int64_t n) {
  int64_t chunks = ceil_div(n, kRankTile);
  if (chunks < 1) chunks = 1;
  if (chunks > kRankMaxChunks) chunks = kRankMaxChunks;
  const int64_t per = ceil_div(ceil_div(n, chunks), kRankTile) * kRankTile;
  const int64_t used = n > 0 ? ceil_div(n, per) : 1;
  return {n, per, static_cast<int>(used)};
}

// Shared memory of the ranking launch: counts per warp and bin, and the next
// place of each bin.
inline size_t rank_smem(int bins) { return static_cast<size_t>(kRankWarps + 1) * bins * 4; }

// counts[bin] of this block's chunk; key(i) < 0 leaves item i out.
template <typename Key>
__device__ void rank_count(const RankSplit& s, int bins, Key key, int32_t* counts) {
  for (int b = threadIdx.x; b < bins; b += kRankThreads) counts[b] = 0;
  __syncthreads();
  const int64_t lo = s.per * blockIdx.x, hi = min(s.n, lo + s.per);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kRankThreads) {
    const int k = key(i);
    if (k >= 0) atomicAdd(&counts[k], 1);
  }
  __syncthreads();
}

// Exclusive sum over the bins of padded(count), in place: begin[b].  Returns
// the sum over all bins.  `work` holds kRankWarps values.
template <int kAlign>
__device__ int32_t rank_begins(int bins, const int32_t* total, int32_t* begin, int32_t* work) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kRankThreads) {
    const int b = b0 + threadIdx.x;
    const int32_t v = b < bins ? (total[b] + kAlign - 1) / kAlign * kAlign : 0;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) work[warp] = x;
    __syncthreads();
    int32_t before = carry;
    for (int w = 0; w < warp; ++w) before += work[w];
    for (int w = 0; w < kRankWarps; ++w) carry += work[w];
    if (b < bins) begin[b] = before + x - v;
    __syncthreads();
  }
  return carry;
}

// Ranks this block's chunk.  next[bin] holds the place of the chunk's first
// item of that bin and is advanced; emit(i, key, place) is called for every
// item with a key >= 0, and emit(i, -1, -1) for the others.
template <typename Key, typename Emit>
__device__ void rank_chunk(const RankSplit& s, int bins, Key key, Emit emit, int32_t* next, int32_t* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lo = s.per * blockIdx.x, hi = min(s.n, lo + s.per);
  int32_t* mine = counts + warp * bins;
  const int bits = 32 - __clz(bins - 1);
  for (int64_t t0 = lo; t0 < hi; t0 += kRankTile) {
    for (int b = threadIdx.x; b < kRankWarps * bins; b += kRankThreads) counts[b] = 0;
    __syncthreads();
    int k[kRankRounds], at[kRankRounds];
    const int64_t i0 = t0 + warp * (32 * kRankRounds) + lane;
#pragma unroll
    for (int r = 0; r < kRankRounds; ++r) k[r] = i0 + 32 * r < hi ? key(i0 + 32 * r) : -1;
#pragma unroll
    for (int r = 0; r < kRankRounds; ++r) {
      const uint32_t same = same_key(k[r], bits);
      const int32_t before = k[r] >= 0 ? mine[k[r]] : 0;
      at[r] = before + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (k[r] >= 0 && lane == 31 - __clz(same)) mine[k[r]] = at[r] + 1;
      __syncwarp();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kRankThreads) {
      int32_t place = next[b];
#pragma unroll
      for (int w = 0; w < kRankWarps; ++w) {
        const int32_t c = counts[w * bins + b];
        counts[w * bins + b] = place;
        place += c;
      }
      next[b] = place;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRankRounds; ++r) {
      const int64_t i = i0 + 32 * r;
      if (i < hi) emit(i, k[r], k[r] >= 0 ? mine[k[r]] + at[r] : -1);
    }
    __syncthreads();
  }
}

// A block's counts for the second launch, one chunk's row of [chunks, bins].
__device__ __forceinline__ void rank_keep_counts(const RankSplit& s, int bins, const int32_t* counts,
                                                 int32_t* chunk_counts, unsigned int* status) {
  for (int b = threadIdx.x; b < bins; b += kRankThreads)
    write_at(chunk_counts, static_cast<int64_t>(blockIdx.x) * bins + b, static_cast<int64_t>(s.chunks) * bins, counts[b], status);
}

// Totals over all chunks and the sum over the chunks before this block's, from
// the [chunks, bins] counts of the first launch.
__device__ __forceinline__ void rank_totals(const RankSplit& s, int bins, const int32_t* chunk_counts,
                                            int32_t* total, int32_t* before, unsigned int* status) {
  for (int b = threadIdx.x; b < bins; b += kRankThreads) {
    int32_t all = 0, mine = 0;
#pragma unroll 8
    for (int c = 0; c < s.chunks; ++c) {
      const int32_t v = read_at(chunk_counts, static_cast<int64_t>(c) * bins + b, static_cast<int64_t>(s.chunks) * bins, 0, status);
      all += v;
      if (c < static_cast<int>(blockIdx.x)) mine += v;
    }
    total[b] = all;
    before[b] = mine;
  }
  __syncthreads();
}

}  // namespace mxq
