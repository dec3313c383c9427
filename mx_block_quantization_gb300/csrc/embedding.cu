// embedding.cu -- scaled lookup of table rows, and the table's gradient.
//
//   lookup     y[t] = scale * table[ids[t]]
//   gradient   dtable[v] = scale * sum over the tokens t with ids[t] = v of dy[t]
//
// The gradient sorts the tokens by id (rank_tile.cuh: stable, one launch pair
// per digit of at most 10 bits), so that the tokens of a row lie side by side,
// and then writes every row of the table once: zero where no token has it, the
// sum in token order otherwise.  A frequent id would keep one block busy for
// long, so a run of more than kChunk tokens is first summed in pieces, one per
// chunk of kChunk sorted places, by a launch of its own; the row then adds the
// pieces in order.  Sums are in fp32 and their order depends on the ids alone.
#include <cuda_runtime.h>
#include <stdint.h>

#include "rank_tile.cuh"
#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_embedding_status = 0;

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = 16;  // table rows a block of the gradient writes
constexpr int kChunk = 32;         // sorted places per piece of a long run
constexpr int kDigitBits = 10;     // at most kRankMaxBins bins

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
struct LookupShape {
  int64_t tokens, rows, D, ldw, ldy;
  int tx;
};

template <typename I, typename T, typename U, int kV>
__global__ void __launch_bounds__(kThreads)
    lookup_kernel(const I* __restrict__ ids, const T* __restrict__ table, const LookupShape s, float scale,
                  U* __restrict__ y) {
  pdl_wait();
  const int ty = kThreads / s.tx;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * ty + threadIdx.x / s.tx;
  if (t >= s.tokens) return;
  const int64_t id = ids[t];
  const bool live = id >= 0 && id < s.rows;
  if (!live) atomicOr(&g_embedding_status, MXQ_DEV_BADINDEX);
  const int64_t nv = s.D / kV;
  const uint64_t in_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldy + s.D) * sizeof(U);
  for (int64_t c = threadIdx.x % s.tx; c < nv; c += s.tx) {
    Vec<T, kV> v = {};
    if (live && in_buf(table + id * s.ldw + c * kV, sizeof v, table, in_bytes, &g_embedding_status))
      v = *reinterpret_cast<const Vec<T, kV>*>(table + id * s.ldw + c * kV);
    Vec<U, kV> out;
#pragma unroll
    for (int i = 0; i < kV; ++i) out.v[i] = live ? narrow<U>(scale * widen(v.v[i])) : U{};
    if (in_buf(y + t * s.ldy + c * kV, sizeof out, y, out_bytes, &g_embedding_status))
      *reinterpret_cast<Vec<U, kV>*>(y + t * s.ldy + c * kV) = out;
  }
}

// ---------------------------------------------------------------------------
// gradient: sort
// ---------------------------------------------------------------------------
// Ids as keys: an id out of range, or the padding id, takes the key `rows`,
// behind every row of the table.
template <typename I>
struct IdKey {
  const I* ids;
  int64_t rows, padding;
  __device__ int full(int64_t i) const {
    const int64_t id = ids[i];
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
  __device__ int full(int64_t i) const { return keys[i]; }
  __device__ int token(int64_t i) const { return tokens[i]; }
};

template <typename Source>
__global__ void __launch_bounds__(kRankThreads)
    digit_count_kernel(const Source src, const RankSplit s, int shift, int bins, int32_t* chunk_counts) {
  extern __shared__ int32_t counts[];
  pdl_wait();
  pdl_launch_dependents();  // as few blocks follow
  rank_count(s, bins, [&](int64_t i) { return (src.full(i) >> shift) & (bins - 1); }, counts);
  for (int b = threadIdx.x; b < bins; b += kRankThreads)
    chunk_counts[static_cast<int64_t>(blockIdx.x) * bins + b] = counts[b];
}

template <typename Source>
__global__ void __launch_bounds__(kRankThreads)
    digit_sort_kernel(const Source src, const RankSplit s, int shift, int bins,
                      const int32_t* __restrict__ chunk_counts, int32_t* __restrict__ keys,
                      int32_t* __restrict__ tokens) {
  extern __shared__ int32_t smem[];
  int32_t* next = smem;
  int32_t* counts = smem + bins;
  __shared__ int32_t total[kRankMaxBins], begin[kRankMaxBins], work[kRankWarps];
  pdl_wait();
  const auto key = [&](int64_t i) { return (src.full(i) >> shift) & (bins - 1); };
  if (s.chunks == 1) {
    rank_count(s, bins, key, total);
    for (int b = threadIdx.x; b < bins; b += kRankThreads) next[b] = 0;
  } else {
    rank_totals(s, bins, chunk_counts, total, next);
  }
  rank_begins<1>(bins, total, begin, work);
  for (int b = threadIdx.x; b < bins; b += kRankThreads) next[b] += begin[b];
  __syncthreads();
  const uint64_t bytes = static_cast<uint64_t>(s.n) * 4;
  rank_chunk(
      s, bins, key,
      [&](int64_t i, int, int32_t place) {
        if (!in_buf(keys + place, 4, keys, bytes, &g_embedding_status)) return;
        keys[place] = src.full(i);
        tokens[place] = src.token(i);
      },
      next, counts);
}

// ---------------------------------------------------------------------------
// gradient: sums
// ---------------------------------------------------------------------------
struct GradShape {
  int64_t tokens, rows, D, ldd, ldw;
  int tx;
};

// First place whose key is >= v, by a whole warp: each step splits the range in
// 33 with 32 probes at once (3 dependent loads for 32768 keys, where a binary
// search has 15).
__device__ __forceinline__ int64_t warp_lower_bound(const int32_t* __restrict__ keys, int64_t n, int64_t v) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo) / 33 + 1;
    const int64_t at = lo + step * (lane + 1) - 1;  // probes lo + step - 1, lo + 2 step - 1, ...
    const bool below = at < hi && keys[at] < v;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));  // the first k probes lie below v
    const int64_t next = lo + step * k;
    hi = min(hi, next + step - 1);
    lo = next;
  }
  return lo;
}

// acc[u] += dy[tokens[p]] over the places [lo, hi), in order, for the kU column
// vectors c, c + tx, ...: kU * kAhead loads before the first is used.
template <typename T, int kV, int kU>
__device__ __forceinline__ void add_tokens(const T* __restrict__ dy, const GradShape& s,
                                           const int32_t* __restrict__ tokens, int64_t lo, int64_t hi, int64_t c,
                                           int tx, int64_t nv, float (&acc)[kU][kV]) {
  const uint64_t bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ldd + s.D) * sizeof(T);
  constexpr int kAhead = 8 / kU;
  for (int64_t p = lo; p < hi; p += kAhead) {
    Vec<T, kV> v[kAhead][kU];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const T* row = dy + (p + a < hi ? static_cast<int64_t>(tokens[p + a]) * s.ldd : 0);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v[a][u] = Vec<T, kV>{};
        const T* src = row + (c + u * tx) * kV;
        if (p + a < hi && c + u * tx < nv && in_buf(src, sizeof v[a][u], dy, bytes, &g_embedding_status))
          v[a][u] = load_once<T, kV>(src);
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

// Column vectors a thread holds at once: more of them where each is narrow.
template <typename T, int kV>
__host__ __device__ constexpr int columns_at_once() {
  return sizeof(T) * kV >= 16 ? 2 : 4;
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
    const int32_t key = keys[at], first = keys[lo];
    // equal keys side by side, up to kChunk of them before the place and from it on
    const bool before = at - 1 - lane >= 0 && keys[at - 1 - lane] == key;
    const bool after = at + lane < s.tokens && keys[at + lane] == key;
    const int left = __ffs(~__ballot_sync(0xFFFFFFFFu, before)) - 1, right = __ffs(~__ballot_sync(0xFFFFFFFFu, after)) - 1;
    const bool next = at + kChunk < s.tokens && keys[at + kChunk] == key;  // one more than a whole chunk
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
    float* out = pieces + (2 * chunk + q) * s.D;
    for (int64_t c = (blockIdx.x % column_blocks) * kPieceThreads + threadIdx.x; c < nv; c += kU * tx) {
      float acc[kU][kV] = {};
      add_tokens<T, kV, kU>(dy, s, tokens, lo + part_lo[q], lo + part_hi[q], c, tx, nv, acc);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c + u * tx < nv)
#pragma unroll
          for (int i = 0; i < kV; ++i) out[(c + u * tx) * kV + i] = acc[u][i];
    }
  }
}

template <typename T, typename U, int kV>
__global__ void __launch_bounds__(kThreads)
    table_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ tokens, const T* __restrict__ dy,
                 const GradShape s, const float* __restrict__ pieces, float scale, U* __restrict__ dtable) {
  __shared__ int64_t range[2];
  __shared__ int64_t run_lo[kRowsPerBlock], run_hi[kRowsPerBlock];
  pdl_wait();
  constexpr int kU = columns_at_once<T, kV>();
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock;
  const int n = static_cast<int>(min(static_cast<int64_t>(kRowsPerBlock), s.rows - v0));
  if (threadIdx.x < 64) {
    const int64_t at = warp_lower_bound(keys, s.tokens, threadIdx.x < 32 ? v0 : v0 + n);
    if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = at;
  } else if (threadIdx.x - 64 < kRowsPerBlock) {
    run_lo[threadIdx.x - 64] = run_hi[threadIdx.x - 64] = 0;
  }
  __syncthreads();
  for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += kThreads) {
    const int32_t key = keys[i];
    if (i == range[0] || keys[i - 1] != key) run_lo[key - v0] = i;
    if (i == range[1] - 1 || keys[i + 1] != key) run_hi[key - v0] = i + 1;
  }
  __syncthreads();
  const int ty = kThreads / s.tx;
  const int64_t nv = s.D / kV;
  const uint64_t out_bytes = (static_cast<uint64_t>(s.rows - 1) * s.ldw + s.D) * sizeof(U);
  for (int r = threadIdx.x / s.tx; r < n; r += ty) {
    const int64_t lo = run_lo[r], hi = run_hi[r];
    U* row = dtable + (v0 + r) * s.ldw;
    for (int64_t c = threadIdx.x % s.tx; c < nv; c += kU * s.tx) {
      float acc[kU][kV] = {};
      if (hi - lo > kChunk) {
        for (int64_t q = lo / kChunk; q * kChunk < hi; ++q) {
          const float* piece = pieces + (2 * q + (q * kChunk < lo ? 1 : 0)) * s.D;
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (c + u * s.tx < nv)
#pragma unroll
              for (int i = 0; i < kV; ++i) acc[u][i] += piece[(c + u * s.tx) * kV + i];
        }
      } else if (hi > lo) {
        add_tokens<T, kV, kU>(dy, s, tokens, lo, hi, c, s.tx, nv, acc);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        Vec<U, kV> out;
#pragma unroll
        for (int i = 0; i < kV; ++i) out.v[i] = narrow<U>(scale * acc[u][i]);
        U* to = row + (c + u * s.tx) * kV;
        if (c + u * s.tx < nv && in_buf(to, sizeof out, dtable, out_bytes, &g_embedding_status))
          *reinterpret_cast<Vec<U, kV>*>(to) = out;
      }
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
  a.s.tx = threads_per_row(a.s.D / kV);
  return launch_pdl(lookup_kernel<I, T, U, kV>, static_cast<unsigned>(ceil_div(a.s.tokens, kThreads / a.s.tx)), kThreads,
                    0, a.stream, static_cast<const I*>(a.ids), static_cast<const T*>(a.table), a.s, a.scale,
                    static_cast<U*>(a.y));
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
template <typename T, typename U, int kV>
int launch_table(GradCall a) {
  const int64_t nv = a.s.D / kV;
  if (a.s.tokens > kChunk) {
    const int64_t blocks = ceil_div(nv, kPieceThreads * columns_at_once<T, kV>());
    const int column_blocks = static_cast<int>(blocks < 8 ? blocks : 8);
    const int rc = launch_pdl(pieces_kernel<T, kV>, static_cast<unsigned>(ceil_div(a.s.tokens, kChunk) * column_blocks),
                              kPieceThreads, 0, a.stream, a.keys, a.tokens, static_cast<const T*>(a.dy), a.s,
                              column_blocks, a.pieces);
    if (rc != MXQ_OK) return rc;
  }
  // a thread of a row holds several column vectors at once
  a.s.tx = threads_per_row(ceil_div(nv, columns_at_once<T, kV>()));
  return launch_pdl(table_kernel<T, U, kV>, static_cast<unsigned>(ceil_div(a.s.rows, kRowsPerBlock)), kThreads, 0,
                    a.stream, a.keys, a.tokens, static_cast<const T*>(a.dy), a.s, a.pieces, a.scale,
                    static_cast<U*>(a.dtable));
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
                 cudaStream_t stream) {
  const int bins = 1 << p.d.bits;
  if (p.s.chunks > 1) {
    const int rc = launch_pdl(digit_count_kernel<Source>, p.s.chunks, kRankThreads, bins * 4, stream, src, p.s, shift,
                              bins, counts);
    if (rc != MXQ_OK) return rc;
  }
  return launch_pdl(digit_sort_kernel<Source>, p.s.chunks, kRankThreads, rank_smem(bins), stream, src, p.s, shift, bins,
                    counts, keys, tokens);
}

template <typename I>
int launch_gradient(const void* ids, const GradPlan& p, int64_t padding, uint8_t* workspace, GradCall a, int dtype,
                    int out_dtype) {
  int32_t* counts = reinterpret_cast<int32_t*>(workspace + p.counts);
  int32_t* buf = reinterpret_cast<int32_t*>(workspace + p.keys);
  const int64_t n = p.s.n;
  int32_t* keys[2] = {buf, buf + 2 * n};
  int32_t* tokens[2] = {buf + n, buf + 3 * n};
  for (int q = 0; q < p.d.passes; ++q) {
    const int shift = q * p.d.bits, to = q & 1;
    const int rc = q == 0 ? launch_digit(IdKey<I>{static_cast<const I*>(ids), a.s.rows, padding}, p, shift, counts,
                                         keys[to], tokens[to], a.stream)
                          : launch_digit(SortedKey{keys[to ^ 1], tokens[to ^ 1]}, p, shift, counts, keys[to],
                                         tokens[to], a.stream);
    if (rc != MXQ_OK) return rc;
  }
  const int last = (p.d.passes - 1) & 1;
  a.keys = keys[last];
  a.tokens = tokens[last];
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
  a.s = {tokens, rows, D, ldd, ldw, 0};
  a.scale = scale;
  a.dtable = dtable;
  a.stream = stream;
  return ids_bytes == 4 ? launch_gradient<int32_t>(ids, p, padding, workspace, a, dtype, out_dtype)
                        : launch_gradient<int64_t>(ids, p, padding, workspace, a, dtype, out_dtype);
}
