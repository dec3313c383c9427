// moe_route.cu -- routing of tokens to experts with the balance loss, and the
// gradient of the logits.
//
// For a token's logits l over E experts:  p = softmax(l);  the k experts with
// the largest logits, ties to the lowest index;  weights p (or p over the
// chosen ones' sum);  counts_e = tokens that chose e;  and over the n routed
// tokens the balance loss  E/(k n^2) sum_e counts_e sum_t p_te.  With
// c_e = dloss E counts_e/(k n^2), the logits' gradient is
//   p_e (c_e - sum p c)  +  the chosen weights' part, which is
//   w_j (dw_j - sum w dw) at the chosen experts for weights over their sum, and
//   p_e ([e chosen] dw_e - sum_chosen p dw) otherwise.
//
// One warp owns a token (eight lanes with at most 32 experts, see below); a lane
// keeps kPer of its logits in registers, so the logits are read once each way, the
// next token's while this one is worked on.
// The k-th largest of the lanes' own maxima is at most the k-th largest logit, so
// only the few logits from there on (k to a dozen of random ones) are gathered,
// one per lane, and each counts those before it by keys that no two share.  With
// more than 32 such logits (many equal ones) every logit takes part in each of k
// rounds of a warp-wide maximum.  A lane also keeps the sums over its tokens of
// the probabilities of its experts; they are added up per block and then over the
// blocks in a fixed order, so the loss has the same bits in every run.
//
// Exponentials and the sums' reciprocals are the hardware's approximations, a few units
// in the last place: the exact forms' steps are worth more here than their last bits
// (131071 x 250: probabilities off by 1.2e-7, 4e-8 with them).
//
// The forward pass is bound by instruction issue, 430 a token with 250 experts in
// 90% of the issue slots: the softmax and the loss's sums take 40 of them for a
// lane's 8 logits, the choice most of the rest.  131071 x 250 fp32, k = 6: 56 us,
// 2.3 TB/s (a float and an index compared instead of one key cost 4 us more, a
// ballot for each of a lane's logits instead of one count 2).  The backward pass
// reads the logits again, as keeping p would cost a write and the same read:
// 48 us, 5.5 TB/s.  7168 x 64 bf16, k = 8: 10 us and 4.7, mostly the latency of
// three launches.
#include "moe_route_common.cuh"

namespace {

using namespace mxq;

template <typename T, int kPer, int kV, int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    route_kernel(const T* __restrict__ logits, const RouteShape s, const uint8_t* __restrict__ mask,
                 float* __restrict__ weights, int32_t* __restrict__ ids, float* part_p,
                 int32_t* part_c, int32_t* part_n, uint32_t* joined, int32_t* counts, float* loss, int32_t* n_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  float* by_warp = reinterpret_cast<float*>(smem);          // [warps, 32 * kPer]
  int32_t* hist = reinterpret_cast<int32_t*>(by_warp + kPer * kThreads);  // [E]
  float* sums = reinterpret_cast<float*>(hist + s.E);       // [E]
  __shared__ int32_t routed_tokens;
  using Key = typename ChoiceKey<T>::type;
  __shared__ int few_n[kWarps];
  __shared__ __align__(16) float2 few[kWarps][32];          // the logits gathered with their experts, then their keys
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < s.E; e += kThreads) hist[e] = 0;
  if (tid == 0) routed_tokens = 0;
  if (lane == 0) few_n[warp] = 0;
  __syncthreads();
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>(s.tokens) * s.k * 4;
  if (gridDim.x > 1) pdl_launch_dependents();  // the join's few blocks wait beside this one
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  int routed_here = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  Row<T, kPer, kV> ahead;
  const auto fetch = [&](int64_t t) {
    if (t < s.tokens && in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status))
      ahead.load(logits + t * s.ld, s.E, lane);
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  fetch(t);
  for (; t < s.tokens; t += step) {
    float x[kPer];
    ahead.values(x);
    fetch(t + step);
    float best = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = fmaxf(best, x[i]);  // skips NaN
    // the k-th largest lane maximum, equal ones counted once; 0 when there are fewer
    uint32_t mine = order_key(best);
    const uint32_t top_key = __reduce_max_sync(0xFFFFFFFFu, mine);
    uint32_t bar = top_key;
#pragma unroll 4
    for (int j = 1; j < s.k; ++j) {
      if (mine == bar) mine = 0u;
      bar = __reduce_max_sync(0xFFFFFFFFu, mine);
    }
    bool routed = mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0;
    if (routed && top_key == 0u) {  // no logit to choose: counted only if one is NaN
      bool nan = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) nan |= x[i] != x[i];
      routed = __any_sync(0xFFFFFFFFu, nan);
    }
    // a lane with a chosen expert: its place among the chosen, its expert and its logit
    int rank = kMaxK, my_id = -1;
    float my_x = 0.0f, my_w = 0.0f;
    if (routed) {
      ++routed_here;
      const float top = top_key != 0u ? key_value(top_key) : -CUDART_INF_F;
      const float from = bar != 0u ? key_value(bar) : -FLT_MAX;
      if (top_key != 0u) {
        // how many of them this lane has, and where it puts them, in any order
        int own_n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) own_n += x[i] >= from ? 1 : 0;  // not NaN and -inf
        int at = 0;
        if (own_n > 0) at = atomicAdd(&few_n[warp], own_n);
        const int n = __reduce_add_sync(0xFFFFFFFFu, own_n);
        __syncwarp();
        if (lane == 0) few_n[warp] = 0;  // for the next token
        if (n <= 32) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (x[i] >= from) few[warp][at++] = make_float2(x[i], __int_as_float(expert_of<kV>(i, lane)));
          __syncwarp();
          const float2 own = few[warp][lane];
          const int e = __float_as_int(own.y);
          const Key key = lane < n ? ChoiceKey<T>::of(own.x, e) : 0;
          Key* keys = reinterpret_cast<Key*>(few[warp]);
          __syncwarp();
          keys[lane] = key;
          __syncwarp();
          int before = 0;
          constexpr int kAtOnce = 16 / sizeof(Key);
          for (int i = 0; i < n; i += kAtOnce) {
            const Vec<Key, kAtOnce> other = *reinterpret_cast<const Vec<Key, kAtOnce>*>(keys + i);
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) before += other.v[q] > key ? 1 : 0;
          }
          if (lane < n && before < s.k) {
            rank = before;
            my_id = e;
            my_x = own.x;
          }
        } else {
          uint32_t key[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) key[i] = order_key(x[i]);
          for (int j = 0; j < s.k; ++j) {
            uint32_t local = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (key[i] > local) local = key[i], at = expert_of<kV>(i, lane);
            const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, local);
            if (m == 0u) break;
            const int e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, local == m ? static_cast<uint32_t>(at) : ~0u));
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (expert_of<kV>(i, lane) == e) key[i] = 0u;
            if (lane == j) {
              rank = j;
              my_id = e;
              my_x = key_value(m);
            }
          }
        }
        __syncwarp();
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] = exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
        sum += x[i];
      }
      const float inv = reciprocal(warp_sum(sum));
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
      if (my_id >= 0) {
        my_w = exp2_ftz((my_x - top) * kLog2E) * inv;  // NaN in a row with NaN or +inf
        atomicAdd(&hist[my_id], 1);
      }
      if (s.renorm) my_w /= warp_sum(my_w);
      if (my_id < 0) my_w = 0.0f;
    }
    // the chosen ones' lanes write their places, and as many others the places left
    const uint32_t chosen = __ballot_sync(0xFFFFFFFFu, my_id >= 0);
    if (my_id < 0) rank = __popc(chosen) + __popc(~chosen & ((1u << lane) - 1u));
    if (rank < s.k && in_buf(weights + t * s.k + rank, 4, weights, out_bytes, &g_route_status) &&
        in_buf(ids + t * s.k + rank, 4, ids, out_bytes, &g_route_status)) {
      weights[t * s.k + rank] = my_w;
      ids[t * s.k + rank] = my_id;
    }
  }
  if (lane == 0 && routed_here) atomicAdd(&routed_tokens, routed_here);
  // the warps' sums side by side, then added up in warp order
#pragma unroll
  for (int i = 0; i < kPer; ++i) by_warp[warp * (32 * kPer) + expert_of<kV>(i, lane)] = acc[i];
  __syncthreads();
  for (int e = tid; e < s.E; e += kThreads) {
    float sum = 0.0f;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) sum += by_warp[w * (32 * kPer) + e];
    sums[e] = sum;
  }
  __syncthreads();
  finish_block(s, sums, hist, routed_tokens, part_p, part_c, part_n, joined, counts, loss, n_out);
}

// At most 32 experts: eight lanes a token, lane l with the experts l, l + 8, ..., four
// tokens a warp.  Every logit counts those before it, so there is nothing to gather.
// (131072 tokens of 8 experts fp32, k = 2: 13.5 us forward and 8.3 backward, 48 and 33
// with a warp a token; of 32, k = 4: 31 and 16, 52 and 35.)
constexpr int kFewThreads = 1024, kFewBackThreads = 256, kFewExperts = 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
template <typename V, typename Op>
__device__ __forceinline__ V over_eight(V v, Op op) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ float sum_eight(float v) {
  return over_eight(v, [](float a, float b) { return a + b; });
}
// A token's logits in its eight lanes: loaded ahead, -inf past E and past the tokens.
template <typename T, int kPer>
struct FewRow {
  T v[kPer];
  __device__ __forceinline__ void load(const T* logits, const RouteShape& s, int64_t t, int sub, uint64_t bytes) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const T* p = logits + t * s.ld + sub + 8 * i;
      v[i] = minus_infinity<T>();
      if (t < s.tokens && sub + 8 * i < s.E && in_buf(p, sizeof(T), logits, bytes, &g_route_status)) v[i] = *p;
    }
  }
};
// The softmax of a token over its eight lanes; whether it takes part.
template <int kPer>
struct FewSoftmax {
  float p[kPer];
  uint32_t key[kPer];
  bool routed;
  template <typename T>
  __device__ __forceinline__ FewSoftmax(const FewRow<T, kPer>& row, bool unmasked) {
    uint32_t best = 0u;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      p[i] = widen(row.v[i]);
      key[i] = order_key(p[i]);
      best = max(best, key[i]);
      nan |= p[i] != p[i];
    }
    best = over_eight(best, [](uint32_t a, uint32_t b) { return max(a, b); });
    const uint32_t nans = __ballot_sync(kAll, nan) >> (threadIdx.x & 24u) & 0xFFu;
    routed = unmasked && (best != 0u || nans != 0u);
    const float top = best != 0u ? key_value(best) : -CUDART_INF_F;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      p[i] = exp2_ftz((p[i] - top) * kLog2E);  // 0 past E: those are -inf
      sum += p[i];
    }
    const float inv = reciprocal(sum_eight(sum));
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] *= inv;
  }
};

template <typename T, int kPer>
__global__ void __launch_bounds__(kFewThreads)
    route_few_kernel(const T* __restrict__ logits, const RouteShape s, const uint8_t* __restrict__ mask,
                     float* __restrict__ weights, int32_t* __restrict__ ids, float* part_p, int32_t* part_c,
                     int32_t* part_n, uint32_t* joined, int32_t* counts, float* loss, int32_t* n_out) {
  __shared__ float by_group[kFewThreads / 8][8 * kPer];
  __shared__ float sums[8 * kPer];
  __shared__ int32_t hist[8 * kPer], routed_tokens;
  const int tid = threadIdx.x, sub = tid & 7, base = tid & 24;
  if (tid < 8 * kPer) hist[tid] = 0;
  if (tid == 0) routed_tokens = 0;
  __syncthreads();
  pdl_wait();
  if (gridDim.x > 1) pdl_launch_dependents();  // the join's few blocks wait beside this one
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>(s.tokens) * s.k * 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kFewThreads / 8);
  float acc[kPer] = {};
  int routed_here = 0;
  FewRow<T, kPer> ahead;
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 8) + tid / 8;
  ahead.load(logits, s, t, sub, in_bytes);
  for (; t - base / 8 < s.tokens; t += step) {  // the warp's first token
    const FewRow<T, kPer> row = ahead;
    ahead.load(logits, s, t + step, sub, in_bytes);
    const bool in = t < s.tokens;
    const FewSoftmax<kPer> soft(row, in && (mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0));
    int rank[kPer] = {};
#pragma unroll
    for (int j = 0; j < 8 * kPer; ++j) {
      const uint32_t other = __shfl_sync(kAll, soft.key[j / 8], base | (j & 7));
#pragma unroll
      for (int i = 0; i < kPer; ++i) rank[i] += other > soft.key[i] || (other == soft.key[i] && j < sub + 8 * i) ? 1 : 0;
    }
    float w[kPer], all = 0.0f;
    int chosen = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool own = soft.routed && soft.key[i] != 0u && rank[i] < s.k;
      if (!own) rank[i] = kFewExperts;
      w[i] = own ? soft.p[i] : 0.0f;
      all += w[i];
      chosen += __popc(__ballot_sync(kAll, own) >> base & 0xFFu);
      if (soft.routed) acc[i] += soft.p[i];
    }
    all = sum_eight(all);
    if (soft.routed && sub == 0) ++routed_here;
    const auto write = [&](int place, float weight, int32_t e) {
      if (in_buf(weights + t * s.k + place, 4, weights, out_bytes, &g_route_status) &&
          in_buf(ids + t * s.k + place, 4, ids, out_bytes, &g_route_status)) {
        weights[t * s.k + place] = weight;
        ids[t * s.k + place] = e;
      }
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (rank[i] < kFewExperts) {
        write(rank[i], s.renorm ? w[i] / all : w[i], sub + 8 * i);
        atomicAdd(&hist[sub + 8 * i], 1);
      }
    for (int place = chosen + sub; in && place < s.k; place += 8) write(place, 0.0f, -1);
  }
  if (routed_here) atomicAdd(&routed_tokens, routed_here);
#pragma unroll
  for (int i = 0; i < kPer; ++i) by_group[tid / 8][sub + 8 * i] = acc[i];
  __syncthreads();
  if (tid < s.E) {
    float sum = 0.0f;
#pragma unroll 16
    for (int g = 0; g < kFewThreads / 8; ++g) sum += by_group[g][tid];
    sums[tid] = sum;
  }
  __syncthreads();
  finish_block(s, sums, hist, routed_tokens, part_p, part_c, part_n, joined, counts, loss, n_out);
}

template <typename T, int kPer>
__global__ void __launch_bounds__(kFewBackThreads)
    route_backward_few_kernel(const T* __restrict__ logits, const RouteShape s, const uint8_t* __restrict__ mask,
                              const int32_t* __restrict__ ids, const int32_t* __restrict__ counts,
                              const int32_t* __restrict__ n_in, const float* __restrict__ dweights,
                              const float* __restrict__ dloss, T* __restrict__ dlogits, int64_t ldd) {
  const int tid = threadIdx.x, sub = tid & 7, base = tid & 24;
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * ldd + s.E) * sizeof(T);
  float c[kPer];
  const float n = static_cast<float>(*n_in);
  const float f = dloss != nullptr && n > 0.0f ? *dloss * (static_cast<float>(s.E) / (static_cast<float>(s.k) * n * n)) : 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) c[i] = dloss != nullptr && sub + 8 * i < s.E ? f * static_cast<float>(read_at(counts, sub + 8 * i, s.E, 0, &g_route_status)) : 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kFewBackThreads / 8);
  FewRow<T, kPer> ahead;
  int32_t e_ahead[kPer];
  float dw_ahead[kPer];
  const auto fetch = [&](int64_t t) {
    ahead.load(logits, s, t, sub, in_bytes);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool there = dweights != nullptr && t < s.tokens && sub + 8 * i < s.k;
      e_ahead[i] = there ? read_at(ids, t * s.k + sub + 8 * i, s.tokens * s.k, -1, &g_route_status) : -1;
      dw_ahead[i] = there ? read_at(dweights, t * s.k + sub + 8 * i, s.tokens * s.k, 0.0f, &g_route_status) : 0.0f;
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kFewBackThreads / 8) + tid / 8;
  fetch(t);
  for (; t - base / 8 < s.tokens; t += step) {  // the warp's first token
    const FewRow<T, kPer> row = ahead;
    int32_t e[kPer];
    float dw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = e_ahead[i], dw[i] = dw_ahead[i];
    fetch(t + step);
    const bool in = t < s.tokens;
    const FewSoftmax<kPer> soft(row, in && (mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0));
    // the chosen experts' gradients in their own lanes
    float own_dw[kPer] = {};
    bool own[kPer] = {};
#pragma unroll
    for (int j = 0; j < 8 * kPer; ++j) {
      if (j >= s.k) break;
      const int32_t id = __shfl_sync(kAll, e[j / 8], base | (j & 7));
      const float d = __shfl_sync(kAll, dw[j / 8], base | (j & 7));
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (id == sub + 8 * i) own[i] = true, own_dw[i] = d;
    }
    float pc = 0.0f, all = 0.0f, part[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pc = fmaf(soft.p[i], c[i], pc);
      all += own[i] ? soft.p[i] : 0.0f;
    }
    if (s.renorm) {
      all = sum_eight(all);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        part[i] = own[i] ? soft.p[i] / all : 0.0f;
        dot = own[i] ? fmaf(part[i], own_dw[i], dot) : dot;
      }
      dot = sum_eight(dot);
#pragma unroll
      for (int i = 0; i < kPer; ++i) part[i] = own[i] ? part[i] * (own_dw[i] - dot) : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        part[i] = own[i] ? soft.p[i] * own_dw[i] : 0.0f;
        pc += part[i];
      }
    }
    const float total = sum_eight(pc);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      T* to = dlogits + t * ldd + sub + 8 * i;
      const float d = soft.routed ? fmaf(soft.p[i], c[i] - total, part[i]) : 0.0f;
      if (in && sub + 8 * i < s.E && in_buf(to, sizeof(T), dlogits, out_bytes, &g_route_status)) *to = narrow<T>(d);
    }
  }
}

template <typename T, int kPer, int kV, int kThreads>
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const T* __restrict__ logits, const RouteShape s, const uint8_t* __restrict__ mask,
                          const int32_t* __restrict__ ids, const int32_t* __restrict__ counts,
                          const int32_t* __restrict__ n_in, const float* __restrict__ dweights,
                          const float* __restrict__ dloss, T* __restrict__ dlogits, int64_t ldd) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the chosen experts' part of a row, zero between rows
  constexpr int kRow = kPer * 32;
  float* chosen = reinterpret_cast<float*>(smem) + warp * 2 * kRow;
  float* probs = chosen + kRow;
  for (int e = lane; e < kRow; e += 32) chosen[e] = 0.0f;
  __syncwarp();
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = (static_cast<uint64_t>(s.tokens - 1) * ldd + s.E) * sizeof(T);
  float c[kPer];
  {
    const float n = static_cast<float>(*n_in);
    const float f = dloss != nullptr && n > 0.0f ? *dloss * (static_cast<float>(s.E) / (static_cast<float>(s.k) * n * n)) : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = expert_of<kV>(i, lane);
      c[i] = dloss != nullptr && e < s.E ? f * static_cast<float>(read_at(counts, e, s.E, 0, &g_route_status)) : 0.0f;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  // the next token's logits, chosen experts and their gradients
  Row<T, kPer, kV> ahead;
  int32_t e_ahead = -1;
  float dw_ahead = 0.0f;
  const auto fetch = [&](int64_t t) {
    if (t >= s.tokens) return;
    if (in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status))
      ahead.load(logits + t * s.ld, s.E, lane);
    if (dweights != nullptr && lane < s.k) {
      e_ahead = read_at(ids, t * s.k + lane, s.tokens * s.k, -1, &g_route_status);
      dw_ahead = read_at(dweights, t * s.k + lane, s.tokens * s.k, 0.0f, &g_route_status);
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  fetch(t);
  for (; t < s.tokens; t += step) {
    const int e = e_ahead >= 0 && e_ahead < s.E ? e_ahead : -1;
    float dw = dw_ahead;
    float x[kPer];
    ahead.values(x);
    fetch(t + step);
    float top = -CUDART_INF_F;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      top = fmaxf(top, x[i]);  // skips NaN
      nan |= x[i] != x[i];
    }
    top = key_value(__reduce_max_sync(0xFFFFFFFFu, order_key(top)));
    const bool some = top > -CUDART_INF_F;  // false for NaN, the value of key 0
    const bool routed = (mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0) && (some || __any_sync(0xFFFFFFFFu, nan));
    T* out = dlogits + t * ldd;
    if (routed) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] = exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
        sum += x[i];
      }
      const float inv = reciprocal(warp_sum(sum));
      float pc = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] *= inv;
        pc = fmaf(x[i], c[i], pc);
      }
      // the probabilities of the chosen experts, from the lanes that hold them
#pragma unroll
      for (int q = 0; q < kPer / kV; ++q) {
        Vec<float, kV> p;
#pragma unroll
        for (int i = 0; i < kV; ++i) p.v[i] = x[q * kV + i];
        *reinterpret_cast<Vec<float, kV>*>(probs + expert_of<kV>(q * kV, lane)) = p;
      }
      __syncwarp();
      float w = e >= 0 ? probs[e] : 0.0f;
      if (e < 0) dw = 0.0f;
      float part = 0.0f;
      if (s.renorm) {
        const float all = warp_sum(w);
        if (e >= 0) w /= all;
        const float dot = warp_sum(w * dw);
        part = w * (dw - dot);
      } else {
        part = w * dw;
        pc += part;
      }
      if (e >= 0) chosen[e] = part;
      __syncwarp();
      const float total = warp_sum(pc);
#pragma unroll
      for (int q = 0; q < kPer / kV; ++q) {
        const Vec<float, kV> add = *reinterpret_cast<const Vec<float, kV>*>(chosen + expert_of<kV>(q * kV, lane));
#pragma unroll
        for (int i = 0; i < kV; ++i) x[q * kV + i] = fmaf(x[q * kV + i], c[q * kV + i] - total, add.v[i]);
      }
      __syncwarp();
      if (e >= 0) chosen[e] = 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = 0.0f;
    }
    if (!in_buf(out, s.E * sizeof(T), dlogits, out_bytes, &g_route_status)) continue;
#pragma unroll
    for (int q = 0; q < kPer / kV; ++q) {
      const int e0 = expert_of<kV>(q * kV, lane);
      if (e0 + kV <= s.E) {
        Vec<T, kV> v;
#pragma unroll
        for (int j = 0; j < kV; ++j) v.v[j] = narrow<T>(x[q * kV + j]);
        *reinterpret_cast<Vec<T, kV>*>(out + e0) = v;
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (e0 + j < s.E) out[e0 + j] = narrow<T>(x[q * kV + j]);
      }
    }
  }
}

// tokens that a block works on at a time, for that many experts
int tokens_at_once(int experts) {
  if (experts <= kFewExperts) return kFewThreads / 8;
  return (experts <= 256 ? route_threads<8>() : experts <= 512 ? route_threads<16>() : route_threads<32>()) / 32;
}
struct RouteCall {
  const void* logits;
  RouteShape s;
  const uint8_t* mask;
  float* weights;
  int32_t *ids, *counts;
  float* loss;
  int32_t* n;
  uint8_t* workspace;
  // backward
  const float *dweights, *dloss;
  void* dlogits;
  int64_t ldd;
  int sms;
  cudaStream_t stream;
};

// A forward kernel of that block size, and the join where there is more than one.
template <typename Kernel>
int launch_forward(const RouteCall& a, Kernel kernel, int threads, size_t smem) {
  const int blocks = route_blocks(a.s.tokens, tokens_at_once(a.s.E), a.sms);
  float* part_p = reinterpret_cast<float*>(a.workspace);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + static_cast<int64_t>(blocks) * a.s.E);
  int32_t* part_n = part_c + static_cast<int64_t>(blocks) * a.s.E;
  uint32_t* joined = reinterpret_cast<uint32_t*>(part_n + blocks);
  float* part_loss = reinterpret_cast<float*>(joined + 1);
  const int rc = kernel(blocks, threads, smem, part_p, part_c, part_n, joined);
  if (rc != MXQ_OK || blocks == 1) return rc;
  return launch_pdl(route_join_kernel, static_cast<unsigned>(ceil_div(a.s.E, 32)), 32 * kJoinWarps, 0, a.stream, a.s, blocks,
                    part_p, part_c, part_n, joined, part_loss, a.counts, a.loss, a.n);
}
template <typename T, int kPer, int kV>
int launch_route(const RouteCall& a) {
  constexpr int kThreads = route_threads<kPer>();
  return launch_forward(a, [&](int blocks, int threads, size_t smem, float* part_p, int32_t* part_c, int32_t* part_n, uint32_t* joined) {
    return launch_pdl(route_kernel<T, kPer, kV, kThreads>, blocks, threads, smem, a.stream, static_cast<const T*>(a.logits), a.s,
                      a.mask, a.weights, a.ids, part_p, part_c, part_n, joined, a.counts, a.loss, a.n);
  }, kThreads, a.s.E * 8 + kPer * kThreads * 4);
}
template <typename T, int kPer, bool kBack>
int launch_few(const RouteCall& a) {
  if constexpr (kBack) {
    const int64_t want = ceil_div(a.s.tokens, kFewBackThreads / 8), cap = static_cast<int64_t>(a.sms) * (2048 / kFewBackThreads);
    return launch_pdl(route_backward_few_kernel<T, kPer>, static_cast<unsigned>(want < cap ? want : cap), kFewBackThreads, 0,
                      a.stream, static_cast<const T*>(a.logits), a.s, a.mask, a.ids, a.counts, a.n, a.dweights, a.dloss,
                      static_cast<T*>(a.dlogits), a.ldd);
  } else {
    return launch_forward(a, [&](int blocks, int threads, size_t smem, float* part_p, int32_t* part_c, int32_t* part_n, uint32_t* joined) {
      return launch_pdl(route_few_kernel<T, kPer>, blocks, threads, smem, a.stream, static_cast<const T*>(a.logits), a.s, a.mask,
                        a.weights, a.ids, part_p, part_c, part_n, joined, a.counts, a.loss, a.n);
    }, kFewThreads, 0);
  }
}

template <typename T, int kPer, int kV>
int launch_route_backward(const RouteCall& a) {
  constexpr int kBackThreads = back_threads<kPer>();
  const int64_t want = ceil_div(a.s.tokens, kBackThreads / 32);
  const int64_t cap = static_cast<int64_t>(a.sms) * (2048 / kBackThreads);
  return launch_pdl(route_backward_kernel<T, kPer, kV, kBackThreads>, static_cast<unsigned>(want < cap ? want : cap),
                    kBackThreads, 2 * kPer * 32 * 4 * (kBackThreads / 32), a.stream, static_cast<const T*>(a.logits), a.s,
                    a.mask, a.ids, a.counts, a.n, a.dweights, a.dloss, static_cast<T*>(a.dlogits), a.ldd);
}

template <typename T, int kPer, int kV, bool kBack>
int launch_one(const RouteCall& a) {
  if constexpr (kBack)
    return launch_route_backward<T, kPer, kV>(a);
  else
    return launch_route<T, kPer, kV>(a);
}

// Vectors of 4 elements (2 for up to 64 experts) where base and row pitch are
// aligned to them, else single elements.
template <typename T, bool kBack>
int launch_typed(const RouteCall& a) {
  const uint64_t pitch = static_cast<uint64_t>(a.s.ld) * sizeof(T);
  const uint64_t dpitch = kBack ? static_cast<uint64_t>(a.ldd) * sizeof(T) : 0;
  const int align = common_alignment({address_of(a.logits), pitch, kBack ? address_of(a.dlogits) : 0, dpitch});
  const bool v4 = align >= static_cast<int>(4 * sizeof(T)), v2 = align >= static_cast<int>(2 * sizeof(T));
  const int E = a.s.E;
  if (E <= 8) return launch_few<T, 1, kBack>(a);
  if (E <= 16) return launch_few<T, 2, kBack>(a);
  if (E <= kFewExperts) return launch_few<T, 4, kBack>(a);
  if (E <= 64) return v2 ? launch_one<T, 2, 2, kBack>(a) : launch_one<T, 2, 1, kBack>(a);
  if (E <= 128) return v4 ? launch_one<T, 4, 4, kBack>(a) : launch_one<T, 4, 1, kBack>(a);
  if (E <= 256) return v4 ? launch_one<T, 8, 4, kBack>(a) : launch_one<T, 8, 1, kBack>(a);
  if (E <= 512) return v4 ? launch_one<T, 16, 4, kBack>(a) : launch_one<T, 16, 1, kBack>(a);
  return v4 ? launch_one<T, 32, 4, kBack>(a) : launch_one<T, 32, 1, kBack>(a);
}

int check_route_shape(int dtype, int64_t tokens, int32_t experts, int32_t k, int64_t ld) {
  if (dtype != MXQ_F32 && dtype != MXQ_BF16) return MXQ_EBADDTYPE;
  if (tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > MXQ_MAX_GROUPS || k < 1 || k > experts ||
      k > kMaxK || ld < experts || ld > INT32_MAX)
    return MXQ_EBADSHAPE;
  return MXQ_OK;
}

}  // namespace

namespace mxq {
int route_status_read(unsigned int* out, bool clear) {
  return read_status_word(g_route_status, out, clear);
}
int route_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

// Sized for blocks of at most kWorkspaceTokens tokens: whether a call needs a workspace
// goes by its tokens, the same for every number of experts up to 256 and whichever
// kernel serves them.  (A block takes 128 tokens where there are at most 32 experts.
// Sized for those, calls of 33 to 128 tokens asked for none, and one with too small a
// workspace, or none, was accepted beside 32 experts and refused beside 33.)
constexpr int kWorkspaceTokens = 32;
extern "C" int64_t mxq_moe_route_workspace(int64_t tokens, int32_t experts) {
  if (tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > MXQ_MAX_GROUPS) return MXQ_EBADSHAPE;
  const int at_once = tokens_at_once(experts);
  const int64_t blocks = ceil_div(tokens, at_once < kWorkspaceTokens ? at_once : kWorkspaceTokens);
  // per block the experts' sums and counts and the routed tokens; the join's counter and losses
  return blocks <= 1 ? 0 : (static_cast<int64_t>(experts) * 8 + 4) * (blocks < kMaxBlocks ? blocks : kMaxBlocks) + 4 * (1 + kMaxJoins);
}

extern "C" int mxq_moe_route(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t k,
                             const uint8_t* mask, int renorm, float* weights, int32_t* ids, int32_t* counts,
                             float* loss, int32_t* routed, uint8_t* workspace, int64_t workspace_bytes,
                             cudaStream_t stream) {
  int rc = check_route_shape(dtype, tokens, experts, k, ld);
  if (rc != MXQ_OK) return rc;
  const int64_t need = mxq_moe_route_workspace(tokens, experts);
  if (workspace_bytes < need) return MXQ_EBADSHAPE;
  if (!counts || !loss || !routed || (need > 0 && !workspace) || (tokens > 0 && (!logits || !weights || !ids))) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(logits, es) || !aligned_to(weights, 4) || !aligned_to(ids, 4) || !aligned_to(counts, 4) ||
      !aligned_to(loss, 4) || !aligned_to(routed, 4) || !aligned_to(workspace, 16))
    return MXQ_EALIGN;
  const uint64_t chosen = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[6] = {range_of(weights, chosen), range_of(ids, chosen), range_of(counts, 4ull * experts),
                            range_of(loss, 4), range_of(routed, 4), range_of(workspace, need)};
  const ByteRange in[2] = {range_of(logits, pitched_bytes(tokens, experts, ld, es)), range_of(mask, tokens)};
  if (outputs_overlap(out, 6, in, 2)) return MXQ_EOVERLAP;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;
  RouteCall a = {};
  a.logits = logits;
  a.s = {tokens, ld, experts, k, renorm != 0};
  a.mask = mask;
  a.weights = weights;
  a.ids = ids;
  a.counts = counts;
  a.loss = loss;
  a.n = routed;
  a.workspace = workspace;
  a.sms = sms < kMaxBlocks ? sms : kMaxBlocks;
  a.stream = stream;
  return dtype == MXQ_F32 ? launch_typed<float, false>(a) : launch_typed<bf16_t, false>(a);
}

extern "C" int mxq_moe_route_backward(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld,
                                      int32_t k, const uint8_t* mask, int renorm, const int32_t* ids,
                                      const int32_t* counts, const int32_t* routed, const float* dweights,
                                      const float* dloss, void* dlogits, int64_t ldd, cudaStream_t stream) {
  int rc = check_route_shape(dtype, tokens, experts, k, ld);
  if (rc != MXQ_OK) return rc;
  if (ldd < experts || ldd > INT32_MAX) return MXQ_EBADSHAPE;
  if (tokens == 0) return MXQ_OK;
  if (!logits || !ids || !counts || !routed || !dlogits) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(ids, 4) || !aligned_to(counts, 4) ||
      !aligned_to(routed, 4) || !aligned_to(dweights, 4) || !aligned_to(dloss, 4))
    return MXQ_EALIGN;
  const uint64_t chosen = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[1] = {range_of(dlogits, pitched_bytes(tokens, experts, ldd, es))};
  const ByteRange in[7] = {range_of(logits, pitched_bytes(tokens, experts, ld, es)), range_of(mask, tokens),
                           range_of(ids, chosen), range_of(counts, 4ull * experts), range_of(routed, 4),
                           range_of(dweights, chosen), range_of(dloss, 4)};
  if (outputs_overlap(out, 1, in, 7)) return MXQ_EOVERLAP;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;
  RouteCall a = {};
  a.logits = logits;
  a.s = {tokens, ld, experts, k, renorm != 0};
  a.mask = mask;
  a.ids = const_cast<int32_t*>(ids);
  a.counts = const_cast<int32_t*>(counts);
  a.n = const_cast<int32_t*>(routed);
  a.dweights = dweights;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.sms = sms;
  a.stream = stream;
  return dtype == MXQ_F32 ? launch_typed<float, true>(a) : launch_typed<bf16_t, true>(a);
}
