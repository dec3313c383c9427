// moe_route_groups.cu -- routing by scores with a bias, among the best groups of experts,
// with the balance loss, and the gradient of the logits.
//
// For a token's logits l over E experts in equal groups of consecutive ones:
//   s = logistic(l) or softmax(l);  c = s + bias;  a group's value is the sum of its two
//   largest c;  the k largest c among the experts of the best groups are chosen;
//   weights w = s (over the chosen ones' sum with renorm), times scale;
//   p = s / sum s, and the balance loss E/(k n^2) sum_e counts_e sum_t p_te.
// With g_j the gradient of s_j through the weights (scale dw_j, or
// (scale dw_j - sum w scale dw) / sum of the chosen s), c_e = dloss E counts_e/(k n^2),
// the logits' gradient is
//   logistic  s (1 - s) (g + (c_e - sum p c) / sum s)
//   softmax   p (h - sum p h)  with  h = g + c.
//
// The choice is that of exact arithmetic: c is computed in fp32, where it is off by a few
// 2^-23, and wherever two values that the choice hangs on lie nearer than that (the last
// of the chosen groups and the first of the others, neighbours among the chosen experts
// and the first of the others) the token is done again in 64 bits (choose_exactly).
// Experts with the same logit and the same bias are equal and go by their index at once.
//
// One warp owns a token, a lane keeps kPer of its logits in registers, and the next
// token's are loaded ahead, as in moe_route.cu.  For the groups the keys of all c go
// through shared memory, rows of a group apart so that the lanes of different groups read
// different banks; 32 / groups lanes find the two largest of a group.
#include "moe_route_common.cuh"

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxGroups = 32;  // a group per lane

struct Grouped {
  int groups, best, size;       // size: experts of a group
  int lanes, pitch;             // lanes that work on a group; floats between groups' keys
  float scale;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// The choice of one token in 64 bits; lane l has the experts l, l + 32, ...  Returns in
// lane j the j-th of the chosen, -1 where there are no more.
template <typename T, int kPer, bool kLogistic>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int k, int groups, int best, int size) {
  const int lane = threadIdx.x & 31;
  const double none = -CUDART_INF;
  double c[kPer];
  double top = none, sum = 0.0;
  if (!kLogistic) {
#pragma unroll 1
    for (int e = lane; e < E; e += 32) top = fmax(top, static_cast<double>(widen(row[e])));
    top = warp_max(top);
#pragma unroll 1
    for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(widen(row[e])) - top);
    sum = warp_sum(sum);
  }
#pragma unroll 1
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    c[i] = none;
    if (e >= E) continue;
    const double x = widen(row[e]);
    if (!(x > none)) continue;
    const double v = (kLogistic ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum) + (bias != nullptr ? bias[e] : 0.0f);
    if (v > none) c[i] = v;
  }
  if (groups > 1) {
    double value = none;  // of the group of this lane
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      double first = none, second = none;
#pragma unroll 1
      for (int i = 0; i < kPer; ++i)
        if ((lane + 32 * i) / size == g) second = fmax(second, fmin(first, c[i])), first = fmax(first, c[i]);
#pragma unroll 1
      for (int d = 16; d > 0; d >>= 1) {
        const double other = __shfl_xor_sync(kAll, first, d), next = __shfl_xor_sync(kAll, second, d);
        second = fmax(fmax(second, next), fmin(first, other));
        first = fmax(first, other);
      }
      if (lane == g) value = second > none ? first + second : first;
    }
    int before = 0;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      const double other = __shfl_sync(kAll, value, g);
      before += other > value || (other == value && g < lane) ? 1 : 0;
    }
    const uint32_t chosen = __ballot_sync(kAll, lane < groups && before < best);
#pragma unroll 1
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E && !(chosen >> ((lane + 32 * i) / size) & 1u)) c[i] = none;
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    double most = none;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) most = fmax(most, c[i]);
    most = warp_max(most);
    if (!(most > none)) break;
    int at = INT32_MAX;
#pragma unroll 1
    for (int i = kPer - 1; i >= 0; --i)
      if (c[i] == most) at = lane + 32 * i;
    at = static_cast<int>(__reduce_min_sync(kAll, static_cast<uint32_t>(at)));
#pragma unroll 1
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == at) c[i] = none;
    if (lane == j) mine = at;
  }
  return mine;
}

// How near two values may be in fp32 and still not be known to be in order: twice what a
// value can be off by.  logistic: 2^-22 for the exponential's and the reciprocal's units in
// the last place and the sum's rounding.  softmax: (kPer + 16) 2^-24 of the score for the
// sum over a lane's values and the lanes, and its exponent's distance from the largest,
// `below`, times 2^-24.  And 2^-24 of c for the addition of the bias.
template <int kPer, bool kLogistic>
__device__ __forceinline__ float doubt(float s, float below, float c) {
  const float of_c = 0x1p-22f * fabsf(c);
  return kLogistic ? 0x1p-21f + of_c : fmaf(s * 0x1p-22f, kPer + 16 + below, of_c);
}

struct Candidate {
  float c, x, b;
  int32_t e;
};

template <typename T, int kPer, int kV, bool kLogistic, int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    route_groups_kernel(const T* __restrict__ logits, const RouteShape s, const Grouped gr, const float* __restrict__ bias,
                        const uint8_t* __restrict__ mask, float* __restrict__ weights, int32_t* __restrict__ ids, float* part_p,
                        int32_t* part_c, int32_t* part_n, uint32_t* joined, int32_t* counts, float* loss, int32_t* n_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  __shared__ int32_t routed_tokens;
  __shared__ int few_n[kWarps];
  __shared__ __align__(16) Candidate few[kWarps][32];
  __shared__ __align__(16) uint64_t order[kWarps][32];
  // the groups' keys while tokens are worked on; after that the warps' sums
  float* by_warp = reinterpret_cast<float*>(smem);                        // [warps, 32 * kPer]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int keys_row = gr.groups > 1 ? gr.groups * gr.pitch : 0;
  const int shared_rows = max(32 * kPer, keys_row);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem) + warp * shared_rows;
  int32_t* hist = reinterpret_cast<int32_t*>(smem) + kWarps * shared_rows;  // [E]
  float* sums = reinterpret_cast<float*>(hist + s.E);                       // [E]
  for (int e = tid; e < s.E; e += kThreads) hist[e] = 0;
  if (tid == 0) routed_tokens = 0;
  if (lane == 0) few_n[warp] = 0;
  __syncthreads();
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>(s.tokens) * s.k * 4;
  if (gridDim.x > 1) pdl_launch_dependents();  // the join's few blocks wait beside this one
  float acc[kPer], b[kPer];
  int group_of[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = expert_of<kV>(i, lane);
    acc[i] = 0.0f;
    b[i] = bias != nullptr && e < s.E ? read_at(bias, e, s.E, 0.0f, &g_route_status) : 0.0f;
    group_of[i] = e < s.E ? e / gr.size : 0;
  }
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
    float x[kPer], sc[kPer];
    ahead.values(x);
    fetch(t + step);
    float top = -CUDART_INF_F;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      top = fmaxf(top, x[i]);  // skips NaN
      nan |= x[i] != x[i];
    }
    top = key_value(max(__reduce_max_sync(kAll, order_key(top)), order_key(-FLT_MAX)));
    const bool unmasked = mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) some |= x[i] > -CUDART_INF_F;
    const bool routed = unmasked && __any_sync(kAll, some || nan);
    int rank = kMaxK, my_id = -1;
    float my_s = 0.0f;
    if (routed) {
      ++routed_here;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        sc[i] = kLogistic ? logistic(x[i]) : exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
        sum += sc[i];
      }
      sum = warp_sum(sum);
      const float inv = sum == 0.0f ? 0.0f : reciprocal(sum);
      uint32_t key[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float p = sc[i] * inv;
        acc[i] += p;
        if (!kLogistic) sc[i] = p;
        key[i] = x[i] > -CUDART_INF_F ? order_key(sc[i] + b[i]) : 0u;
      }
      bool certain = true;
      if (gr.groups > 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = expert_of<kV>(i, lane);
          if (e < s.E) keys[group_of[i] * gr.pitch + e - group_of[i] * gr.size] = key[i];
        }
        __syncwarp();
        const int g = lane / gr.lanes;
        uint32_t first = 0u, second = 0u;
        if (g < gr.groups)
          for (int m = lane % gr.lanes; m < gr.size; m += gr.lanes) {
            const uint32_t v = keys[g * gr.pitch + m];
            second = max(second, min(first, v));
            first = max(first, v);
          }
        for (int d = gr.lanes / 2; d > 0; d >>= 1) {
          const uint32_t other = __shfl_xor_sync(kAll, first, d), next = __shfl_xor_sync(kAll, second, d);
          second = max(max(second, next), min(first, other));
          first = max(first, other);
        }
        const float value = key_value(first) + (second != 0u ? key_value(second) : 0.0f);
        const uint32_t own = first != 0u ? order_key(value) : 0u;
        int before = 0;
        for (int o = 0; o < gr.groups; ++o) {
          const uint32_t other = __shfl_sync(kAll, own, o * gr.lanes);
          before += other > own || (other == own && o < g) ? 1 : 0;
        }
        const bool in = own != 0u && before < gr.best;
        const uint32_t chosen = __ballot_sync(kAll, in);
        const uint32_t last = __reduce_min_sync(kAll, in ? own : ~0u), next = __reduce_max_sync(kAll, in ? 0u : own);
        // a sum of two values, and of which two: four times what one is off by, and its rounding
        if (next != 0u) certain = key_value(last) - key_value(next) > 0x1p-18f * (1.0f + fabsf(key_value(last)));
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (!(chosen >> (group_of[i] * gr.lanes) & 1u)) key[i] = 0u;
      }
      uint32_t mine = 0u;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine = max(mine, key[i]);
      // the k-th largest lane maximum, equal ones counted once; 0 when there are fewer
      uint32_t bar = __reduce_max_sync(kAll, mine);
      const bool any = bar != 0u;
#pragma unroll 4
      for (int j = 1; j < s.k; ++j) {
        if (mine == bar) mine = 0u;
        bar = __reduce_max_sync(kAll, mine);
      }
      if (any && certain) {
        const float low = bar != 0u ? key_value(bar) : -FLT_MAX;
        const uint32_t from = order_key(low - 0x1p-18f * (1.0f + fabsf(low)));
        int own_n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) own_n += key[i] != 0u && key[i] >= from ? 1 : 0;
        int at = 0;
        if (own_n > 0) at = atomicAdd(&few_n[warp], own_n);
        const int n = __reduce_add_sync(kAll, own_n);
        __syncwarp();
        if (lane == 0) few_n[warp] = 0;  // for the next token
        if (n <= 32) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (key[i] != 0u && key[i] >= from) few[warp][at++] = Candidate{key_value(key[i]), x[i], b[i], expert_of<kV>(i, lane)};
          __syncwarp();
          const Candidate own = few[warp][lane];
          const uint64_t own_key = lane < n ? ChoiceKey<float>::of(own.c, own.e) : 0;
          order[warp][lane] = own_key;
          __syncwarp();
          int before = 0;
          for (int i = 0; i < n; i += 2) {
            const Vec<uint64_t, 2> other = *reinterpret_cast<const Vec<uint64_t, 2>*>(&order[warp][i]);
            before += (other.v[0] > own_key ? 1 : 0) + (other.v[1] > own_key ? 1 : 0);
          }
          if (lane < n) few[warp][before] = own;
          __syncwarp();
          bool clear = true;
          if (lane < n && before < s.k) {
            rank = before;
            my_id = own.e;
            my_s = kLogistic ? logistic(own.x) : exp2_ftz((own.x - top) * kLog2E) * inv;
            if (before + 1 < n) {
              const Candidate after = few[warp][before + 1];
              clear = own.c - after.c > doubt<kPer, kLogistic>(my_s, top - own.x, own.c) || (own.x == after.x && own.b == after.b);
            }
          }
          certain = __all_sync(kAll, clear);
        } else {
          certain = false;
        }
        __syncwarp();
      }
      if (any && !certain) {
        const T* row = logits + t * s.ld;
        my_id = in_buf(row, s.E * sizeof(T), logits, in_bytes, &g_route_status)
                    ? choose_exactly<T, kPer, kLogistic>(row, bias, s.E, s.k, gr.groups, gr.best, gr.size) : -1;
        rank = my_id >= 0 ? lane : kMaxK;
        const float own = my_id >= 0 ? widen(row[my_id]) : 0.0f;
        my_s = my_id < 0 ? 0.0f : kLogistic ? logistic(own) : exp2_ftz((own - top) * kLog2E) * inv;
      }
      if (my_id >= 0) atomicAdd(&hist[my_id], 1);
    }
    float w = my_id >= 0 ? my_s : 0.0f;
    if (s.renorm) {
      const float all = warp_sum(w);
      w = all == 0.0f ? 0.0f : w / all;
    }
    w *= gr.scale;
    // the chosen ones' lanes write their places, and as many others the places left
    const uint32_t chosen = __ballot_sync(kAll, my_id >= 0);
    if (my_id < 0) {
      rank = __popc(chosen) + __popc(~chosen & ((1u << lane) - 1u));
      w = 0.0f;
    }
    if (rank < s.k && in_buf(weights + t * s.k + rank, 4, weights, out_bytes, &g_route_status) &&
        in_buf(ids + t * s.k + rank, 4, ids, out_bytes, &g_route_status)) {
      weights[t * s.k + rank] = w;
      ids[t * s.k + rank] = my_id;
    }
  }
  if (lane == 0 && routed_here) atomicAdd(&routed_tokens, routed_here);
  __syncthreads();  // the keys' last readers
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

template <typename T, int kPer, int kV, bool kLogistic, int kThreads>
__global__ void __launch_bounds__(kThreads)
    route_groups_backward_kernel(const T* __restrict__ logits, const RouteShape s, float scale, const uint8_t* __restrict__ mask,
                                 const int32_t* __restrict__ ids, const int32_t* __restrict__ counts, const int32_t* __restrict__ n_in,
                                 const float* __restrict__ dweights, const float* __restrict__ dloss, T* __restrict__ dlogits,
                                 int64_t ldd) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the scores of a row, and the chosen experts' gradients, zero between rows
  constexpr int kRow = kPer * 32;
  float* chosen = reinterpret_cast<float*>(smem) + warp * 2 * kRow;
  float* scores = chosen + kRow;
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
    if (in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status)) ahead.load(logits + t * s.ld, s.E, lane);
    if (dweights != nullptr && lane < s.k) {
      e_ahead = read_at(ids, t * s.k + lane, s.tokens * s.k, -1, &g_route_status);
      dw_ahead = read_at(dweights, t * s.k + lane, s.tokens * s.k, 0.0f, &g_route_status);
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  fetch(t);
  for (; t < s.tokens; t += step) {
    const int e = e_ahead >= 0 && e_ahead < s.E ? e_ahead : -1;
    const float dw = e >= 0 ? dw_ahead * scale : 0.0f;
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
    const uint32_t top_key = __reduce_max_sync(kAll, order_key(top));
    top = key_value(max(top_key, order_key(-FLT_MAX)));
    const bool routed =
        (mask == nullptr || read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status) != 0) && (top_key != 0u || __any_sync(kAll, nan));
    T* out = dlogits + t * ldd;
    float d[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) d[i] = 0.0f;
    if (routed) {
      float sc[kPer], rest[kPer], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (kLogistic)
          logistic_pair(x[i], sc[i], rest[i]);
        else
          sc[i] = exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
        sum += sc[i];
      }
      sum = warp_sum(sum);
      const float inv = sum == 0.0f ? 0.0f : reciprocal(sum);
      float pc = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float p = sc[i] * inv;
        if (!kLogistic) sc[i] = p;
        pc = fmaf(p, c[i], pc);
      }
      // the scores of the chosen experts, from the lanes that hold them
#pragma unroll
      for (int q = 0; q < kPer / kV; ++q) {
        Vec<float, kV> v;
#pragma unroll
        for (int i = 0; i < kV; ++i) v.v[i] = sc[q * kV + i];
        *reinterpret_cast<Vec<float, kV>*>(scores + expert_of<kV>(q * kV, lane)) = v;
      }
      __syncwarp();
      const float own = e >= 0 ? scores[e] : 0.0f;
      float part = dw;
      if (s.renorm) {
        const float all = warp_sum(own), back = all == 0.0f ? 0.0f : 1.0f / all;
        const float dot = warp_sum(own * back * dw);
        part = (dw - dot) * back;
      }
      if (e >= 0) chosen[e] = part;
      if (!kLogistic) pc = fmaf(own, e >= 0 ? part : 0.0f, pc);
      __syncwarp();
      const float total = warp_sum(pc);
#pragma unroll
      for (int q = 0; q < kPer / kV; ++q) {
        const Vec<float, kV> add = *reinterpret_cast<const Vec<float, kV>*>(chosen + expert_of<kV>(q * kV, lane));
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int j = q * kV + i;
          d[j] = kLogistic ? sc[j] * rest[j] * fmaf(c[j] - total, inv, add.v[i]) : sc[j] * (add.v[i] + c[j] - total);
        }
      }
      __syncwarp();
      if (e >= 0) chosen[e] = 0.0f;
    }
    if (!in_buf(out, s.E * sizeof(T), dlogits, out_bytes, &g_route_status)) continue;
#pragma unroll
    for (int q = 0; q < kPer / kV; ++q) {
      const int e0 = expert_of<kV>(q * kV, lane);
      if (e0 + kV <= s.E) {
        Vec<T, kV> v;
#pragma unroll
        for (int j = 0; j < kV; ++j) v.v[j] = narrow<T>(d[q * kV + j]);
        *reinterpret_cast<Vec<T, kV>*>(out + e0) = v;
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (e0 + j < s.E) out[e0 + j] = narrow<T>(d[q * kV + j]);
      }
    }
  }
}

struct GroupsCall {
  const void* logits;
  RouteShape s;
  Grouped gr;
  const float* bias;
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

template <typename T, int kPer, int kV, bool kLogistic>
int launch_groups(const GroupsCall& a) {
  constexpr int kThreads = route_threads<kPer>(), kWarps = kThreads / 32;
  const int blocks = route_blocks(a.s.tokens, kWarps, a.sms);
  float* part_p = reinterpret_cast<float*>(a.workspace);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + static_cast<int64_t>(blocks) * a.s.E);
  int32_t* part_n = part_c + static_cast<int64_t>(blocks) * a.s.E;
  uint32_t* joined = reinterpret_cast<uint32_t*>(part_n + blocks);
  float* part_loss = reinterpret_cast<float*>(joined + 1);
  const int keys = a.gr.groups > 1 ? a.gr.groups * a.gr.pitch : 0;
  const size_t smem = static_cast<size_t>(kWarps) * (keys > 32 * kPer ? keys : 32 * kPer) * 4 + static_cast<size_t>(a.s.E) * 8;
  const auto kernel = route_groups_kernel<T, kPer, kV, kLogistic, kThreads>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024) != cudaSuccess) return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  const int rc = launch_pdl(kernel, static_cast<unsigned>(blocks), kThreads, smem, a.stream, static_cast<const T*>(a.logits), a.s, a.gr,
                            a.bias, a.mask, a.weights, a.ids, part_p, part_c, part_n, joined, a.counts, a.loss, a.n);
  if (rc != MXQ_OK || blocks == 1) return rc;
  return launch_pdl(route_join_kernel, static_cast<unsigned>(ceil_div(a.s.E, 32)), 32 * kJoinWarps, 0, a.stream, a.s, blocks, part_p,
                    part_c, part_n, joined, part_loss, a.counts, a.loss, a.n);
}
template <typename T, int kPer, int kV, bool kLogistic>
int launch_groups_backward(const GroupsCall& a) {
  constexpr int kThreads = back_threads<kPer>();
  const int64_t want = ceil_div(a.s.tokens, kThreads / 32), cap = static_cast<int64_t>(a.sms) * (2048 / kThreads);
  return launch_pdl(route_groups_backward_kernel<T, kPer, kV, kLogistic, kThreads>, static_cast<unsigned>(want < cap ? want : cap),
                    kThreads, 2 * kPer * 32 * 4 * (kThreads / 32), a.stream, static_cast<const T*>(a.logits), a.s, a.gr.scale, a.mask,
                    a.ids, a.counts, a.n, a.dweights, a.dloss, static_cast<T*>(a.dlogits), a.ldd);
}
template <typename T, int kPer, int kV, bool kBack>
int launch_scores(const GroupsCall& a, int scores) {
  if constexpr (kBack)
    return scores == MXQ_SCORES_SIGMOID ? launch_groups_backward<T, kPer, kV, true>(a) : launch_groups_backward<T, kPer, kV, false>(a);
  else
    return scores == MXQ_SCORES_SIGMOID ? launch_groups<T, kPer, kV, true>(a) : launch_groups<T, kPer, kV, false>(a);
}

// Vectors of 4 elements (2 for up to 64 experts) where base and row pitch are
// aligned to them, else single elements.
template <typename T, bool kBack>
int launch_grouped(const GroupsCall& a, int scores) {
  const uint64_t pitch = static_cast<uint64_t>(a.s.ld) * sizeof(T);
  const uint64_t dpitch = kBack ? static_cast<uint64_t>(a.ldd) * sizeof(T) : 0;
  const int align = common_alignment({address_of(a.logits), pitch, kBack ? address_of(a.dlogits) : 0, dpitch});
  const bool v4 = align >= static_cast<int>(4 * sizeof(T)), v2 = align >= static_cast<int>(2 * sizeof(T));
  const int E = a.s.E;
  if (E <= 32) return launch_scores<T, 1, 1, kBack>(a, scores);
  if (E <= 64) return v2 ? launch_scores<T, 2, 2, kBack>(a, scores) : launch_scores<T, 2, 1, kBack>(a, scores);
  if (E <= 128) return v4 ? launch_scores<T, 4, 4, kBack>(a, scores) : launch_scores<T, 4, 1, kBack>(a, scores);
  if (E <= 256) return v4 ? launch_scores<T, 8, 4, kBack>(a, scores) : launch_scores<T, 8, 1, kBack>(a, scores);
  if (E <= 512) return v4 ? launch_scores<T, 16, 4, kBack>(a, scores) : launch_scores<T, 16, 1, kBack>(a, scores);
  return v4 ? launch_scores<T, 32, 4, kBack>(a, scores) : launch_scores<T, 32, 1, kBack>(a, scores);
}

int check_groups_shape(int dtype, int64_t tokens, int32_t experts, int32_t k, int64_t ld, int scores, float scale) {
  if (dtype != MXQ_F32 && dtype != MXQ_BF16) return MXQ_EBADDTYPE;
  if (tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > MXQ_MAX_GROUPS || k < 1 || k > experts || k > kMaxK ||
      ld < experts || ld > INT32_MAX || (scores != MXQ_SCORES_SIGMOID && scores != MXQ_SCORES_SOFTMAX) || !isfinite(scale))
    return MXQ_EBADSHAPE;
  return MXQ_OK;
}

}  // namespace

namespace mxq {
int route_groups_status_read(unsigned int* out, bool clear) { return read_status_word(g_route_status, out, clear); }
int route_groups_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int mxq_moe_route_groups(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t k,
                                    const float* bias, int scores, int32_t groups, int32_t best, const uint8_t* mask, int renorm,
                                    float scale, float* weights, int32_t* ids, int32_t* counts, float* loss, int32_t* routed,
                                    uint8_t* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  int rc = check_groups_shape(dtype, tokens, experts, k, ld, scores, scale);
  if (rc != MXQ_OK) return rc;
  if (groups < 1 || groups > kMaxGroups || experts % groups != 0 || best < 1 || best > groups || k > experts / groups * best)
    return MXQ_EBADSHAPE;
  const int64_t need = mxq_moe_route_workspace(tokens, experts);
  if (workspace_bytes < need) return MXQ_EBADSHAPE;
  if (!counts || !loss || !routed || (need > 0 && !workspace) || (tokens > 0 && (!logits || !weights || !ids))) return MXQ_ENULL;
  const int es = element_bytes(dtype);
  if (!aligned_to(logits, es) || !aligned_to(bias, 4) || !aligned_to(weights, 4) || !aligned_to(ids, 4) || !aligned_to(counts, 4) ||
      !aligned_to(loss, 4) || !aligned_to(routed, 4) || !aligned_to(workspace, 16))
    return MXQ_EALIGN;
  const uint64_t chosen = static_cast<uint64_t>(tokens) * k * 4;
  const ByteRange out[6] = {range_of(weights, chosen), range_of(ids, chosen), range_of(counts, 4ull * experts),
                            range_of(loss, 4), range_of(routed, 4), range_of(workspace, need)};
  const ByteRange in[3] = {range_of(logits, pitched_bytes(tokens, experts, ld, es)), range_of(mask, tokens), range_of(bias, 4ull * experts)};
  if (outputs_overlap(out, 6, in, 3)) return MXQ_EOVERLAP;
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;
  GroupsCall a = {};
  a.logits = logits;
  a.s = {tokens, ld, experts, k, renorm != 0};
  a.gr.groups = best == groups ? 1 : groups;  // all of them: no choice
  a.gr.best = best == groups ? 1 : best;
  a.gr.size = experts / a.gr.groups;
  int wide = 1;
  while (wide < a.gr.groups) wide *= 2;
  a.gr.lanes = 32 / wide;
  // the next number of floats that is `lanes` past a multiple of 32 banks: neighbouring
  // groups' lanes then read neighbouring banks
  a.gr.pitch = a.gr.size + ((a.gr.lanes - a.gr.size) % 32 + 32) % 32;
  a.gr.scale = scale;
  a.bias = bias;
  a.mask = mask;
  a.weights = weights;
  a.ids = ids;
  a.counts = counts;
  a.loss = loss;
  a.n = routed;
  a.workspace = workspace;
  a.sms = sms < kMaxBlocks ? sms : kMaxBlocks;
  a.stream = stream;
  return dtype == MXQ_F32 ? launch_grouped<float, false>(a, scores) : launch_grouped<bf16_t, false>(a, scores);
}

extern "C" int mxq_moe_route_groups_backward(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t k,
                                             int scores, const uint8_t* mask, int renorm, float scale, const int32_t* ids,
                                             const int32_t* counts, const int32_t* routed, const float* dweights,
                                             const float* dloss, void* dlogits, int64_t ldd, cudaStream_t stream) {
  int rc = check_groups_shape(dtype, tokens, experts, k, ld, scores, scale);
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
  GroupsCall a = {};
  a.logits = logits;
  a.s = {tokens, ld, experts, k, renorm != 0};
  a.gr.scale = scale;
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
  return dtype == MXQ_F32 ? launch_grouped<float, true>(a, scores) : launch_grouped<bf16_t, true>(a, scores);
}
