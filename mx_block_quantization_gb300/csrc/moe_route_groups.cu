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
// The choice is that of 64-bit arithmetic: c is computed in fp32, where it is off by a few
// 2^-23, and wherever two values that the choice hangs on lie nearer than that (the chosen
// groups and the others, neighbours among the chosen experts and the first of the others)
// they are compared again: by their own errors, which are small for small scores (settle,
// groups_clear), the candidates in 64 bits (rank_exactly), and at last the whole row in 64
// bits (choose_exactly).  Experts with the same logit and the same bias are equal and go by
// their index at once.  131071 tokens of 256 experts in 8 groups take 113 us; with logits
// around -20 118, with one bias of -inf or -1e9 112, of 1e9 or inf 120; if all of them
// went by 64 bits, 1895.  That is left for rows whose scores vanish beside a bias of all
// experts: logits around -20 with biases of -0.01.
//
// One warp owns a token, a lane keeps some of its logits in registers, and the next
// token's are loaded ahead, as in moe_route.cu.  Up to eight experts of one group a lane:
// route_owned_kernel; else (more than 256 experts, or groups that fill their lanes badly)
// route_groups_kernel.  Both are bound by the instructions they issue, at three quarters
// of the issue slots: 131071 tokens, 256 experts in 8 groups, fp32, takes 113 us forward
// (about 615 instructions a token; the logits' bytes alone take 20) and 52 backward
// (40 for the bytes of logits and gradient); 10007 tokens, 150 experts in 5 groups,
// bf16, softmax, 25 us, and some 10 more where a single token has to be done again in 64
// bits, backward 13.  More than 256 experts: 131071 x 512 in 8 groups, k 8, 206 and 99 us,
// 65536 x 1024 in 32 groups 269 and 107.
#include "moe_route_common.cuh"

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxGroups = 32;  // a group per lane

struct Grouped {
  int groups, best, size;       // size: experts of a group
  int lanes, shift, pitch;      // lanes that work on a group, their logarithm; floats between groups' rows
  float scale;
};

// Keys in the order of values of 64 bits, 0 for -inf and NaN: what is compared, so that
// the slow pipe for 64 bits sees the scores alone.
__device__ __forceinline__ uint64_t wide_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return v > -CUDART_INF ? b ^ ((b >> 63) != 0 ? ~0ull : 1ull << 63) : 0ull;
}
__device__ __forceinline__ double wide_value(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) != 0 ? k ^ 1ull << 63 : ~k));
}
__device__ __forceinline__ uint64_t wide_max(uint64_t k) {
  const uint32_t high = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
  const uint32_t low = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == high ? static_cast<uint32_t>(k) : 0u);
  return static_cast<uint64_t>(high) << 32 | low;
}
__device__ __forceinline__ double wide_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// The choice of one token in 64 bits; lane l has the experts l, l + 32, ...  Returns in
// lane j the j-th of the chosen, -1 where there are no more.
template <typename T, int kPer, bool kLogistic>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int k, int groups, int best, int size) {
  constexpr int kAtOnce = kPer < 4 ? kPer : 4;  // chains of the scores in flight
  const int lane = threadIdx.x & 31;
  // a router that begins with zeros: all alike, the lowest ones (131071 such tokens with
  // 256 experts: 1700 us without this)
  const float x0 = widen(row[0]), b0 = bias != nullptr ? bias[0] : 0.0f;
  bool alike = fabsf(x0) < CUDART_INF_F && fabsf(b0) < CUDART_INF_F;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) alike = alike && widen(row[e]) == x0 && (bias == nullptr || bias[e] == b0);
  if (__all_sync(kAll, alike)) return lane < k ? lane : -1;
  double c[kPer];
  uint64_t key[kPer];
  float top = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = fmaxf(top, lane + 32 * i < E ? widen(row[lane + 32 * i]) : -CUDART_INF_F);
  top = key_value(max(__reduce_max_sync(kAll, order_key(top)), order_key(-FLT_MAX)));
  double sum = 0.0;
#pragma unroll 1
  for (int i = 0; i < kPer; i += kAtOnce)
#pragma unroll
    for (int j = i; j < i + kAtOnce; ++j) {
      const double x = lane + 32 * j < E ? widen(row[lane + 32 * j]) : -CUDART_INF_F;
      c[j] = exp(kLogistic ? -x : x - top);
      sum += c[j];
    }
  if (!kLogistic) sum = 1.0 / wide_sum(sum);
#pragma unroll 1
  for (int i = 0; i < kPer; i += kAtOnce)
#pragma unroll
    for (int j = i; j < i + kAtOnce; ++j) {
      const int e = lane + 32 * j;
      // the product rounded by itself: fused with the addition in some of a lane's experts
      // and not in others, equal ones would differ
      const double v = __dadd_rn(kLogistic ? 1.0 / (1.0 + c[j]) : __dmul_rn(c[j], sum), bias != nullptr && e < E ? bias[e] : 0.0f);
      key[j] = e < E && widen(row[e]) > -CUDART_INF_F ? wide_key(v) : 0ull;
    }
  if (groups > 1) {
    uint64_t value = 0;  // of the group of this lane
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      uint64_t first = 0, second = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if ((lane + 32 * i) / size == g) second = max(second, min(first, key[i])), first = max(first, key[i]);
      const uint64_t most = wide_max(first);
      const int owner = __ffs(__ballot_sync(kAll, first == most)) - 1;
      const uint64_t next = wide_max(lane == owner ? second : first);
      if (lane == g && most != 0) value = next != 0 ? wide_key(wide_value(most) + wide_value(next)) : most;
    }
    uint32_t chosen = 0;
#pragma unroll 1
    for (int r = 0; r < best; ++r) {
      const uint64_t most = wide_max(value);
      if (most == 0) break;
      const int g = __ffs(__ballot_sync(kAll, value == most)) - 1;
      chosen |= 1u << g;
      if (lane == g) value = 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E && !(chosen >> ((lane + 32 * i) / size) & 1u)) key[i] = 0;
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint64_t own = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > own) own = key[i], at = lane + 32 * i;
    const uint64_t most = wide_max(own);
    if (most == 0) break;
    at = static_cast<int>(__reduce_min_sync(kAll, own == most ? static_cast<uint32_t>(at) : ~0u));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == at) key[i] = 0;
    if (lane == j) mine = at;
  }
  return mine;
}

// What fp32 may be off by.  A logistic score s: 2^-22, for the exponential's and the
// reciprocal's units in the last place and the sum's rounding; where s is small 2^-24 of it
// times 7 and 1.25 of its logit's size, `below` 0, for the exponent.  A softmax's score, in
// 2^-24 of it: 4 for its exponential and 2.25 of its distance `below` the largest logit, as
// much for the sum's terms on their mean (14 at most with 1024 of them), kPer + 4 for their
// additions, 3 for reciprocal and product.  And the addition of the bias 2^-24 of c, taken
// twice.
template <int kPer, bool kLogistic>
__device__ __forceinline__ float off_by(float s, float below, float c) {
  const float of_c = fminf(0x1p-23f * fabsf(c), FLT_MAX);  // an infinite c is exact
  if (kLogistic) return fminf(s * 0x1p-24f * fmaf(1.25f, fmaxf(below, 0.0f), 7.0f), 0x1p-22f) + of_c;
  return fmaf(s * 0x1p-24f, fmaf(2.25f, below, kPer + 25), of_c);
}
// Twice what any score may be off by whose c is not above this one.  It goes by the scores'
// size: s = c - bias is at most c - least, and at most 1 or a softmax's largest, `cap`.  What is
// said above grows with s; it is taken for no less than 2^-40, where a logistic's exponent
// counts 35, or 2^-16 cap, where a softmax's counts 25.  Biases up to kFarBias are not in
// `least`, so that an expert that is left out by one does not count: their c are below -1 and
// not near one from -1/2 on.
constexpr float kFarBias = -2.0f;
template <int kPer, bool kLogistic>
__device__ __forceinline__ float scores_doubt(float c, float cap, float least) {
  if (kLogistic) cap = 1.0f;
  const float most = c >= -0.5f ? fmaxf(fminf(c - least, cap), (kLogistic ? 0x1p-40f : 0x1p-16f) * cap) : cap;
  return kLogistic ? fminf(most * (0x1p-23f * (7 + 35)), 0x1p-21f) : most * (0x1p-23f * (kPer + 25 + 25));
}
// How far above the next value one has to lie to be known to be above it and all others
// behind, c the larger one: these may have larger scores than it, with biases below its.
// `cut` is added; an infinite c lies above every finite one.
template <int kPer, bool kLogistic>
__device__ __forceinline__ float doubt(float c, float cap, float least, float cut) {
  return fminf(fmaf(0x1p-22f, fabsf(c), scores_doubt<kPer, kLogistic>(c, cap, least)) + cut, FLT_MAX);
}
// The same for any scores of a logistic, which nearly always tells as much.
__device__ __forceinline__ float any_doubt(float c, float cut) { return fminf(fmaf(0x1p-22f, fabsf(c), 0x1p-21f) + cut, FLT_MAX); }
// Whether all lanes' c are known to be above what comes behind them, `gap` lower.
template <int kPer, bool kLogistic>
__device__ __forceinline__ bool all_clear(bool no_matter, float gap, float c, float cap, float least, float cut) {
  if (!kLogistic) return __all_sync(kAll, no_matter || gap > doubt<kPer, false>(c, cap, least, cut));
  const bool clear = no_matter || gap > any_doubt(c, cut);
  return __all_sync(kAll, clear) || __all_sync(kAll, clear || gap > doubt<kPer, true>(c, cap, least, cut));
}
// The same for two groups' values, sums of two c, none of whose sizes add up to more than
// `size`: two of a logistic's or of the row's largest score in each value, and 2^-24 of the c
// for the additions of their biases and again for their sums.
template <int kPer, bool kLogistic>
__device__ __forceinline__ float group_doubt(float size, float cap) {
  return fmaf(size, 0x1p-22f, kLogistic ? 0x1p-20f : cap * (0x1p-22f * (kPer + 25)));
}
// Whether the chosen groups are known to lie above the others where that does not say so,
// as one group's large bias is no other's doubt, nor are scores larger than its own: each
// value with what it may be off by itself.  A lane has a group's value, its largest c and
// the size of its two, `cut` more that the value may lack; `there`: the group has an expert.
template <int kPer, bool kLogistic>
__device__ __noinline__ bool groups_clear(bool there, bool chosen, float value, float first, float size, float cut, float cap,
                                          float least) {
  const float off = fabsf(value) < FLT_MAX ? fmaf(size, 0x1p-23f, scores_doubt<kPer, kLogistic>(first, cap, least)) + cut : 0.0f;
  const uint32_t low = __reduce_min_sync(kAll, there && chosen ? order_key(value - off) : ~0u);
  const uint32_t high = __reduce_max_sync(kAll, there && !chosen ? order_key(value + off) : 0u);
  return low > high;
}

// The place in 64 bits of each of n candidates, one a lane, with logistic scores.
__device__ __noinline__ int rank_exactly(float x, float b, int e, int n) {
  const int lane = threadIdx.x & 31;
  const uint64_t own = wide_key(1.0 / (1.0 + exp(-static_cast<double>(x))) + b);
  int before = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint64_t other = __shfl_sync(kAll, own, i);
    const int o = __shfl_sync(kAll, e, i);
    before += other > own || (other == own && o < e) ? 1 : 0;
  }
  return lane < n ? before : kMaxK;
}

// The places of n candidates, one a lane, some perhaps nearer than fp32 can tell: equal ones
// go by their index where logit and bias are alike, and where two others are nearer than
// they may be off by all go by 64 bits.  Less than 0 where that takes the whole row
// (choose_exactly).
template <int kPer, bool kLogistic>
__device__ __noinline__ int settle(int e, float x, float b, float score, float below, int n, int k) {
  const int lane = threadIdx.x & 31;
  const float c = lane < n ? score + b : -CUDART_INF_F, off = off_by<kPer, kLogistic>(score, below, c);
  const float low = c - off, high = c + off;
  int before = 0;
  bool clear = true;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const float other = __shfl_sync(kAll, c, i), other_high = __shfl_sync(kAll, high, i);
    const float other_x = __shfl_sync(kAll, x, i), other_b = __shfl_sync(kAll, b, i);
    const int o = __shfl_sync(kAll, e, i);
    const bool first = other > c || (other == c && o < e);
    before += first ? 1 : 0;
    clear = clear && (first || other_high < low || (other_x == x && other_b == b));
  }
  if (__all_sync(kAll, clear || lane >= n || before >= k)) return lane < n ? before : kMaxK;
  return kLogistic ? rank_exactly(x, b, e, n) : -1;
}

// Puts v at `at` and moves on where x >= from, under one predicate: as branches, each with
// a few lanes, the slots of a lane cost three times as much.
__device__ __forceinline__ void put_from(uint32_t& at, int32_t v, float x, float from) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %2, %3;\n\t@p st.shared.b32 [%0], %1;\n\t@p add.u32 %0, %0, 4;\n\t}"
               : "+r"(at)
               : "r"(v), "f"(x), "f"(from)
               : "memory");
}
// A token's logits in the lanes, vectors that end past E left at -inf (E is a multiple of
// kV); each load under its own predicate.
template <typename T, int kPer, int kV>
struct Ahead {
  Vec<T, kV> v[kPer / kV];
  uint32_t there;  // a bit for each vector
  __device__ __forceinline__ Ahead(int E, int lane) : there(0u) {
#pragma unroll
    for (int q = 0; q < kPer / kV; ++q) {
      if (expert_of<kV>(q * kV, lane) < E) there |= 1u << q;
#pragma unroll
      for (int j = 0; j < kV; ++j) v[q].v[j] = minus_infinity<T>();
    }
  }
  __device__ __forceinline__ void load(const T* row, int lane) {
#pragma unroll
    for (int q = 0; q < kPer / kV; ++q) {
      const T* at = row + expert_of<kV>(q * kV, lane);
      const uint32_t p = there >> q & 1u;
      if constexpr (sizeof v[q] == 16) {
        uint4& w = *reinterpret_cast<uint4*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                     : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w) : "l"(at), "r"(p));
      } else if constexpr (sizeof v[q] == 8) {
        uint2& w = *reinterpret_cast<uint2*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];\n\t}"
                     : "+r"(w.x), "+r"(w.y) : "l"(at), "r"(p));
      } else if constexpr (sizeof v[q] == 4) {
        uint32_t& w = *reinterpret_cast<uint32_t*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.L1::no_allocate.b32 %0, [%1];\n\t}" : "+r"(w) : "l"(at), "r"(p));
      } else {
        uint16_t& w = *reinterpret_cast<uint16_t*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.L1::no_allocate.b16 %0, [%1];\n\t}" : "+h"(w) : "l"(at), "r"(p));
      }
    }
  }
};

// For the groups all c go through shared memory, the groups' rows so far apart that the
// lanes of different groups read different banks; 32 / groups lanes find the two largest
// of a group.  The k-th largest of the lanes' maxima bounds the candidates from below;
// those from there on go side by side and count the larger ones.
template <typename T, int kPer, int kV, bool kLogistic, int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    route_groups_kernel(const T* __restrict__ logits, const RouteShape s, const Grouped gr, const float* __restrict__ bias,
                        const uint8_t* __restrict__ mask, float* __restrict__ weights, int32_t* __restrict__ ids, float* part_p,
                        int32_t* part_c, int32_t* part_n, uint32_t* joined, int32_t* counts, float* loss, int32_t* n_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  __shared__ int32_t routed_tokens;
  __shared__ int32_t few[kWarps][32];                // experts near the top, in any order
  __shared__ __align__(16) float few_c[kWarps][32];  // their c, then in order
  // the groups' rows while tokens are worked on; after that the warps' sums
  float* by_warp = reinterpret_cast<float*>(smem);                        // [warps, 32 * kPer]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int shared_rows = max(32 * kPer, gr.groups > 1 ? gr.groups * gr.pitch : 0);
  float* rows = reinterpret_cast<float*>(smem) + warp * shared_rows;
  float* own_x = reinterpret_cast<float*>(smem) + kWarps * shared_rows + warp * (32 * kPer);  // the token's logits
  float* sums = reinterpret_cast<float*>(smem) + kWarps * (shared_rows + 32 * kPer);  // [32 * kPer]: the biases while tokens are worked on
  int32_t* hist = reinterpret_cast<int32_t*>(sums + 32 * kPer);                       // [E]
  for (int e = tid; e < s.E; e += kThreads) hist[e] = 0;
  if (tid == 0) routed_tokens = 0;
  __syncthreads();
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>(s.tokens) * s.k * 4;
  if (gridDim.x > 1) pdl_launch_dependents();  // the join's few blocks wait beside this one
  constexpr int kVectors = kPer / kV;
  float acc[kPer], least = CUDART_INF_F;
  int first_lane[kVectors], place[kVectors];  // of the vector's group, and in the groups' rows
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  for (int e = lane; e < 32 * kPer; e += 32) {
    const float b = bias != nullptr && e < s.E ? read_at(bias, e, s.E, 0.0f, &g_route_status) : 0.0f;
    if (e < s.E && b > kFarBias) least = fminf(least, b);
    if (warp == 0) sums[e] = b;
  }
  least = key_value(__reduce_min_sync(kAll, order_key(least)));
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kVectors; ++q) {
    const int e = expert_of<kV>(q * kV, lane), g = e < s.E ? e / gr.size : 0;
    first_lane[q] = g << gr.shift;
    place[q] = e < s.E ? g * gr.pitch + e - g * gr.size : -1;
  }
  int routed_here = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  Ahead<T, kPer, kV> ahead(s.E, lane);
  uint32_t wanted_ahead = 1u;
  const auto fetch = [&](int64_t t) {
    if (t >= s.tokens) return;
    if (in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status)) ahead.load(logits + t * s.ld, lane);
    if (mask != nullptr) wanted_ahead = read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status);
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  fetch(t);
  for (; t < s.tokens; t += step) {
    float x[kPer], c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = widen(ahead.v[i / kV].v[i % kV]);
    bool routed = wanted_ahead != 0u;
    fetch(t + step);
    float top = 0.0f, sum = 0.0f;
    if (!kLogistic) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);  // skips NaN
      top = key_value(max(__reduce_max_sync(kAll, order_key(top)), order_key(-FLT_MAX)));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = kLogistic ? logistic(x[i]) : exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
      sum += c[i];
    }
    sum = warp_sum(sum);
    if (sum == 0.0f) {  // no expert at all, or scores below fp32's range
      bool alive = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) alive |= x[i] != -CUDART_INF_F;
      routed = __any_sync(kAll, alive) && routed;
    }
    int rank = kMaxK, my_id = -1;
    float my_s = 0.0f;
    if (routed) {
      ++routed_here;
      const float inv = sum == 0.0f ? 0.0f : reciprocal(sum);
#pragma unroll
      for (int q = 0; q < kVectors; ++q) {
        const Vec<float, kV> b = *reinterpret_cast<const Vec<float, kV>*>(sums + expert_of<kV>(q * kV, lane));
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const int i = q * kV + j;
          if (kLogistic) {
            acc[i] = fmaf(c[i], inv, acc[i]);
            c[i] += b.v[j];
          } else {
            const float p = c[i] * inv;
            acc[i] += p;
            c[i] = p + b.v[j];
          }
          c[i] = x[i] > -CUDART_INF_F ? fmaxf(c[i], -CUDART_INF_F) : -CUDART_INF_F;  // not NaN
        }
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kVectors; ++q) {
        Vec<float, kV> v;
#pragma unroll
        for (int i = 0; i < kV; ++i) v.v[i] = x[q * kV + i];
        *reinterpret_cast<Vec<float, kV>*>(own_x + expert_of<kV>(q * kV, lane)) = v;
      }
      bool certain = true;
      if (gr.groups > 1) {
#pragma unroll
        for (int q = 0; q < kVectors; ++q) {
          Vec<float, kV> v;
#pragma unroll
          for (int i = 0; i < kV; ++i) v.v[i] = c[q * kV + i];
          if (place[q] >= 0) *reinterpret_cast<Vec<float, kV>*>(rows + place[q]) = v;
        }
        __syncwarp();
        const int g = lane >> gr.shift;
        float first = -CUDART_INF_F, second = -CUDART_INF_F;
        if (g < gr.groups) {
          const float* row = rows + g * gr.pitch;
#pragma unroll 1
          for (int m = (lane & (gr.lanes - 1)) * kV; m < gr.size; m += gr.lanes * kV) {
            const Vec<float, kV> v = *reinterpret_cast<const Vec<float, kV>*>(row + m);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
              second = fmaxf(second, fminf(first, v.v[i]));
              first = fmaxf(first, v.v[i]);
            }
          }
        }
#pragma unroll 1
        for (int d = gr.lanes >> 1; d > 0; d >>= 1) {
          const float other = __shfl_xor_sync(kAll, first, d), next = __shfl_xor_sync(kAll, second, d);
          second = fmaxf(fmaxf(second, next), fminf(first, other));
          first = fmaxf(first, other);
        }
        // the sum of two of the type's lowest values is a group's all the same
        const float value = fmaxf(second > -CUDART_INF_F ? first + second : first, -FLT_MAX);
        uint32_t left = first > -CUDART_INF_F ? order_key(value) : 0u, last = 0u, chosen = 0u;
#pragma unroll 1
        for (int r = 0; r < gr.best; ++r) {
          const uint32_t most = __reduce_max_sync(kAll, left);
          if (most == 0u) break;
          const int lead = __ffs(__ballot_sync(kAll, left == most)) - 1;  // the first lane of the lowest of them
          chosen |= 1u << lead;
          if (g == lead >> gr.shift) left = 0u;
          last = most;
        }
        const uint32_t next = __reduce_max_sync(kAll, left);
        if (next != 0u) {
          const float size = first > -CUDART_INF_F ? fabsf(first) + (second > -CUDART_INF_F ? fabsf(second) : 0.0f) : 0.0f;
          const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));  // not negative: ordered as its bits
          certain = key_value(last) - key_value(next) > group_doubt<kPer, kLogistic>(most, inv) ||
                    groups_clear<kPer, kLogistic>(first > -CUDART_INF_F, chosen >> (g << gr.shift) & 1u, value, first, size, 0.0f, inv, least);
        }
#pragma unroll
        for (int q = 0; q < kVectors; ++q) {
          const bool in = chosen >> first_lane[q] & 1u;
#pragma unroll
          for (int i = 0; i < kV; ++i) c[q * kV + i] = in ? c[q * kV + i] : -CUDART_INF_F;
        }
      }
      float most = c[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) most = fmaxf(most, c[i]);
      uint32_t mine = order_key(most);
      // the k-th largest lane maximum, equal ones counted once; 0 when there are fewer
      uint32_t bar = __reduce_max_sync(kAll, mine);
      const uint32_t first_key = bar;
      const bool any = bar != 0u;
#pragma unroll 4
      for (int j = 1; j < s.k; ++j) {
        if (mine == bar) mine = 0u;
        bar = __reduce_max_sync(kAll, mine);
      }
      if (any && certain) {
        float from;
        int own_n, upto, n;
        const auto gather = [&](float low) {  // those from there on side by side, the lanes' one behind the other
          from = fmaxf(low - 4.0f * doubt<kPer, kLogistic>(low, inv, least, 0.0f), -FLT_MAX);
          own_n = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) own_n += c[i] >= from ? 1 : 0;
          upto = own_n;
#pragma unroll
          for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(kAll, upto, d);
            if (lane >= d) upto += other;
          }
          n = __shfl_sync(kAll, upto, 31);
        };
        gather(bar != 0u ? key_value(bar) : -FLT_MAX);
        if (n > 32) {  // lanes with several of the largest, as when k is near 32: from the k-th of all on, by halving
          uint32_t below = bar, above = first_key + 1u;
          int count = n;
#pragma unroll 1
          while (count != s.k && above - below > 1u) {
            const uint32_t mid = below + (above - below) / 2u;
            int own = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) own += c[i] >= key_value(mid) ? 1 : 0;
            own = __reduce_add_sync(kAll, own);
            if (own >= s.k) below = mid, count = own;
            else above = mid;
          }
          gather(key_value(max(below, order_key(-FLT_MAX))));
        }
        if (n <= 32) {
          uint32_t at = smem_u32(&few[warp][upto - own_n]);
#pragma unroll
          for (int i = 0; i < kPer; ++i) put_from(at, expert_of<kV>(i, lane), c[i], from);
          __syncwarp();
          const int e = lane < n ? few[warp][lane] : 0;
          const float x_e = own_x[e], own_b = sums[e];
          my_s = kLogistic ? logistic(x_e) : exp2_ftz((x_e - top) * kLog2E) * inv;
          const float own_c = lane < n ? my_s + own_b : -CUDART_INF_F;
          few_c[warp][lane] = own_c;
          __syncwarp();
          int before = 0;
          for (int i = 0; i < n; i += 4) {
            const float4 other = *reinterpret_cast<const float4*>(&few_c[warp][i]);
            before += (other.x > own_c ? 1 : 0) + (other.y > own_c ? 1 : 0) + (other.z > own_c ? 1 : 0) + (other.w > own_c ? 1 : 0);
          }
          // equal ones by their index
          const uint32_t places = __reduce_or_sync(kAll, lane < n ? 1u << before : 0u);
          if (__popc(places) != n)
            for (int i = 0; i < n; ++i) {
              const float other = __shfl_sync(kAll, own_c, i);
              const int o = __shfl_sync(kAll, e, i);
              if (other == own_c && o < e) ++before;
            }
          __syncwarp();
          if (lane < n) few_c[warp][before] = own_c;
          __syncwarp();
          const bool no_matter = lane >= n || before >= s.k || before + 1 >= n;
          const float gap = no_matter ? 0.0f : own_c - few_c[warp][before + 1];
          if (!all_clear<kPer, kLogistic>(no_matter, gap, own_c, inv, least, 0.0f)) {
            before = settle<kPer, kLogistic>(e, x_e, own_b, my_s, top - x_e, n, s.k);
            certain = !__any_sync(kAll, before < 0);
          }
          if (certain && lane < n && before < s.k) {
            rank = before;
            my_id = e;
          }
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
        my_s = kLogistic ? logistic(own) : exp2_ftz((own - top) * kLog2E) * inv;
      }
      if (my_id >= 0) atomicAdd(&hist[my_id], 1);
    }
    float w = my_id >= 0 ? my_s : 0.0f;
    if (s.renorm) {
      const float all = warp_sum(w);
      w = all == 0.0f ? 0.0f : w * reciprocal(all);
    }
    w *= gr.scale;
    const uint32_t chosen = __ballot_sync(kAll, my_id >= 0);
    if (__popc(chosen) < s.k && my_id < 0) {  // as many other lanes write the places left
      rank = __popc(chosen) + __popc(~chosen & ((1u << lane) - 1u));
      w = 0.0f;
    }
    if (rank < s.k) {
      const int64_t at = t * s.k + rank;
      if (in_buf(weights + at, 4, weights, out_bytes, &g_route_status) && in_buf(ids + at, 4, ids, out_bytes, &g_route_status)) {
        weights[at] = w;
        ids[at] = my_id;
      }
    }
  }
  if (lane == 0 && routed_here) atomicAdd(&routed_tokens, routed_here);
  __syncthreads();  // the last readers of the groups' rows and the biases
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

// At most eight experts a lane: a lane's are consecutive ones of one group (gr.lanes lanes
// a group), so that a group's two largest are two shuffles a step away from the lanes' own,
// a group that is not chosen leaves its lanes out, and nothing goes by single experts.  A
// lane sorts its experts' keys; each of the k + 1 rounds takes the largest of the lanes'
// heads and moves one lane on.  A key's lowest bits give way to the expert's place in its
// lane, lower places first, and what they held is added to the doubt.
// A group's best is known without a pass through shared memory and a candidate without a
// pass over all: 615 instructions a token in place of 860 with the kernel above.  131071
// tokens by this kernel and by that: 16 experts 47 and 54 us, 64 in 8 groups 74 and 95, 64
// without groups, softmax, 62 and 74, 128 in 8 groups 83 and 108, 150 bf16 in 5 groups,
// softmax, 128 and 165, 256 in 8 groups 114 and 132, in 32 groups 126 and 156, bf16 without
// groups, softmax, 93 and 102.
template <int kW>
__device__ __forceinline__ void sort_down(uint32_t (&k)[kW]) {
  const auto order = [&](int a, int b) {
    const uint32_t high = max(k[a], k[b]), low = min(k[a], k[b]);
    k[a] = high, k[b] = low;
  };
  if constexpr (kW == 2) order(0, 1);
  if constexpr (kW == 4) order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  if constexpr (kW == 8) {
    order(0, 1), order(2, 3), order(4, 5), order(6, 7);
    order(0, 2), order(1, 3), order(4, 6), order(5, 7);
    order(1, 2), order(5, 6), order(0, 4), order(3, 7);
    order(1, 5), order(2, 6);
    order(1, 4), order(3, 6);
    order(2, 4), order(3, 5);
    order(3, 4);
  }
}

// A token's logits, kW consecutive ones a lane: in vectors where kVector (each lane has all
// of its experts or none), else one by one; those that are not there stay -inf.
template <typename T, int kW, bool kVector>
struct OwnedAhead {
  static constexpr int kV = kVector ? (kW * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : kW) : 1;
  Vec<T, kV> v[kW / kV];
  __device__ __forceinline__ OwnedAhead() {
#pragma unroll
    for (int i = 0; i < kW; ++i) v[i / kV].v[i % kV] = minus_infinity<T>();
  }
  __device__ __forceinline__ void load(const T* first, int there) {
#pragma unroll
    for (int q = 0; q < kW / kV; ++q) {
      const T* at = first + q * kV;
      const uint32_t p = q * kV < there ? 1u : 0u;
      if constexpr (sizeof v[q] == 16) {
        uint4& w = *reinterpret_cast<uint4*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                     : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w) : "l"(at), "r"(p));
      } else if constexpr (sizeof v[q] == 8) {
        uint2& w = *reinterpret_cast<uint2*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p ld.global.nc.v2.b32 {%0, %1}, [%2];\n\t}"
                     : "+r"(w.x), "+r"(w.y) : "l"(at), "r"(p));
      } else if constexpr (sizeof v[q] == 4) {
        uint32_t& w = *reinterpret_cast<uint32_t*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}" : "+r"(w) : "l"(at), "r"(p));
      } else {
        uint16_t& w = *reinterpret_cast<uint16_t*>(&v[q]);
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.b16 %0, [%1];\n\t}" : "+h"(w) : "l"(at), "r"(p));
      }
    }
  }
};

// Where shared memory holds the value of place i of a lane: vectors side by side.
template <int kW>
__device__ __forceinline__ int owned_at(int lane, int i) {
  constexpr int kU = kW < 4 ? kW : 4;
  return i / kU * (32 * kU) + lane * kU + i % kU;
}
// Of c, which is neither NaN nor -0, at place i of its lane.
template <int kW>
__device__ __forceinline__ uint32_t owned_key(float c, int i) {
  const uint32_t b = __float_as_uint(c);
  return ((b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u)) & ~static_cast<uint32_t>(kW - 1)) |
         static_cast<uint32_t>(kW - 1 - i);
}
template <int kW>
__device__ __forceinline__ int owned_place(uint32_t key) { return kW - 1 - static_cast<int>(key & (kW - 1)); }
template <int kW>
__device__ __forceinline__ float owned_value(uint32_t key) { return key_value(key & ~static_cast<uint32_t>(kW - 1)); }
// What a key may lack of the value.
template <int kW>
__device__ __forceinline__ float owned_cut(float v) { return kW > 1 ? fmaf(fabsf(v), kW * 0x1p-23f, kW * 0x1p-149f) : 0.0f; }

// A token some of whose candidates have like keys or lie too near one another: the rounds
// once more, a lane at a time, on until one is clearly behind the k-th or none is left, and
// then by settle.  Lane j returns an expert and its place among the chosen, place << 16 |
// expert, -1 where it has none; all -2 where it takes the whole row.
template <int kW, bool kLogistic>
__device__ __noinline__ int settle_owned(const uint32_t* lists, bool in, const float* own_x, const float* own_b, float top, float inv,
                                         float least, int k, int size, int lanes, int shift) {
  const int lane = threadIdx.x & 31;
  uint32_t head = in ? lists[lane] : 0u, kept = 0u;
  int from = 0, taken = 1, n = 0;
  const auto far = [&] {  // the last one from the k-th
    const float low = owned_value<kW>(__shfl_sync(kAll, kept, k - 1)), end = owned_value<kW>(__shfl_sync(kAll, kept, n - 1));
    return low - end > 4.0f * doubt<kW, kLogistic>(low, inv, least, owned_cut<kW>(low));
  };
  bool all = false;
  while (!all) {
    const uint32_t most = __reduce_max_sync(kAll, head);
    if (most == 0u) break;
    if (n == 32) return -2;
    const int lead = __ffs(__ballot_sync(kAll, head == most)) - 1;
    if (lane == n) kept = most, from = lead;
    if (lane == lead) head = lists[32 * taken++ + lane];
    all = ++n > k && far();
  }
  const int place = owned_place<kW>(kept);
  const int e = (from >> shift) * size + (from & (lanes - 1)) * kW + place;
  const float x = own_x[owned_at<kW>(from, place)], b = own_b[owned_at<kW>(from, place)];
  const float score = kLogistic ? logistic(x) : exp2_ftz((x - top) * kLog2E) * inv;
  const int before = settle<kW, kLogistic>(e, x, b, score, top - x, n, k);
  if (__any_sync(kAll, before < 0)) return -2;
  return lane < n && before < k ? before << 16 | e : -1;
}

template <typename T, int kW, bool kVector, bool kLogistic>
__global__ void __launch_bounds__(1024, 1)
    route_owned_kernel(const T* __restrict__ logits, const RouteShape s, const Grouped gr, const float* __restrict__ bias,
                       const uint8_t* __restrict__ mask, float* __restrict__ weights, int32_t* __restrict__ ids, float* part_p,
                       int32_t* part_c, int32_t* part_n, uint32_t* joined, int32_t* counts, float* loss, int32_t* n_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = 32, kLane = 32 * kW, kU = kW < 4 ? kW : 4;
  __shared__ int32_t routed_tokens;
  __shared__ uint2 slots[kWarps][kMaxK + 1];  // the candidates' keys and lanes, largest first
  float* own_x = reinterpret_cast<float*>(smem);          // [warps][kW of 32 lanes]: the token's logits; then the warps' sums
  uint32_t* lists = reinterpret_cast<uint32_t*>(own_x + kWarps * kLane);  // [warps][kW + 1, 32]: the lanes' keys, largest first, and 0
  float* own_b = reinterpret_cast<float*>(lists + kWarps * (kLane + 32)); // [kW of 32 lanes]: the biases
  float* sums = own_b + kLane;                                            // [E]
  int32_t* hist = reinterpret_cast<int32_t*>(sums + s.E);                 // [E]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> gr.shift, at_g = (lane & (gr.lanes - 1)) * kW;    // the lane's group and its first expert's place there
  const int there = g < gr.groups ? min(max(gr.size - at_g, 0), kW) : 0, e0 = there > 0 ? g * gr.size + at_g : 0;
  for (int e = tid; e < s.E; e += 32 * kWarps) hist[e] = 0;
  if (tid == 0) routed_tokens = 0;
  own_x += warp * kLane, lists += warp * (kLane + 32);
  lists[kLane + lane] = 0u;
  pdl_wait();
  const uint64_t in_bytes = (static_cast<uint64_t>(s.tokens - 1) * s.ld + s.E) * sizeof(T);
  const uint64_t out_bytes = static_cast<uint64_t>(s.tokens) * s.k * 4;
  if (gridDim.x > 1) pdl_launch_dependents();  // the join's few blocks wait beside this one
  float least = CUDART_INF_F, acc[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    acc[i] = 0.0f;
    const float b = bias != nullptr && i < there ? read_at(bias, e0 + i, s.E, 0.0f, &g_route_status) : 0.0f;
    if (warp == 0) own_b[owned_at<kW>(lane, i)] = b;
    if (i < there && b > kFarBias) least = fminf(least, b);
  }
  least = key_value(__reduce_min_sync(kAll, order_key(least)));
  __syncthreads();
  int routed_here = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  OwnedAhead<T, kW, kVector> ahead;
  uint32_t wanted_ahead = 1u;
  const auto fetch = [&](int64_t t) {
    if (t >= s.tokens) return;
    if (in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status)) ahead.load(logits + t * s.ld + e0, there);
    if (mask != nullptr) wanted_ahead = read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status);
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  fetch(t);
  for (; t < s.tokens; t += step) {
    float x[kW], c[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) x[i] = widen(ahead.v[i / ahead.kV].v[i % ahead.kV]);
    bool routed = wanted_ahead != 0u;
    float top = 0.0f, sum = 0.0f;
    if (!kLogistic) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < kW; ++i) top = fmaxf(top, x[i]);  // skips NaN
      top = key_value(max(__reduce_max_sync(kAll, order_key(top)), order_key(-FLT_MAX)));
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      c[i] = kLogistic ? logistic(x[i]) : exp2_ftz((x[i] - top) * kLog2E);  // 0 where there is no expert: those are -inf
      sum += c[i];
    }
    sum = warp_sum(sum);
    if (sum == 0.0f) {  // no expert at all, or scores below fp32's range
      bool alive = false;
#pragma unroll
      for (int i = 0; i < kW; ++i) alive |= x[i] != -CUDART_INF_F;
      routed = __any_sync(kAll, alive) && routed;
    }
    int rank = kMaxK, my_id = -1;
    float my_s = 0.0f;
    if (routed) {
      ++routed_here;
      const float inv = sum == 0.0f ? 0.0f : reciprocal(sum);
      __syncwarp();
      slots[warp][lane] = make_uint2(0u, 0u);
      slots[warp][lane + 1] = make_uint2(0u, 0u);
      uint32_t key[kW];
#pragma unroll
      for (int q = 0; q < kW; q += kU) {
        const Vec<float, kU> b = *reinterpret_cast<const Vec<float, kU>*>(own_b + owned_at<kW>(lane, q));
        Vec<float, kU> v;
#pragma unroll
        for (int j = 0; j < kU; ++j) {
          const int i = q + j;
          v.v[j] = x[i];
          if (kLogistic)
            acc[i] = fmaf(c[i], inv, acc[i]);
          else
            acc[i] += c[i] *= inv;
          c[i] += b.v[j];
          key[i] = x[i] > -CUDART_INF_F && c[i] > -CUDART_INF_F ? owned_key<kW>(c[i], i) : 0u;  // not NaN
        }
        *reinterpret_cast<Vec<float, kU>*>(own_x + owned_at<kW>(lane, q)) = v;
      }
      fetch(t + step);  // not before: x and c have taken the registers
      sort_down<kW>(key);
#pragma unroll
      for (int i = 0; i < kW; ++i) lists[i * 32 + lane] = key[i];
      bool certain = true, in = true;
      if (gr.groups > 1) {
        uint32_t first = key[0], second = kW > 1 ? key[kW > 1 ? 1 : 0] : 0u;
#pragma unroll 1
        for (int d = gr.lanes >> 1; d > 0; d >>= 1) {
          const uint32_t other = __shfl_xor_sync(kAll, first, d), next = __shfl_xor_sync(kAll, second, d);
          second = max(max(second, next), min(first, other));
          first = max(first, other);
        }
        const float of_first = owned_value<kW>(first), of_second = second != 0u ? owned_value<kW>(second) : 0.0f;
        const float value = fmaxf(of_first + of_second, -FLT_MAX);
        uint32_t left = first != 0u ? order_key(value) : 0u, last = 0u;
        in = false;
#pragma unroll 1
        for (int r = 0; r < gr.best; ++r) {  // groups of like values at once
          last = __reduce_max_sync(kAll, left);
          if (left == last) in = true, left = 0u;
        }
        const uint32_t next = __reduce_max_sync(kAll, left);
        if (next != 0u) {
          const float size = first != 0u ? fabsf(of_first) + fabsf(of_second) : 0.0f;
          const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));  // not negative: ordered as its bits
          certain = key_value(last) - key_value(next) > group_doubt<kW, kLogistic>(most, inv) + owned_cut<kW>(most) ||
                    groups_clear<kW, kLogistic>(first != 0u, in, value, of_first, size, owned_cut<kW>(size), inv, least);
        }
        if (__popc(__ballot_sync(kAll, in && first != 0u)) > gr.best << gr.shift) certain = false;
      }
      if (certain) {
        uint32_t head = in ? key[0] : 0u, at = smem_u32(lists + 32 + lane), slot = smem_u32(&slots[warp][0]);
        const uint32_t begin = at;
        __syncwarp();
#pragma unroll 3
        for (int r = 0; r <= s.k; ++r) {  // all lanes whose head is the largest: nearly always one
          const uint32_t most = __reduce_max_sync(kAll, head);
          asm volatile(
              "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\tsetp.eq.and.u32 p, %0, %2, p;\n\t@p st.shared.v2.b32 [%3], {%2, %4};\n\t"
              "@p ld.shared.b32 %0, [%1];\n\t@p add.u32 %1, %1, 128;\n\t}"
              : "+r"(head), "+r"(at)
              : "r"(most), "r"(slot + 8 * r), "r"(lane)
              : "memory");
        }
        __syncwarp();
        const uint2 own = slots[warp][lane];
        const uint32_t next = slots[warp][lane + 1].x;
        const int n = __popc(__ballot_sync(kAll, own.x != 0u)) + (__ballot_sync(kAll, next != 0u) >> 31);
        const int place = owned_place<kW>(own.x), from = static_cast<int>(own.y);
        const float x_e = own_x[owned_at<kW>(from, place)];
        my_s = kLogistic ? logistic(x_e) : exp2_ftz((x_e - top) * kLog2E) * inv;
        const float own_c = my_s + own_b[owned_at<kW>(from, place)];
        const bool clear = all_clear<kW, kLogistic>(lane >= s.k || own.x == 0u || next == 0u, own_c - owned_value<kW>(next), own_c, inv,
                                                    least, 2.0f * owned_cut<kW>(own_c));
        if (clear && __reduce_add_sync(kAll, at - begin) == 128u * n) {
          if (lane < s.k && own.x != 0u) rank = lane, my_id = (from >> gr.shift) * gr.size + (from & (gr.lanes - 1)) * kW + place;
        } else if (n > 0) {
          const int found = settle_owned<kW, kLogistic>(lists, in, own_x, own_b, top, inv, least, s.k, gr.size, gr.lanes, gr.shift);
          certain = found != -2;
          if (found >= 0) {
            rank = found >> 16, my_id = found & 0xFFFF;
            const int g_e = my_id / gr.size, j = my_id - g_e * gr.size;
            const float chosen_x = own_x[owned_at<kW>((g_e << gr.shift) + j / kW, j % kW)];
            my_s = kLogistic ? logistic(chosen_x) : exp2_ftz((chosen_x - top) * kLog2E) * inv;
          }
        }
      }
      if (!certain) {
        const T* row = logits + t * s.ld;
        my_id = in_buf(row, s.E * sizeof(T), logits, in_bytes, &g_route_status)
                    ? choose_exactly<T, kW, kLogistic>(row, bias, s.E, s.k, gr.groups, gr.best, gr.size) : -1;
        rank = my_id >= 0 ? lane : kMaxK;
        const float own = my_id >= 0 ? widen(row[my_id]) : 0.0f;
        my_s = kLogistic ? logistic(own) : exp2_ftz((own - top) * kLog2E) * inv;
      }
      if (my_id >= 0) atomicAdd(&hist[my_id], 1);
    } else {
      fetch(t + step);
    }
    float w = my_id >= 0 ? my_s : 0.0f;
    if (s.renorm) {
      const float all = warp_sum(w);
      w = all == 0.0f ? 0.0f : w * reciprocal(all);
    }
    w *= gr.scale;
    const uint32_t chosen = __ballot_sync(kAll, my_id >= 0);
    if (__popc(chosen) < s.k && my_id < 0) {  // as many other lanes write the places left
      rank = __popc(chosen) + __popc(~chosen & ((1u << lane) - 1u));
      w = 0.0f;
    }
    if (rank < s.k) {
      const int64_t at = t * s.k + rank;
      if (in_buf(weights + at, 4, weights, out_bytes, &g_route_status) && in_buf(ids + at, 4, ids, out_bytes, &g_route_status)) {
        weights[at] = w;
        ids[at] = my_id;
      }
    }
  }
  if (lane == 0 && routed_here) atomicAdd(&routed_tokens, routed_here);
  __syncwarp();
  // the warps' sums side by side, then added up in warp order
#pragma unroll
  for (int i = 0; i < kW; ++i) own_x[owned_at<kW>(lane, i)] = acc[i];
  __syncthreads();
  for (int e = tid; e < s.E; e += 32 * kWarps) {
    const int g_e = e / gr.size, j = e - g_e * gr.size;
    const float* at = reinterpret_cast<const float*>(smem) + owned_at<kW>((g_e << gr.shift) + j / kW, j % kW);
    float sum = 0.0f;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) sum += at[w * kLane];
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
  Ahead<T, kPer, kV> ahead(s.E, lane);
  uint32_t wanted_ahead = 1u;
  int32_t e_ahead = -1;
  float dw_ahead = 0.0f;
  const auto fetch = [&](int64_t t) {
    if (t >= s.tokens) return;
    if (in_buf(logits + t * s.ld, s.E * sizeof(T), logits, in_bytes, &g_route_status)) ahead.load(logits + t * s.ld, lane);
    if (mask != nullptr) wanted_ahead = read_at(mask, t, s.tokens, uint8_t{0}, &g_route_status);
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
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = widen(ahead.v[i / kV].v[i % kV]);
    bool routed = wanted_ahead != 0u;
    fetch(t + step);
    float top = 0.0f;
    if (!kLogistic) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);  // skips NaN
      top = key_value(max(__reduce_max_sync(kAll, order_key(top)), order_key(-FLT_MAX)));
    }
    T* out = dlogits + t * ldd;
    float d[kPer], rest[kPer], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kLogistic)
        logistic_pair(x[i], d[i], rest[i]);
      else
        d[i] = exp2_ftz((x[i] - top) * kLog2E);  // 0 past E: those are -inf
      sum += d[i];
    }
    sum = warp_sum(sum);
    // with a sum of 0 every score is 0, and so is every gradient
    if (routed && sum != 0.0f) {
      float (&sc)[kPer] = d;
      const float inv = reciprocal(sum);
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
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] = 0.0f;
    }
    if (!in_buf(out, s.E * sizeof(T), dlogits, out_bytes, &g_route_status)) continue;
#pragma unroll
    for (int q = 0; q < kPer / kV; ++q) {
      const int e0 = expert_of<kV>(q * kV, lane);
      if (e0 >= s.E) continue;
      Vec<T, kV> v;
#pragma unroll
      for (int j = 0; j < kV; ++j) v.v[j] = narrow<T>(d[q * kV + j]);
      *reinterpret_cast<Vec<T, kV>*>(out + e0) = v;
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

// A forward kernel over blocks of so many warps, and the join where there is more than one.
template <typename T, typename Kernel>
int launch_choice(const GroupsCall& a, const Grouped& gr, Kernel* kernel, int warps, size_t smem, bool (&attr_done)[64]) {
  const int blocks = route_blocks(a.s.tokens, warps, a.sms);
  float* part_p = reinterpret_cast<float*>(a.workspace);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + static_cast<int64_t>(blocks) * a.s.E);
  int32_t* part_n = part_c + static_cast<int64_t>(blocks) * a.s.E;
  uint32_t* joined = reinterpret_cast<uint32_t*>(part_n + blocks);
  float* part_loss = reinterpret_cast<float*>(joined + 1);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 184 * 1024) != cudaSuccess) return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  const int rc = launch_pdl(kernel, static_cast<unsigned>(blocks), 32 * warps, smem, a.stream, static_cast<const T*>(a.logits), a.s, gr,
                            a.bias, a.mask, a.weights, a.ids, part_p, part_c, part_n, joined, a.counts, a.loss, a.n);
  if (rc != MXQ_OK || blocks == 1) return rc;
  return launch_pdl(route_join_kernel, static_cast<unsigned>(ceil_div(a.s.E, 32)), 32 * kJoinWarps, 0, a.stream, a.s, blocks, part_p,
                    part_c, part_n, joined, part_loss, a.counts, a.loss, a.n);
}
template <typename T, int kPer, int kV, bool kLogistic>
int launch_groups(const GroupsCall& a) {
  constexpr int kThreads = route_threads<kPer>(), kWarps = kThreads / 32;
  // the next number of floats that is a group's lanes' vectors past a multiple of 32 banks:
  // neighbouring groups' lanes then read neighbouring banks
  Grouped gr = a.gr;
  gr.pitch = gr.size + ((gr.lanes * kV - gr.size) % 32 + 32) % 32;
  const int rows = gr.groups > 1 ? gr.groups * gr.pitch : 0;
  const size_t smem = static_cast<size_t>(kWarps) * ((rows > 32 * kPer ? rows : 32 * kPer) + 32 * kPer) * 4 + 32 * kPer * 4 +
                      static_cast<size_t>(a.s.E) * 4;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  return launch_choice<T>(a, gr, route_groups_kernel<T, kPer, kV, kLogistic, kThreads>, kWarps, smem, attr_done);
}
template <typename T, int kW, bool kVector>
int launch_owned(const GroupsCall& a, int scores) {
  const size_t smem = ((2 * 32 + 1) * 32 * kW + 32 * 32) * 4 + static_cast<size_t>(a.s.E) * 8;
  static bool attr_done[2][64] = {};  // benign race: the same attribute set twice
  return scores == MXQ_SCORES_SIGMOID ? launch_choice<T>(a, a.gr, route_owned_kernel<T, kW, kVector, true>, 32, smem, attr_done[0])
                                      : launch_choice<T>(a, a.gr, route_owned_kernel<T, kW, kVector, false>, 32, smem, attr_done[1]);
}
// Vectors where every lane has all of its kW experts or none, at aligned places.
template <typename T, int kW>
int launch_owned_width(const GroupsCall& a, int scores, int align) {
  constexpr int kBytes = kW * static_cast<int>(sizeof(T));
  if constexpr (kW > 1)
    if (a.gr.size % kW != 0 || align < (kBytes < 16 ? kBytes : 16)) return launch_owned<T, kW, false>(a, scores);
  return launch_owned<T, kW, true>(a, scores);
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

// Vectors of 4 elements (2 for up to 64 experts) where base and row pitch are aligned to
// them and the experts, and those of a group, are whole vectors; else single elements.
template <typename T, bool kBack>
int launch_grouped(const GroupsCall& a, int scores) {
  const uint64_t pitch = static_cast<uint64_t>(a.s.ld) * sizeof(T);
  const uint64_t dpitch = kBack ? static_cast<uint64_t>(a.ldd) * sizeof(T) : 0;
  const int align = common_alignment({address_of(a.logits), pitch, kBack ? address_of(a.dlogits) : 0, dpitch});
  const int size = kBack ? a.s.E : a.gr.size;
  const bool v4 = align >= static_cast<int>(4 * sizeof(T)) && size % 4 == 0, v2 = align >= static_cast<int>(2 * sizeof(T)) && size % 2 == 0;
  const int E = a.s.E;
  if constexpr (kBack) {
    if (E <= 32) return launch_scores<T, 1, 1, true>(a, scores);
    if (E <= 64) return v2 ? launch_scores<T, 2, 2, true>(a, scores) : launch_scores<T, 2, 1, true>(a, scores);
    if (E <= 128) return v4 ? launch_scores<T, 4, 4, true>(a, scores) : launch_scores<T, 4, 1, true>(a, scores);
  } else {  // by a lane's part of a group, which is at most 8 for up to 128 experts
    const int64_t part = ceil_div(a.gr.size, a.gr.lanes);
    if (part <= 1) return launch_owned_width<T, 1>(a, scores, align);
    if (part <= 2) return launch_owned_width<T, 2>(a, scores, align);
    if (part <= 4) return launch_owned_width<T, 4>(a, scores, align);
    if (part <= 8) return launch_owned_width<T, 8>(a, scores, align);
  }
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
  a.gr.shift = 5;
  while (32 >> a.gr.shift < a.gr.groups) --a.gr.shift;
  a.gr.lanes = 1 << a.gr.shift;
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
