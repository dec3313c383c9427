// moe_route_common.cuh -- what the routing kernels share: keys in the order of the values,
// a token's logits in the lanes of a warp, and the sums over tokens: each block's in its
// own part of the workspace, joined in a fixed order.
#pragma once

#include <cuda_runtime.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_route_status = 0;

constexpr int kMaxK = 32;  // a chosen expert per lane

// Unsigned key in the order of the values: 0 for -inf and NaN (never chosen),
// the same for both zeros.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return x > -CUDART_INF_F ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// A key in the order in which experts are chosen, no two of a row alike: the
// larger logit, then the lower expert.  The logits of one type take 32 bits where
// their own keys leave 16 for the expert.
template <typename T>
struct ChoiceKey {
  using type = uint64_t;
  static __device__ __forceinline__ type of(float x, int e) {
    return (static_cast<uint64_t>(order_key(x)) << 32) | static_cast<uint32_t>(~e);
  }
};
template <>
struct ChoiceKey<bf16_t> {
  using type = uint32_t;
  static __device__ __forceinline__ type of(float x, int e) {
    return (order_key(x) & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(e));
  }
};

// Expert of register i of a lane: vectors of kV consecutive experts per lane.
template <int kV>
__device__ __forceinline__ int expert_of(int i, int lane) {
  return (i / kV) * (32 * kV) + lane * kV + i % kV;
}

// A lane's logits of one row as they are stored; experts past E are -inf and
// stay so.
template <typename T>
__device__ __forceinline__ T minus_infinity();
template <>
__device__ __forceinline__ float minus_infinity<float>() {
  return -CUDART_INF_F;
}
template <>
__device__ __forceinline__ bf16_t minus_infinity<bf16_t>() {
  return 0xFF80u;
}
template <typename T, int kPer, int kV>
struct Row {
  Vec<T, kV> v[kPer / kV];
  __device__ __forceinline__ Row() {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i / kV].v[i % kV] = minus_infinity<T>();
  }
  __device__ __forceinline__ void load(const T* row, int E, int lane) {
#pragma unroll
    for (int c = 0; c < kPer / kV; ++c) {
      const int e0 = expert_of<kV>(c * kV, lane);
      if (e0 + kV <= E) {
        v[c] = load_once<T, kV>(row + e0);
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (e0 + j < E) v[c].v[j] = row[e0 + j];
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = widen(v[i / kV].v[i % kV]);
  }
};

struct RouteShape {
  int64_t tokens, ld;
  int E, k, renorm;
};

// The loss from sum_e counts_e sum_t p_te over n tokens.
__device__ __forceinline__ float loss_of(const RouteShape& s, float sum, int n) {
  const float f = static_cast<float>(n);
  return n > 0 ? sum * (static_cast<float>(s.E) / (static_cast<float>(s.k) * f * f)) : 0.0f;
}

// Counts, routed tokens and loss of a grid of one block, from its sums.
__device__ __forceinline__ void finish_alone(const RouteShape& s, const float* p, const int32_t* c, int n, int32_t* counts,
                                             float* loss, int32_t* n_out) {
  __shared__ float by_warp[32];
  const int tid = threadIdx.x;
  float sum = 0.0f;
  for (int e = tid; e < s.E; e += blockDim.x) {
    write_at(counts, e, s.E, c[e], &g_route_status);
    sum += static_cast<float>(c[e]) * p[e];
  }
  sum = warp_sum(sum);
  if ((tid & 31) == 0) by_warp[tid >> 5] = sum;
  __syncthreads();
  if (tid >= 32) return;
  sum = warp_sum(tid < static_cast<int>(blockDim.x) / 32 ? by_warp[tid] : 0.0f);
  if (tid == 0) {
    *loss = loss_of(s, sum, n);
    *n_out = n;
  }
}

// A block's sums, counts and tokens: its part for the join, or the results.
__device__ __forceinline__ void finish_block(const RouteShape& s, const float* sums, const int32_t* hist, int tokens,
                                             float* part_p, int32_t* part_c, int32_t* part_n, uint32_t* joined,
                                             int32_t* counts, float* loss, int32_t* n_out) {
  if (gridDim.x == 1) {
    finish_alone(s, sums, hist, tokens, counts, loss, n_out);
    return;
  }
  const int64_t base = static_cast<int64_t>(blockIdx.x) * s.E;
  for (int e = threadIdx.x; e < s.E; e += blockDim.x) {
    write_at(part_p, base + e, static_cast<int64_t>(gridDim.x) * s.E, sums[e], &g_route_status);
    write_at(part_c, base + e, static_cast<int64_t>(gridDim.x) * s.E, hist[e], &g_route_status);
  }
  if (threadIdx.x == 0) {
    write_at(part_n, blockIdx.x, gridDim.x, tokens, &g_route_status);
    if (blockIdx.x == 0) *joined = 0u;
  }
}

// Sums over the blocks, part_p and part_c [blocks, E], part_n [blocks]: a block
// for 32 experts, whose warps take every kJoinWarps-th block of the grid before
// and are added in order.  The block that is last to write its part of the loss
// adds the parts up.  (With one block for all experts the forward pass takes 64.6 us
// instead of 58.3 at 131071 tokens x 250 experts, 87.8 instead of 59.3 at 32768 x
// 1024: its threads' loads come in several turns.)
constexpr int kJoinWarps = 16, kMaxBlocks = 256, kMaxJoins = 32;
static_assert(MXQ_MAX_GROUPS <= 32 * kMaxJoins, "a lane for each block's part of the loss");
__global__ void __launch_bounds__(32 * kJoinWarps)
    route_join_kernel(const RouteShape s, int blocks, const float* part_p, const int32_t* part_c,
                      const int32_t* part_n, uint32_t* joined, float* part_loss, int32_t* counts, float* loss,
                      int32_t* n_out) {
  __shared__ float sum_p[kJoinWarps][32];
  __shared__ int32_t sum_c[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  pdl_wait();
  float p = 0.0f;
  int c = 0, n = 0;
  if (e < s.E)
#pragma unroll 10
    for (int b = warp; b < blocks; b += kJoinWarps) {
      p += read_at(part_p, static_cast<int64_t>(b) * s.E + e, static_cast<int64_t>(blocks) * s.E, 0.0f, &g_route_status);
      c += read_at(part_c, static_cast<int64_t>(b) * s.E + e, static_cast<int64_t>(blocks) * s.E, 0, &g_route_status);
    }
  if (warp == 0)
    for (int b = lane; b < blocks; b += 32) n += read_at(part_n, b, blocks, 0, &g_route_status);
  sum_p[warp][lane] = p;
  sum_c[warp][lane] = c;
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < kJoinWarps; ++w) {
    p += sum_p[w][lane];
    c += sum_c[w][lane];
  }
  if (e < s.E) write_at(counts, e, s.E, c, &g_route_status);
  const float own = warp_sum(e < s.E ? static_cast<float>(c) * p : 0.0f);
  uint32_t before = 0;
  if (lane == 0) {
    write_at(part_loss, blockIdx.x, gridDim.x, own, &g_route_status);
    __threadfence();
    before = atomicAdd(joined, 1u);
    __threadfence();
  }
  if (__shfl_sync(0xFFFFFFFFu, before, 0) + 1 != gridDim.x) return;
  const float all = warp_sum(
      lane < static_cast<int>(gridDim.x) && in_array(part_loss, lane, gridDim.x, &g_route_status) ? __ldcg(part_loss + lane) : 0.0f);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if (lane == 0) {
    *loss = loss_of(s, all, n);
    *n_out = n;
  }
}

// kPer registers of logits per lane hold up to 32 * kPer experts; the block is
// as large as the registers allow, so that there are few partial sums.
template <int kPer>
constexpr int route_threads() {
  return kPer <= 8 ? 1024 : kPer == 16 ? 512 : 256;
}
// threads of a block of the backward pass: its shared rows stay within 32 KB
template <int kPer>
constexpr int back_threads() {
  return kPer <= 16 ? 256 : 128;
}

int route_blocks(int64_t tokens, int warps, int sms) {
  const int64_t want = ceil_div(tokens, warps);
  return static_cast<int>(want < 1 ? 1 : want < sms ? want : sms);
}

}  // namespace
