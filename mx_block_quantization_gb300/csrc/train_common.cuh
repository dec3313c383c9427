// train_common.cuh -- element types, vector access and warp sums shared by the
// training kernels (routing, exchange, embedding table, orthogonalisation).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "mxq.h"
#define MXQ_WATCHED 1
#include "mxq_check.cuh"
#include "mxq_device.cuh"
#include "mxq_host.h"

namespace mxq {

// bf16 values are handled as their bits; widening is exact, rounding is to
// nearest even.
using bf16_t = uint16_t;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// kN elements of T as one access of kN * sizeof(T) bytes (at most 16).
template <typename T, int kN>
struct alignas(sizeof(T) * kN) Vec {
  T v[kN];
};

// Element i of an array of n elements, checked like every computed access: `other`
// where it lies outside, and nothing written there.
template <typename T>
__device__ __forceinline__ bool in_array(const T* a, int64_t i, int64_t n, unsigned int* status) {
  return in_buf(a + i, sizeof(T), a, static_cast<uint64_t>(n) * sizeof(T), status);
}
template <typename T>
__device__ __forceinline__ T read_at(const T* a, int64_t i, int64_t n, T other, unsigned int* status) {
  return in_array(a, i, n, status) ? a[i] : other;
}
template <typename T>
__device__ __forceinline__ void write_at(T* a, int64_t i, int64_t n, T v, unsigned int* status) {
  if (in_array(a, i, n, status)) a[i] = v;
}

// Load of data that this launch does not write, not kept in L1; zero where `wanted`
// is false.  The condition is the load's own predicate: as a branch around each
// load it makes the loads wait for one another.
template <typename T, int kN>
__device__ __forceinline__ Vec<T, kN> load_if(const T* p, bool wanted) {
  Vec<T, kN> v;
  const uint32_t w = wanted ? 1u : 0u;
  if constexpr (sizeof v == 16) {
    uint4 q;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
        : "l"(p), "r"(w));
    *reinterpret_cast<uint4*>(&v) = q;
  } else if constexpr (sizeof v == 8) {
    uint2 q;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];\n\t}"
        : "=&r"(q.x), "=&r"(q.y)
        : "l"(p), "r"(w));
    *reinterpret_cast<uint2*>(&v) = q;
  } else if constexpr (sizeof v == 4) {
    uint32_t q;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.b32 %0, [%1];\n\t}"
        : "=&r"(q)
        : "l"(p), "r"(w));
    *reinterpret_cast<uint32_t*>(&v) = q;
  } else {
    uint16_t q;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.b16 %0, [%1];\n\t}"
        : "=&h"(q)
        : "l"(p), "r"(w));
    *reinterpret_cast<uint16_t*>(&v) = q;
  }
  return v;
}
template <typename T, int kN>
__device__ __forceinline__ Vec<T, kN> load_once(const T* p) {
  return load_if<T, kN>(p, true);
}

// Rows that begin anywhere, written in whole 16-byte units out of shared memory.
// A group of tx threads stages the elements of a row, or of a tile of one, at
// `even` (4-byte aligned), at most kUnits units a thread; where rows can begin at any
// 2 bytes also at `odd`, a second copy's base 2 bytes past a word, so that every unit
// begins at a word of one of them.  A group takes kUnits * 16 * tx bytes and a word.
constexpr int kUnits = 4;

// Writes n staged elements to `row`, by thread `own` of the group's tx; may(address,
// bytes) says whether an access is allowed.
template <typename T, bool kTwo, typename May>
__device__ __forceinline__ void write_staged(const T* even, const T* odd, T* row, int n, int own, int tx, const May& may) {
  constexpr int kSize = static_cast<int>(sizeof(T));
  const int bytes = n * kSize, turn = threadIdx.x >> 3 & 3;
  const int before = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);  // bytes of the first unit before the row
  uint8_t* to = reinterpret_cast<uint8_t*>(row);
  const uint8_t* from = reinterpret_cast<const uint8_t*>(kTwo && (before & 2) != 0 ? odd : even);
  for (int u = own; u < (bytes + before + 15) / 16; u += tx) {
    const int start = 16 * u - before;
    if (start >= 0 && start + 16 <= bytes) {
      // four words, every eight lanes in another order: no two in one bank
      const uint32_t* w = reinterpret_cast<const uint32_t*>(from + start);
      uint32_t a = w[turn], b = w[(1 + turn) & 3], c = w[(2 + turn) & 3], d = w[(3 + turn) & 3];
      if (turn & 1) {
        const uint32_t last = d;
        d = c, c = b, b = a, a = last;
      }
      if (may(to + start, 16)) *reinterpret_cast<uint4*>(to + start) = turn & 2 ? make_uint4(c, d, a, b) : make_uint4(a, b, c, d);
    } else {
      const int end = start + 16 < bytes ? start + 16 : bytes;
      for (int i = start > 0 ? start : 0; i < end; i += kSize)
        if (may(to + i, kSize)) *reinterpret_cast<T*>(to + i) = even[i / kSize];
    }
  }
}

// Threads for a row's units, and a unit less for where it begins; longer rows in
// equal tiles of whole accesses of kV elements.
struct StagedTiles {
  int tx, tiles, tile;  // tile: elements
};
inline StagedTiles staged_tiles(int64_t D, int esize, int kV, int threads) {
  StagedTiles s;
  const int64_t bytes = D * esize;
  s.tx = 8;
  while (s.tx < threads && 16 * kUnits * s.tx - 16 < bytes) s.tx *= 2;
  const int64_t tiles = (bytes + 16 * kUnits * s.tx - 17) / (16 * kUnits * s.tx - 16);
  const int64_t pieces = D / kV;
  s.tiles = static_cast<int>(tiles);
  s.tile = static_cast<int>((pieces + tiles - 1) / tiles * kV);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// 2^x, subnormal results flushed to zero.
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2E = 1.4426950408889634f;

// The widest power of two of bytes, up to 16, that divides every value.
inline int common_alignment(std::initializer_list<uint64_t> values) {
  uint64_t all = 16;
  for (uint64_t v : values) all |= v;
  return static_cast<int>(all & (~all + 1));
}
inline uint64_t address_of(const void* p) { return reinterpret_cast<uintptr_t>(p); }

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes of a [rows, cols] matrix with `ld` elements between its rows.
inline uint64_t pitched_bytes(int64_t rows, int64_t cols, int64_t ld, int esize) {
  return rows > 0 ? (static_cast<uint64_t>(rows - 1) * ld + cols) * esize : 0;
}

inline int element_bytes(int dtype) { return dtype == MXQ_F32 ? 4 : 2; }

// Launch with programmatic stream serialization (see allow_programmatic_launch).
template <typename... Params, typename... Args>
inline int launch_pdl(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                      cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  allow_programmatic_launch(&cfg, &attr);
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) == cudaSuccess ? MXQ_OK : MXQ_ECUDA;
}

// The output ranges must overlap neither one another nor an input; inputs may
// share storage.
inline bool outputs_overlap(const ByteRange* out, int n_out, const ByteRange* in, int n_in) {
  if (ranges_overlap(out, n_out)) return true;
  for (int i = 0; i < n_in; ++i)
    for (int o = 0; o < n_out; ++o) {
      const ByteRange two[2] = {out[o], in[i]};
      if (ranges_overlap(two, 2)) return true;
    }
  return false;
}

inline ByteRange range_of(const void* p, uint64_t bytes) { return {address_of(p), p ? bytes : 0}; }

// Reads (and with `clear` zeroes) a kernel file's status word.
inline int read_status_word(const unsigned int& symbol, unsigned int* out, bool clear) {
  if (cudaMemcpyFromSymbol(out, symbol, sizeof *out) != cudaSuccess) return MXQ_ECUDA;
  const unsigned int zero = 0;
  if (clear && cudaMemcpyToSymbol(symbol, &zero, sizeof zero) != cudaSuccess) return MXQ_ECUDA;
  return MXQ_OK;
}

// Sets the address that this file's checks take as outside (mxq_selftest_watch).
static inline int watch_address(uint64_t address) {
#if MXQ_DEBUG_BOUNDS
  const unsigned long long v = address;
  return cudaMemcpyToSymbol(g_watched, &v, sizeof v) == cudaSuccess ? MXQ_OK : MXQ_ECUDA;
#else
  (void)address;
  return MXQ_OK;
#endif
}

}  // namespace mxq
