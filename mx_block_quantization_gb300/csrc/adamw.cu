// adamw.cu -- an AdamW step over many tensors at once, with moments in 32 bits or in MXFP8.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// One launch takes up to MXQ_ADAMW_TENSORS tensors, whose addresses are the kernel's own
// parameters: nothing is copied to the device first, and a captured call replays.  A block
// takes 4096 elements of one tensor.
//
// Moments in 8 bits are kept as E4M3 with one E8M0 per 32 elements, the cast's format and
// its rule for the scale: m, and the root of v, whose exponents span half of v's.  A step
// changes v by (1 - b2) of it, far less than half a step of E4M3, so rounding to nearest
// would never let it fall; both are rounded at random instead, up with the probability of
// what lies above the value below, so that their mean is the exact value's.  A root that
// is not 0 is never rounded to 0: m over eps would be no step that the gradients ask for.
// The random bits are a mixing of the element's place, the step and the seed (two rounds
// of shift, exclusive or and product with the fractional digits of the roots of 2 and 3),
// 16 of them for each moment: the same call gives the same bits.
//
// m, v and the root are computed with the roundings of the formulas as they stand, one for
// each operation, so that the bytes are a function of the inputs alone.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_adamw_status = 0;

constexpr int kThreads = 256, kV = 4, kAhead = 4;
constexpr int kChunk = kThreads * kV * kAhead;  // elements of a block
constexpr int kScaleBlock = 32, kStartAlign = 128;
constexpr int kFew = 32;                        // tensors of the smaller parameter list

struct Entry {
  void *p, *copy;
  const void* g;
  int64_t n, start;   // elements, and where its moments begin
  int32_t first;      // block of the launch
  uint8_t p_bf16, g_bf16, vector, unused;
};
template <int kTensors>
struct Entries {
  Entry e[kTensors];
};
struct Step {
  void *m, *v;
  uint8_t *ms, *vs;
  int64_t total;       // elements of the moments
  int32_t count;
  float b1, b2, rest1, rest2, log_b1, log_b2, eps, wd, lr, decay;
  const float *lr_at, *grad_scale;
  const int64_t* step_at;
  int64_t step;
  uint32_t seed_low, seed_high;
};

__device__ __forceinline__ uint32_t mixed(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Four elements as floats; `left` of them there, zero for the others.
template <typename T>
__device__ __forceinline__ float4 load_four(const T* p, int left, bool vector, const void* base, uint64_t bytes) {
  float f[kV] = {};
  if (vector && left >= kV) {
    if (in_buf(p, kV * sizeof(T), base, bytes, &g_adamw_status)) {
      const Vec<T, kV> v = *reinterpret_cast<const Vec<T, kV>*>(p);
#pragma unroll
      for (int i = 0; i < kV; ++i) f[i] = widen(v.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (i < left && in_buf(p + i, sizeof(T), base, bytes, &g_adamw_status)) f[i] = widen(p[i]);
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}
template <typename T>
__device__ __forceinline__ void store_four(T* p, const float (&f)[kV], int left, bool vector, const void* base, uint64_t bytes) {
  if (vector && left >= kV) {
    Vec<T, kV> v;
#pragma unroll
    for (int i = 0; i < kV; ++i) v.v[i] = narrow<T>(f[i]);
    if (in_buf(p, sizeof v, base, bytes, &g_adamw_status)) *reinterpret_cast<Vec<T, kV>*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (i < left && in_buf(p + i, sizeof(T), base, bytes, &g_adamw_status)) p[i] = narrow<T>(f[i]);
  }
}

// The values of four E4M3 bytes times the block's power of two, exact.
__device__ __forceinline__ void decode_four(uint32_t bytes, uint32_t scale, float (&f)[kV]) {
  const float s = __uint_as_float(scale == 0u ? 0x00400000u : scale << 23);
#pragma unroll
  for (int i = 0; i < kV; i += 2) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes >> (8 * i))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
    f[i] = fmul_rn_noftz(lo, s);
    f[i + 1] = fmul_rn_noftz(hi, s);
  }
}

// Four values of a block of 32 (eight lanes) to bytes and the block's scale, rounded at
// random by 16 bits each.  A block with a value that is not finite becomes NaN, scale 255.
template <bool kKeep>
__device__ __forceinline__ uint32_t encode_four(const float (&x)[kV], const uint32_t (&random)[kV], int shift, uint32_t& scale) {
  uint32_t most = 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
  if (most >= 0x7F800000u) {
    scale = 255u;
    return 0x7F7F7F7Fu;
  }
  const int e = static_cast<int>(most >> 23) - 8 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  scale = static_cast<uint32_t>(max(e, 0));
  const float up = e8m0_multiplier(scale);
  float q[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const float a = fmul_rn_noftz(fabsf(x[i]), up);
    // 2^-place and 2^place of the last place that E4M3 keeps of a
    const int place = max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -6) - 3;
    const float u = static_cast<float>(random[i] >> shift & 0xFFFFu) * (1.0f / 65536.0f);
    float n = floorf(__fadd_rn(a * __uint_as_float(static_cast<uint32_t>(127 - place) << 23), u));
    if (kKeep) n = a > 0.0f && n < 1.0f ? 1.0f : n;
    q[i] = copysignf(n * __uint_as_float(static_cast<uint32_t>(127 + place) << 23), x[i]);
  }
  return cvt_e4m3x2(q[1], q[0]) | cvt_e4m3x2(q[3], q[2]) << 16;
}

template <int kBits, int kTensors>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Entries<kTensors> list, const __grid_constant__ Step s) {
  pdl_wait();
  int32_t at = 0, most = s.count - 1;  // the last tensor whose first block is not behind this one
  while (at < most) {
    const int32_t mid = (at + most + 1) / 2;
    if (list.e[mid].first <= static_cast<int32_t>(blockIdx.x)) at = mid;
    else most = mid - 1;
  }
  const Entry& t = list.e[at];
  const int64_t base = static_cast<int64_t>(static_cast<int32_t>(blockIdx.x) - t.first) * kChunk;
  const int64_t n = t.n;
  const bool vector = t.vector != 0;
  const uint64_t p_bytes = static_cast<uint64_t>(n) * (t.p_bf16 ? 2 : 4), g_bytes = static_cast<uint64_t>(n) * (t.g_bf16 ? 2 : 4);

  float4 p4[kAhead], g4[kAhead], m4[kAhead], v4[kAhead];
  uint32_t mq[kAhead], vq[kAhead], ms[kAhead], vs[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t i = base + (u * kThreads + threadIdx.x) * kV, at_m = t.start + i;
    const int left = static_cast<int>(min(n - i, static_cast<int64_t>(kV)));
    p4[u] = t.p_bf16 ? load_four(static_cast<const bf16_t*>(t.p) + i, left, vector, t.p, p_bytes)
                     : load_four(static_cast<const float*>(t.p) + i, left, vector, t.p, p_bytes);
    g4[u] = t.g_bf16 ? load_four(static_cast<const bf16_t*>(t.g) + i, left, vector, t.g, g_bytes)
                     : load_four(static_cast<const float*>(t.g) + i, left, vector, t.g, g_bytes);
    if (kBits == 32) {
      m4[u] = load_four(static_cast<const float*>(s.m) + at_m, left, true, s.m, static_cast<uint64_t>(s.total) * 4);
      v4[u] = load_four(static_cast<const float*>(s.v) + at_m, left, true, s.v, static_cast<uint64_t>(s.total) * 4);
    } else {
      mq[u] = vq[u] = ms[u] = vs[u] = 0u;
      if (left > 0) {  // a block of 32 is there in whole
        const uint8_t *m = static_cast<const uint8_t*>(s.m) + at_m, *v = static_cast<const uint8_t*>(s.v) + at_m;
        if (in_buf(m, kV, s.m, s.total, &g_adamw_status)) mq[u] = *reinterpret_cast<const uint32_t*>(m);
        if (in_buf(v, kV, s.v, s.total, &g_adamw_status)) vq[u] = *reinterpret_cast<const uint32_t*>(v);
        ms[u] = read_at(s.ms, at_m / kScaleBlock, s.total / kScaleBlock, uint8_t{0}, &g_adamw_status);
        vs[u] = read_at(s.vs, at_m / kScaleBlock, s.total / kScaleBlock, uint8_t{0}, &g_adamw_status);
      }
    }
  }
  const float gs = s.grad_scale != nullptr ? *s.grad_scale : 1.0f;
  const int64_t step = s.step_at != nullptr ? *s.step_at : s.step;
  const float lr = s.lr_at != nullptr ? *s.lr_at : s.lr;
  const float decay = s.lr_at != nullptr ? fmaf(-lr, s.wd, 1.0f) : s.decay;
  // 1 - b^t, without the cancellation
  const float c1 = -expm1f(static_cast<float>(step) * s.log_b1), c2 = -expm1f(static_cast<float>(step) * s.log_b2);
  const float rate = lr / c1, back = 1.0f / sqrtf(c2);
  const uint32_t key = mixed(mixed(mixed(s.seed_low) ^ s.seed_high) ^ static_cast<uint32_t>(step));
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t i = base + (u * kThreads + threadIdx.x) * kV, at_m = t.start + i;
    const int left = static_cast<int>(min(n - i, static_cast<int64_t>(kV)));
    float p[kV] = {p4[u].x, p4[u].y, p4[u].z, p4[u].w}, g[kV] = {g4[u].x, g4[u].y, g4[u].z, g4[u].w};
    float m[kV], v[kV], root[kV];
    if (kBits == 32) {
      m[0] = m4[u].x, m[1] = m4[u].y, m[2] = m4[u].z, m[3] = m4[u].w;
      v[0] = v4[u].x, v[1] = v4[u].y, v[2] = v4[u].z, v[3] = v4[u].w;
    } else {
      decode_four(mq[u], ms[u], m);
      decode_four(vq[u], vs[u], root);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[j] = __fmul_rn(root[j], root[j]);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const float d = j < left ? __fmul_rn(g[j], gs) : 0.0f;
      m[j] = __fadd_rn(__fmul_rn(s.b1, m[j]), __fmul_rn(s.rest1, d));
      v[j] = __fadd_rn(__fmul_rn(s.b2, v[j]), __fmul_rn(s.rest2, __fmul_rn(d, d)));
      root[j] = sqrtf(v[j]);
      p[j] = p[j] * decay - rate * __fdividef(m[j], fmaf(root[j], back, s.eps));
    }
    if (t.p_bf16)
      store_four(static_cast<bf16_t*>(t.p) + i, p, left, vector, t.p, p_bytes);
    else
      store_four(static_cast<float*>(t.p) + i, p, left, vector, t.p, p_bytes);
    if (t.copy != nullptr) store_four(static_cast<bf16_t*>(t.copy) + i, p, left, vector, t.copy, static_cast<uint64_t>(n) * 2);
    if (kBits == 32) {
      store_four(static_cast<float*>(s.m) + at_m, m, left, true, s.m, static_cast<uint64_t>(s.total) * 4);
      store_four(static_cast<float*>(s.v) + at_m, v, left, true, s.v, static_cast<uint64_t>(s.total) * 4);
    } else {
      uint32_t random[kV], scale_m, scale_v;
      const uint32_t high = static_cast<uint32_t>(at_m >> 32), own = key ^ (high != 0u ? mixed(high) : 0u);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        random[j] = mixed((static_cast<uint32_t>(at_m) + j) ^ own);
        if (j >= left) m[j] = root[j] = 0.0f;
      }
      const uint32_t bytes_m = encode_four<false>(m, random, 0, scale_m);
      const uint32_t bytes_v = encode_four<true>(root, random, 16, scale_v);
      // the last block of 32 is written in whole
      if (i < ceil_div(n, kScaleBlock) * kScaleBlock) {
        uint8_t *to_m = static_cast<uint8_t*>(s.m) + at_m, *to_v = static_cast<uint8_t*>(s.v) + at_m;
        if (in_buf(to_m, kV, s.m, s.total, &g_adamw_status)) *reinterpret_cast<uint32_t*>(to_m) = bytes_m;
        if (in_buf(to_v, kV, s.v, s.total, &g_adamw_status)) *reinterpret_cast<uint32_t*>(to_v) = bytes_v;
        if ((threadIdx.x & 7) == 0) {
          write_at(s.ms, at_m / kScaleBlock, s.total / kScaleBlock, static_cast<uint8_t>(scale_m), &g_adamw_status);
          write_at(s.vs, at_m / kScaleBlock, s.total / kScaleBlock, static_cast<uint8_t>(scale_v), &g_adamw_status);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Marked {
  uintptr_t lo;
  uint64_t bytes;
  bool out;
};
// Whether an output overlaps anything (see ranges_overlap); n log n, as there can be
// thousands of ranges.
bool marked_overlap(Marked* r, int n) {
  int kept = 0;
  for (int i = 0; i < n; ++i)
    if (r[i].lo != 0 && r[i].bytes != 0) {
      if (r[i].lo + r[i].bytes <= r[i].lo) return true;
      r[kept++] = r[i];
    }
  std::sort(r, r + kept, [](const Marked& a, const Marked& b) { return a.lo < b.lo; });
  uintptr_t end_in = 0, end_out = 0;
  for (int i = 0; i < kept; ++i) {
    if (r[i].lo < end_out || (r[i].out && r[i].lo < end_in)) return true;
    uintptr_t& end = r[i].out ? end_out : end_in;
    if (r[i].lo + r[i].bytes > end) end = r[i].lo + r[i].bytes;
  }
  return false;
}

template <int kBits, int kTensors>
int launch_adamw(const mxq_adamw_tensor* tensors, int32_t count, Step s, unsigned blocks, cudaStream_t stream) {
  Entries<kTensors> list;
  int32_t first = 0, used = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mxq_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const bool p16 = t.dtype == MXQ_BF16, g16 = t.grad_dtype == MXQ_BF16;
    const bool vector = aligned_to(t.p, p16 ? 8 : 16) && aligned_to(t.grad, g16 ? 8 : 16) && aligned_to(t.copy, 8);
    list.e[used++] = Entry{t.p, t.copy, t.grad, t.n, t.start, first, p16, g16, vector, 0};
    first += static_cast<int32_t>(ceil_div(t.n, kChunk));
  }
  s.count = used;
  return launch_pdl(adamw_kernel<kBits, kTensors>, blocks, kThreads, 0, stream, list, s);
}

}  // namespace

namespace mxq {
int adamw_status_read(unsigned int* out, bool clear) { return read_status_word(g_adamw_status, out, clear); }
int adamw_watch(uint64_t address) { return watch_address(address); }
}  // namespace mxq

extern "C" int mxq_adamw(const mxq_adamw_tensor* tensors, int32_t count, int32_t bits, void* m, void* v, uint8_t* m_scale,
                         uint8_t* v_scale, int64_t total, int64_t step, const int64_t* step_at, double lr, const float* lr_at,
                         double beta1, double beta2, double eps, double weight_decay, const float* grad_scale, uint64_t seed,
                         cudaStream_t stream) {
  if (bits != 8 && bits != 32) return MXQ_EBADDTYPE;
  if (count < 0 || count > MXQ_ADAMW_TENSORS || total < 0 || total > (int64_t{1} << 44) || total % kStartAlign != 0 ||
      (!step_at && (step < 1 || step > INT32_MAX)) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
      !isfinite(eps) || !isfinite(weight_decay) || (!lr_at && !isfinite(lr)))
    return MXQ_EBADSHAPE;
  if (count == 0) return MXQ_OK;
  if (!tensors) return MXQ_ENULL;
  const int es = bits == 32 ? 4 : 1;
  Marked ranges[4 * MXQ_ADAMW_TENSORS + 6];
  int n = 0;
  int64_t blocks = 0;
  int32_t used = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mxq_adamw_tensor& t = tensors[i];
    if ((t.dtype != MXQ_F32 && t.dtype != MXQ_BF16) || (t.grad_dtype != MXQ_F32 && t.grad_dtype != MXQ_BF16)) return MXQ_EBADDTYPE;
    if (t.n < 0 || t.start < 0 || t.start % kStartAlign != 0 || t.start > total || t.n > total - t.start) return MXQ_EBADSHAPE;
    if (t.n == 0) continue;
    if (!t.p || !t.grad) return MXQ_ENULL;
    const int ps = element_bytes(t.dtype), gs = element_bytes(t.grad_dtype);
    if (!aligned_to(t.p, ps) || !aligned_to(t.grad, gs) || !aligned_to(t.copy, 2)) return MXQ_EALIGN;
    ranges[n++] = {address_of(t.p), static_cast<uint64_t>(t.n) * ps, true};
    ranges[n++] = {address_of(t.copy), static_cast<uint64_t>(t.n) * 2, true};
    ranges[n++] = {address_of(t.grad), static_cast<uint64_t>(t.n) * gs, false};
    ranges[n++] = {m ? address_of(m) + static_cast<uint64_t>(t.start) * es : 0,
                   static_cast<uint64_t>(ceil_div(t.n, kScaleBlock) * kScaleBlock) * es, true};
    blocks += ceil_div(t.n, kChunk);
    ++used;
  }
  if (used == 0) return MXQ_OK;
  if (blocks > INT32_MAX) return MXQ_EBADSHAPE;
  if (!m || !v || (bits == 8 && (!m_scale || !v_scale))) return MXQ_ENULL;
  if (!aligned_to(m, 16) || !aligned_to(v, 16) || !aligned_to(lr_at, 4) || !aligned_to(grad_scale, 4) || !aligned_to(step_at, 8))
    return MXQ_EALIGN;
  ranges[n++] = {address_of(v), static_cast<uint64_t>(total) * es, true};
  ranges[n++] = {bits == 8 ? address_of(m_scale) : 0, static_cast<uint64_t>(total) / kScaleBlock, true};
  ranges[n++] = {bits == 8 ? address_of(v_scale) : 0, static_cast<uint64_t>(total) / kScaleBlock, true};
  ranges[n++] = {address_of(lr_at), 4, false};
  ranges[n++] = {address_of(grad_scale), 4, false};
  ranges[n++] = {address_of(step_at), 8, false};
  if (marked_overlap(ranges, n)) return MXQ_EOVERLAP;
  Step s = {};
  s.m = m, s.v = v, s.ms = m_scale, s.vs = v_scale;
  s.total = total;
  s.b1 = static_cast<float>(beta1), s.b2 = static_cast<float>(beta2);
  s.rest1 = static_cast<float>(1 - beta1), s.rest2 = static_cast<float>(1 - beta2);
  s.log_b1 = static_cast<float>(log(beta1)), s.log_b2 = static_cast<float>(log(beta2));
  s.eps = static_cast<float>(eps), s.wd = static_cast<float>(weight_decay);
  s.lr = static_cast<float>(lr), s.decay = static_cast<float>(1 - lr * weight_decay);
  s.lr_at = lr_at, s.grad_scale = grad_scale, s.step_at = step_at;
  s.step = step;
  s.seed_low = static_cast<uint32_t>(seed), s.seed_high = static_cast<uint32_t>(seed >> 32);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (bits == 32)
    return used <= kFew ? launch_adamw<32, kFew>(tensors, count, s, grid, stream)
                        : launch_adamw<32, MXQ_ADAMW_TENSORS>(tensors, count, s, grid, stream);
  return used <= kFew ? launch_adamw<8, kFew>(tensors, count, s, grid, stream)
                      : launch_adamw<8, MXQ_ADAMW_TENSORS>(tensors, count, s, grid, stream);
}
