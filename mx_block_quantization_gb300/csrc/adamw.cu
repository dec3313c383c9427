// adamw.cu -- an AdamW step over many tensors at once, with moments in 32 bits or in MXFP8.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// One launch takes up to MXQ_ADAMW_TENSORS tensors of one pair of types, whose addresses
// are the kernel's own parameters: nothing is copied to the device first, and a captured
// call replays.  Every block takes a run of chunks of 2048 elements, through the tensors
// that they lie in.  Whole chunks of aligned tensors come by bulk copies into a ring of
// stages in shared memory, so that loads are in flight while the arithmetic runs; with
// loads into registers the 8-bit step took 950 to 1080 us where it takes 811 (loads that
// the registers do not have room for, or that the compiler moves down to their use).
//
// Moments in 8 bits are kept as E4M3 with one E8M0 per 32 elements, the cast's format and
// its rule for the scale: m, and the root of v, whose exponents span half of v's.  A step
// changes v by (1 - b2) of it, far less than half a step of E4M3, so rounding to nearest
// would never let it fall; both are rounded at random instead, up with the probability of
// what lies above the value below, so that the mean of m and of the root is the exact one's.
// v is the root's square, and gains the variance of its roundings: with normal gradients it
// is 2.5% too high on the mean for b2 0.95 and 4.2% for 0.999, single elements 0.2 to 3.6 of
// the exact one.  A root that is not 0 is never rounded to 0, as m over eps would be no step
// that the gradients ask for: elements 2^-17 of their block's largest and below have the
// smallest root of the block, and steps as much smaller as theirs would be.
// The random bits are a mixing of the element's place, the step and the seed (two rounds
// of shift, exclusive or and product with the fractional digits of the roots of 2 and 3),
// 16 of them for each moment: the same call gives the same bits.
//
// m, v and the root are computed with the roundings of the formulas as they stand, one for
// each operation, so that the bytes are a function of the inputs alone (but for a root in
// 2^16, see roots()).  Where rounding does not reach a byte, two values share an
// instruction (f32x2), and a reciprocal is the hardware's, one unit in the last place.
//
// 297M parameters fp32 with bf16 gradients and copies: 1285 us and 6.0 TB/s with moments
// in 32 bits (28 bytes an element, the copy rate would be 1138), bound by DRAM with its
// reads and writes mixed; 811 us and 5.5 TB/s with 8 bits (16.1 bytes an element, 655),
// bound by instruction issue: 78 an element, half of them on the integer pipe, most of them
// for the random bits (10) and the two encodings (22).  A tensor whose addresses are no
// multiples of 16 bytes (the copy's of 8) goes by loads of single elements without the ring:
// 60M parameters 306 to 332 us in place of 265, in 8 bits 306 in place of 167.
#include <cuda_runtime.h>
#include <math.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "train_common.cuh"

namespace {

using namespace mxq;

__device__ unsigned int g_adamw_status = 0;

constexpr int kThreads = 256, kV = 4, kAhead = 2;
constexpr int kChunk = kThreads * kV * kAhead;  // elements that a block takes at a time
// Stages of a block's ring: with two blocks on an SM 160 KB (8 bits) or 192 of its shared
// memory.  (8 bits: 3 blocks of 3 stages 847 us, 2 of 4 811; 32 bits: 3 of 2 1300, 2 of 3
// 1285.)
template <int kBits>
constexpr int kStages = kBits == 32 ? 3 : 4;
constexpr int kBlocksPerSM = 2;
constexpr int kScaleBlock = 32, kStartAlign = 128;
constexpr int kFew = 32;                        // tensors of the smaller parameter list

struct Entry {
  void *p, *copy;
  const void* g;
  int64_t n, start;   // elements, and where its moments begin
  int32_t first;      // chunk of the launch
  int32_t aligned;    // every address to 16 bytes, the copy's to 8
};
template <int kTensors>
struct Entries {
  Entry e[kTensors];
};
struct Step {
  void *m, *v;
  uint8_t *ms, *vs;
  int64_t total;       // elements of the moments
  int32_t count, chunks;
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

// Four elements, `left` of them there and zero for the others, as they are stored; kVector:
// all there, and aligned.
template <typename T, bool kVector>
__device__ __forceinline__ Vec<T, kV> load_four(const T* p, int left, const void* base, uint64_t bytes) {
  Vec<T, kV> v = {};
  if (kVector) {
    if (in_buf(p, sizeof v, base, bytes, &g_adamw_status)) v = *reinterpret_cast<const Vec<T, kV>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (i < left && in_buf(p + i, sizeof(T), base, bytes, &g_adamw_status)) v.v[i] = p[i];
  }
  return v;
}
template <typename T, bool kVector>
__device__ __forceinline__ void store_four(T* p, const float (&f)[kV], int left, const void* base, uint64_t bytes) {
  if (kVector) {
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

// Two fp32 operations in one instruction, rounded to nearest, subnormals kept.  A product
// that goes into a sum may be contracted with it all the same; mul_apart() is for products
// whose rounding counts.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
#define MXQ_PAIR_OP(name, op)                                                                                               \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                                                              \
    float2 r;                                                                                                               \
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t" op                                   \
        ".rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"                                                                  \
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                                   \
    return r;                                                                                                               \
  }
MXQ_PAIR_OP(mul2, "mul")
MXQ_PAIR_OP(add2, "add")
#undef MXQ_PAIR_OP
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 mul_apart(float a, float2 b) { return make_float2(__fmul_rn(a, b.x), __fmul_rn(a, b.y)); }

// Square roots by Newton's iteration, r + (v - r^2) / 2 sqrt(v), from the hardware's
// approximate 1 / sqrt(v): the correction is right to 2^-40, so the sum is rounded as the
// root itself but for one value in 2^16.  v is not below kLeastSquare and at most 2^127.
constexpr float kLeastSquare = 0x1p-100f;
__device__ __forceinline__ float2 roots(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  const float2 r = mul2(v, y), minus = make_float2(-r.x, -r.y);
  return fma2(fma2(minus, r, v), mul2(y, both(0.5f)), r);
}

// max(a, |b|), NaN kept.
__device__ __forceinline__ float max_size(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The values of four E4M3 bytes times the block's power of two, exact.
__device__ __forceinline__ void decode_four(uint32_t bytes, uint32_t scale, float2 (&f)[kV / 2]) {
  const float2 s = both(__uint_as_float(max(scale << 23, 0x00400000u)));  // 2^-127 is a subnormal
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes >> (16 * i))));
    float2 v;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(v.x), "=f"(v.y) : "r"(h));
    f[i] = mul2(v, s);
  }
}

// A size's exponent field, one more where its mantissa is above 1.75: 8 more than the scale
// byte of a block whose largest size it is, which is at least 0.  From kRareField on the
// size may not be finite.
__device__ __forceinline__ uint32_t scale_field(float size) { return (__float_as_uint(size) + 0x1FFFFFu) >> 23; }
constexpr uint32_t kRareField = 255u;

// Four values of a block of 32 (eight lanes) with its scale to bytes, rounded at random by
// 16 bits each.  Adding the random bits below the last place that E4M3 keeps, and cutting
// there, rounds a value that E4M3 holds as a normal number; a zero stays one.
template <bool kKeep>
__device__ __forceinline__ uint32_t encode_four(const float2 (&x)[kV / 2], const uint32_t (&random)[kV], uint32_t scale) {
  const float2 up = both(__uint_as_float((254u << 23) - scale * (1u << 23)));
  float a[kV], q[kV];
  bool small = false;  // some value may be E4M3's subnormal
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) {
    const float2 y = mul2(x[i], up);
    a[2 * i] = y.x, a[2 * i + 1] = y.y;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const uint32_t low = kKeep ? random[i] >> 16 : random[i] & 0xFFFFu;  // of the 20 bits below
    q[i] = __uint_as_float((__float_as_uint(a[i]) + 16u * low) & 0xFFF00000u);
    small |= fabsf(a[i]) < 0x1p-6f;
  }
  if (small)
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (fabsf(a[i]) < 0x1p-6f && a[i] != 0.0f) {  // whole steps of 2^-9
        const uint32_t low = kKeep ? random[i] >> 16 : random[i] & 0xFFFFu;
        float n = floorf(__fadd_rn(fabsf(a[i]) * 512.0f, static_cast<float>(low) * 0x1p-16f));
        if (kKeep && n < 1.0f) n = 1.0f;
        q[i] = copysignf(n * 0x1p-9f, a[i]);
      }
  return cvt_e4m3x2(q[1], q[0]) | cvt_e4m3x2(q[3], q[2]) << 16;
}

// What is the same for all elements of a step.
struct Rates {
  float gs, decay, rate, back;
  uint32_t key;
};

// What a thread has of a chunk, as it is stored.
template <int kBits, typename P, typename G>
struct Chunk {
  Vec<P, kV> p[kAhead];
  Vec<G, kV> g[kAhead];
  Vec<float, kV> m[kBits == 32 ? kAhead : 1], v[kBits == 32 ? kAhead : 1];
  uint32_t mq[kAhead], vq[kAhead], ms[kAhead], vs[kAhead];
};
constexpr int kStep = kThreads * kV;

// The scale bytes of the chunk that begins at `base`, of which `there` elements are there.
template <typename C>
__device__ __forceinline__ void load_scales(C& c, const Entry& t, const Step& s, int64_t base, int there) {
  const int own = static_cast<int>(threadIdx.x) * kV;
  const int64_t at = (t.start + base + own) / kScaleBlock;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    c.ms[u] = c.vs[u] = 0u;
    if (there - own - u * kStep > 0) {
      c.ms[u] = read_at(s.ms, at + u * (kStep / kScaleBlock), s.total / kScaleBlock, uint8_t{0}, &g_adamw_status);
      c.vs[u] = read_at(s.vs, at + u * (kStep / kScaleBlock), s.total / kScaleBlock, uint8_t{0}, &g_adamw_status);
    }
  }
}
// The chunk by loads of each thread: one that ends within it, or that is not aligned.
template <int kBits, typename P, typename G>
__device__ __forceinline__ void load_chunk(Chunk<kBits, P, G>& c, const Entry& t, const Step& s, int64_t base, int there) {
  const int own = static_cast<int>(threadIdx.x) * kV;
  const int64_t at = base + own, at_m = t.start + at;
  const P* const p = static_cast<const P*>(t.p) + at;
  const G* const g = static_cast<const G*>(t.g) + at;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int left = there - own - u * kStep;
    c.p[u] = load_four<P, false>(p + u * kStep, left, t.p, static_cast<uint64_t>(t.n) * sizeof(P));
    c.g[u] = load_four<G, false>(g + u * kStep, left, t.g, static_cast<uint64_t>(t.n) * sizeof(G));
    if constexpr (kBits == 32) {
      c.m[u] = load_four<float, false>(static_cast<const float*>(s.m) + at_m + u * kStep, left, s.m, static_cast<uint64_t>(s.total) * 4);
      c.v[u] = load_four<float, false>(static_cast<const float*>(s.v) + at_m + u * kStep, left, s.v, static_cast<uint64_t>(s.total) * 4);
    } else {
      c.mq[u] = c.vq[u] = 0u;
      if (left > 0) {  // a block of 32 is there in whole
        const uint8_t *m = static_cast<const uint8_t*>(s.m) + at_m + u * kStep, *v = static_cast<const uint8_t*>(s.v) + at_m + u * kStep;
        if (in_buf(m, kV, s.m, s.total, &g_adamw_status)) c.mq[u] = *reinterpret_cast<const uint32_t*>(m);
        if (in_buf(v, kV, s.v, s.total, &g_adamw_status)) c.vq[u] = *reinterpret_cast<const uint32_t*>(v);
      }
    }
  }
  if (kBits == 8) load_scales(c, t, s, base, there);
}

// Whole chunks ahead of the arithmetic: bulk copies into the stages of a ring, issued by
// one thread, each stage with its barrier.
constexpr int kArray = kChunk * 4;  // room for the parameters, and for the gradients
template <int kBits>
constexpr int kMomentBytes = kChunk * (kBits == 32 ? 4 : 1);
template <int kBits>
constexpr int kStageBytes = 2 * kArray + 2 * kMomentBytes<kBits>;
struct Ring {
  uint32_t smem, bars;              // addresses
  volatile uint32_t* abort_flag;
  uint32_t issued, used;            // stages, from the beginning of the launch
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
template <int kBits, typename P, typename G>
__device__ __forceinline__ void issue_chunk(Ring& ring, const Entry& t, const Step& s, int64_t base) {
  if (threadIdx.x == 0) {
    const uint32_t slot = ring.issued % kStages<kBits>, to = ring.smem + slot * kStageBytes<kBits>, bar = ring.bars + 8 * slot;
    constexpr uint32_t kP = kChunk * sizeof(P), kG = kChunk * sizeof(G), kM = kMomentBytes<kBits>;
    const auto load = [&](uint32_t at, const void* src, uint32_t bytes, const void* buf, uint64_t size) {
      if (in_buf(src, bytes, buf, size, &g_adamw_status)) bulk_load(at, src, bytes, bar);
      else mbar_complete_tx(bar, bytes);
    };
    const int64_t at_m = (t.start + base) * (kM / kChunk), all_m = s.total * (kM / kChunk);
    mbar_arrive_expect_tx(bar, kP + kG + 2 * kM);
    load(to, static_cast<const P*>(t.p) + base, kP, t.p, static_cast<uint64_t>(t.n) * sizeof(P));
    load(to + kArray, static_cast<const G*>(t.g) + base, kG, t.g, static_cast<uint64_t>(t.n) * sizeof(G));
    load(to + 2 * kArray, static_cast<const uint8_t*>(s.m) + at_m, kM, s.m, all_m);
    load(to + 2 * kArray + kM, static_cast<const uint8_t*>(s.v) + at_m, kM, s.v, all_m);
  }
  ++ring.issued;
}
template <typename V>
__device__ __forceinline__ V shared_vector(uint32_t at) {
  V v;
  if constexpr (sizeof(V) == 16) {
    *reinterpret_cast<uint4*>(&v) = lds128(at);
  } else if constexpr (sizeof(V) == 8) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(reinterpret_cast<uint2*>(&v)->x), "=r"(reinterpret_cast<uint2*>(&v)->y) : "r"(at));
  } else {
    *reinterpret_cast<uint32_t*>(&v) = lds32(at);
  }
  return v;
}
// This thread's part of the next stage; false where the wait for it ran out.
template <int kBits, typename P, typename G>
__device__ __forceinline__ bool take_chunk(const Ring& ring, Chunk<kBits, P, G>& c) {
  const uint32_t slot = ring.used % kStages<kBits>, round = ring.used / kStages<kBits>;
  if (!mbar_wait_bounded(ring.bars + 8 * slot, round & 1u, ring.abort_flag, &g_adamw_status, MXQ_DEV_TIMEOUT)) return false;
  const uint32_t from = ring.smem + slot * kStageBytes<kBits>, own = threadIdx.x * kV;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    c.p[u] = shared_vector<Vec<P, kV>>(from + (own + u * kStep) * sizeof(P));
    c.g[u] = shared_vector<Vec<G, kV>>(from + kArray + (own + u * kStep) * sizeof(G));
    const uint32_t m = from + 2 * kArray + (own + u * kStep) * (kMomentBytes<kBits> / kChunk);
    if constexpr (kBits == 32) {
      c.m[u] = shared_vector<Vec<float, kV>>(m);
      c.v[u] = shared_vector<Vec<float, kV>>(m + kMomentBytes<kBits>);
    } else {
      c.mq[u] = lds32(m);
      c.vq[u] = lds32(m + kMomentBytes<kBits>);
    }
  }
  return true;
}

// kWhole: all of the chunk's elements are there, and aligned.
template <int kBits, typename P, typename G, bool kWhole>
__device__ __forceinline__ void step_chunk(const Chunk<kBits, P, G>& c, const Entry& t, const Step& s, const Rates& r, int64_t base,
                                           int there) {
  const int own = static_cast<int>(threadIdx.x) * kV;
  const int64_t at = base + own, at_m = t.start + at, at_s = at_m / kScaleBlock;
  P* const p_at = static_cast<P*>(t.p) + at;
  const uint64_t p_bytes = static_cast<uint64_t>(t.n) * sizeof(P);
  float *const m32 = static_cast<float*>(s.m) + at_m, *const v32 = static_cast<float*>(s.v) + at_m;
  uint8_t *const m8 = static_cast<uint8_t*>(s.m) + at_m, *const v8 = static_cast<uint8_t*>(s.v) + at_m;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int left = there - own - u * kStep;
    float2 m[kV / 2], v[kV / 2], root[kV / 2];
    if constexpr (kBits == 32) {
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) {
        m[j] = make_float2(c.m[u].v[2 * j], c.m[u].v[2 * j + 1]);
        v[j] = make_float2(c.v[u].v[2 * j], c.v[u].v[2 * j + 1]);
      }
    } else {
      decode_four(c.mq[u], c.ms[u], m);
      decode_four(c.vq[u], c.vs[u], root);
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) v[j] = mul2(root[j], root[j]);
    }
#pragma unroll
    for (int j = 0; j < kV / 2; ++j) {
      const float2 d = mul2(make_float2(widen(c.g[u].v[2 * j]), widen(c.g[u].v[2 * j + 1])), both(r.gs));
      m[j] = add2(mul_apart(s.b1, m[j]), mul_apart(s.rest1, d));
      v[j] = add2(mul_apart(s.b2, v[j]), mul_apart(s.rest2, mul2(d, d)));
      root[j] = roots(v[j]);
    }
    const float least = fminf(fminf(v[0].x, v[0].y), fminf(v[1].x, v[1].y));
    if (!(least >= kLeastSquare && max_size(max_size(v[0].x, v[0].y), max_size(v[1].x, v[1].y)) <= 0x1p127f))  // out of its range
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) root[j] = make_float2(sqrtf(v[j].x), sqrtf(v[j].y));
    float p[kV];
#pragma unroll
    for (int j = 0; j < kV / 2; ++j) {
      const float2 denom = fma2(root[j], both(r.back), both(s.eps));
      const float2 update = mul2(m[j], make_float2(reciprocal(denom.x), reciprocal(denom.y)));
      const float2 old = mul2(make_float2(widen(c.p[u].v[2 * j]), widen(c.p[u].v[2 * j + 1])), both(r.decay));
      const float2 now = fma2(update, both(-r.rate), old);
      p[2 * j] = now.x, p[2 * j + 1] = now.y;
    }
    store_four<P, kWhole>(p_at + u * kStep, p, left, t.p, p_bytes);
    if (t.copy != nullptr)
      store_four<bf16_t, kWhole>(static_cast<bf16_t*>(t.copy) + at + u * kStep, p, left, t.copy, static_cast<uint64_t>(t.n) * 2);
    if (kBits == 32) {
      const float flat_m[kV] = {m[0].x, m[0].y, m[1].x, m[1].y}, flat_v[kV] = {v[0].x, v[0].y, v[1].x, v[1].y};
      store_four<float, kWhole>(m32 + u * kStep, flat_m, left, s.m, static_cast<uint64_t>(s.total) * 4);
      store_four<float, kWhole>(v32 + u * kStep, flat_v, left, s.v, static_cast<uint64_t>(s.total) * 4);
    } else {
      // four places from a multiple of four on share their high part
      const int64_t place = at_m + u * kStep;
      const uint32_t high = static_cast<uint32_t>(place >> 32), key = r.key ^ (high != 0u ? mixed(high) : 0u);
      uint32_t random[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) random[j] = mixed((static_cast<uint32_t>(place) + j) ^ key);
      if (!kWhole && left < kV)
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (j >= left) (j & 1 ? m[j / 2].y : m[j / 2].x) = (j & 1 ? root[j / 2].y : root[j / 2].x) = 0.0f;
      // both fields at once, as halves of a word
      uint32_t fields = scale_field(max_size(max_size(fabsf(m[0].x), m[0].y), max_size(fabsf(m[1].x), m[1].y))) |
                        scale_field(max_size(max_size(root[0].x, root[0].y), max_size(root[1].x, root[1].y))) << 16;
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) fields = __vmaxu2(fields, __shfl_xor_sync(0xFFFFFFFFu, fields, d));
      uint32_t scale_m = max(fields & 0xFFFFu, 8u) - 8u, scale_v = max(fields >> 16, 8u) - 8u;
      uint32_t bytes_m = encode_four<false>(m, random, scale_m), bytes_v = encode_four<true>(root, random, scale_v);
      // a block with a value that is not finite becomes NaN
      const bool rare = max(fields & 0xFFFFu, fields >> 16) >= kRareField;
      if (__any_sync(0xFFFFFFFFu, rare)) {
        const float all_m = max_size(max_size(fabsf(m[0].x), m[0].y), max_size(fabsf(m[1].x), m[1].y));
        const float all_v = max_size(max_size(root[0].x, root[0].y), max_size(root[1].x, root[1].y));
        const uint32_t group = 0xFFu << (threadIdx.x & 24u);
        if (__ballot_sync(0xFFFFFFFFu, !(all_m < CUDART_INF_F)) & group) scale_m = 255u, bytes_m = 0x7F7F7F7Fu;
        if (__ballot_sync(0xFFFFFFFFu, !(all_v < CUDART_INF_F)) & group) scale_v = 255u, bytes_v = 0x7F7F7F7Fu;
      }
      // the last block of 32 is written in whole
      if (kWhole || own + u * kStep < (there + kScaleBlock - 1) / kScaleBlock * kScaleBlock) {
        if (in_buf(m8 + u * kStep, kV, s.m, s.total, &g_adamw_status)) *reinterpret_cast<uint32_t*>(m8 + u * kStep) = bytes_m;
        if (in_buf(v8 + u * kStep, kV, s.v, s.total, &g_adamw_status)) *reinterpret_cast<uint32_t*>(v8 + u * kStep) = bytes_v;
        if ((threadIdx.x & 7) == 0) {
          write_at(s.ms, at_s + u * (kStep / kScaleBlock), s.total / kScaleBlock, static_cast<uint8_t>(scale_m), &g_adamw_status);
          write_at(s.vs, at_s + u * (kStep / kScaleBlock), s.total / kScaleBlock, static_cast<uint8_t>(scale_v), &g_adamw_status);
        }
      }
    }
  }
}

// Chunks [from, to) of one tensor; false where a wait ran out.
template <int kBits, typename P, typename G>
__device__ __forceinline__ bool step_tensor(Ring& ring, const Entry& t, const Step& s, const Rates& r, int32_t from, int32_t to) {
  Chunk<kBits, P, G> c;
  if (t.aligned) {
    const int32_t whole = static_cast<int32_t>(min(static_cast<int64_t>(to), t.n / kChunk));
    int32_t next = from;
    for (; next < whole && next < from + kStages<kBits>; ++next) issue_chunk<kBits, P, G>(ring, t, s, static_cast<int64_t>(next) * kChunk);
    Chunk<8, bf16_t, bf16_t> ahead;  // its scales alone
    if (kBits == 8 && from < whole) load_scales(ahead, t, s, static_cast<int64_t>(from) * kChunk, kChunk);
    for (; from < whole; ++from) {
      const bool ok = take_chunk<kBits, P, G>(ring, c);
      if (kBits == 8)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) c.ms[u] = ahead.ms[u], c.vs[u] = ahead.vs[u];
      if (!__syncthreads_and(ok)) return false;  // and all have taken their part
      ++ring.used;
      if (next < whole) issue_chunk<kBits, P, G>(ring, t, s, static_cast<int64_t>(next++) * kChunk);
      if (kBits == 8 && from + 1 < whole) load_scales(ahead, t, s, static_cast<int64_t>(from + 1) * kChunk, kChunk);
      step_chunk<kBits, P, G, true>(c, t, s, r, static_cast<int64_t>(from) * kChunk, kChunk);
    }
  }
  for (; from < to; ++from) {
    const int64_t base = static_cast<int64_t>(from) * kChunk;
    const int there = static_cast<int>(min(t.n - base, static_cast<int64_t>(kChunk)));
    load_chunk<kBits, P, G>(c, t, s, base, there);
    step_chunk<kBits, P, G, false>(c, t, s, r, base, there);
  }
  return true;
}

// A block takes a run of chunks, and the tensors that they lie in one after another.
template <int kBits, typename P, typename G, int kTensors>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM)
    adamw_kernel(const __grid_constant__ Entries<kTensors> list, const __grid_constant__ Step s) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kStages<kBits>];
  __shared__ uint32_t abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages<kBits>; ++i) mbar_init(smem_u32(&bars[i]), 1);
    abort_flag = 0u;
    mbar_init_fence();
  }
  __syncthreads();
  Ring ring = {smem_u32(smem), smem_u32(bars), &abort_flag, 0u, 0u};
  const int32_t begin = static_cast<int32_t>(static_cast<int64_t>(s.chunks) * blockIdx.x / gridDim.x);
  const int32_t end = static_cast<int32_t>(static_cast<int64_t>(s.chunks) * (blockIdx.x + 1) / gridDim.x);
  int32_t at = 0, most = s.count - 1;  // the last tensor whose first chunk is not behind this block's
  while (at < most) {
    const int32_t mid = (at + most + 1) / 2;
    if (list.e[mid].first <= begin) at = mid;
    else most = mid - 1;
  }
  pdl_wait();
  Rates r;
  r.gs = s.grad_scale != nullptr ? *s.grad_scale : 1.0f;
  r.decay = s.decay;
  float lr = s.lr;
  if (s.lr_at != nullptr) {
    lr = *s.lr_at;
    r.decay = fmaf(-lr, s.wd, 1.0f);
  }
  // 1 - b^t without the cancellation, here for either t: the same bits
  const int64_t step = s.step_at != nullptr ? *s.step_at : s.step;
  r.rate = lr / -expm1f(static_cast<float>(step) * s.log_b1);
  r.back = 1.0f / sqrtf(-expm1f(static_cast<float>(step) * s.log_b2));
  r.key = mixed(mixed(mixed(s.seed_low) ^ s.seed_high) ^ static_cast<uint32_t>(step));
  bool ok = true;
  for (int32_t chunk = begin; ok && chunk < end; ++at) {
    const Entry& t = list.e[at];
    const int32_t stop = at + 1 < s.count ? min(end, list.e[at + 1].first) : end, from = chunk - t.first, to = stop - t.first;
    chunk = stop;
    ok = step_tensor<kBits, P, G>(ring, t, s, r, from, to);
  }
  if (!ok && threadIdx.x == 0)  // copies in flight end before the block's memory is given away
    for (uint32_t n = ring.used; n < ring.issued; ++n)
      mbar_wait_drain(ring.bars + 8 * (n % kStages<kBits>), n / kStages<kBits> & 1u);
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

// The tensors of one pair of types, a launch of their own.
template <int kBits, typename P, typename G, int kTensors>
int launch_tensors(const mxq_adamw_tensor* tensors, int32_t count, Step s, int sms, cudaStream_t stream) {
  Entries<kTensors> list;
  int32_t first = 0, used = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mxq_adamw_tensor& t = tensors[i];
    if (t.n == 0 || element_bytes(t.dtype) != sizeof(P) || element_bytes(t.grad_dtype) != sizeof(G)) continue;
    const bool aligned = aligned_to(t.p, 16) && aligned_to(t.grad, 16) && aligned_to(t.copy, 8);
    list.e[used++] = Entry{t.p, t.copy, t.grad, t.n, t.start, first, aligned};
    first += static_cast<int32_t>(ceil_div(t.n, kChunk));
  }
  s.count = used;
  s.chunks = first;
  const auto kernel = adamw_kernel<kBits, P, G, kTensors>;
  constexpr int kSmem = kStages<kBits> * kStageBytes<kBits>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ECUDA;
  static bool attr_done[64] = {};  // benign race: the same attribute set twice
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MXQ_ECUDA;
    attr_done[dev] = true;
  }
  const int most = sms * kBlocksPerSM;
  return launch_pdl(kernel, static_cast<unsigned>(s.chunks < most ? s.chunks : most), kThreads, kSmem, stream, list, s);
}

template <int kBits, typename P, typename G>
int launch_pair(const mxq_adamw_tensor* tensors, int32_t count, const Step& s, int sms, cudaStream_t stream) {
  int32_t used = 0;
  for (int32_t i = 0; i < count; ++i)
    used += tensors[i].n > 0 && element_bytes(tensors[i].dtype) == sizeof(P) && element_bytes(tensors[i].grad_dtype) == sizeof(G);
  if (used == 0) return MXQ_OK;
  return used <= kFew ? launch_tensors<kBits, P, G, kFew>(tensors, count, s, sms, stream)
                      : launch_tensors<kBits, P, G, MXQ_ADAMW_TENSORS>(tensors, count, s, sms, stream);
}
template <int kBits>
int launch_adamw(const mxq_adamw_tensor* tensors, int32_t count, const Step& s, int sms, cudaStream_t stream) {
  for (const auto launch : {launch_pair<kBits, float, float>, launch_pair<kBits, float, bf16_t>, launch_pair<kBits, bf16_t, float>,
                            launch_pair<kBits, bf16_t, bf16_t>}) {
    const int rc = launch(tensors, count, s, sms, stream);
    if (rc != MXQ_OK) return rc;
  }
  return MXQ_OK;
}

// The buffers of a list of tensors: their types, sizes, places and overlaps.  `ranges` holds
// 4 count + 6.  *used: tensors with elements.
int check_buffers(const mxq_adamw_tensor* tensors, int32_t count, int32_t bits, const void* m, const void* v, const uint8_t* m_scale,
                  const uint8_t* v_scale, int64_t total, const int64_t* step_at, const float* lr_at, const float* grad_scale, Marked* ranges,
                  int32_t* used) {
  const int es = bits == 32 ? 4 : 1;
  int n = 0;
  *used = 0;
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
    ++*used;
  }
  if (*used == 0) return MXQ_OK;
  if (!m || !v || (bits == 8 && (!m_scale || !v_scale))) return MXQ_ENULL;
  if (!aligned_to(m, 16) || !aligned_to(v, 16) || !aligned_to(lr_at, 4) || !aligned_to(grad_scale, 4) || !aligned_to(step_at, 8))
    return MXQ_EALIGN;
  ranges[n++] = {address_of(v), static_cast<uint64_t>(total) * es, true};
  ranges[n++] = {bits == 8 ? address_of(m_scale) : 0, static_cast<uint64_t>(total) / kScaleBlock, true};
  ranges[n++] = {bits == 8 ? address_of(v_scale) : 0, static_cast<uint64_t>(total) / kScaleBlock, true};
  ranges[n++] = {address_of(lr_at), 4, false};
  ranges[n++] = {address_of(grad_scale), 4, false};
  ranges[n++] = {address_of(step_at), 8, false};
  return marked_overlap(ranges, n) ? MXQ_EOVERLAP : MXQ_OK;
}
bool total_ok(int64_t total) { return total >= 0 && total <= (int64_t{1} << 44) && total % kStartAlign == 0; }

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
  if (count < 0 || count > MXQ_ADAMW_TENSORS || !total_ok(total) || (!step_at && (step < 1 || step > INT32_MAX)) ||
      !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || !isfinite(eps) || !isfinite(weight_decay) ||
      (!lr_at && !isfinite(lr)))
    return MXQ_EBADSHAPE;
  if (count == 0) return MXQ_OK;
  if (!tensors) return MXQ_ENULL;
  Marked ranges[4 * MXQ_ADAMW_TENSORS + 6];
  int32_t used = 0;
  const int rc = check_buffers(tensors, count, bits, m, v, m_scale, v_scale, total, step_at, lr_at, grad_scale, ranges, &used);
  if (rc != MXQ_OK || used == 0) return rc;
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) chunks += ceil_div(tensors[i].n, kChunk);
  if (chunks > INT32_MAX) return MXQ_EBADSHAPE;
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
  const int sms = sm_count_current_device(nullptr);
  if (sms <= 0) return MXQ_ECUDA;
  return bits == 32 ? launch_adamw<32>(tensors, count, s, sms, stream) : launch_adamw<8>(tensors, count, s, sms, stream);
}

extern "C" int mxq_adamw_check(const mxq_adamw_tensor* tensors, int64_t count, int32_t bits, const void* m, const void* v,
                               const uint8_t* m_scale, const uint8_t* v_scale, int64_t total, const int64_t* step_at, const float* lr_at,
                               const float* grad_scale) {
  if (bits != 8 && bits != 32) return MXQ_EBADDTYPE;
  if (count < 0 || count > (1 << 24) || !total_ok(total)) return MXQ_EBADSHAPE;
  if (count == 0) return MXQ_OK;
  if (!tensors) return MXQ_ENULL;
  const std::unique_ptr<Marked[]> ranges(new (std::nothrow) Marked[4 * count + 6]);
  if (!ranges) return MXQ_EBADSHAPE;
  int32_t used = 0;
  return check_buffers(tensors, static_cast<int32_t>(count), bits, m, v, m_scale, v_scale, total, step_at, lr_at, grad_scale, ranges.get(),
                       &used);
}
