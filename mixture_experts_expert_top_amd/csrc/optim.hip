// The step that uses the gradients: their global norm, and AdamW over many
// tensors in one launch.
//
//   norm = sqrt(sum over all tensors of g^2)
//   g' = g min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr wd p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Both kernels are bound by memory: a value's gradient, parameter and moments
// are read once and the parameter and moments written once.  The table of
// tensors travels in the kernel's arguments (kTensors a launch), so a call
// copies nothing to the device and can be captured.
//
// 8-bit moments.  m and r = sqrt(v) are held as E4M3 codes with an fp32 scale
// for each 256 values (the block's largest magnitude stands at 256, so nothing
// reaches the format's end).  Rounding to nearest would hold a moment that
// moves by less than half a code a step where it is for good (sqrt(v) falls by
// 0.05% a step at b2 = 0.999, a code is 6 to 12%), so before a value is cut a
// fraction of the last bit that it keeps is added, which depends on the step
// alone (multiples of the golden ratio modulo 1): over the steps the cuts of a
// value average out, and no random numbers are read.  All values of a step get
// the same fraction, so equal values move together and a tensor's mean moves
// with them (in the oracle, 2048 log-normal values of r at b2 = 0.999: after
// 3000 steps without gradients, beside live values, 0.88 to 0.98 of the true
// mean by the step they start from; with steady gradients 0.94 to 1.08).
// r is held rather than v because it spans half the exponents: 2^17 from the
// scale's top to the smallest code, which is also the least that a second
// moment above zero is held as, so that it never divides as zero.

#include "optim.h"

#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

// every fp32 operation of the moments is rounded by itself, so that codes and
// scales are defined to the bit
#pragma clang fp contract(off)

constexpr int kThreads = 256;
// A thread takes kVec values in runs of R: all of them in a row (R = 8, for
// tensors of one and two bytes a value: 8- and 16-byte accesses), or two runs
// of four, kStateBlock apart (R = 4, for fp32), so that a wave's access is
// always a run of whole cache lines.  Every value is touched once, so the
// accesses are non-temporal.  With 554 M values (bf16 parameters and
// gradients): fp32 moments and copies 2814 us with R = 4, 3094 with R = 8, and
// 2915 with R = 8 and ordinary accesses; 8-bit moments 1605, 1329 and 1398.
constexpr int kVec = 8;
constexpr int kChunk = kThreads * kVec;         // values a workgroup and pass
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;
// Passes a workgroup of the 8-bit form, which the vector units bound (74
// instructions a value with one pass, 60 with eight: what all values share,
// the corrections' exponentials among it, is computed once a workgroup): as
// many as leave the CUs 16 rounds of workgroups, up to eight.  554 M values
// 1420 -> 1208 us with the norm; 45 M, where eight passes would leave 11
// workgroups a CU, 143 us with one and 163 with eight.  The fp32 form is bound
// by memory and stays at one (2820 us for 2986).
constexpr int kMostPasses = 8;
constexpr int64_t kRoundsChunks = int64_t{16} * 256 * 8;

// first value of the thread in its chunk
template <int R>
__device__ __forceinline__ int thread_first() {
  static_assert(R == 8 || R == 4, "runs");
  return R == 8 ? threadIdx.x * 8
                : (threadIdx.x >> 6) * (2 * kStateBlock) +
                      (threadIdx.x & 63) * 4;
}

template <typename V>
__device__ __forceinline__ V load_nt(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
}
template <typename V>
__device__ __forceinline__ void store_nt(void* p, V v) {
  __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
}

template <int R>
__device__ __forceinline__ void load_run(const float* p, float* v) {
#pragma unroll
  for (int h = 0; h < R / 4; ++h) {
    const f32x4 a = load_nt<f32x4>(p + 4 * h);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * h + i] = a[i];
  }
}
template <int R>
__device__ __forceinline__ void store_run(float* p, const float* v) {
#pragma unroll
  for (int h = 0; h < R / 4; ++h)
    store_nt(p + 4 * h, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2],
                              v[4 * h + 3]});
}
template <int R>
__device__ __forceinline__ void load_run(const bf16_t* p, float* v) {
  typedef int vec __attribute__((ext_vector_type(R / 2)));
  const vec r = load_nt<vec>(p);
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    v[2 * i] = bf_lo(static_cast<uint32_t>(r[i]));
    v[2 * i + 1] = bf_hi(static_cast<uint32_t>(r[i]));
  }
}
template <int R>
__device__ __forceinline__ void store_run(bf16_t* p, const float* v) {
  typedef int vec __attribute__((ext_vector_type(R / 2)));
  vec o;
#pragma unroll
  for (int i = 0; i < R / 2; ++i)
    o[i] = static_cast<int>(pack_bf16x2(v[2 * i], v[2 * i + 1]));
  store_nt(p, o);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t* p) { return bf2f(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { *p = f2bf(v); }

// A thread's values from p on; with `left` values from p to the tensor's end
// those past it are zero, and not stored.
template <int R, typename T>
__device__ __forceinline__ void load_some(const T* p, int64_t left, float* v) {
#pragma unroll
  for (int h = 0; h < kVec / R; ++h) {
    const T* const q = p + h * kStateBlock;
    const int64_t l = left - h * kStateBlock;
    if (l >= R) {
      load_run<R>(q, v + R * h);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) v[R * h + i] = i < l ? load1(q + i) : 0.0f;
    }
  }
}
template <int R, typename T>
__device__ __forceinline__ void store_some(T* p, int64_t left,
                                           const float* v) {
#pragma unroll
  for (int h = 0; h < kVec / R; ++h) {
    T* const q = p + h * kStateBlock;
    const int64_t l = left - h * kStateBlock;
    if (l >= R) {
      store_run<R>(q, v + R * h);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < l) store1(q + i, v[R * h + i]);
    }
  }
}

// The last entry of first[0 .. count) that is not above `chunk`.
__device__ __forceinline__ int find_tensor(const uint32_t* first, int count,
                                           uint32_t chunk) {
  int lo = 0, n = count;
  while (n > 1) {
    const int half = n >> 1;
    if (first[lo + half] <= chunk) lo += half;
    n -= half;
  }
  return lo;
}

// ------------------------------------------------------------------- norm
// fp64 sums of squares: the vector units add doubles at the rate of floats,
// and the clip factor then depends on no order of summation.
constexpr int kNormTensors = 160;
constexpr int kNormGroups = 1024;
constexpr int kNormBytes = kThreads * 32;       // a chunk: 32 bytes a thread
constexpr int kNormAhead = 2;                   // chunks in flight
// Gradients of more than the memory-side cache holds are read as non-temporal
// (64 experts of 2048 x 1408, 1.1 GB: 181 -> 173 us); smaller ones are left
// where the step that follows finds them (three blocks of 7 experts of 1032 x
// 680, norm and step 142 us, and 149 with the mark).
constexpr int64_t kNormCached = int64_t{256} << 20;

struct NormTable {
  const void* g[kNormTensors];
  int64_t bytes[kNormTensors];
  uint32_t first[kNormTensors];       // first chunk
  uint8_t fp32[kNormTensors];
  int count;
  uint32_t chunks;
  int add;                            // to what an earlier launch left
};

// The sum over a wave's lanes, in a fixed order, in every lane.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

__device__ __forceinline__ double square_add(float v, double s) {
  const double x = v;
  return fma(x, x, s);
}

// Chunks are counted in bytes, so that what is in flight does not depend on a
// tensor's type; a resource that ends with the tensor zeroes what lies past
// it.
template <bool NT>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(
    NormTable P, double* __restrict__ part) {
  __shared__ double red[kThreads / kWave];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < P.chunks; c += kNormAhead * gridDim.x) {
    i32x4 raw[kNormAhead][2];
    bool fp32[kNormAhead];
#pragma unroll
    for (int u = 0; u < kNormAhead; ++u) {
      const uint32_t cu = c + u * gridDim.x;
      const bool in = cu < P.chunks;
      const int i = in ? find_tensor(P.first, P.count, cu) : 0;
      const int64_t at =
          in ? static_cast<int64_t>(cu - P.first[i]) * kNormBytes : 0;
      const int64_t left = in ? P.bytes[i] - at : 0;
      const uint32_t bytes =
          left < kNormBytes ? static_cast<uint32_t>(left) : kNormBytes;
      // an odd number of bf16 values: the last one's word is read whole and
      // its upper half cleared
      const auto rs = make_rsrc(static_cast<const char*>(P.g[i]) + at,
                                (bytes + 3) & ~3u);
      fp32[u] = P.fp32[i] != 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t off = (h * kThreads + threadIdx.x) * 16;
        constexpr int kNonTemporal = 2;
        raw[u][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rs, off, 0, NT ? kNonTemporal : 0);
        if (bytes & 2)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (off + q * 4 + 2 == bytes) raw[u][h][q] &= 0xffff;
      }
    }
#pragma unroll
    for (int u = 0; u < kNormAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t w = static_cast<uint32_t>(raw[u][h][q]);
          if (fp32[u]) {
            s = square_add(__uint_as_float(w), s);
          } else {
            s = square_add(bf_lo(w), s);
            s = square_add(bf_hi(w), s);
          }
        }
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = P.add ? part[blockIdx.x] : 0.0;
    for (int w = 0; w < kThreads / kWave; ++w) s += red[w];
    part[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(kThreads) void grad_norm_finish_kernel(
    const double* __restrict__ part, int count, float* __restrict__ norm) {
  __shared__ double red[kThreads / kWave];
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s += part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < kThreads / kWave; ++w) s += red[w];
    norm[0] = static_cast<float>(sqrt(s));
  }
}

// ------------------------------------------------------------------ AdamW
constexpr int kTensors = 48;

struct AdamwTable {
  void* p[kTensors];
  float* master[kTensors];
  const void* g[kTensors];
  void* m[kTensors];
  void* v[kTensors];
  float* ms[kTensors];
  float* vs[kTensors];
  int64_t n[kTensors];
  uint32_t first[kTensors];           // first chunk
  float decay[kTensors];
  uint8_t p_fp32[kTensors], g_fp32[kTensors];
  int count;
  int passes;
  AdamwHyper h;
};
static_assert(sizeof(AdamwTable) <= 4096, "kernel arguments");
static_assert(sizeof(NormTable) <= 4096, "kernel arguments");

// What every value of a step shares.
struct Shared {
  float b1, c1, b2, c2, coef, size, root, eps, lr;
  uint32_t dither;
  bool clip;
};

// 1 - b^t, to about an ulp for every t (t log b is rounded once, and expm1
// keeps its relative precision)
__device__ __forceinline__ float one_minus_power(double log_b, int64_t t) {
  return -expm1f(static_cast<float>(static_cast<double>(t) * log_b));
}

// Eight E4M3 codes, and their values.  With `left` codes from p to the
// tensor's end those past it are zero, and not stored.
static_assert(kVec == 8, "codes are read and written in eights");
__device__ __forceinline__ i32x2 load_codes(const uint8_t* p, int64_t left) {
  if (left >= kVec) return load_nt<i32x2>(p);
  i32x2 c = {};
#pragma unroll
  for (int q = 0; q < kVec; ++q)
    if (q < left) c[q / 4] |= p[q] << (q % 4 * 8);
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left,
                                            i32x2 c) {
  if (left >= kVec) {
    store_nt(p, c);
  } else {
#pragma unroll
    for (int q = 0; q < kVec; ++q)
      if (q < left) p[q] = static_cast<uint8_t>(c[q / 4] >> (q % 4 * 8));
  }
}
__device__ __forceinline__ void decode(i32x2 c, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
}
template <typename F>
__device__ __forceinline__ i32x2 encode(F value) {
  i32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(value(4 * i),
                                                  value(4 * i + 1), 0, false);
    c[i] = __builtin_amdgcn_cvt_pk_fp8_f32(value(4 * i + 2), value(4 * i + 3),
                                           w, true);
  }
  return c;
}

// A moment, cut to four significant bits: `y` in units of the block's scale.
__device__ __forceinline__ float cut(float y, uint32_t dither) {
  return __uint_as_float((__float_as_uint(y) + dither) & ~0xfffffu);
}

// The codes of values y over their block's scale; old: those that they had.
// Below 2^-6 codes are 2^-9 apart, more than the unit of four significant bits.
// Where the nearest of them is the one that the value has, it would stay for
// good: there the fraction is added to the distance between codes, which from
// 2^-6 to 2^-5 is that of the four bits, so the value is moved there and back.
// Elsewhere the nearest code is taken, whose error is half as large.
__device__ __forceinline__ i32x2 new_codes(const float* y, i32x2 old,
                                           uint32_t dither) {
  const i32x2 c = encode([&](int q) { return cut(y[q], dither); });
  // a zero byte: a code below 2^-5 that is the old one
  uint32_t held = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = static_cast<uint32_t>((c[i] ^ old[i]) |
                                             (c[i] & 0x70707070));
    held |= (v - 0x01010101u) & ~v;
  }
  if (!__any(held & 0x80808080u)) return c;
  return encode([&](int q) {
    const bool same = (((c[q / 4] ^ old[q / 4]) >> (q % 4 * 8)) & 0xff) == 0;
    const float low = copysignf(0x1p-6f, y[q]);
    return same && fabsf(y[q]) < 0x1p-6f ? cut(y[q] + low, dither) - low
                                         : cut(y[q], dither);
  });
}

// The correctly rounded root of x >= 2^-96, by the last step of Newton's
// method on a root and half its reciprocal (each good to about an ulp) with
// the residual x - s^2 exact: five instructions where the library's root for
// every float takes 14 (60 instructions a value for 71; 554 M values with the
// norm 1208 us for 1249).
__device__ __forceinline__ float root(float x) {
  const float y = __builtin_amdgcn_rsqf(x);
  const float s = x * y;
  return fmaf(fmaf(-s, s, x), 0.5f * y, s);
}

// The largest of 32 lanes' values, in each of them.
__device__ __forceinline__ float max32(float v) {
  v = dpp_group_max<16>(v);
  return fmaxf(v, shfl_xor(v, 16));
}

// A thread's values of one tensor, from `at` on.  kBits8: 32 lanes hold a
// block, and lanes past the tensor's end hold zeros.
template <bool kBits8, typename TP, bool kMaster, typename TG>
__device__ __forceinline__ void update(const AdamwTable& P, int i, int64_t at,
                                       const Shared& S) {
  constexpr int R = kBits8 ? 8 : 4;
  at += thread_first<R>();
  const int64_t left = P.n[i] - at;
  if (!kBits8 && left <= 0) return;
  TP* const p = static_cast<TP*>(P.p[i]) + at;
  float* const master = P.master[i] + at;
  float g[kVec], x[kVec], m[kVec], r[kVec];
  load_some<R>(static_cast<const TG*>(P.g[i]) + at, left, g);
  if constexpr (kMaster)
    load_some<R>(master, left, x);
  else
    load_some<R>(p, left, x);
  using TS = typename std::conditional<kBits8, uint8_t, float>::type;
  TS* const pm = static_cast<TS*>(P.m[i]) + at;
  TS* const pv = static_cast<TS*>(P.v[i]) + at;
  if constexpr (kBits8) {
    const i32x2 cm = load_codes(pm, left), cr = load_codes(pv, left);
    decode(cm, m);
    decode(cr, r);
    const int64_t b = at / kStateBlock;
    const float sm = left > 0 ? P.ms[i][b] : 0.0f;
    const float sv = left > 0 ? P.vs[i][b] : 0.0f;
    if (S.clip)
#pragma unroll
      for (int q = 0; q < kVec; ++q) g[q] *= S.coef;
    float tm = 0.0f, tr = 0.0f;
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      m[q] = m[q] * sm * S.b1 + g[q] * S.c1;
      const float ro = r[q] * sv;
      const float v = ro * ro * S.b2 + g[q] * g[q] * S.c2;
      r[q] = v >= 0x1p-96f ? root(v) : 0.0f;
      tm = fmaxf(tm, fabsf(m[q]));
      tr = fmaxf(tr, r[q]);
    }
    tm = max32(tm);
    tr = max32(tr);
    const float im = tm >= 1e-30f ? 256.0f / tm : 0.0f;
    const float ir = tr >= 1e-30f ? 256.0f / tr : 0.0f;
    float ym[kVec], yr[kVec];
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      ym[q] = m[q] * im;
      yr[q] = r[q] > 0.0f ? fmaxf(r[q] * ir, 0x1p-9f) : 0.0f;
    }
    store_codes(pm, left, new_codes(ym, cm, S.dither));
    store_codes(pv, left, new_codes(yr, cr, S.dither));
    if ((threadIdx.x & 31) == 0 && left > 0) {
      P.ms[i][b] = tm >= 1e-30f ? tm * 0x1p-8f : 0.0f;
      P.vs[i][b] = tr >= 1e-30f ? tr * 0x1p-8f : 0.0f;
    }
  } else {
    load_some<R>(pm, left, m);
    load_some<R>(pv, left, r);
    if (S.clip)
#pragma unroll
      for (int q = 0; q < kVec; ++q) g[q] *= S.coef;
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      m[q] = m[q] * S.b1 + g[q] * S.c1;
      r[q] = r[q] * S.b2 + g[q] * g[q] * S.c2;
    }
    store_some<R>(pm, left, m);
    store_some<R>(pv, left, r);
#pragma unroll
    for (int q = 0; q < kVec; ++q) r[q] = sqrtf(r[q]);
  }
  const float shrink = S.lr * P.decay[i];
#pragma unroll
  for (int q = 0; q < kVec; ++q) {
    const float d = fmaf(r[q], S.root, S.eps);
    const float u = m[q] * __builtin_amdgcn_rcpf(d);
    x[q] = fmaf(-S.size, u, fmaf(-shrink, x[q], x[q]));
  }
  if constexpr (kMaster) store_some<R>(master, left, x);
  store_some<R>(p, left, x);
}

template <bool kBits8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwTable P) {
  Shared S;
  S.clip = P.h.norm != nullptr;
  S.coef = 1.0f;
  if (S.clip) {
    const float norm = *P.h.norm;
    // an infinite or NaN norm: the step is left out
    if (!(fabsf(norm) < INFINITY)) return;
    S.coef = fminf(P.h.max_norm / (norm + 1e-6f), 1.0f);
  }
  const int64_t t = *P.h.step;
  S.b1 = P.h.b1;
  S.c1 = P.h.c1;
  S.b2 = P.h.b2;
  S.c2 = P.h.c2;
  S.eps = P.h.eps;
  S.lr = *P.h.lr;
  S.size = S.lr / one_minus_power(P.h.log_b1, t);
  S.root = 1.0f / sqrtf(one_minus_power(P.h.log_b2, t));
  S.dither = (static_cast<uint32_t>(t) * 0x9e3779b1u) >> 12;
  const int i = find_tensor(P.first, P.count, blockIdx.x);
  const int64_t chunk = static_cast<int64_t>(P.passes) * kChunk;
  int64_t at = (blockIdx.x - P.first[i]) * chunk;
  const int64_t end = min(at + chunk, P.n[i]);
  for (; at < end; at += kChunk) {
    if (P.p_fp32[i]) {
      if (P.g_fp32[i])
        update<kBits8, float, false, float>(P, i, at, S);
      else
        update<kBits8, float, false, bf16_t>(P, i, at, S);
    } else if (P.master[i]) {
      if (P.g_fp32[i])
        update<kBits8, bf16_t, true, float>(P, i, at, S);
      else
        update<kBits8, bf16_t, true, bf16_t>(P, i, at, S);
    } else {
      if (P.g_fp32[i])
        update<kBits8, bf16_t, false, float>(P, i, at, S);
      else
        update<kBits8, bf16_t, false, bf16_t>(P, i, at, S);
    }
  }
}

}  // namespace

size_t grad_norm_workspace() { return kNormGroups * sizeof(double); }

hipError_t launch_grad_norm(const moe_grad* grads, int count, float* norm,
                            void* ws, hipStream_t s) {
  double* part = static_cast<double*>(ws);
  const auto bytes = [&](int i) {
    return grads[i].n * (grads[i].g_fp32 ? 4 : 2);
  };
  const auto chunks_of = [&](int i) {
    return (bytes(i) + kNormBytes - 1) / kNormBytes;
  };
  int64_t all = 0, total = 0;
  for (int i = 0; i < count; ++i) {
    all += chunks_of(i);
    total += bytes(i);
  }
  const auto kernel =
      total > kNormCached ? grad_norm_kernel<true> : grad_norm_kernel<false>;
  const int groups = static_cast<int>(
      all < 1 ? 1 : all < kNormGroups ? all : kNormGroups);
  // each launch adds to what the ones before it left
  int i = 0;
  bool first = true;
  do {
    NormTable P{};
    int64_t chunks = 0;
    for (; i < count && P.count < kNormTensors; ++i) {
      if (grads[i].n == 0) continue;
      const int64_t c = chunks_of(i);
      // chunk numbers, also those past the end that a group asks for
      if (chunks + c > 0xffffffff - kNormAhead * kNormGroups) break;
      const int q = P.count++;
      P.g[q] = grads[i].g;
      P.bytes[q] = bytes(i);
      P.fp32[q] = grads[i].g_fp32 != 0;
      P.first[q] = static_cast<uint32_t>(chunks);
      chunks += c;
    }
    P.chunks = static_cast<uint32_t>(chunks);
    P.add = !first;
    first = false;
    hipLaunchKernelGGL(kernel, dim3(groups), dim3(kThreads), 0, s,
                       P, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (i < count);
  hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(kThreads), 0, s,
                     part, groups, norm);
  return hipGetLastError();
}

hipError_t launch_adamw(bool bits8, const moe_adamw_tensor* t, int count,
                        const AdamwHyper& h, hipStream_t s) {
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += t[i].n;
  const int passes = static_cast<int>(
      bits8 ? std::max<int64_t>(1, std::min<int64_t>(
                                       kMostPasses,
                                       all / kChunk / kRoundsChunks))
            : 1);
  const int64_t chunk = static_cast<int64_t>(passes) * kChunk;
  int i = 0;
  while (i < count) {
    AdamwTable P{};
    P.h = h;
    P.passes = passes;
    int64_t chunks = 0;
    for (; i < count && P.count < kTensors; ++i) {
      if (t[i].n == 0) continue;
      const int64_t c = (t[i].n + chunk - 1) / chunk;
      if (chunks + c > kMaxGroups) break;
      const int q = P.count++;
      P.p[q] = t[i].p;
      P.master[q] = t[i].master;
      P.g[q] = t[i].g;
      P.m[q] = t[i].m;
      P.v[q] = t[i].v;
      P.ms[q] = t[i].m_scale;
      P.vs[q] = t[i].v_scale;
      P.n[q] = t[i].n;
      P.decay[q] = t[i].weight_decay;
      P.p_fp32[q] = t[i].p_fp32 != 0;
      P.g_fp32[q] = t[i].g_fp32 != 0;
      P.first[q] = static_cast<uint32_t>(chunks);
      chunks += c;
    }
    if (P.count == 0) break;
    const dim3 grid(static_cast<uint32_t>(chunks));
    if (bits8)
      hipLaunchKernelGGL(adamw_kernel<true>, grid, dim3(kThreads), 0, s, P);
    else
      hipLaunchKernelGGL(adamw_kernel<false>, grid, dim3(kThreads), 0, s, P);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
