// Dropout with an optional residual sum; the mask comes from a
// counter-based generator and is never stored.
//
//   out[i] = res[i] + (keep_i ? x[i] * scale : 0)
// The backward pass is the same call on the upstream gradient without res:
// it draws the same mask from the same counters.
//
// Generator: Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E.
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11) under the
// 64-bit key rng[0], on the counter (element index / 8, rng[1] + delta).
// Its four 32-bit words are eight 16-bit draws, one for each element of a
// 16-byte bf16 chunk: half i % 2 (low first) of word (i % 8) / 2 decides
// element i, which is kept when the draw is at least thr = p * 65536
// (rounded to an integer); scale = 65536 / (65536 - thr), so the mean is
// kept exactly for the probability that is drawn.  16 bits a draw are half
// the integer work of 32-bit draws (20 widening multiplies a counter); both
// hide behind the memory traffic on MI355X (8192 x 4096 bf16 with a
// residual: 37.5 us, and 37.1 with 32-bit draws).
// A dropped element adds exactly 0, whatever x holds there.
//
// Bound by memory: x, res and out once, 16-byte accesses, a chunk a thread
// (8192 x 4096 bf16: 37.5 us with a residual, 5.4 TB/s, and 23.9 without, 5.6
// TB/s; 8 chunks a thread 39.3 and 25.8 us).  All times: calls in a captured
// sequence over data that leaves the caches.

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kDropThreads = 256;

struct Philox {
  uint32_t w[4];
  __device__ __forceinline__ void run(uint64_t block, uint64_t offset,
                                      uint64_t key) {
    uint32_t c0 = static_cast<uint32_t>(block);
    uint32_t c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset);
    uint32_t c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(key);
    uint32_t k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
      const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
      c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
      c1 = static_cast<uint32_t>(b);
      c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
      c3 = static_cast<uint32_t>(a);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
  }
  __device__ __forceinline__ uint32_t draw(int i) const {
    return (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
  }
};

__device__ __forceinline__ void load8(const bf16_t* p, float* v) {
  const i32x4 r = *reinterpret_cast<const i32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf_lo(static_cast<uint32_t>(r[i]));
    v[2 * i + 1] = bf_hi(static_cast<uint32_t>(r[i]));
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8(bf16_t* p, const float* v) {
  i32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = static_cast<int>(pack_bf16x2(v[2 * i], v[2 * i + 1]));
  *reinterpret_cast<i32x4*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float to_f(bf16_t v) { return bf2f(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// One chunk of 8 elements a thread and turn.  out may be x (of its type) or
// res: a chunk is read before the thread that read it writes it.
template <typename XT, typename OT, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(
    const XT* x, const OT* res, int64_t n, uint32_t thr, float scale,
    const uint64_t* __restrict__ rng, uint64_t delta, OT* out) {
  const uint64_t key = rng[0];
  const uint64_t off = rng[1] + delta;
  const int64_t nfull = n >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kDropThreads;
  int64_t c = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x;
  for (; c < nfull; c += step) {
    float v[8], r[8], o[8];
    load8(x + c * 8, v);
    if constexpr (RES) load8(res + c * 8, r);
    Philox g;
    g.run(static_cast<uint64_t>(c), off, key);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float base = RES ? r[i] : 0.0f;
      o[i] = g.draw(i) >= thr ? fmaf(v[i], scale, base) : base;
    }
    store8(out + c * 8, o);
  }
  // the last, partial chunk belongs to the thread whose turn it is
  if (c == nfull && (n & 7)) {
    Philox g;
    g.run(static_cast<uint64_t>(c), off, key);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t j = c * 8 + i;
      if (j < n) {
        const float base = RES ? to_f(res[j]) : 0.0f;
        put(out + j,
            g.draw(i) >= thr ? fmaf(to_f(x[j]), scale, base) : base);
      }
    }
  }
}

template <typename XT, typename OT>
hipError_t dropout(const void* x, const void* res, int64_t n, uint32_t thr,
                   float scale, const uint64_t* rng, uint64_t delta,
                   void* out, hipStream_t s) {
  const int64_t chunks = (n + 7) / 8;
  int64_t nb = (chunks + kDropThreads - 1) / kDropThreads;
  if (nb > 65536) nb = 65536;
  if (res)
    hipLaunchKernelGGL((dropout_kernel<XT, OT, true>),
                       dim3(static_cast<uint32_t>(nb)), dim3(kDropThreads),
                       0, s, static_cast<const XT*>(x),
                       static_cast<const OT*>(res), n, thr, scale, rng,
                       delta, static_cast<OT*>(out));
  else
    hipLaunchKernelGGL((dropout_kernel<XT, OT, false>),
                       dim3(static_cast<uint32_t>(nb)), dim3(kDropThreads),
                       0, s, static_cast<const XT*>(x),
                       static_cast<const OT*>(nullptr), n, thr, scale, rng,
                       delta, static_cast<OT*>(out));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int x_fp32, const void* res,
                          int out_fp32, int64_t n, uint32_t thr, float scale,
                          const uint64_t* rng, uint64_t delta, void* out,
                          hipStream_t s) {
  if (x_fp32)
    return out_fp32 ? dropout<float, float>(x, res, n, thr, scale, rng,
                                            delta, out, s)
                    : dropout<float, bf16_t>(x, res, n, thr, scale, rng,
                                             delta, out, s);
  return out_fp32 ? dropout<bf16_t, float>(x, res, n, thr, scale, rng, delta,
                                           out, s)
                  : dropout<bf16_t, bf16_t>(x, res, n, thr, scale, rng,
                                            delta, out, s);
}

}  // namespace moe
