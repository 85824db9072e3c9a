// The whole expert layer for up to 64 tokens (generation, the end of a
// prompt): router, top-k, gate and up projections with SwiGLU, down
// projection, combine.
//
//   z = x W_g^T + b, (i_j, p_j) = top-k softmax of z
//   S_j = p_j silu(x G_{i_j}^T) (x U_{i_j}^T),  y = y_add + sum_j S_j W2_{i_j}^T
//
// Bound by reading the weights of the experts that are reached, once: nothing
// is permuted or staged, weights go from global memory straight into MFMA
// fragments.
//
//  * few_route_kernel, a workgroup a token: its scores, their order, the
//    routing weights.
//  * few_up_kernel, a workgroup for 8 gate and 8 up rows of an expert: S for
//    all of the expert's tokens.
//  * few_down_kernel, a workgroup for 8 rows of y: the sum over all experts
//    that are reached, in order, so nothing is added twice or in another
//    order.
//
// A tile is 8 weight rows x 64 k (bf16), one 16-byte load a lane that covers
// whole 128-byte lines of a row: lanes 0-7 of each 16 hold the rows' first 32
// k and lanes 8-15 the rows' other 32.  As the A operand of a 16 x 16 x 32
// MFMA, with 8 tokens' same two halves as B, the two 8 x 8 blocks on the
// diagonal of the product are the two halves' sums.  MXFP8 weights: a load is
// 8 rows x 128 codes, widened in registers to two such tiles of bf16 (exact:
// a code has four significant bits, its scale is a power of two).

#include "decode.h"

#include <math.h>

#include "common.cuh"

namespace moe {
namespace {

// --------------------------------------------------------------- routing
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;

// Scores in the order of the choice, as integers: a larger key is a better
// score, +0 and -0 are equal, NaN is below every number.
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);    // -0 becomes +0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_group_sum<16>(v);
  v += shfl_xor(v, 16);
  return v + shfl_xor(v, 32);
}

__global__ __launch_bounds__(kRouteThreads) void few_route_kernel(
    const bf16_t* __restrict__ x, const bf16_t* __restrict__ w_g,
    const float* __restrict__ bias, const float* __restrict__ logits, int d,
    int E, int k, int renorm, int32_t* __restrict__ idx,
    float* __restrict__ wt) {
  __shared__ float s_z[kMaxExperts];
  __shared__ uint32_t s_key[kMaxExperts];
  __shared__ int s_idx[kMaxTopK];
  __shared__ float s_p[kMaxTopK];
  __shared__ float s_sum[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = blockIdx.x;
  if (w_g) {
    const auto rx = make_rsrc(x + static_cast<int64_t>(t) * d, d * 2);
    // four experts a wave at a time
    for (int e0 = wave * 4; e0 < E; e0 += kRouteWaves * 4) {
      const int ne = min(4, E - e0);
      const auto rw = make_rsrc(w_g + static_cast<int64_t>(e0) * d,
                                static_cast<uint32_t>(ne) * d * 2);
      float acc[4] = {};
      for (int k0 = lane * 8; k0 < d; k0 += 512) {
        const i32x4 xv = buf_load16(rx, k0 * 2);
        i32x4 wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wv[i] = buf_load16(rw, i < ne ? (i * d + k0) * 2 : kOob);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t a = xv[q], b = wv[i][q];
            acc[i] = fmaf(bf_lo(a), bf_lo(b), acc[i]);
            acc[i] = fmaf(bf_hi(a), bf_hi(b), acc[i]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = wave_sum(acc[i]);
        if (lane == 0 && i < ne)
          s_z[e0 + i] = bias ? z + bias[e0 + i] : z;
      }
    }
  } else if (tid < E) {
    s_z[tid] = logits[static_cast<int64_t>(t) * E + tid];
  }
  __syncthreads();
  if (tid < E) s_key[tid] = score_key(s_z[tid]);
  __syncthreads();
  // an expert's place is the number of better ones
  if (tid < E) {
    const uint32_t key = s_key[tid];
    int place = 0;
    for (int e = 0; e < E; ++e) {
      const uint32_t o = s_key[e];
      place += o > key || (o == key && e < tid);
    }
    if (place < k) s_idx[place] = tid;
  }
  __syncthreads();
  const float top = s_z[s_idx[0]];
  if (tid < k) s_p[tid] = expf(s_z[s_idx[tid]] - top);
  if (!renorm) {
    const float z = wave_sum(tid < E ? expf(s_z[tid] - top) : 0.0f);
    if (lane == 0) s_sum[wave] = z;
  }
  __syncthreads();
  if (tid < k) {
    float sum = 0.0f;
    if (renorm)
      for (int j = 0; j < k; ++j) sum += s_p[j];
    else
      for (int w = 0; w < kRouteWaves; ++w) sum += s_sum[w];
    idx[t * k + tid] = s_idx[tid];
    wt[t * k + tid] = s_p[tid] / sum;
  }
}

// ---------------------------------------------------------------- weights
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 8;              // weight rows of a tile
constexpr int kTok = 8;               // tokens of a block
constexpr int kChunkK = 256;          // k a wave takes at a time

// A wave's place in a tile: row or token lane & 7 of each, and first k.
template <bool MX>
struct Lane {
  int r, k;
  __device__ __forceinline__ Lane() {
    const int lane = lane_id(), fr = lane & 15, g = lane >> 4;
    r = fr & 7;
    k = MX ? ((fr >> 3) * 4 + g) * 16 : (fr >> 3) * 32 + g * 8;
  }
};

// The k of a chunk of kChunkK for 8 weight rows, as loaded.
template <bool MX>
struct Weights {
  static constexpr int kSteps = MX ? 2 : 4;      // loads
  static constexpr int kStepK = kChunkK / kSteps;
  static constexpr int kFrags = MX ? 4 : 4;      // MFMA operands
  i32x4 w[kSteps];
  i32x2 s;                                       // MX: the 8 scale bytes

  // row0: byte offset of the lane's row; k0: first k of the chunk
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r,
                                       __amdgpu_buffer_rsrc_t rs,
                                       uint32_t row, int k0, int K,
                                       const Lane<MX>& L) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = k0 + i * kStepK + L.k;
      w[i] = buf_load16(r, k < K ? row + static_cast<uint32_t>(k) *
                                             (MX ? 1 : 2)
                                 : kOob);
    }
    if constexpr (MX)
      s = __builtin_amdgcn_raw_buffer_load_b64(
          rs, row / 32 + static_cast<uint32_t>(k0) / 32, 0, 0);
  }
  __device__ __forceinline__ bf16x8_v frag(int i, const Lane<MX>& L) const {
    if constexpr (!MX) {
      return __builtin_bit_cast(bf16x8_v, w[i]);
    } else {
      // codes 8 (i % 2) .. + 7 of load i / 2; its scale byte, of 4 a load,
      // as the exponent of a float
      const uint32_t sb = static_cast<uint32_t>(s[i >> 1]);
      const float sc =
          __uint_as_float(((sb >> ((L.k >> 5) * 8)) & 0xff) << 23);
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
      i32x4 o;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t c = static_cast<uint32_t>(w[i >> 1][2 * (i & 1) + q]);
        const bf16x2_t lo =
            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, false);
        const bf16x2_t hi =
            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, true);
        o[2 * q] = __builtin_bit_cast(int, lo);
        o[2 * q + 1] = __builtin_bit_cast(int, hi);
      }
      return __builtin_bit_cast(bf16x8_v, o);
    }
  }
};

// The same k of one block of tokens: fragment i matches Weights' i.
template <bool MX>
struct Tokens {
  i32x4 v[4];
  // row: byte offset of the lane's token, or kOob for none
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row,
                                       int k0, int K, const Lane<MX>& L) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = MX ? k0 + (i >> 1) * 128 + L.k + (i & 1) * 8
                       : k0 + i * 64 + L.k;
      v[i] = buf_load16(r, k < K && row != kOob
                               ? row + static_cast<uint32_t>(k) * 2
                               : kOob);
    }
  }
  __device__ __forceinline__ bf16x8_v frag(int i) const {
    return __builtin_bit_cast(bf16x8_v, v[i]);
  }
};

__device__ __forceinline__ f32x4 mma(bf16x8_v a, bf16x8_v b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// bytes of n x K weights, and of their scales
template <bool MX>
__device__ __forceinline__ uint32_t weight_bytes(int64_t n, int K) {
  return static_cast<uint32_t>(n * K * (MX ? 1 : 2));
}

// ---------------------------------------------------------------- gate, up
struct FewParams {
  const bf16_t* x;
  const uint8_t* w_gu;
  const uint8_t* w_gu_scales;
  const uint8_t* w2;
  const uint8_t* w2_scales;
  const int32_t* idx;                 // [T][k]
  const float* wt;
  bf16_t* s;                          // [T k][f]
  const bf16_t* y_add;
  bf16_t* y;
  int T, d, f, E, k;
  int slots;                          // units are slots (T k < E), or experts
};

// S of one expert for the NB blocks of its tokens.  slot: of member `lane`.
template <bool MX, int NB>
__device__ __forceinline__ void up_tile(const FewParams& P, int e, int n0,
                                        int members, int slot,
                                        float* __restrict__ red) {
  const Lane<MX> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int K = P.d;
  const int64_t per = static_cast<int64_t>(2) * P.f * K;   // values an expert
  const auto rw = make_rsrc(P.w_gu + e * per * (MX ? 1 : 2),
                            weight_bytes<MX>(2 * P.f, K));
  const auto rs = MX ? make_rsrc(P.w_gu_scales + e * (per / 32),
                                 static_cast<uint32_t>(per / 32))
                     : rw;
  const auto rx = make_rsrc(P.x, static_cast<uint32_t>(P.T) * K * 2);
  const uint32_t gate = static_cast<uint32_t>(n0 + L.r) * K * (MX ? 1 : 2);
  const uint32_t up = gate + static_cast<uint32_t>(P.f) * K * (MX ? 1 : 2);
  uint32_t tok[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int m = b * kTok + L.r;
    const int sl = __shfl(slot, m, kWave);
    tok[b] = m < members ? static_cast<uint32_t>(sl / P.k) * K * 2 : kOob;
  }
  f32x4 ag[NB], au[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) ag[b] = au[b] = f32x4{};
  Weights<MX> g, u;
  Tokens<MX> x[NB];
  int k0 = wave * kChunkK;
  if (k0 < K) {
    g.load(rw, rs, gate, k0, K, L);
    u.load(rw, rs, up, k0, K, L);
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b].load(rx, tok[b], k0, K, L);
  }
  while (k0 < K) {
    const int k1 = k0 + kWaves * kChunkK;
    const Weights<MX> cg = g, cu = u;
    Tokens<MX> cx[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) cx[b] = x[b];
    if (k1 < K) {
      g.load(rw, rs, gate, k1, K, L);
      u.load(rw, rs, up, k1, K, L);
#pragma unroll
      for (int b = 0; b < NB; ++b) x[b].load(rx, tok[b], k1, K, L);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8_v fg = cg.frag(i, L), fu = cu.frag(i, L);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        ag[b] = mma(fg, cx[b].frag(i), ag[b]);
        au[b] = mma(fu, cx[b].frag(i), au[b]);
      }
    }
    k0 = k1;
  }
  // red[wave][gate, up][lane][4]: row 4 (lane / 16) + v, token lane % 16
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b) __syncthreads();
    *reinterpret_cast<f32x4*>(red + (wave * 2 * 64 + lane) * 4) = ag[b];
    *reinterpret_cast<f32x4*>(red + ((wave * 2 + 1) * 64 + lane) * 4) = au[b];
    __syncthreads();
    if (tid < kRows * kTok) {
      const int row = tid & 7, c = tid >> 3;
      // the two halves of k: rows and tokens 0-7, and 8-15
      const int o1 = ((row >> 2) * 16 + c) * 4 + (row & 3);
      const int o2 = (((row >> 2) + 2) * 16 + c + 8) * 4 + (row & 3);
      float a = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* q = red + w * 2 * 256;
        a += q[o1] + q[o2];
        v += q[256 + o1] + q[256 + o2];
      }
      const int m = b * kTok + c;
      const int sl = __shfl(slot, m, kWave);
      if (m < members) {
        const float h = a * sigmoidf_(a) * v * P.wt[sl];
        P.s[static_cast<int64_t>(sl) * P.f + n0 + row] = f2bf(h);
      }
    }
  }
}

// MAXB: blocks that T tokens can fill.
template <bool MX, int MAXB>
__global__ __launch_bounds__(kThreads) void few_up_kernel(FewParams P) {
  __shared__ __attribute__((aligned(16))) float red[kWaves * 2 * 256];
  const int lane = threadIdx.x & 63;
  const int tiles = P.f / kRows;
  const int unit = blockIdx.x / tiles;
  const int n0 = (blockIdx.x - unit * tiles) * kRows;
  // lane t looks for the unit's expert among token t's choices
  const int e = __builtin_amdgcn_readfirstlane(P.slots ? P.idx[unit] : unit);
  int slot = -1;
  if (lane < P.T)
    for (int j = 0; j < P.k; ++j)
      if (P.idx[lane * P.k + j] == e) slot = lane * P.k + j;
  const uint64_t mask = __ballot(slot >= 0);
  if (mask == 0) return;
  // a slot whose expert an earlier token has too is left to that token's
  if (P.slots && __ffsll(static_cast<unsigned long long>(mask)) - 1 !=
                     unit / P.k)
    return;
  const int members = __popcll(mask);
  // member m's slot to lane m
  const int rank = __popcll(mask & ((uint64_t{1} << lane) - 1));
  slot = __builtin_amdgcn_ds_permute((slot >= 0 ? rank : 63) * 4, slot);
  if (members <= 8) {
    up_tile<MX, 1>(P, e, n0, members, slot, red);
  } else if (MAXB >= 2 && members <= 16) {
    up_tile<MX, MAXB >= 2 ? 2 : 1>(P, e, n0, members, slot, red);
  } else if (MAXB >= 4 && members <= 32) {
    up_tile<MX, MAXB >= 4 ? 4 : 1>(P, e, n0, members, slot, red);
  } else if (MAXB >= 8) {
    up_tile<MX, MAXB >= 8 ? 8 : 1>(P, e, n0, members, slot, red);
  }
}

// -------------------------------------------------------------------- down
// What every wave of few_down_kernel knows of the experts that are reached.
struct Units {
  uint64_t mask[kMaxExperts];         // tokens of an expert
  uint16_t first[kMaxExperts];        // its first place in `slot`
  uint16_t expert[kMaxExperts];       // reached experts in order
  uint16_t slot[kFewTokens * kMaxTopK];
  int count;
};

__device__ __forceinline__ void find_units(const FewParams& P, Units& U) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int n = P.T * P.k;
  for (int e = tid; e < P.E; e += kThreads) U.mask[e] = 0;
  int mine[kFewTokens * kMaxTopK / kThreads];
#pragma unroll
  for (int q = 0; q < kFewTokens * kMaxTopK / kThreads; ++q) {
    const int i = tid + q * kThreads;
    mine[q] = i < n ? P.idx[i] : -1;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kFewTokens * kMaxTopK / kThreads; ++q)
    if (mine[q] >= 0)
      atomicOr(reinterpret_cast<unsigned long long*>(&U.mask[mine[q]]),
               1ull << ((tid + q * kThreads) / P.k));
  __syncthreads();
  if (tid < 64) {
    int count = 0, first = 0;
    for (int e0 = 0; e0 < P.E; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < P.E ? __popcll(U.mask[e]) : 0;
      const uint64_t act = __ballot(c > 0);
      int incl = c;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(incl, m, kWave);
        if (lane >= m) incl += o;
      }
      if (e < P.E) U.first[e] = static_cast<uint16_t>(first + incl - c);
      if (c)
        U.expert[count + __popcll(act & ((uint64_t{1} << lane) - 1))] =
            static_cast<uint16_t>(e);
      count += __popcll(act);
      first += __shfl(incl, 63, kWave);
    }
    if (lane == 0) U.count = count;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kFewTokens * kMaxTopK / kThreads; ++q)
    if (mine[q] >= 0) {
      const int i = tid + q * kThreads, t = i / P.k;
      const uint64_t below = (uint64_t{1} << t) - 1;
      U.slot[U.first[mine[q]] + __popcll(U.mask[mine[q]] & below)] =
          static_cast<uint16_t>(i);
    }
  __syncthreads();
}

// Adds a wave's sums of the expert's members b * 8 .. + 7 to its own plane
// [half of k][token][8 rows].
__device__ __forceinline__ void add_members(float* plane, int T, f32x4 acc,
                                            int token) {
  const int lane = lane_id(), c = lane & 15, q = lane >> 4;
  // the diagonal blocks: rows 0-7 with tokens 0-7, rows 8-15 with 8-15
  if ((q >> 1) != (c >> 3) || token < 0) return;
  f32x4* p = reinterpret_cast<f32x4*>(
      plane + (((q >> 1) * T + token) * kRows + (q & 1) * 4));
  *p += acc;
}

template <bool MX, int MAXB>
__global__ __launch_bounds__(kThreads) void few_down_kernel(FewParams P) {
  __shared__ Units U;
  // [wave][half][T][8]
  extern __shared__ __attribute__((aligned(16))) float planes[];
  const Lane<MX> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = blockIdx.x * kRows;
  const int K = P.f, T = P.T;
  for (int i = tid; i < kWaves * 2 * T * kRows; i += kThreads) planes[i] = 0;
  find_units(P, U);
  float* const plane = planes + wave * 2 * T * kRows;
  const int chunks = (K + kChunkK - 1) / kChunkK;      // of an expert
  const int total = U.count * chunks;
  const auto rx =
      make_rsrc(P.s, static_cast<uint32_t>(T) * P.k * K * 2);
  const int64_t per = static_cast<int64_t>(P.d) * K;
  const uint32_t row = static_cast<uint32_t>(L.r) * K * (MX ? 1 : 2);

  // (unit, chunk) pairs in order, dealt to the waves in turn
  for (int q = wave; q < total; q += kWaves) {
    const int un = q / chunks, k0 = (q - un * chunks) * kChunkK;
    const int e = __builtin_amdgcn_readfirstlane(U.expert[un]);
    const int members = __builtin_amdgcn_readfirstlane(
        __popcll(U.mask[e]));
    const int first = U.first[e];
    const auto rw = make_rsrc(
        P.w2 + (e * per + static_cast<int64_t>(n0) * K) * (MX ? 1 : 2),
        weight_bytes<MX>(kRows, K));
    const auto rs =
        MX ? make_rsrc(P.w2_scales +
                           (e * per + static_cast<int64_t>(n0) * K) / 32,
                       static_cast<uint32_t>(kRows) * K / 32)
           : rw;
    Weights<MX> w;
    w.load(rw, rs, row, k0, K, L);
    for (int b = 0; b * kTok < members; ++b) {
      const int m = b * kTok + L.r;
      const int sl = m < members ? U.slot[first + m] : -1;
      Tokens<MX> x;
      x.load(rx, sl >= 0 ? static_cast<uint32_t>(sl) * K * 2 : kOob, k0, K,
             L);
      f32x4 acc = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = mma(w.frag(i, L), x.frag(i), acc);
      add_members(plane, T, acc, sl >= 0 ? sl / P.k : -1);
    }
  }
  __syncthreads();
  for (int i = tid; i < T * kRows; i += kThreads) {
    const int t = i >> 3, r = i & 7;
    float v = 0.0f;
    for (int p = 0; p < kWaves * 2; ++p) v += planes[(p * T + t) * kRows + r];
    const int64_t o = static_cast<int64_t>(t) * P.d + n0 + r;
    if (P.y_add) v += bf2f(P.y_add[o]);
    P.y[o] = f2bf(v);
  }
}

template <bool MX, int MAXB>
hipError_t launch_few(const FewParams& P, hipStream_t s) {
  const int units = P.slots ? P.T * P.k : P.E;
  hipLaunchKernelGGL((few_up_kernel<MX, MAXB>),
                     dim3(static_cast<uint32_t>(units) * (P.f / kRows)),
                     dim3(kThreads), 0, s, P);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((few_down_kernel<MX, MAXB>), dim3(P.d / kRows),
                     dim3(kThreads),
                     kWaves * 2 * P.T * kRows * sizeof(float), s, P);
  return hipGetLastError();
}

template <bool MX>
hipError_t launch_blocks(const FewParams& P, hipStream_t s) {
  if (P.T <= 8) return launch_few<MX, 1>(P, s);
  if (P.T <= 16) return launch_few<MX, 2>(P, s);
  if (P.T <= 32) return launch_few<MX, 4>(P, s);
  return launch_few<MX, 8>(P, s);
}

}  // namespace

size_t layer_fwd_workspace(int64_t T, int E, int k, int64_t f) {
  return (static_cast<size_t>(T * k * f * 2) + 255) & ~size_t{255};
}

hipError_t launch_layer_fwd(bool mx, const LayerArgs& a, void* ws,
                            hipStream_t s) {
  hipLaunchKernelGGL(few_route_kernel, dim3(a.T), dim3(kRouteThreads), 0, s,
                     a.x, a.w_g, a.bias, a.logits, a.d, a.E, a.k, a.renorm,
                     a.topk_idx, a.topk_w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  FewParams P{};
  P.x = a.x;
  P.w_gu = static_cast<const uint8_t*>(a.w_gu);
  P.w_gu_scales = a.w_gu_scales;
  P.w2 = static_cast<const uint8_t*>(a.w2);
  P.w2_scales = a.w2_scales;
  P.idx = a.topk_idx;
  P.wt = a.topk_w;
  P.s = static_cast<bf16_t*>(ws);
  P.y_add = a.y_add;
  P.y = a.y;
  P.T = a.T;
  P.d = a.d;
  P.f = a.f;
  P.E = a.E;
  P.k = a.k;
  P.slots = a.T * a.k < a.E;
  return mx ? launch_blocks<true>(P, s) : launch_blocks<false>(P, s);
}

}  // namespace moe
