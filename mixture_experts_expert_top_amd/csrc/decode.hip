// The whole expert layer for up to 64 tokens (generation, the end of a
// prompt): router, top-k, gate and up projections with SwiGLU, down
// projection, combine.
//
//   z = x W_g^T + b, (i_j, p_j) = top-k softmax of z
//   S_j = p_j silu(x G_{i_j}^T) (x U_{i_j}^T),  y = y_add + sum_j S_j W2_{i_j}^T
//
// Bound by reading the weights of the experts that are reached, once (w2 twice
// for an expert of more than 32 tokens): nothing is permuted, weights go from
// global memory straight into MFMA fragments.
// A kernel that only reads gets 6.1 TB/s here; times below are of kernels
// alone, traced, weights not in any cache.
//
//  * few_logits_kernel: the scores.
//  * few_topk_kernel: the choice, where the first product does not make it.
//  * the first product, S for the tokens of each expert: few_up_kernel (up to
//    8 tokens, bf16 weights) or few_up_batch_kernel.
//  * the second, the sums over all experts: few_down_kernel (few tokens, few
//    weights) or few_down_batch_kernel.
//  * few_sum_kernel, where the second product is cut into parts: y.
//
// S is held as the sum of two bf16 values, the second what the first leaves:
// 16 significant bits, so that y has the error of its own rounding alone.
// The second product multiplies both as two columns of the same MFMA, which
// has columns to spare.  (As one bf16 value S would lose up to 2^-8 of each
// term, more than y's own rounding where terms cancel.)
//
// All sums are made in one order, so that equal calls give equal bits.
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

#include <type_traits>

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

// x[t] . w_g[e] by one wave, 4 KB of both in flight; in every lane.
__device__ __forceinline__ float score(const bf16_t* __restrict__ x,
                                       const bf16_t* __restrict__ w_g, int d,
                                       int t, int e) {
  const auto rx = make_rsrc(x + static_cast<int64_t>(t) * d, d * 2);
  const auto rw = make_rsrc(w_g + static_cast<int64_t>(e) * d, d * 2);
  // loads past the row read zeros
  float acc = 0.0f;
  for (int k0 = lane_id() * 16; k0 < d * 2; k0 += 4096) {
    i32x4 xv[4], wv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      xv[u] = buf_load16(rx, k0 + u * 1024);
      wv[u] = buf_load16(rw, k0 + u * 1024);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a = xv[u][q], b = wv[u][q];
        acc = fmaf(bf_lo(a), bf_lo(b), acc);
        acc = fmaf(bf_hi(a), bf_hi(b), acc);
      }
  }
  return wave_sum(acc);
}

// Scores: a wave an expert and token.  64 experts of 2048: 3 us for one token,
// 4.7 for 24, of which a kernel that does next to nothing takes 2 to 4.
constexpr int kLogitThreads = 256;
constexpr int kLogitWaves = kLogitThreads / kWave;

__global__ __launch_bounds__(kLogitThreads) void few_logits_kernel(
    const bf16_t* __restrict__ x, const bf16_t* __restrict__ w_g,
    const float* __restrict__ bias, int d, int E, float* __restrict__ logits) {
  const int e = __builtin_amdgcn_readfirstlane(
      blockIdx.x * kLogitWaves + (threadIdx.x >> 6));
  const int t = blockIdx.y;
  if (e >= E) return;
  const float z = score(x, w_g, d, t, e);
  if (lane_id() == 0)
    logits[static_cast<int64_t>(t) * E + e] = bias ? z + bias[e] : z;
}

// The choice of one token from its scores, any number of experts.  4.6 us
// for 24 tokens of 64 experts.  logits null: the scores too, which saves a
// launch and pays where a wave has one expert (whole layers: 16 tokens, 8
// experts of 4096 x 256 35.7 -> 34.3 us, 24 tokens, 16 of 1024 x 256 25.2 ->
// 24.2; 24 tokens, 64 of 1024 x 256 31.3 -> 33.0).
__global__ __launch_bounds__(kRouteThreads) void few_topk_kernel(
    const float* __restrict__ logits, const bf16_t* __restrict__ x,
    const bf16_t* __restrict__ w_g, const float* __restrict__ bias, int d,
    int E, int k, int renorm, int32_t* __restrict__ idx,
    float* __restrict__ wt) {
  __shared__ float s_z[kMaxExperts];
  __shared__ __attribute__((aligned(16))) uint32_t s_key[kMaxExperts];
  __shared__ int s_place[kMaxExperts];
  __shared__ int s_idx[kMaxTopK];
  __shared__ float s_p[kMaxTopK];
  __shared__ float s_sum[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = blockIdx.x;
  // An expert's place is the number of better ones.  The keys (padded to a
  // multiple of four that nothing is worse than) are compared by `segs`
  // threads an expert, each with its share of them.
  const int E4 = (E + 3) & ~3;
  if (!logits) {
    for (int e = __builtin_amdgcn_readfirstlane(wave); e < E;
         e += kRouteWaves) {
      const float z = score(x, w_g, d, t, e);
      if (lane == 0) s_z[e] = bias ? z + bias[e] : z;
    }
    __syncthreads();
  }
  if (tid < E4) {
    const float z = tid >= E ? 0.0f
                    : logits ? logits[static_cast<int64_t>(t) * E + tid]
                             : s_z[tid];
    s_z[tid] = z;
    s_key[tid] = tid < E ? score_key(z) : 0;
    s_place[tid] = 0;
  }
  __syncthreads();
  int width = 64;
  while (width < E) width *= 2;
  const int me = tid & (width - 1), seg = tid / width;
  if (me < E) {
    const int fours = E4 / 4, segs = kRouteThreads / width;
    const int per = (fours + segs - 1) / segs;
    const uint32_t key = s_key[me];
    int place = 0;
    for (int q = seg * per; q < min(fours, (seg + 1) * per); ++q) {
      const uint4 o = reinterpret_cast<const uint4*>(s_key)[q];
      const uint32_t ok[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        place += ok[i] > key || (ok[i] == key && q * 4 + i < me);
    }
    if (place) atomicAdd(&s_place[me], place);
  }
  __syncthreads();
  if (tid < E && s_place[tid] < k) s_idx[s_place[tid]] = tid;
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

// The largest of a wave's values.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
#define MOE_DPP_MAX(ctrl)                                                    \
  v = step(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(             \
                  0, static_cast<int>(v), ctrl, 0xf, 0xf, false)))
  MOE_DPP_MAX(kDppXor1);
  MOE_DPP_MAX(kDppXor2);
  MOE_DPP_MAX(kDppHalfMirror);
  MOE_DPP_MAX(kDppMirror);
#undef MOE_DPP_MAX
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    m = step(m, static_cast<uint32_t>(__builtin_amdgcn_readlane(
                    static_cast<int>(v), r * 16)));
  return m;
}

// The same by one wave for up to 64 N experts, N a lane: its choices go to
// idx[0 .. k) and wt.
template <int N>
__device__ __forceinline__ void choose(const float* __restrict__ z, int E,
                                       int k, int renorm, int* idx,
                                       float* wt) {
  const int lane = lane_id();
  float v[N];
  uint32_t key[N];                    // 0: none, or chosen already
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * kWave + lane;
    v[i] = e < E ? z[e] : 0.0f;
    key[i] = e < E ? max(score_key(v[i]), 1u) : 0;
  }
  int mine = 0;                       // choice `lane`, and its score
  float score = 0.0f, top = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = max(m, key[i]);
    m = wave_max(m);
    // the lowest expert with that key
    bool found = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t b = __ballot(key[i] == m);
      if (found || b == 0) continue;
      found = true;
      const int l = __ffsll(static_cast<unsigned long long>(b)) - 1;
      const float s = __int_as_float(
          __builtin_amdgcn_readlane(__float_as_int(v[i]), l));
      if (j == 0) top = s;
      if (lane == j) {
        mine = i * kWave + l;
        score = s;
      }
      if (lane == l) key[i] = 0;
    }
  }
  const float p = expf(score - top);
  float part = 0.0f;
  if (renorm) {
    part = lane < k ? p : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * kWave + lane < E) part += expf(v[i] - top);
  }
  const float sum = wave_sum(part);
  if (lane < k) {
    idx[lane] = mine;
    wt[lane] = p / sum;
  }
}

// ---------------------------------------------------------------- weights
constexpr int kRows = 8;              // weight rows of a tile
constexpr int kChunkK = 256;          // k a wave takes at a time

// Workgroups of the two products: four waves for a tile of gate and up (the
// tiles are many, and small workgroups start and end independently); for a
// tile of y, whose reduction is long, kDownThreads.
constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / kWave;

struct FewParams {
  const bf16_t* x;
  const uint8_t* w_gu;
  const uint8_t* w_gu_scales;
  const uint8_t* w2;
  const uint8_t* w2_scales;
  int32_t* idx;                       // [T][k]
  float* wt;
  const float* logits;                // to choose from, or null: idx, wt given
  int renorm;
  bf16_t* s;                          // [T k][2][f]: S in two parts
  const bf16_t* y_add;
  bf16_t* y;
  float* part;                        // [part][T][d]
  int T, d, f, E, k;
  int parts;                          // of the reduction of a tile of y
  uint32_t inv_k;                     // ceil(2^16 / k)

  // i / k for slots below 2048 and k up to 32: i (k - 1) stays below 2^16
  __device__ __forceinline__ int token(int i) const {
    return static_cast<int>((static_cast<uint32_t>(i) * inv_k) >> 16);
  }
};

// A wave's place in a tile of 8 rows: the lane's row (and token), and its
// first k in a load.
template <bool MX>
struct Lane {
  int r, k;
  __device__ __forceinline__ Lane() {
    const int lane = lane_id(), fr = lane & 15, g = lane >> 4;
    r = fr & 7;
    k = MX ? ((fr >> 3) * 4 + g) * 16 : (fr >> 3) * 32 + g * 8;
  }
};

// bf16 values of eight E4M3 codes; `scale`: 4 scale bytes of 32 codes each,
// `block`: which of them, as the exponent of a float.
__device__ __forceinline__ bf16x8_v widen(int c0, int c1, uint32_t scale,
                                          int block) {
  const float sc = __uint_as_float(((scale >> (block * 8)) & 0xff) << 23);
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  i32x4 o;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t c = static_cast<uint32_t>(q ? c1 : c0);
    const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc,
                                                                  false);
    const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc,
                                                                  true);
    o[2 * q] = __builtin_bit_cast(int, lo);
    o[2 * q + 1] = __builtin_bit_cast(int, hi);
  }
  return __builtin_bit_cast(bf16x8_v, o);
}

// 16 bytes of weights.  NT: rows of whole 128-byte lines; no one else reads
// these, and marked as non-temporal they come faster (24 tokens, 64 experts of
// 2048 x 1408 in MXFP8: the first product 70 -> 62 us; one token of 2 experts
// of 4096 x 14336: 81 -> 73).  Lines that two rows share are read twice, and
// then the mark costs (61 tokens, 41 experts of 1032 x 680: 28 -> 30 us).
template <bool NT>
__device__ __forceinline__ i32x4 weight16(__amdgpu_buffer_rsrc_t r,
                                          uint32_t off) {
  constexpr int kNonTemporal = 2;
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0,
                                               NT ? kNonTemporal : 0);
}

// KC k of 8 weight rows, as loaded; KC / 64 MFMA operands.
template <bool MX, bool NT, int KC = kChunkK>
struct Weights {
  static constexpr int kLoadK = MX ? 128 : 64;
  static constexpr int kLoads = KC / kLoadK;
  static constexpr int kFrags = KC / 64;
  i32x4 w[kLoads];
  uint32_t s[MX ? kLoads : 1];         // MX: 4 scale bytes a load
  int end;                            // MX: k from k0 to the row's end

  // row: byte offset of the lane's row (MX: of a byte a value)
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r,
                                       __amdgpu_buffer_rsrc_t rs,
                                       uint32_t row, int k0, int K,
                                       const Lane<MX>& L) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = k0 + i * kLoadK + L.k;
      w[i] = weight16<NT>(
          r, k < K ? row + static_cast<uint32_t>(k) * (MX ? 1 : 2) : kOob);
    }
    if constexpr (MX) {
      end = K - k0;
      const uint32_t at =
          k0 < K ? row / 32 + static_cast<uint32_t>(k0) / 32 : kOob;
      if constexpr (kLoads == 4) {
        const i32x4 v = buf_load16(rs, at);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = static_cast<uint32_t>(v[i]);
      } else if constexpr (kLoads == 1) {
        s[0] = buf_load4(rs, at);
      } else {
        static_assert(kLoads == 2, "128, 256 or 512 codes");
        const i32x2 v = __builtin_bit_cast(
            i32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0));
        s[0] = static_cast<uint32_t>(v[0]);
        s[1] = static_cast<uint32_t>(v[1]);
      }
    }
  }
  __device__ __forceinline__ bf16x8_v frag(int i, const Lane<MX>& L) const {
    if constexpr (!MX) {
      return __builtin_bit_cast(bf16x8_v, w[i]);
    } else {
      // where the row ends inside the chunk the scales behind it are the next
      // row's: one that is NaN would make NaN of the zeros that stand there
      const uint32_t sc =
          (i >> 1) == 0 || (i >> 1) * kLoadK < end ? s[i >> 1] : 0;
      return widen(w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1], sc,
                   L.k >> 5);
    }
  }
};

// The same k of a block of 8 tokens: fragment i matches Weights' i.
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

// --------------------------------------------------------- reached experts
// The experts that are reached, in order, with the slots of their tokens, in
// the front of a kernel's dynamic LDS.
struct Expert {
  uint16_t id, first, members, tokens;  // tokens: the mask of tokens 0 to 15
};
struct Units {
  uint64_t* mask;       // [E] tokens of an expert
  Expert* expert;       // [E] reached experts, in order
  float* wt;            // [T k] weight of a slot
  uint16_t* slot;       // [T k] slots, those of an expert in a row
  uint16_t* first;      // [E] where an expert's are
  int count;

  // bytes for E experts and n slots, a multiple of 16
  __host__ __device__ static int bytes(int E, int n) {
    return (E * 18 + n * 6 + 4 + 15) & ~15;
  }
};

// The direct forms, in which the waves of a workgroup divide the reduction and
// read the tokens' values themselves, against the batch forms, which stage
// them in LDS (us):
//   first product, bf16         direct   batch
//     8 tokens, 64 x 2048 x 1408    83      96
//     8 tokens, 8 x 4096 x 14336   262     272
//     1 token, 64 x 2048 x 1408     20      23
//   first product, MXFP8, where a token's values are as many loads as the
//   weights
//     8 tokens, 64 x 2048 x 1408    55      47
//     1 token, 8 x 4096 x 14336     50      46
//     1 token, 64 x 2048 x 1408     14      15
//   second product, to which the batch form adds few_sum_kernel's 4.7
//     1 token, bf16, 8 x 4096 x 14336     43    38 + 4.7
//     4 tokens, bf16, 8 x 4096 x 14336   135   117 + 4.7
//     2 tokens, bf16, 64 x 2048 x 1408    18    18 + 4.7
//     4 tokens, MXFP8, 64 x 2048 x 1408   25    20 + 4.7
// So: the first product direct for bf16 weights up to the 8 columns that a
// tile has, the second up to the 4 whose two parts fit and as long as few_sum
// weighs more, by the values that it may have to read (one limit for both
// types; between 46 and 92 million values neither was measured).
constexpr int kDirectUp = 8;
constexpr int kDirectDown = 4;
constexpr int64_t kDirectValues = 80000000;
// Up to kChooseTokens and 64 kChooseLanes experts: the waves of a workgroup
// of the first product choose for the tokens themselves, and the first one
// writes the choices down: two tokens a wave cost less than few_topk_kernel
// and its launch (one token of 64 experts, the whole layer 36.8 -> 34.7 us).
// With six tokens a wave (24 of 64 experts, 8 each) the first product takes 6
// to 10 us longer, more than the kernel's 4.6; with sixteen (61 of 41, 3
// each) 13 longer.
constexpr int kChooseTokens = 8;
constexpr int kChooseLanes = 4;

struct Choices {
  int* idx;
  float* wt;
};

// Chooses into LDS at `to` (8 bytes a slot) where the call left that to the
// kernel.
template <int kThreads>
__device__ __forceinline__ Choices choose_here(const FewParams& P,
                                               uint8_t* to) {
  Choices c{P.idx, P.wt};
  if (!P.logits) return c;
  const int n = P.T * P.k;
  c.idx = reinterpret_cast<int*>(to);
  c.wt = reinterpret_cast<float*>(c.idx + n);
  for (int t = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); t < P.T;
       t += kThreads / kWave) {
    const float* const z = P.logits + t * P.E;
    int* const i = c.idx + t * P.k;
    float* const w = c.wt + t * P.k;
    if (P.E <= kWave)
      choose<1>(z, P.E, P.k, P.renorm, i, w);
    else
      choose<kChooseLanes>(z, P.E, P.k, P.renorm, i, w);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < n; i += kThreads) {
      P.idx[i] = c.idx[i];
      P.wt[i] = c.wt[i];
    }
  return c;
}

template <int kThreads>
__device__ __forceinline__ void find_units(const FewParams& P,
                                           const Choices& chosen, uint8_t* lds,
                                           Units* out) {
  constexpr int kPer = kFewTokens * kMaxTopK / kThreads;
  const int tid = threadIdx.x, lane = tid & 63;
  const int n = P.T * P.k, E = P.E;
  const int* const idx = chosen.idx;
  const float* const weights = chosen.wt;
  Units U;
  U.mask = reinterpret_cast<uint64_t*>(lds);
  U.expert = reinterpret_cast<Expert*>(U.mask + E);
  U.wt = reinterpret_cast<float*>(U.expert + E);
  int* const count_at = reinterpret_cast<int*>(U.wt + n);
  U.slot = reinterpret_cast<uint16_t*>(count_at + 1);
  U.first = U.slot + n;
  if (P.T == 1) {                     // every slot, in its own order
    if (tid < n) {
      const uint16_t i = static_cast<uint16_t>(tid);
      U.wt[tid] = weights[tid];
      U.expert[tid] = Expert{static_cast<uint16_t>(idx[tid]), i, 1, 1};
      U.slot[tid] = i;
    }
    __syncthreads();
    U.count = n;
    *out = U;
    return;
  }
  int mine[kPer];
  float wt[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid + q * kThreads;
    mine[q] = i < n ? idx[i] : -1;
    wt[q] = i < n ? weights[i] : 0.0f;
  }
  for (int e = tid; e < E; e += kThreads) U.mask[e] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (mine[q] >= 0) {
      const int i = tid + q * kThreads;
      U.wt[i] = wt[q];
      atomicOr(reinterpret_cast<unsigned long long*>(&U.mask[mine[q]]),
               1ull << P.token(i));
    }
  __syncthreads();
  if (tid < 64) {
    int count = 0, first = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint64_t mask = e < E ? U.mask[e] : 0;
      const int c = __popcll(mask);
      const uint64_t act = __ballot(c > 0);
      int incl = c;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(incl, m, kWave);
        if (lane >= m) incl += o;
      }
      const uint16_t at = static_cast<uint16_t>(first + incl - c);
      if (e < E) U.first[e] = at;
      if (c)
        U.expert[count + __popcll(act & ((uint64_t{1} << lane) - 1))] =
            Expert{static_cast<uint16_t>(e), at, static_cast<uint16_t>(c),
                   static_cast<uint16_t>(mask)};
      count += __popcll(act);
      first += __shfl(incl, 63, kWave);
    }
    if (lane == 0) *count_at = count;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (mine[q] >= 0) {
      const int i = tid + q * kThreads;
      const uint64_t below = (uint64_t{1} << P.token(i)) - 1;
      U.slot[U.first[mine[q]] + __popcll(U.mask[mine[q]] & below)] =
          static_cast<uint16_t>(i);
    }
  __syncthreads();
  U.count = __builtin_amdgcn_readfirstlane(*count_at);
  *out = U;
}

// A reached expert in scalar registers.
struct Reached {
  int id, first, members, tokens;
  __device__ __forceinline__ void read(const Units& U, int un) {
    const i32x2 v = *reinterpret_cast<const i32x2*>(&U.expert[un]);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(v[0]);
    const uint32_t hi = __builtin_amdgcn_readfirstlane(v[1]);
    id = static_cast<int>(lo & 0xffff);
    first = static_cast<int>(lo >> 16);
    members = static_cast<int>(hi & 0xffff);
    tokens = static_cast<int>(hi >> 16);
  }
};

// ---------------------------------------------------------------- gate, up
// The weights of an expert's gate and up projection.
template <bool MX>
struct UpWeights {
  __amdgpu_buffer_rsrc_t rw, rs;
  __device__ __forceinline__ UpWeights(const FewParams& P, int e) {
    const int64_t per = static_cast<int64_t>(2) * P.f * P.d;
    rw = make_rsrc(P.w_gu + e * per * (MX ? 1 : 2),
                   static_cast<uint32_t>(per * (MX ? 1 : 2)));
    rs = MX ? make_rsrc(P.w_gu_scales + e * (per / 32),
                        static_cast<uint32_t>(per / 32))
            : rw;
  }
  // byte offset of row n of gate, or of up
  __device__ __forceinline__ static uint32_t row(const FewParams& P, int n,
                                                 bool up) {
    return (static_cast<uint32_t>(n) + (up ? P.f : 0)) * P.d * (MX ? 1 : 2);
  }
};

// S = wt silu(a) u, held in two bf16 parts, the second what the first leaves.
__device__ __forceinline__ float swiglu(float a, float u, float wt) {
  return a * sigmoidf_(a) * u * wt;
}
// What the first part is rounded from: always finite in bf16, so that the
// second is infinite or NaN where S is, and not by taking infinities apart.
__device__ __forceinline__ float first_part(float h) {
  constexpr float kMost = 0x1.fep127f;          // bf16's largest value
  return __builtin_amdgcn_fmed3f(h, -kMost, kMost);
}

// Tiles [t0, t1) of an expert, 8 gate and 8 up rows each, for up to 8 members;
// the waves divide the reduction.  red: two buffers, `flip` tells which is
// next.
template <bool NT>
__device__ __forceinline__ void up_tiles(const FewParams& P, const Units& U,
                                         int un, int t0, int t1,
                                         float* __restrict__ red, int* flip) {
  const Lane<false> L;
  Reached X;
  X.read(U, un);
  const UpWeights<false> W(P, X.id);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = P.d;
  const auto rx = make_rsrc(P.x, static_cast<uint32_t>(P.T) * K * 2);
  const uint32_t tok =
      L.r < X.members
          ? static_cast<uint32_t>(P.token(U.slot[X.first + L.r])) * K * 2
          : kOob;
  // the member that the lane stores for, and its weight
  const int mine = lane >> 3;
  const int slot = mine < X.members ? U.slot[X.first + mine] : -1;
  const float wt = slot >= 0 ? U.wt[slot] : 0.0f;
  // A wave's chunks of a tile, then the next tile's: one is in flight while
  // the one before it is multiplied.  The last is taken out of the loop: a
  // branch around its loads would make the compiler wait for all that is in
  // flight, every time.
  struct Item {
    Weights<false, NT> g, u;
    Tokens<false> x;
  };
  auto load = [&](Item& it, int tile, int k0) {
    const int n = tile * kRows + L.r;
    it.g.load(W.rw, W.rs, W.row(P, n, false), k0, K, L);
    it.u.load(W.rw, W.rs, W.row(P, n, true), k0, K, L);
    it.x.load(rx, tok, k0, K, L);
    __builtin_amdgcn_sched_barrier(0);
  };
  const int rounds = (K + kUpWaves * kChunkK - 1) / (kUpWaves * kChunkK);
  Item nxt;
  load(nxt, t0, wave * kChunkK);
  f32x4 ag = {}, au = {};
  auto multiply = [&](const Item& cur) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ag = mma(cur.g.frag(i, L), cur.x.frag(i), ag);
      au = mma(cur.u.frag(i, L), cur.x.frag(i), au);
    }
  };
  auto finish = [&](int tile) {
    // red[wave][gate, up][lane][4]: row 4 (lane / 16) + v, token lane % 16.
    // A wave that still adds up one buffer passes the next barrier before
    // anyone writes to that buffer again.
    float* const r = red + *flip * (kUpWaves * 512);
    *flip ^= 1;
    *reinterpret_cast<f32x4*>(r + (wave * 128 + lane) * 4) = ag;
    *reinterpret_cast<f32x4*>(r + (wave * 128 + 64 + lane) * 4) = au;
    __syncthreads();
    if (wave == (tile & (kUpWaves - 1))) {
      const int row = lane & 7;
      // the two halves of k: rows and tokens 0-7, and 8-15
      const int o1 = ((row >> 2) * 16 + mine) * 4 + (row & 3);
      const int o2 = (((row >> 2) + 2) * 16 + mine + 8) * 4 + (row & 3);
      float a = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kUpWaves; ++w) {
        const float* q = r + w * 512;
        a += q[o1] + q[o2];
        v += q[256 + o1] + q[256 + o2];
      }
      if (slot >= 0) {
        const float h = swiglu(a, v, wt);
        const bf16_t hi = f2bf(first_part(h));
        bf16_t* const o =
            P.s + static_cast<int64_t>(slot) * 2 * P.f + tile * kRows + row;
        o[0] = hi;
        o[P.f] = f2bf(h - bf2f(hi));
      }
    }
    ag = au = f32x4{};
  };
  int tile = t0, c = 0;
  for (int left = (t1 - t0) * rounds; left > 1; --left) {
    const Item cur = nxt;
    const bool last = c + 1 == rounds;
    const int now = tile;
    c = last ? 0 : c + 1;
    tile += last;
    load(nxt, tile, (c * kUpWaves + wave) * kChunkK);
    multiply(cur);
    if (last) finish(now);
  }
  multiply(nxt);
  finish(tile);
}

// All tiles of all reached experts in order, divided evenly over the
// workgroups (what the CUs hold at once, so that starting and finding the
// experts is paid once).  One token: 8 experts of 2048 x 1408, 92 MB, 20.6 us;
// 2 of 4096 x 14336, 470 MB, 73 us (6.4 TB/s).
template <bool NT>
__global__ __launch_bounds__(kUpThreads, 4) void few_up_kernel(FewParams P) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ __attribute__((aligned(16))) float red[2 * kUpWaves * 512];
  static_assert(sizeof(red) >= kChooseTokens * kMaxTopK * 8, "room for choices");
  Units U;
  find_units<kUpThreads>(
      P, choose_here<kUpThreads>(P, reinterpret_cast<uint8_t*>(red)), lds, &U);
  const int tiles = P.f / kRows;
  const int total = U.count * tiles;
  const int groups = gridDim.x, me = blockIdx.x;
  const int per = total / groups, more = total - per * groups;
  int at = me * per + min(me, more);
  const int end = at + per + (me < more);
  int flip = 0;
  while (at < end) {
    const int un = at / tiles;
    const int t0 = at - un * tiles, t1 = min(tiles, t0 + end - at);
    up_tiles<NT>(P, U, un, t0, t1, red, &flip);
    at += t1 - t0;
  }
}

// ------------------------------------------------------------------- batch
// More tokens.  The waves of a workgroup own rows and go through the same k
// in step: the tokens' k (x, or S) are staged in LDS once for all of them,
// and a wave holds the sums of its two 8-row tiles whole, so nothing is added
// across waves.  Tokens stand in blocks of eight columns.
//
// kAhead steps of kStepK k are in flight, 16 KB a wave and 128 KB a CU; twice
// as many are no faster, since a CU's rate stops at 25 GB/s for every count of
// CUs at work (64 workgroups on 64 CUs take four times as long as 256 on
// 256).  The columns of step s + 2 are requested before the weights of step
// s + kAhead, since loads return in order and waiting for the columns must not
// wait for those.
//
// First product: two workgroups of four waves a CU.  One of eight waves is
// faster where all experts are large and 5% slower where they are many (24
// tokens, 64 experts of 2048 x 1408 62 against 64 us; 64 tokens, 8 of 4096 x
// 14336 306 against 300).  Second product: one of eight waves, for S's columns
// are as many bytes as the weights and 128 rows share them (64 tokens, 8 of
// 4096 x 14336 192 -> 169 us; 24 tokens, 64 of 2048 x 1408 in MXFP8 42 -> 40).
constexpr int kUpBatchThreads = 256;
constexpr int kUpBatchWaves = kUpBatchThreads / kWave;
constexpr int kUpBatchRows = kUpBatchWaves * kRows;
constexpr int kDownBatchThreads = 512;
constexpr int kDownBatchWaves = kDownBatchThreads / kWave;
constexpr int kBatchRows = kDownBatchWaves * 2 * kRows;

// Fewer k a step, and more steps in flight, keep the columns of many blocks
// within 16 KB a buffer: with 32 KB for eight blocks a CU held one workgroup
// (61 tokens, 41 experts of 1032 x 680: the second product 30 us).
template <bool MX, int NB>
struct BatchShape {
  static constexpr int kStepK =
      MX ? (NB <= 2 ? 512 : NB == 4 ? 256 : 128) : (NB <= 4 ? 256 : 128);
  static constexpr int kAhead = kStepK == (MX ? 512 : 256) ? 2 : 4;
  static constexpr int kPieces = kStepK / 8;            // of 16 bytes a column
  static constexpr int kColumns = NB * 8 * kPieces;     // pieces of a step
  static constexpr int kBytes = NB * 8 * kPieces * 16;  // of a buffer
};
// the most of them up to `blocks`
template <bool MX>
constexpr int batch_bytes(int blocks) {
  return MX ? 8192 * (blocks < 2 ? blocks : 2)
            : 4096 * (blocks < 4 ? blocks : 4);
}

// The columns' k in LDS: 16-byte piece p of column c lies at p ^ swizzle(c),
// so that the sixteen lanes of a fragment read that share a cycle (8 columns
// x 2 pieces, 4 (bf16) or 8 apart) meet every bank once.
template <bool MX>
__device__ __forceinline__ int swizzle(int c) {
  return MX ? c : (c & 3) | ((c & 4) << 1);
}

// Where a batch stands: step (expert, group of rows, round of k), one for the
// columns, one for the weights and one for the sums.
struct Cursor {
  int left, un, mid, r;               // left: steps from here on
  Reached X;
  __device__ __forceinline__ Cursor(const Units& U, int begin, int end,
                                    int mids, int rounds)
      : left(end - begin) {
    const int t = begin / rounds;
    r = begin - t * rounds;
    un = t / mids;
    mid = t - un * mids;
    X.read(U, un);
  }
  // true where another expert begins
  __device__ __forceinline__ bool next(const Units& U, int mids, int rounds) {
    --left;
    if (++r < rounds) return false;
    r = 0;
    if (++mid < mids) return false;
    mid = 0;
    ++un;
    if (left <= 0) return false;
    X.read(U, un);
    return true;
  }
};

// Steps [begin, end) of a Source, which says what a step reads and what
// becomes of the sums:
//   weights(cursor, a, b): loads the wave's two tiles
//   column(cursor, c, b): byte offset of column c of block b in rx, kOob for
//     none; K: the columns' length
//   done(cursor, a, b): called at every step; true clears the sums
template <bool MX, bool NT, int NB, class Source>
__device__ __forceinline__ void batch(Source& src, const Units& U, int begin,
                                      int end, uint8_t* xs) {
  using H = BatchShape<MX, NB>;
  constexpr int D = H::kAhead;
  constexpr int kThreads = Source::kThreads;
  // columns' pieces of a thread; a small step leaves some threads none
  constexpr int kLoads =
      H::kColumns < kThreads ? 1 : H::kColumns / kThreads;
  static_assert(H::kColumns % kThreads == 0 || H::kColumns < kThreads,
                "whole loads");
  static_assert(D % 2 == 0, "the LDS buffer is a compile-time constant");
  const Lane<MX> L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int fr = lane & 15, g = lane >> 4, col = fr & 7;
  struct Columns {
    i32x4 v[kLoads];
  };
  Columns cx[2];
  Weights<MX, NT, H::kStepK> wa[D], wb[D];
  Cursor at_x(U, begin, end, src.mids, src.rounds), at_w = at_x, at = at_x;
  // piece i of the thread: 16 bytes of column `col_of(i)` (8 a block)
  auto col_of = [&](int i) { return (tid + i * kThreads) / H::kPieces; };
  auto piece_of = [&](int i) { return (tid + i * kThreads) % H::kPieces; };
  // byte offsets of the thread's pieces at k = 0, which change with the
  // expert; kOob: none
  uint32_t from[kLoads];
  const bool has_column = H::kColumns >= kThreads || tid < H::kColumns;
  auto find_columns = [&]() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      from[i] = has_column ? src.column(at_x, col_of(i) & 7, col_of(i) >> 3)
                           : kOob;
  };
  find_columns();
  auto load_columns = [&](Columns& x) {
    const int k0 = at_x.left > 0 ? at_x.r * H::kStepK : src.K;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = k0 + piece_of(i) * 8;
      x.v[i] = buf_load16(src.rx, k < src.K && from[i] != kOob
                                      ? from[i] + static_cast<uint32_t>(k) * 2
                                      : kOob);
    }
    if (at_x.next(U, src.mids, src.rounds)) find_columns();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_weights = [&](int u) {
    src.weights(at_w, wa[u], wb[u]);
    at_w.next(U, src.mids, src.rounds);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto store_columns = [&](const Columns& x, uint8_t* to) {
    if (!has_column) return;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = col_of(i);
      *reinterpret_cast<i32x4*>(
          to + (c * H::kPieces + (piece_of(i) ^ swizzle<MX>(c & 7))) * 16) =
          x.v[i];
    }
  };
  // byte offset of fragment i of the lane's column of a block
  auto piece = [&](int i) {
    const int p = MX ? (i >> 1) * 16 + (fr >> 3) * 8 + g * 2 + (i & 1)
                     : i * 8 + (fr >> 3) * 4 + g;
    return (col * H::kPieces + (p ^ swizzle<MX>(col))) * 16;
  };
  load_columns(cx[0]);
  load_columns(cx[1]);
#pragma unroll
  for (int i = 0; i < D; ++i) load_weights(i);
  store_columns(cx[0], xs);
  __syncthreads();
  f32x4 a[NB], b[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) a[i] = b[i] = f32x4{};
  // D steps; the last of a batch (kMore false) request nothing
  auto steps = [&](auto more) {
    constexpr bool kMore = decltype(more)::value;
#pragma unroll
    for (int u = 0; u < D; ++u) {
      uint8_t* const now = xs + (u & 1) * H::kBytes;
      uint8_t* const then = xs + ((u & 1) ^ 1) * H::kBytes;
      if (kMore || u + 2 < D) load_columns(cx[u & 1]);
#pragma unroll
      for (int i = 0; i < H::kStepK / 64; ++i) {
        const bf16x8_v fa = wa[u].frag(i, L), fb = wb[u].frag(i, L);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const bf16x8_v x = __builtin_bit_cast(
              bf16x8_v, *reinterpret_cast<const i32x4*>(
                            now + n * 8 * H::kPieces * 16 + piece(i)));
          a[n] = mma(fa, x, a[n]);
          b[n] = mma(fb, x, b[n]);
        }
      }
      if (kMore) load_weights(u);
      if (at.left > 0 && src.done(at, a, b))
#pragma unroll
        for (int i = 0; i < NB; ++i) a[i] = b[i] = f32x4{};
      at.next(U, src.mids, src.rounds);
      if (kMore || u + 1 < D) {
        // the other buffer: its last reads were before the last barrier
        store_columns(cx[(u & 1) ^ 1], then);
        __syncthreads();
      }
    }
  };
  for (int q = begin; q + D < end; q += D) steps(std::true_type{});
  steps(std::false_type{});
}

// Adds the two halves of k: rows 0-7 with columns 0-7 (lanes below 32 of
// columns 0-7, where the sum is left) and rows 8-15 with columns 8-15, by a
// rotation of each 16 lanes by 8 and an exchange of the wave's halves.
__device__ __forceinline__ f32x4 join_halves(f32x4 v) {
  constexpr int kDppRor8 = 0x128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = __float_as_uint(dpp_move<kDppRor8>(v[i]));
    const auto s = __builtin_amdgcn_permlane32_swap(t, t, false, false);
    v[i] += __uint_as_float(s[1]);
  }
  return v;
}

// Gate and up: steps are (expert, group of 32 rows each, k), a wave's tiles
// its gate and its up rows.
template <bool MX, bool NT, int NB>
struct UpSource {
  static constexpr int kThreads = kUpBatchThreads;
  using H = BatchShape<MX, NB>;
  const FewParams& P;
  const Units& U;
  __amdgpu_buffer_rsrc_t rx;
  int K, rounds, mids, wave;
  Lane<MX> L;

  __device__ __forceinline__ UpSource(const FewParams& p, const Units& u)
      : P(p), U(u),
        rx(make_rsrc(p.x, static_cast<uint32_t>(p.T) * p.d * 2)), K(p.d),
        rounds((p.d + H::kStepK - 1) / H::kStepK),
        mids((p.f + kUpBatchRows - 1) / kUpBatchRows),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {}
  __device__ __forceinline__ uint32_t column(const Cursor& at, int c,
                                             int b) const {
    const int m = b * 8 + c;
    return m < at.X.members
               ? static_cast<uint32_t>(P.token(U.slot[at.X.first + m])) * K * 2
               : kOob;
  }
  __device__ __forceinline__ void weights(const Cursor& at,
                                          Weights<MX, NT, H::kStepK>& a,
                                          Weights<MX, NT, H::kStepK>& b) const {
    const UpWeights<MX> W(P, at.X.id);
    const int n = (at.mid * kUpBatchWaves + wave) * kRows;
    const int k0 = at.left > 0 && n < P.f ? at.r * H::kStepK : K;
    a.load(W.rw, W.rs, W.row(P, n + L.r, false), k0, K, L);
    b.load(W.rw, W.rs, W.row(P, n + L.r, true), k0, K, L);
  }
  __device__ __forceinline__ bool done(const Cursor& at, const f32x4* a,
                                       const f32x4* b) const {
    if (at.r + 1 < rounds) return false;
    const int lane = lane_id(), c = lane & 15, qr = lane >> 4;
    const int n = (at.mid * kUpBatchWaves + wave) * kRows;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (i * 8 >= at.X.members) break;
      const f32x4 ga = join_halves(a[i]), up = join_halves(b[i]);
      const int m = i * 8 + c;
      if (c >= 8 || qr >= 2 || m >= at.X.members || n >= P.f) continue;
      const int slot = U.slot[at.X.first + m];
      const float wt = U.wt[slot];
      float h[4], l[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float S = swiglu(ga[v], up[v], wt);
        h[v] = first_part(S);
        l[v] = S - bf2f(f2bf(h[v]));
      }
      bf16_t* const o =
          P.s + static_cast<int64_t>(slot) * 2 * P.f + n + qr * 4;
      *reinterpret_cast<i32x2*>(o) =
          i32x2{static_cast<int>(pack_bf16x2(h[0], h[1])),
                static_cast<int>(pack_bf16x2(h[2], h[3]))};
      *reinterpret_cast<i32x2*>(o + P.f) =
          i32x2{static_cast<int>(pack_bf16x2(l[0], l[1])),
                static_cast<int>(pack_bf16x2(l[2], l[3]))};
    }
    return true;
  }
};

// The largest number of members of the experts [u0, u1).
__device__ __forceinline__ int most_members(const Units& U, int u0, int u1) {
  int most = 0;
  for (int u = u0 + lane_id(); u < u1; u += kWave)
    most = max(most, static_cast<int>(U.expert[u].members));
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) most = max(most, shfl_xor(most, m));
  return __builtin_amdgcn_readfirstlane(most);
}

template <bool MX, bool NT, int NB>
__device__ __forceinline__ void up_batch(const FewParams& P, const Units& U,
                                         int first, int last, uint8_t* xs) {
  UpSource<MX, NT, NB> src(P, U);
  batch<MX, NT, NB>(src, U, first * src.rounds, last * src.rounds, xs);
}

// MAXB: blocks of 8 that T tokens can fill.  24 tokens, 64 experts of 2048 x
// 1408 in MXFP8, 358 MB: 63 us (5.7 TB/s); 64 tokens, 8 of 4096 x 14336 in
// bf16, 1.88 GB: 305 us (6.2 TB/s).  What is left: 2 us until the experts are
// found, 5 to 15 until the first weights come, and workgroups that have 6
// groups of rows where others have 5.
template <bool MX, bool NT, int MAXB>
__global__ __launch_bounds__(kUpBatchThreads, 2) void few_up_batch_kernel(
    FewParams P) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  Units U;
  uint8_t* const xs = lds + Units::bytes(P.E, P.T * P.k);
  static_assert(2 * 4096 >= kChooseTokens * kMaxTopK * 8, "room for choices");
  find_units<kUpBatchThreads>(P, choose_here<kUpBatchThreads>(P, xs), lds, &U);
  const int groups = (P.f + kUpBatchRows - 1) / kUpBatchRows;
  const int total = U.count * groups;
  const int n = gridDim.x, me = blockIdx.x;
  const int per = total / n, more = total - per * n;
  const int first = me * per + min(me, more);
  const int last = first + per + (me < more);
  if (first >= last) return;
  const int most = most_members(U, first / groups, (last - 1) / groups + 1);
  if (MAXB == 1 || most <= 8)
    up_batch<MX, NT, 1>(P, U, first, last, xs);
  else if (MAXB == 2 || most <= 16)
    up_batch<MX, NT, MAXB >= 2 ? 2 : 1>(P, U, first, last, xs);
  else if (MAXB == 4 || most <= 32)
    up_batch<MX, NT, MAXB >= 4 ? 4 : 1>(P, U, first, last, xs);
  else
    up_batch<MX, NT, MAXB >= 8 ? 8 : 1>(P, U, first, last, xs);
}

// Down: steps are (expert, k), a wave's tiles 16 rows of y.  A block holds
// four members, each as two columns, S's larger and smaller part; members
// past what NB blocks hold are left to further passes.
template <bool MX, bool NT, int NB>
struct DownSource {
  static constexpr int kThreads = kDownBatchThreads;
  using H = BatchShape<MX, NB>;
  const FewParams& P;
  const Units& U;
  __amdgpu_buffer_rsrc_t rx;
  int K, rounds, mids, n0, skip;      // skip: members of earlier passes
  float* plane;                       // [T][16], the wave's
  Lane<MX> L;

  __device__ __forceinline__ DownSource(const FewParams& p, const Units& u,
                                        int rows, int row0, int members,
                                        float* sums)
      : P(p), U(u),
        rx(make_rsrc(p.s, static_cast<uint32_t>(p.T) * p.k * 4 * p.f)),
        K(p.f), rounds(rows), mids(1), n0(row0), skip(members), plane(sums) {}
  __device__ __forceinline__ uint32_t column(const Cursor& at, int c,
                                             int b) const {
    const int m = skip + b * 4 + (c >> 1);
    return m < at.X.members
               ? (static_cast<uint32_t>(U.slot[at.X.first + m]) * 2 +
                  (c & 1)) * K * 2
               : kOob;
  }
  __device__ __forceinline__ void weights(const Cursor& at,
                                          Weights<MX, NT, H::kStepK>& a,
                                          Weights<MX, NT, H::kStepK>& b) const {
    // an expert without members in this pass is not read
    const bool in = at.left > 0 && n0 < P.d && skip < at.X.members;
    const int64_t o = (at.X.id * static_cast<int64_t>(P.d) + (in ? n0 : 0)) *
                      K;
    const uint32_t rows = static_cast<uint32_t>(in ? min(16, P.d - n0) : 0);
    const auto rw = make_rsrc(P.w2 + o * (MX ? 1 : 2),
                              rows * K * (MX ? 1 : 2));
    const auto rs =
        MX ? make_rsrc(P.w2_scales + o / 32, rows * K / 32) : rw;
    const uint32_t row = static_cast<uint32_t>(L.r) * K * (MX ? 1 : 2);
    const int k0 = in ? at.r * H::kStepK : K;
    a.load(rw, rs, row, k0, K, L);
    b.load(rw, rs, row + static_cast<uint32_t>(kRows) * K * (MX ? 1 : 2),
           rows > kRows ? k0 : K, K, L);
  }
  __device__ __forceinline__ bool done(const Cursor& at, const f32x4* a,
                                       const f32x4* b) const {
    if (at.r + 1 < rounds && at.left > 1) return false;
    const int lane = lane_id(), c = lane & 15, qr = lane >> 4;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (skip + i * 4 >= at.X.members) break;
      f32x4 s0 = join_halves(a[i]), s1 = join_halves(b[i]);
      // S's two parts stand in neighbouring columns
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        s0[v] += dpp_move<kDppXor1>(s0[v]);
        s1[v] += dpp_move<kDppXor1>(s1[v]);
      }
      const int m = skip + i * 4 + (c >> 1);
      if (c >= 8 || (c & 1) || qr >= 2 || m >= at.X.members) continue;
      f32x4* const o = reinterpret_cast<f32x4*>(
          plane + P.token(U.slot[at.X.first + m]) * 16 + qr * 4);
      o[0] += s0;
      o[2] += s1;
    }
    return true;
  }
};

// Pieces of kPartK k of the experts' reductions, [begin, end) of them; a unit
// that does not depend on NB, so that neighbouring parts meet.
template <bool MX>
constexpr int kPartK = MX ? 512 : 256;

// Experts of more than the 4 NB members that the columns hold, NB 8 at most,
// are read again for the others (64 tokens of one expert of 4096 x 14336 in
// bf16 123 us for the layer, 32 tokens 86; of two, all chosen, 216 and 150).
template <bool MX, bool NT, int NB>
__device__ __forceinline__ void down_batch(const FewParams& P, const Units& U,
                                           int begin, int end, int most,
                                           int n0, float* plane,
                                           uint8_t* xs) {
  constexpr int kSteps = kPartK<MX> / BatchShape<MX, NB>::kStepK;
  const int rounds = (P.f + kPartK<MX> - 1) / kPartK<MX> * kSteps;
  for (int skip = 0; skip < most; skip += 4 * NB) {
    if (skip) __syncthreads();        // xs is free again
    DownSource<MX, NT, NB> src(P, U, rounds, n0, skip, plane);
    batch<MX, NT, NB>(src, U, begin * kSteps, end * kSteps, xs);
  }
}

// MAXB: blocks of 4 members that T tokens can fill, up to 8.  24 tokens, 64
// experts of 2048 x 1408 in MXFP8, 181 MB: 41 us; 64 tokens, 8 of 4096 x 14336
// in bf16, 0.94 GB: 168 us.
template <bool MX, bool NT, int MAXB>
__global__ __launch_bounds__(kDownBatchThreads, 2) void few_down_batch_kernel(
    FewParams P) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, T = P.T;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = blockIdx.x / P.parts, part = blockIdx.x - group * P.parts;
  float* const planes =
      reinterpret_cast<float*>(lds + Units::bytes(P.E, T * P.k));
  for (int i = tid; i < kDownBatchWaves * T * 16; i += kDownBatchThreads)
    planes[i] = 0;
  Units U;
  find_units<kDownBatchThreads>(P, Choices{P.idx, P.wt}, lds, &U);
  float* const plane = planes + wave * T * 16;
  uint8_t* const xs =
      reinterpret_cast<uint8_t*>(planes + kDownBatchWaves * T * 16);
  const int n0 = group * kBatchRows + wave * 16;
  const int pieces = (P.f + kPartK<MX> - 1) / kPartK<MX>;
  const int64_t total = static_cast<int64_t>(U.count) * pieces;
  const int begin = static_cast<int>(total * part / P.parts);
  const int end = static_cast<int>(total * (part + 1) / P.parts);
  if (begin < end) {
    const int most =
        most_members(U, begin / pieces, (end - 1) / pieces + 1);
    if (most <= 4)
      down_batch<MX, NT, 1>(P, U, begin, end, most, n0, plane, xs);
    else if (MAXB == 2 || most <= 8)
      down_batch<MX, NT, 2>(P, U, begin, end, most, n0, plane, xs);
    else if (MAXB == 4 || most <= 16)
      down_batch<MX, NT, MAXB >= 4 ? 4 : 2>(P, U, begin, end, most, n0, plane, xs);
    else
      down_batch<MX, NT, MAXB >= 8 ? 8 : 2>(P, U, begin, end, most, n0, plane, xs);
  }
  // the wave's own rows of the part's sums
  for (int i = lane; i < T * 4; i += kWave) {
    const int t = i >> 2, r = (i & 3) * 4;
    if (n0 + r < P.d)
      *reinterpret_cast<f32x4*>(
          P.part + (static_cast<int64_t>(part) * T + t) * P.d + n0 + r) =
          *reinterpret_cast<const f32x4*>(plane + t * 16 + r);
  }
}

// -------------------------------------------------------------------- down
// The direct form: the columns of a tile are the tokens, each as two, S's
// larger and smaller part, and a wave's sums run over all experts.  One token,
// 8 experts of 2048 x 1408, 46 MB: 10.0 us.
constexpr int kDownThreads = 1024;
constexpr int kDownWaves = kDownThreads / kWave;
constexpr int kAhead = 3;             // chunks of a wave in flight

// A workgroup of sixteen waves a CU goes through its tiles of y: (tile,
// expert, chunk) in order, dealt in turn to the waves, the next tile's loads
// in flight while one is added up.
template <bool MX, bool NT>
__global__ __launch_bounds__(kDownThreads, 4) void few_down_kernel(
    FewParams P) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ __attribute__((aligned(16))) float red[2 * kDownWaves * 256];
  const Lane<MX> L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = blockIdx.x / P.parts, part = blockIdx.x - group * P.parts;
  const int groups = gridDim.x / P.parts, tiles = P.d / kRows;
  const int K = P.f, T = P.T;
  Units U;
  find_units<kDownThreads>(P, Choices{P.idx, P.wt}, lds, &U);
  const int chunks = (K + kChunkK - 1) / kChunkK;      // of an expert
  const int total = U.count * chunks;
  const auto rx = make_rsrc(P.s, static_cast<uint32_t>(T) * P.k * 2 * K * 2);
  const int64_t per = static_cast<int64_t>(P.d) * K;
  const uint32_t row = static_cast<uint32_t>(L.r) * K * (MX ? 1 : 2);
  const int t = L.r >> 1;              // the token of the lane's column

  struct Item {
    Weights<MX, NT> w;
    Tokens<MX> x;
    bool has;                         // the lane's token, this expert
  };
  // items of a tile are dealt in turn to the waves of all parts; a wave makes
  // `rounds` of them, the last one masked where there are fewer
  const int step = kDownWaves * P.parts;
  const int rounds = (total + step - 1) / step;
  int l_tile = group, l_left = rounds, l_q = part * kDownWaves + wave;
  auto load = [&](Item& it) {
    const bool in = l_q < total && l_tile < tiles;
    const int un = in ? l_q / chunks : 0;
    const int k0 = in ? (l_q - un * chunks) * kChunkK : K;
    Reached X;
    X.read(U, un);
    const int64_t at =
        X.id * per + static_cast<int64_t>(in ? l_tile * kRows : 0) * K;
    const auto rw = make_rsrc(
        P.w2 + at * (MX ? 1 : 2),
        static_cast<uint32_t>(kRows) * K * (MX ? 1 : 2));
    const auto rs = MX ? make_rsrc(P.w2_scales + at / 32,
                                   static_cast<uint32_t>(kRows) * K / 32)
                       : rw;
    it.w.load(rw, rs, row, k0, K, L);
    const bool has = (X.tokens >> t) & 1;
    it.has = has;
    const int sl = U.slot[X.first +
                          (has ? __popc(X.tokens & ((1 << t) - 1)) : 0)];
    it.x.load(rx,
              has ? static_cast<uint32_t>(sl * 2 + (L.r & 1)) * K * 2 : kOob,
              k0, K, L);
    l_q += step;
    if (--l_left == 0) {
      l_left = rounds;
      l_q = part * kDownWaves + wave;
      l_tile += groups;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  Item it[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(it[i]);
  f32x4 acc = {};
  int flip = 0;
  auto finish = [&](int tile) {
    float* const r = red + flip * (kDownWaves * 256);
    *reinterpret_cast<f32x4*>(r + (wave * 64 + lane) * 4) = acc;
    __syncthreads();
    // as in up_tiles a buffer is free again after the next barrier
    if (wave == flip) {
      const int n = lane & 7, c = lane >> 3;
      // the two halves of k: rows and columns 0-7, and 8-15
      const int o1 = ((n >> 2) * 16 + c) * 4 + (n & 3);
      const int o2 = (((n >> 2) + 2) * 16 + c + 8) * 4 + (n & 3);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w)
        v += r[w * 256 + o1] + r[w * 256 + o2];
      v += shfl_xor(v, 8);              // S's two parts
      if (!(c & 1) && (c >> 1) < T) {
        const int64_t o = static_cast<int64_t>(c >> 1) * P.d + tile * kRows +
                          n;
        if (P.parts > 1) {
          P.part[static_cast<int64_t>(part) * T * P.d + o] = v;
        } else {
          if (P.y_add) v += bf2f(P.y_add[o]);
          P.y[o] = f2bf(v);
        }
      }
    }
    flip ^= 1;
    acc = f32x4{};
  };
  // Columns of tokens that are not the expert's are left out: 0 times one of
  // its infinities or NaN is no 0.
  auto multiply = [&](const Item& i) {
    f32x4 sum = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) sum = mma(i.w.frag(s, L), i.x.frag(s), sum);
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += i.has ? sum[v] : 0.0f;
  };
  int tile = group, c = 0;
  auto one = [&](const Item& i) {
    multiply(i);
    if (++c < rounds) return;
    finish(tile);
    tile += groups;
    c = 0;
  };
  // kAhead items a time; the last are taken out of the loop, as in up_tiles
  int left = (tiles - group + groups - 1) / groups * rounds;
  for (; left > kAhead; left -= kAhead)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      one(it[i]);
      load(it[i]);
    }
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < left) one(it[i]);
}

// y = y_add + the parts; n values, a multiple of 8.  4.7 us, as for any kernel
// that waits for memory once after a large one.  Four lanes share four
// values, each with every fourth part.
__global__ __launch_bounds__(256) void few_sum_kernel(
    const float* __restrict__ part, int parts, int64_t n, const bf16_t* y_add,
    bf16_t* y) {
  const int lane = threadIdx.x & 63, share = lane >> 4;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 4 +
                     (threadIdx.x >> 6)) * 64 + (lane & 15) * 4;
  if (i >= n) return;                 // all four lanes of a value
  i32x2 a = {};
  if (y_add) a = *reinterpret_cast<const i32x2*>(y_add + i);
  f32x4 v = {};
#pragma unroll 4
  for (int p = share; p < parts; p += 4)
    v += *reinterpret_cast<const f32x4*>(part + p * n + i);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] += shfl_xor(v[q], 16);
    v[q] += shfl_xor(v[q], 32);
  }
  if (share) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    v[2 * q] += bf_lo(static_cast<uint32_t>(a[q]));
    v[2 * q + 1] += bf_hi(static_cast<uint32_t>(a[q]));
  }
  *reinterpret_cast<i32x2*>(y + i) =
      i32x2{static_cast<int>(pack_bf16x2(v[0], v[1])),
            static_cast<int>(pack_bf16x2(v[2], v[3]))};
}

// ---------------------------------------------------------------- launches
// Experts that T tokens can reach.
int most_units(int T, int k, int E) { return T * k < E ? T * k : E; }

// Whether a product of T tokens takes its direct form.
bool direct_up(bool mx, int T) { return !mx && T <= kDirectUp; }
bool direct_down(int64_t T, int k, int E, int64_t d, int64_t f) {
  return T <= kDirectDown &&
         most_units(static_cast<int>(T), k, E) * d * f <= kDirectValues;
}

template <bool NT>
hipError_t launch_up(const FewParams& P, hipStream_t s) {
  // four workgroups a CU, or fewer where the tiles cannot be more
  const int64_t most =
      static_cast<int64_t>(most_units(P.T, P.k, P.E)) * (P.f / kRows);
  hipLaunchKernelGGL(few_up_kernel<NT>,
                     dim3(static_cast<uint32_t>(most < 1024 ? most : 1024)),
                     dim3(kUpThreads), Units::bytes(P.E, P.T * P.k), s, P);
  return hipGetLastError();
}

template <bool MX, bool NT, int MAXB>
hipError_t launch_up_batch(const FewParams& P, hipStream_t s) {
  // two workgroups a CU, or fewer where the groups cannot be more
  const int64_t most = static_cast<int64_t>(most_units(P.T, P.k, P.E)) *
                       ((P.f + kUpBatchRows - 1) / kUpBatchRows);
  hipLaunchKernelGGL(
      (few_up_batch_kernel<MX, NT, MAXB>),
      dim3(static_cast<uint32_t>(most < 512 ? most : 512)),
      dim3(kUpBatchThreads),
      Units::bytes(P.E, P.T * P.k) + 2 * batch_bytes<MX>(MAXB), s, P);
  return hipGetLastError();
}

template <bool MX, bool NT>
hipError_t launch_first(const FewParams& P, hipStream_t s) {
  if constexpr (!MX)
    if (direct_up(MX, P.T)) return launch_up<NT>(P, s);
  if constexpr (MX)
    if (P.T <= 8) return launch_up_batch<MX, NT, 1>(P, s);
  return P.T <= 16   ? launch_up_batch<MX, NT, 2>(P, s)
         : P.T <= 32 ? launch_up_batch<MX, NT, 4>(P, s)
                     : launch_up_batch<MX, NT, 8>(P, s);
}

template <bool MX, bool NT, int MAXB>
hipError_t launch_down_batch(const FewParams& P, hipStream_t s) {
  const uint32_t groups = (P.d + kBatchRows - 1) / kBatchRows;
  hipLaunchKernelGGL(
      (few_down_batch_kernel<MX, NT, MAXB>), dim3(groups * P.parts),
      dim3(kDownBatchThreads),
      Units::bytes(P.E, P.T * P.k) + kDownBatchWaves * P.T * 64 +
          2 * batch_bytes<MX>(MAXB),
      s, P);
  return hipGetLastError();
}

template <bool MX, bool NT>
hipError_t launch_second(const FewParams& P, hipStream_t s) {
  if (direct_down(P.T, P.k, P.E, P.d, P.f)) {
    const uint32_t tiles = P.d / kRows;
    hipLaunchKernelGGL((few_down_kernel<MX, NT>),
                       dim3((tiles < 256 ? tiles : 256) * P.parts),
                       dim3(kDownThreads), Units::bytes(P.E, P.T * P.k), s, P);
    return hipGetLastError();
  }
  return P.T <= 8    ? launch_down_batch<MX, NT, 2>(P, s)
         : P.T <= 16 ? launch_down_batch<MX, NT, 4>(P, s)
                     : launch_down_batch<MX, NT, 8>(P, s);
}

template <bool MX>
hipError_t launch_few(const FewParams& P, hipStream_t s) {
  // rows of whole 128-byte lines
  hipError_t e = MX || P.d % 64 == 0 ? launch_first<MX, true>(P, s)
                                     : launch_first<MX, MX>(P, s);
  if (e != hipSuccess) return e;
  e = MX || P.f % 64 == 0 ? launch_second<MX, true>(P, s)
                          : launch_second<MX, MX>(P, s);
  if (e != hipSuccess || P.parts == 1) return e;
  const int64_t n = static_cast<int64_t>(P.T) * P.d;
  hipLaunchKernelGGL(few_sum_kernel,
                     dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256),
                     0, s, P.part, P.parts, n, P.y_add, P.y);
  return hipGetLastError();
}

// Parts that the reduction of y is cut into.  The direct form: so that all
// CUs have work, but a round of the waves at least.  The batch form always
// leaves its sums to few_sum_kernel: one workgroup a CU, a step each at least
// (34 tokens, 11 experts of 1664 x 160: 11 parts 11.7 us, 5 parts 18.6, 2
// parts 27; 61 tokens, 41 experts of 1032 x 680: 28 parts 20.5, 8 parts 26),
// and up to kMaxParts, past which few_sum_kernel takes what the product gains
// (11 tokens, 111 experts of 512 x 2688 in MXFP8: 64 parts 20 us, 32 30).
constexpr int kMaxParts = 64;
int down_parts(int64_t T, int k, int E, int64_t d, int64_t f) {
  const int64_t most = most_units(static_cast<int>(T), k, E);
  if (direct_down(T, k, E, d, f)) {
    const int64_t items = most * ((f + kChunkK - 1) / kChunkK);
    int parts = 1;
    while (parts < 8 && d / kRows * parts * 2 <= 256 &&
           items >= parts * 2 * kDownWaves)
      parts *= 2;
    return parts;
  }
  const int64_t steps = most * ((f + 255) / 256);
  const int64_t groups = (d + kBatchRows - 1) / kBatchRows;
  int64_t parts = 256 / groups < steps ? 256 / groups : steps;
  parts = parts < kMaxParts ? parts : kMaxParts;
  return static_cast<int>(parts > 2 ? parts : 2);
}

// Workspace: S, the parts' sums, the scores.
struct FewLayout {
  int parts;
  size_t part, logits, total;
};
size_t up256(size_t v) { return (v + 255) & ~size_t{255}; }
FewLayout few_layout(int64_t T, int k, int E, int64_t d, int64_t f) {
  FewLayout w;
  w.parts = down_parts(T, k, E, d, f);
  w.part = up256(static_cast<size_t>(T * k * f * 4));
  w.logits = w.part + up256(static_cast<size_t>(
                          w.parts > 1 ? w.parts * T * d * 4 : 0));
  w.total = w.logits + up256(static_cast<size_t>(T * E * 4));
  return w;
}

}  // namespace

size_t layer_fwd_workspace(int64_t T, int k, int E, int64_t d, int64_t f) {
  return few_layout(T, k, E, d, f).total;
}

hipError_t launch_layer_fwd(bool mx, const LayerArgs& a, void* ws,
                            hipStream_t s) {
  const FewLayout w = few_layout(a.T, a.k, a.E, a.d, a.f);
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
  P.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.part);
  P.T = a.T;
  P.d = a.d;
  P.f = a.f;
  P.E = a.E;
  P.k = a.k;
  P.parts = w.parts;
  P.renorm = a.renorm;
  P.inv_k = (65536 + a.k - 1) / a.k;
  const bool here = a.T <= kChooseTokens && a.E <= kWave * kChooseLanes;
  const float* logits = a.logits;
  if (!logits && (here || a.E > kRouteWaves)) {
    float* const z = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                              w.logits);
    hipLaunchKernelGGL(few_logits_kernel,
                       dim3((a.E + kLogitWaves - 1) / kLogitWaves, a.T),
                       dim3(kLogitThreads), 0, s, a.x, a.w_g, a.bias, a.d, a.E,
                       z);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    logits = z;
  }
  if (here) {
    P.logits = logits;
  } else {
    hipLaunchKernelGGL(few_topk_kernel, dim3(a.T), dim3(kRouteThreads), 0, s,
                       logits, a.x, a.w_g, a.bias, a.d, a.E, a.k, a.renorm,
                       a.topk_idx, a.topk_w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return mx ? launch_few<true>(P, s) : launch_few<false>(P, s);
}

}  // namespace moe
