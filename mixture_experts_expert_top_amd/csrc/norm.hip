// Layer norm and RMS norm, forward and backward, one row per token.
//
//   mean = sum_i x_i / d                      (layer norm; 0 for RMS norm)
//   rstd = 1 / sqrt(sum_i (x_i - mean)^2 / d + eps)
//   y    = (x - mean) rstd gamma + beta
// and with xh = (x - mean) rstd, g = dy gamma:
//   dx     = dres + rstd (g - mean(g) - xh mean(g xh))   (RMS: no mean(g))
//   dgamma = sum_t dy xh,   dbeta = sum_t dy
//
// Both passes are bound by memory: the forward moves x and y once, the
// backward x, dy, dres and dx once.  A row is held in registers by the
// lanes that own its columns (8 columns a 16-byte chunk, at most two chunks
// a lane, so up to 16384 columns by 16 waves): the variance is summed from
// centred values, and nothing is read twice.  Every lane keeps its columns
// for all rows its workgroup takes, so gamma and beta are read once a
// workgroup and the weight gradients are summed in registers; the sums of
// the workgroups go to the workspace and a second kernel adds them in a
// fixed order (no atomics: equal inputs give equal bits).  The next row's
// loads are issued before the current row's sums are exchanged.
// Statistics, sums and weight gradients are fp32; y and a bf16 dx are
// rounded once.
//
// On MI355X, 8192 x 4096 bf16 RMS: forward 24.6 us (5.5 TB/s), backward 48.6
// (5.7 TB/s) and 4.7 us for the weight gradient's second kernel; 16384 x 2048
// fp32 layer norm: 38.4, 82.5 and 4.7 us (kernel times; as calls in a captured
// sequence over data that leaves the caches 27 and 57 us, 41 and 89 us).  A
// copy moves 5.1 TB/s.
//
// Above d = 8192 a row takes 16 waves, which leave a lane 128 registers, and
// the backward of layer norm with its two column sums spills: 35 registers
// for fp32, 4 for bf16; RMS norm none.  2048 x 16384, backward calls in a
// captured sequence: layer norm fp32 138 us (its bytes at a copy's rate are
// 92), bf16 72 (52); RMS norm fp32 98, bf16 61.

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// 8 consecutive values as loaded: one 16-byte piece of bf16, two of fp32.
template <typename XT>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  i32x4 v;
  __device__ __forceinline__ void load(const bf16_t* p) {
    v = *reinterpret_cast<const i32x4*>(p);
  }
  __device__ __forceinline__ void zero() { v = i32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = static_cast<uint32_t>(v[i >> 1]);
    return (i & 1) ? bf_hi(w) : bf_lo(w);
  }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void zero() {
    a = f32x4{0, 0, 0, 0};
    b = a;
  }
  __device__ __forceinline__ float at(int i) const {
    return i < 4 ? a[i] : b[i - 4];
  }
};

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

// How a row is spread: LPR lanes of each of NW waves, NV chunks a lane;
// a workgroup takes kRows rows at a time.
template <int LPR_, int NW_, int NV_>
struct Map {
  static constexpr int LPR = LPR_, NW = NW_, NV = NV_;
  static constexpr int kThreads = NW * 64 > 256 ? NW * 64 : 256;
  static constexpr int kRowLanes = NW * LPR;
  static constexpr int kRows = kThreads / kRowLanes;
  static_assert(NW == 1 || (LPR == 64 && kRows * NW * 64 == kThreads),
                "several waves share a row only whole");
};

// Sums of N values over the lanes of a row, the result in each of them.
// Rows that span waves go through red[2][waves][N]; `buf` alternates
// between calls, so that one barrier a call is enough: a wave that writes a
// buffer has passed the barrier of the call in between, which every wave
// reaches after its last read of that buffer.
template <class M, int N>
__device__ __forceinline__ void row_sums(float (&v)[N],
                                         float (*red)[M::kThreads / 64][N],
                                         int& buf) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = dpp_group_sum<16>(v[n]);
  if constexpr (M::LPR == 64) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] += __shfl_xor(v[n], 16, 64);
      v[n] += __shfl_xor(v[n], 32, 64);
    }
  }
  if constexpr (M::NW > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[buf][wave][n] = v[n];
    __syncthreads();
    const int w0 = wave / M::NW * M::NW;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = red[buf][w0][n];
#pragma unroll
      for (int w = 1; w < M::NW; ++w) s += red[buf][w0 + w][n];
      v[n] = s;
    }
    buf ^= 1;
  }
}

template <typename XT, bool LAYER, class M>
__global__ __launch_bounds__(M::kThreads) void norm_fwd_kernel(
    const XT* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, int64_t T, int d,
    bf16_t* __restrict__ y, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float red[2][M::kThreads / 64][1];
  const int grp = threadIdx.x / M::kRowLanes;
  const int li = threadIdx.x % M::kRowLanes;
  const int nc = d >> 3;
  const float inv_d = 1.0f / static_cast<float>(d);
  int buf = 0;

  bool cok[M::NV];
  float ga[M::NV][8], be[M::NV][8];
#pragma unroll
  for (int i = 0; i < M::NV; ++i) {
    const int c = i * M::kRowLanes + li;
    cok[i] = c < nc;
    Raw8<float> rg, rb;
    rg.zero();
    rb.zero();
    if (cok[i]) rg.load(gamma + c * 8);
    if (LAYER && beta && cok[i]) rb.load(beta + c * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ga[i][j] = rg.at(j);
      be[i][j] = rb.at(j);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * M::kRows;
  Raw8<XT> cur[M::NV], nxt[M::NV];
  auto load = [&](Raw8<XT>* r, int64_t row) {
#pragma unroll
    for (int i = 0; i < M::NV; ++i) {
      r[i].zero();
      if (cok[i] && row < T)
        r[i].load(x + row * d + (i * M::kRowLanes + li) * 8);
    }
  };
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * M::kRows;
  load(cur, row0 + grp);
  for (; row0 < T; row0 += step) {
    const int64_t row = row0 + grp;
    if (row0 + step < T) load(nxt, row + step);
    float mu = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < M::NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += cur[i].at(j);
      row_sums<M, 1>(s, red, buf);
      mu = s[0] * inv_d;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < M::NV; ++i)
      if (cok[i])
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = cur[i].at(j) - mu;
          q[0] = fmaf(c, c, q[0]);
        }
    row_sums<M, 1>(q, red, buf);
    // IEEE square root and division: rstd is the row's common factor
    const float r = 1.0f / sqrtf(q[0] * inv_d + eps);
    if (row < T) {
#pragma unroll
      for (int i = 0; i < M::NV; ++i)
        if (cok[i]) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = fmaf((cur[i].at(j) - mu) * r, ga[i][j], be[i][j]);
          store8(y + row * d + (i * M::kRowLanes + li) * 8, o);
        }
      if (li == 0) {
        if (LAYER && mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
      }
    }
#pragma unroll
    for (int i = 0; i < M::NV; ++i) cur[i] = nxt[i];
  }
}

// part: [gridDim.x][2][d] sums of this workgroup's rows (dgamma, dbeta);
// null when neither gradient is asked for.
template <typename XT, bool LAYER, class M>
__global__ __launch_bounds__(M::kThreads) void norm_bwd_kernel(
    const bf16_t* __restrict__ dy, const XT* __restrict__ x,
    const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const XT* dres, int64_t T, int d, XT* dx,
    float* __restrict__ part) {
  __shared__ float red[2][M::kThreads / 64][2];
  // rows taken side by side leave one sum each; they are joined in LDS
  constexpr int kCols = M::kRowLanes * M::NV * 8;
  constexpr bool kJoin = M::kRows > 1;
  __shared__ float join[kJoin ? M::kRows * kCols : 1];
  const int grp = threadIdx.x / M::kRowLanes;
  const int li = threadIdx.x % M::kRowLanes;
  const int nc = d >> 3;
  const float inv_d = 1.0f / static_cast<float>(d);
  int buf = 0;

  bool cok[M::NV];
  float ga[M::NV][8], dg[M::NV][8], db[M::NV][8];
#pragma unroll
  for (int i = 0; i < M::NV; ++i) {
    const int c = i * M::kRowLanes + li;
    cok[i] = c < nc;
    Raw8<float> rg;
    rg.zero();
    if (cok[i]) rg.load(gamma + c * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ga[i][j] = rg.at(j);
      dg[i][j] = 0.0f;
      db[i][j] = 0.0f;
    }
  }
  // the next row's loads in flight; 16 waves have no registers for it
  constexpr bool kAhead = M::NW < 16;
  struct Row {
    Raw8<XT> x[M::NV], r[M::NV];
    Raw8<bf16_t> dy[M::NV];
    float mu, rs;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * M::kRows;
  Row cur, nxt;
  auto load = [&](Row& w, int64_t row) {
    const bool rok = row < T;
    w.mu = (LAYER && rok) ? mean[row] : 0.0f;
    w.rs = rok ? rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < M::NV; ++i) {
      const int64_t o = row * d + (i * M::kRowLanes + li) * 8;
      w.x[i].zero();
      w.dy[i].zero();
      w.r[i].zero();
      if (cok[i] && rok) {
        w.x[i].load(x + o);
        w.dy[i].load(dy + o);
        if (dres) w.r[i].load(dres + o);
      }
    }
  };
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * M::kRows;
  if (kAhead) load(cur, row0 + grp);
  for (; row0 < T; row0 += step) {
    const int64_t row = row0 + grp;
    if (!kAhead) load(cur, row);
    else if (row0 + step < T) load(nxt, row + step);
    // dy of masked chunks and rows is 0, so they add nothing to the sums
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < M::NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (cur.x[i].at(j) - cur.mu) * cur.rs;
        const float v = cur.dy[i].at(j);
        const float g = v * ga[i][j];
        s[0] = fmaf(g, xh, s[0]);
        if (LAYER) s[1] += g;
        dg[i][j] = fmaf(v, xh, dg[i][j]);
        if (LAYER) db[i][j] += v;
      }
    if constexpr (LAYER) {
      row_sums<M, 2>(s, red, buf);
    } else {
      float s1[1] = {s[0]};
      row_sums<M, 1>(
          s1, reinterpret_cast<float(*)[M::kThreads / 64][1]>(red), buf);
      s[0] = s1[0];
    }
    const float c0 = s[0] * inv_d, c1 = LAYER ? s[1] * inv_d : 0.0f;
    if (row < T) {
#pragma unroll
      for (int i = 0; i < M::NV; ++i)
        if (cok[i]) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (cur.x[i].at(j) - cur.mu) * cur.rs;
            const float g = cur.dy[i].at(j) * ga[i][j];
            o[j] = fmaf(cur.rs, (g - c1) - xh * c0, cur.r[i].at(j));
          }
          store8(dx + row * d + (i * M::kRowLanes + li) * 8, o);
        }
    }
    if (kAhead) cur = nxt;
  }
  if (part == nullptr) return;
  float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
  for (int h = 0; h < (LAYER ? 2 : 1); ++h) {
    if constexpr (kJoin) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < M::NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          join[grp * kCols + (i * M::kRowLanes + li) * 8 + j] =
              h ? db[i][j] : dg[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += M::kThreads) {
        float sum = join[c];
#pragma unroll
        for (int r = 1; r < M::kRows; ++r) sum += join[r * kCols + c];
        pg[h * d + c] = sum;
      }
    } else {
#pragma unroll
      for (int i = 0; i < M::NV; ++i)
        if (cok[i])
          store8(pg + h * d + (i * M::kRowLanes + li) * 8,
                 h ? db[i] : dg[i]);
    }
  }
}

// Columns of dgamma (blockIdx.y 0) and dbeta (1): 64 columns a workgroup,
// 16 waves each adding every 16th partial, then the waves in order.
constexpr int kRedWaves = 16;
__global__ __launch_bounds__(64 * kRedWaves) void norm_wgrad_kernel(
    const float* __restrict__ part, int n, int d, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[kRedWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.y;
  float* out = h ? dbeta : dgamma;
  if (out == nullptr) return;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < d) {
    const float* p = part + static_cast<int64_t>(h) * d + c;
#pragma unroll 8
    for (int i = wave; i < n; i += kRedWaves)
      s += p[static_cast<int64_t>(i) * 2 * d];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    float t = red[0][lane];
#pragma unroll
    for (int w = 1; w < kRedWaves; ++w) t += red[w][lane];
    out[c] = t;
  }
}

// Calls f with the Map of width d.
template <typename F>
auto with_map(int64_t d, F&& f) {
  if (d <= 128) return f(Map<16, 1, 1>{});
  if (d <= 512) return f(Map<64, 1, 1>{});
  if (d <= 1024) return f(Map<64, 1, 2>{});
  if (d <= 2048) return f(Map<64, 4, 1>{});
  if (d <= 4096) return f(Map<64, 4, 2>{});
  if (d <= 8192) return f(Map<64, 8, 2>{});
  return f(Map<64, 16, 2>{});
}

// Workgroups of the two passes, by the threads they put on a CU, and no more
// than there are rows.  The backward takes few: every workgroup leaves two
// rows of partial sums, and with the next row's loads in flight 8 waves a CU
// keep up with the memory (both kernels of the backward, calls in a captured
// sequence, 8192 x 4096 bf16 RMS: 57 us with 512 threads a CU, 63 with 1024,
// 68 with 2048, 59 with 256; 1003 x 2056: 12.4, 17.2, 17.2 and 11.3 us).  The
// forward is within 2% from 1024 to 16384.
template <class M>
int64_t blocks(int64_t T, int per_cu_threads) {
  const int per_cu = per_cu_threads / M::kThreads;
  const int64_t want = 256 * (per_cu > 1 ? per_cu : 1);
  const int64_t have = (T + M::kRows - 1) / M::kRows;
  return have < want ? have : want;
}
constexpr int kFwdThreads = 2048, kBwdThreads = 512;

template <typename XT, bool LAYER>
hipError_t fwd(const void* x, const float* gamma, const float* beta,
               float eps, int64_t T, int64_t d, bf16_t* y, float* mean,
               float* rstd, hipStream_t s) {
  return with_map(d, [&](auto m) {
    using M = decltype(m);
    hipLaunchKernelGGL((norm_fwd_kernel<XT, LAYER, M>),
                       dim3(static_cast<uint32_t>(
                           blocks<M>(T, kFwdThreads))),
                       dim3(M::kThreads), 0, s, static_cast<const XT*>(x),
                       gamma, beta, eps, T, static_cast<int>(d), y, mean,
                       rstd);
    return hipGetLastError();
  });
}

template <typename XT, bool LAYER>
hipError_t bwd(const bf16_t* dy, const void* x, const float* gamma,
               const float* mean, const float* rstd, const void* dres,
               int64_t T, int64_t d, void* dx, float* dgamma, float* dbeta,
               float* part, hipStream_t s) {
  return with_map(d, [&](auto m) {
    using M = decltype(m);
    const int nb = static_cast<int>(blocks<M>(T, kBwdThreads));
    float* p = (dgamma || dbeta) ? part : nullptr;
    hipLaunchKernelGGL((norm_bwd_kernel<XT, LAYER, M>), dim3(nb),
                       dim3(M::kThreads), 0, s, dy,
                       static_cast<const XT*>(x), gamma, mean, rstd,
                       static_cast<const XT*>(dres), T, static_cast<int>(d),
                       static_cast<XT*>(dx), p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p) return e;
    hipLaunchKernelGGL(norm_wgrad_kernel,
                       dim3(static_cast<uint32_t>((d + 63) / 64),
                            LAYER ? 2 : 1),
                       dim3(64 * kRedWaves), 0, s, p, nb,
                       static_cast<int>(d), dgamma, dbeta);
    return hipGetLastError();
  });
}

}  // namespace

size_t norm_bwd_workspace(int64_t T, int64_t d) {
  const int64_t nb = with_map(d, [&](auto m) {
    return blocks<decltype(m)>(T, kBwdThreads);
  });
  return static_cast<size_t>(nb) * 2 * static_cast<size_t>(d) * 4;
}

hipError_t launch_norm_fwd(int layer, const void* x, int x_fp32,
                           const float* gamma, const float* beta, float eps,
                           int64_t T, int64_t d, bf16_t* y, float* mean,
                           float* rstd, hipStream_t s) {
  if (x_fp32)
    return layer ? fwd<float, true>(x, gamma, beta, eps, T, d, y, mean, rstd,
                                    s)
                 : fwd<float, false>(x, gamma, beta, eps, T, d, y, mean,
                                     rstd, s);
  return layer
             ? fwd<bf16_t, true>(x, gamma, beta, eps, T, d, y, mean, rstd, s)
             : fwd<bf16_t, false>(x, gamma, beta, eps, T, d, y, mean, rstd,
                                  s);
}

hipError_t launch_norm_bwd(int layer, const bf16_t* dy, const void* x,
                           int x_fp32, const float* gamma, const float* mean,
                           const float* rstd, const void* dres, int64_t T,
                           int64_t d, void* dx, float* dgamma, float* dbeta,
                           void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  if (x_fp32)
    return layer ? bwd<float, true>(dy, x, gamma, mean, rstd, dres, T, d, dx,
                                    dgamma, dbeta, part, s)
                 : bwd<float, false>(dy, x, gamma, mean, rstd, dres, T, d,
                                     dx, dgamma, dbeta, part, s);
  return layer ? bwd<bf16_t, true>(dy, x, gamma, mean, rstd, dres, T, d, dx,
                                   dgamma, dbeta, part, s)
               : bwd<bf16_t, false>(dy, x, gamma, mean, rstd, dres, T, d, dx,
                                    dgamma, dbeta, part, s);
}

}  // namespace moe
