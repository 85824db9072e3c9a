// Dense gated feed-forward block (the "shared expert" beside the routed
// ones, or a dense layer's MLP), forward and backward, bf16 with fp32 sums:
//
//   A = x W_g^T, U = x W_u^T, S = act(A) U, y = y_add + S W2^T
//   dS = dy W2, dA = dS U act'(A), dU = dS act(A)
//   dW2 = dy^T S, dW_gu = [dA dU]^T x, dx = dx_add + [dA dU] W_gu
// with act(a) = a s(z(a)), s the logistic function, and z(a) = a (SiLU) or
// 2 sqrt(2 / pi) (a + 0.044715 a^3) (tanh GELU, as (1 + tanh(z/2)) / 2 =
// s(z)); act'(a) = s + a s (1 - s) z'(a).
//
// Three forms, by what bounds them:
//  * thin (few tokens): bound by reading the weights once.  ffn_thin_kernel
//    streams them from global memory straight into MFMA fragments.
//  * tile: bound by the latency of the K-loop and by how many CUs have a
//    tile.  ffn_tile_kernel, 128 x 128 or 64 x 64 output tiles, optionally
//    with the reduction split over workgroups.
//  * large: bound by the matrix cores.  The grouped GEMM's 256 x 256 kernel
//    without its routing plan (gemm.hip, gemm_dense_*).

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

enum Epi { kAct = 0, kDAct = 1, kRow = 2, kPlane = 3 };

// ------------------------------------------------------------ activations
template <int ACT>
__device__ __forceinline__ float act_val(float a) {
  return a * sigmoidf_(act_arg<ACT>(a));
}

// ------------------------------------------------------------------ tiles
// C[m][n] = sum_k A(m, k) B(n, k).  A K-contiguous operand (KC) is stored
// [rows][ld] with k along the row; otherwise it is stored [k][ld] with the
// row along the memory row.
struct TileParams {
  const bf16_t* A;
  int64_t lda;
  const bf16_t* B;
  int64_t ldb;
  int64_t b_rows;      // KC: rows of B as stored (kAct: 2f)
  int M, N, K;         // kAct: N = f
  int mtn, ntn;        // tiles along M and N
  int kchunk;          // reduction length of one split, a multiple of 64
  bf16_t* C;           // kAct: AB (may be null); kDAct: dAB; kRow: C
  int64_t ldc;
  bf16_t* S;           // kAct
  const bf16_t* AB;    // kDAct: saved AB; kRow: addend [M][ldc] (may be null)
  float* Cf;           // kPlane: [split][M][N]
};

constexpr int kBK = 64;

__device__ __forceinline__ int swz8(int r) { return (r >> 1) & 7; }

// LDS byte offset of 16-byte chunk c of row r of a K-contiguous tile
// (128-byte rows).
__device__ __forceinline__ int kc_off(int r, int c) {
  return r * 128 + ((c ^ swz8(r)) << 4);
}

// The same of a [64 k][W] tile kept as it lies in memory: the chunk XOR
// puts the four k-rows that one transposed read takes from a 64-byte column
// block into different quarters of the 64 banks.
template <int W>
__device__ __forceinline__ int mn_swz(int r) {
  static_assert(W == 128 || W == 64, "tile widths");
  return W == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}
template <int W>
__device__ __forceinline__ int mn_off(int r, int c) {
  return r * (2 * W) + ((c ^ mn_swz<W>(r)) << 4);
}

// Moves one operand's W x 64 tile: global -> registers -> LDS, W / 32
// 16-byte pieces for each of 256 threads.
template <int W, bool KC>
struct TileMover {
  static constexpr int NP = W / 32;
  uint32_t voff[NP];   // byte offset of each piece, without the k part
  int k_lane;          // KC: first k of the thread's chunk inside a tile
  int lds0;
  const char* base;    // KC: the tile's rows; else the operand
  int64_t ld2;         // bytes of a memory row
  uint32_t bytes;      // KC: bytes from base to the end of the tile's rows
  __device__ __forceinline__ void init(int t, const bf16_t* p, int64_t ld,
                                       int64_t row0, int64_t rows,
                                       bool dual, int f) {
    ld2 = ld * 2;
    if constexpr (KC) {
      // rows row0 .. of the operand; with `dual` the tile's first half is
      // rows row0 .. and its second half rows f + row0 ..
      const int64_t left = (dual ? rows - row0 : min(rows - row0,
                                                     (int64_t)W));
      base = reinterpret_cast<const char*>(p) + row0 * ld2;
      bytes = static_cast<uint32_t>(left * ld2);
      k_lane = (t & 7) * 8;
      lds0 = kc_off(t >> 3, t & 7);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int r = (t >> 3) + 32 * i;
        const int64_t gr = !dual ? r : (r < W / 2 ? r : f + r - W / 2);
        voff[i] = static_cast<uint32_t>(gr * ld2 + (t & 7) * 16);
      }
    } else {
      constexpr int CPR = W / 8;            // chunks a k-row
      constexpr int RPP = 256 / CPR;        // k-rows a piece
      base = reinterpret_cast<const char*>(p);
      const int64_t col = row0 + (t % CPR) * 8;
      lds0 = mn_off<W>(t / CPR, t % CPR);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        voff[i] = col < rows ? static_cast<uint32_t>(
                                   (t / CPR + RPP * i) * ld2 + col * 2)
                             : kOob;
      bytes = 0;
      k_lane = 0;
    }
  }
  // k0: first k of the tile; K: end of the reduction range
  __device__ __forceinline__ void load(i32x4* v, int k0, int K) const {
    if constexpr (KC) {
      const auto rs = make_rsrc(base, bytes);
      const bool ok = k0 + k_lane < K;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        v[i] = buf_load16(rs, ok ? voff[i] + static_cast<uint32_t>(k0) * 2
                                 : kOob);
    } else {
      // the resource spans the k-rows that are left
      const int rows = max(0, min(kBK, K - k0));
      const auto rs = make_rsrc(base + k0 * ld2,
                                static_cast<uint32_t>(rows * ld2));
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = buf_load16(rs, voff[i]);
    }
  }
  // piece i lies 32 rows (KC: 4096 bytes) or RPP k-rows (4096 bytes too)
  // after piece 0, with the same swizzle
  __device__ __forceinline__ void store(const i32x4* v, uint8_t* tile) const {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      *reinterpret_cast<i32x4*>(tile + lds0 + i * 4096) = v[i];
  }
};

// Fragment reads of one operand: 32 rows x 16 k of block blk and k-slice kk.
template <int W, bool KC>
struct TileFrag {
  int off;       // KC: row part; else lane part
  int fr, fk, R;
  __device__ __forceinline__ void init(int lane) {
    fr = lane & 31;
    fk = lane >> 5;
    const int g = lane >> 4, j = lane & 15;
    R = j >> 2;
    const int m = j & 3;
    off = KC ? fr * 128
             : ((g >> 1) * 8 + R) * (2 * W) +
                   (2 * (g & 1) + (m >> 1)) * 16 + (m & 1) * 8;
  }
  __device__ __forceinline__ bf16x8_v read(const uint8_t* tile, int blk,
                                           int kk) const {
    if constexpr (KC) {
      return __builtin_bit_cast(
          bf16x8_v,
          *reinterpret_cast<const i32x4*>(
              tile + blk * 4096 + off + (((2 * kk + fk) ^ swz8(fr)) << 4)));
    } else {
      const int x = W == 128 ? R : (R >> 1);
      const uint8_t* p = tile + off + ((blk ^ x) << 6) + kk * 16 * (2 * W);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(p + 4 * (2 * W)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x8 v = {lo[0], lo[1], lo[2], lo[3],
                       hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(bf16x8_v, v);
    }
  }
};

__device__ __forceinline__ void unpack8(i32x4 r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf_lo(static_cast<uint32_t>(r[i]));
    v[2 * i + 1] = bf_hi(static_cast<uint32_t>(r[i]));
  }
}
__device__ __forceinline__ i32x4 pack8(const float* v) {
  i32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = static_cast<int>(pack_bf16x2(v[2 * i], v[2 * i + 1]));
  return o;
}
__device__ __forceinline__ void lds8(const float* p, float* v) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// 256 threads, 2 x 2 waves, each (W / 2) x (W / 2) of a W x W tile.
template <int W, bool AKC, bool BKC, int EPI, int ACT>
__global__ __launch_bounds__(256, 2) void ffn_tile_kernel(TileParams P) {
  constexpr int BI = W / 64;                      // 32-blocks a wave and side
  constexpr int kTile = W * kBK * 2;              // bytes of one operand tile
  constexpr int kLd = W + 4;                      // fp32 stage stride
  constexpr int kSmem =
      4 * kTile > W * kLd * 4 ? 4 * kTile : W * kLd * 4;
  constexpr bool kDual = EPI == kAct;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmem];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  // tiles an XCD gets are consecutive; blocks of 8 m-tiles, m fastest, so
  // that they share B columns and A rows in its L2
  const int id = xcd_remap(blockIdx.x, P.mtn * P.ntn);
  const int per = 8 * P.ntn;
  const int mb = id / per;
  const int mh = min(8, P.mtn - mb * 8);
  const int rem = id - mb * per;
  const int mt = mb * 8 + rem % mh, nt = rem / mh;
  const int m0 = mt * W;
  const int n0 = nt * (kDual ? W / 2 : W);
  const int kbeg = blockIdx.y * P.kchunk;
  const int kend = min(P.K, kbeg + P.kchunk);
  const int nk = (kend - kbeg + kBK - 1) / kBK;

  TileMover<W, AKC> ma;
  TileMover<W, BKC> mb_;
  ma.init(tid, P.A, P.lda, m0, P.M, false, 0);
  mb_.init(tid, P.B, P.ldb, n0, BKC ? P.b_rows : P.N, kDual, P.N);
  TileFrag<W, AKC> fa;
  TileFrag<W, BKC> fb;
  fa.init(lane);
  fb.init(lane);

  f32x16 acc[BI][BI];
#pragma unroll
  for (int i = 0; i < BI; ++i)
#pragma unroll
    for (int j = 0; j < BI; ++j) acc[i][j] = f32x16{};
  i32x4 va[TileMover<W, AKC>::NP], vb[TileMover<W, BKC>::NP];

  // LDS: [A 0][A 1][B 0][B 1].  Iteration kt computes on stage kt & 1; the
  // registers hold tile kt + 1, which goes to the other stage (last read
  // before the previous barrier) half way through, and are refilled with
  // tile kt + 2.
  ma.load(va, kbeg, kend);
  mb_.load(vb, kbeg, kend);
  ma.store(va, smem);
  mb_.store(vb, smem + 2 * kTile);
  ma.load(va, kbeg + kBK, kend);
  mb_.load(vb, kbeg + kBK, kend);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int cs = kt & 1, ns = cs ^ 1;
    const uint8_t* ta = smem + cs * kTile;
    const uint8_t* tb = smem + 2 * kTile + cs * kTile;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8_v a[BI], b[BI];
#pragma unroll
      for (int i = 0; i < BI; ++i) a[i] = fa.read(ta, wm * BI + i, kk);
#pragma unroll
      for (int j = 0; j < BI; ++j) b[j] = fb.read(tb, wn * BI + j, kk);
#pragma unroll
      for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < BI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              a[i], b[j], acc[i][j], 0, 0, 0);
      if (kk == 1) {
        ma.store(va, smem + ns * kTile);
        mb_.store(vb, smem + 2 * kTile + ns * kTile);
        const int k2 = kbeg + (kt + 2) * kBK;
        ma.load(va, k2, kend);
        mb_.load(vb, k2, kend);
      }
    }
    __syncthreads();
  }

  // The whole tile goes through LDS as fp32 (the K-loop's last barrier
  // freed it), then each thread takes 8 columns of a row at a time.
  float* st = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < BI; ++i)
#pragma unroll
    for (int j = 0; j < BI; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = (wm * BI + i) * 32 + (v >> 2) * 8 + (lane >> 5) * 4 +
                      (v & 3);
        st[r * kLd + (wn * BI + j) * 32 + (lane & 31)] = acc[i][j][v];
      }
  __syncthreads();
  constexpr int kCols = kDual ? W / 2 : W;
  constexpr int kCh = kCols / 8;                  // chunks a row
  constexpr int kIt = W * kCh / 256;
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int idx = tid + 256 * it;
    const int r = idx / kCh, c = (idx % kCh) * 8;
    const int row = m0 + r, col = n0 + c;
    if (row >= P.M || col >= P.N) continue;
    float x[8];
    lds8(st + r * kLd + c, x);
    const int64_t ro = static_cast<int64_t>(row);
    if constexpr (EPI == kAct) {
      float u[8], s[8];
      lds8(st + r * kLd + W / 2 + c, u);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = act_val<ACT>(x[q]) * u[q];
      if (P.C) {
        *reinterpret_cast<i32x4*>(P.C + ro * P.ldc + col) = pack8(x);
        *reinterpret_cast<i32x4*>(P.C + ro * P.ldc + P.N + col) = pack8(u);
      }
      *reinterpret_cast<i32x4*>(P.S + ro * P.N + col) = pack8(s);
    } else if constexpr (EPI == kDAct) {
      float a[8], u[8], dg[8], du[8];
      const bf16_t* ab = P.AB + ro * P.ldc + col;
      unpack8(*reinterpret_cast<const i32x4*>(ab), a);
      unpack8(*reinterpret_cast<const i32x4*>(ab + P.N), u);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float h, slope;
        act_both<ACT>(a[q], &h, &slope);
        dg[q] = x[q] * u[q] * slope;
        du[q] = x[q] * h;
      }
      *reinterpret_cast<i32x4*>(P.C + ro * P.ldc + col) = pack8(dg);
      *reinterpret_cast<i32x4*>(P.C + ro * P.ldc + P.N + col) = pack8(du);
    } else if constexpr (EPI == kRow) {
      if (P.AB) {
        float a[8];
        unpack8(*reinterpret_cast<const i32x4*>(P.AB + ro * P.ldc + col), a);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] += a[q];
      }
      *reinterpret_cast<i32x4*>(P.C + ro * P.ldc + col) = pack8(x);
    } else {
      float* o = P.Cf + (blockIdx.y * static_cast<int64_t>(P.M) + ro) * P.N +
                 col;
      *reinterpret_cast<f32x4*>(o) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
  }
}

// out = bf16(add + the planes in order); n values, a multiple of 8.
__global__ __launch_bounds__(256) void ffn_rows_kernel(
    const float* __restrict__ pl, int planes, int64_t n,
    const bf16_t* add, bf16_t* out) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
       i < n; i += step) {
    float s[8], v[8];
    lds8(pl + i, s);
    for (int p = 1; p < planes; ++p) {
      lds8(pl + p * n + i, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += v[q];
    }
    if (add) {
      unpack8(*reinterpret_cast<const i32x4*>(add + i), v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += v[q];
    }
    *reinterpret_cast<i32x4*>(out + i) = pack8(s);
  }
}

// ------------------------------------------------------------------- thin
// Few tokens: out[t][n] = sum_k W[n][k] x[t][k] for up to 16 NTB tokens.
// A workgroup takes RT outputs (gate and up rows of the same index for
// kAct); its waves split the reduction in interleaved chunks of 128 k, so
// that together they read long runs of each weight row.  Weights are the
// MFMA's A operand (16 rows x 32 k, one 16-byte load a lane straight from
// global memory) and tokens its B operand; the next chunk's loads are in
// flight during the current chunk's products.  The waves' sums are added
// in wave order through LDS.
//   RT = 16: kAct has a gate and an up tile; RT = 8: kAct packs 8 gate and
//   8 up rows into one tile, kRow leaves half of its tile empty.  8 doubles
//   the workgroups where 16 would leave CUs without one.
struct ThinParams {
  const bf16_t* W;     // kAct: [2f][K]; kRow: [N][K]
  const bf16_t* X;     // [T][K]
  int T, N, K;         // kAct: N = f
  bf16_t* C;           // kAct: AB [T][2f] or null; kRow: out [T][N]
  bf16_t* S;           // kAct: S [T][f]
  const bf16_t* add;   // kRow: [T][N] or null
};

template <int NTB, int NWV, int RT, int EPI, int ACT>
__global__ __launch_bounds__(64 * NWV) void ffn_thin_kernel(ThinParams P) {
  constexpr int NWT = (EPI == kAct && RT == 16) ? 2 : 1;   // weight tiles
  __shared__ float red[NWV][NWT][NTB][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int fr = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * RT;
  const uint32_t ld2 = static_cast<uint32_t>(P.K) * 2;
  const int nr = min(RT, P.N - n0);              // rows of this workgroup

  // Weight resources start at the tile's first row; rows past it (and
  // tokens past T) get the masked offset or lie past the range.
  __amdgpu_buffer_rsrc_t rw[NWT];
  uint32_t wv;
  if constexpr (NWT == 2) {
    rw[0] = make_rsrc(P.W + static_cast<int64_t>(n0) * P.K,
                      static_cast<uint32_t>(nr) * ld2);
    rw[1] = make_rsrc(P.W + static_cast<int64_t>(P.N + n0) * P.K,
                      static_cast<uint32_t>(nr) * ld2);
    wv = fr < nr ? fr * ld2 : kOob;
  } else if constexpr (EPI == kAct) {
    // N is a multiple of 8: all 8 rows exist
    rw[0] = make_rsrc(P.W, static_cast<uint32_t>(2 * P.N) * ld2);
    wv = static_cast<uint32_t>(fr < 8 ? n0 + fr : P.N + n0 + fr - 8) * ld2;
  } else {
    rw[0] = make_rsrc(P.W + static_cast<int64_t>(n0) * P.K,
                      static_cast<uint32_t>(nr) * ld2);
    wv = fr < nr ? fr * ld2 : kOob;
  }
  __amdgpu_buffer_rsrc_t rx[NTB];
  uint32_t xv[NTB];
#pragma unroll
  for (int b = 0; b < NTB; ++b) {
    const int nt = max(0, min(16, P.T - 16 * b));
    rx[b] = make_rsrc(P.X + static_cast<int64_t>(16 * b) * P.K,
                      static_cast<uint32_t>(nt) * ld2);
    xv[b] = fr < nt ? fr * ld2 : kOob;
  }

  struct Chunk {
    i32x4 w[NWT][4], x[NTB][4];
  };
  Chunk cur, nxt;
  auto load = [&](Chunk& c, int kc) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = kc * 128 + s * 32 + g * 8;
      const bool ok = k < P.K;
      const uint32_t kb = static_cast<uint32_t>(k) * 2;
#pragma unroll
      for (int i = 0; i < NWT; ++i)
        c.w[i][s] = buf_load16(rw[i], ok && wv != kOob ? wv + kb : kOob);
#pragma unroll
      for (int b = 0; b < NTB; ++b)
        c.x[b][s] = buf_load16(rx[b], ok && xv[b] != kOob ? xv[b] + kb
                                                          : kOob);
    }
  };
  f32x4 acc[NWT][NTB];
#pragma unroll
  for (int i = 0; i < NWT; ++i)
#pragma unroll
    for (int b = 0; b < NTB; ++b) acc[i][b] = f32x4{};
  const int nkc = (P.K + 127) / 128;
  int kc = wave;
  if (kc < nkc) load(cur, kc);
  for (; kc < nkc; kc += NWV) {
    if (kc + NWV < nkc) load(nxt, kc + NWV);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < NWT; ++i)
#pragma unroll
        for (int b = 0; b < NTB; ++b)
          acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_v, cur.w[i][s]),
              __builtin_bit_cast(bf16x8_v, cur.x[b][s]), acc[i][b], 0, 0, 0);
    cur = nxt;
  }
#pragma unroll
  for (int i = 0; i < NWT; ++i)
#pragma unroll
    for (int b = 0; b < NTB; ++b)
      *reinterpret_cast<f32x4*>(&red[wave][i][b][lane * 4]) = acc[i][b];
  __syncthreads();
  // acc element v of lane l is output row 4 (l / 16) + v, token l % 16
  auto sum = [&](int tile, int b, int row, int tok) {
    const int o = ((row >> 2) * 16 + tok) * 4 + (row & 3);
    float s = red[0][tile][b][o];
#pragma unroll
    for (int w = 1; w < NWV; ++w) s += red[w][tile][b][o];
    return s;
  };
  for (int idx = tid; idx < NTB * 16 * RT; idx += 64 * NWV) {
    const int row = idx % RT, t = idx / RT;
    const int b = t >> 4, tok = t & 15;
    if (t >= P.T || row >= nr) continue;
    const int col = n0 + row;
    if constexpr (EPI == kAct) {
      const float a = sum(0, b, row, tok);
      const float u = NWT == 2 ? sum(NWT - 1, b, row, tok)
                               : sum(0, b, row + 8, tok);
      if (P.C) {
        bf16_t* ab = P.C + static_cast<int64_t>(t) * 2 * P.N + col;
        ab[0] = f2bf(a);
        ab[P.N] = f2bf(u);
      }
      P.S[static_cast<int64_t>(t) * P.N + col] = f2bf(act_val<ACT>(a) * u);
    } else {
      const int64_t o = static_cast<int64_t>(t) * P.N + col;
      float v = sum(0, b, row, tok);
      if (P.add) v += bf2f(P.add[o]);
      P.C[o] = f2bf(v);
    }
  }
}

template <int NTB, int RT, int EPI, int ACT>
hipError_t thin_rt(const ThinParams& P, hipStream_t s) {
  constexpr int NWV = 8;
  hipLaunchKernelGGL((ffn_thin_kernel<NTB, NWV, RT, EPI, ACT>),
                     dim3((P.N + RT - 1) / RT), dim3(64 * NWV), 0, s, P);
  return hipGetLastError();
}

template <int EPI, int ACT>
hipError_t thin(const ThinParams& P, hipStream_t s) {
  const int ntb = (P.T + 15) / 16;
  const bool narrow = P.N < 16 * 256;
  if (ntb == 1)
    return narrow ? thin_rt<1, 8, EPI, ACT>(P, s)
                  : thin_rt<1, 16, EPI, ACT>(P, s);
  if (ntb == 2)
    return narrow ? thin_rt<2, 8, EPI, ACT>(P, s)
                  : thin_rt<2, 16, EPI, ACT>(P, s);
  return narrow ? thin_rt<4, 8, EPI, ACT>(P, s)
                : thin_rt<4, 16, EPI, ACT>(P, s);
}

// ---------------------------------------------------------- tile launches
template <int W, bool AKC, bool BKC, int EPI, int ACT>
hipError_t tile_w(TileParams P, int splits, hipStream_t s) {
  constexpr int wn = EPI == kAct ? W / 2 : W;
  P.mtn = (P.M + W - 1) / W;
  P.ntn = (P.N + wn - 1) / wn;
  hipLaunchKernelGGL((ffn_tile_kernel<W, AKC, BKC, EPI, ACT>),
                     dim3(static_cast<uint32_t>(P.mtn) * P.ntn, splits),
                     dim3(256), 0, s, P);
  return hipGetLastError();
}

// 128 x 128 tiles once they give every CU about one; below that 64 x 64
// ones spread the product over four times as many CUs.
constexpr int64_t kWideTiles = 192;
bool wide_tiles(int64_t M, int64_t N, int cols) {
  return ((M + 127) / 128) * ((N + cols - 1) / cols) >= kWideTiles;
}

template <bool AKC, bool BKC, int EPI, int ACT>
hipError_t tile(const TileParams& P, int splits, bool wide, hipStream_t s) {
  return wide ? tile_w<128, AKC, BKC, EPI, ACT>(P, splits, s)
              : tile_w<64, AKC, BKC, EPI, ACT>(P, splits, s);
}

// Splits of a row output's reduction (fc2 and the data gradient), and the
// tile width: with few tiles the reduction is cut so that about two
// workgroups a CU run, each with at least 4 k-steps.
struct RowPlan {
  bool wide;
  int splits, kchunk;
};
RowPlan row_plan(int64_t T, int64_t N, int64_t K) {
  RowPlan r;
  r.wide = wide_tiles(T, N, 128);
  const int64_t w = r.wide ? 128 : 64;
  const int64_t tiles = ((T + w - 1) / w) * ((N + w - 1) / w);
  const int64_t steps = (K + kBK - 1) / kBK;
  int64_t sp = 512 / tiles;
  if (sp > steps / 4) sp = steps / 4;
  if (sp > 8) sp = 8;
  if (sp < 1) sp = 1;
  const int64_t per = (steps + sp - 1) / sp;
  r.kchunk = static_cast<int>(per * kBK);
  r.splits = static_cast<int>((steps + per - 1) / per);
  return r;
}

hipError_t finish_rows(const float* planes, int n_planes, int64_t n,
                       const bf16_t* add, bf16_t* out, hipStream_t s) {
  int64_t nb = (n / 8 + 255) / 256;
  if (nb > 4096) nb = 4096;
  hipLaunchKernelGGL(ffn_rows_kernel, dim3(static_cast<uint32_t>(nb)),
                     dim3(256), 0, s, planes, n_planes, n, add, out);
  return hipGetLastError();
}

// Tokens up to which the weight-streaming form runs.
constexpr int64_t kThinRows = 64;

size_t up256(int64_t v) {
  return (static_cast<size_t>(v) + 255) & ~static_cast<size_t>(255);
}

// out[T][N] = add + A . B (B K-contiguous or not) by tiles.
template <bool BKC>
hipError_t row_product(const bf16_t* A, const bf16_t* B, int64_t ldb,
                       int64_t T, int64_t N, int64_t K, const bf16_t* add,
                       bf16_t* out, float* planes, hipStream_t s) {
  TileParams P{};
  P.A = A; P.lda = K;
  P.B = B; P.ldb = ldb; P.b_rows = N;
  P.M = static_cast<int>(T); P.N = static_cast<int>(N);
  P.K = static_cast<int>(K);
  const RowPlan r = row_plan(T, N, K);
  P.kchunk = r.kchunk;
  if (r.splits == 1) {
    P.C = out; P.ldc = N; P.AB = add;
    return tile<true, BKC, kRow, kActSilu>(P, 1, r.wide, s);
  }
  P.Cf = planes;
  hipError_t e =
      tile<true, BKC, kPlane, kActSilu>(P, r.splits, r.wide, s);
  if (e != hipSuccess) return e;
  return finish_rows(planes, r.splits, T * N, add, out, s);
}

// c[M][N] = sum_t a[t][m] b[t][n]
hipError_t weight_product(const bf16_t* a, const bf16_t* b, int64_t T,
                          int64_t M, int64_t N, bf16_t* c, hipStream_t s) {
  TileParams P{};
  P.A = a; P.lda = M;
  P.B = b; P.ldb = N;
  P.M = static_cast<int>(M); P.N = static_cast<int>(N);
  P.K = static_cast<int>(T);
  P.kchunk = (P.K + kBK - 1) / kBK * kBK;
  P.C = c; P.ldc = N;
  return tile<false, false, kRow, kActSilu>(P, 1, wide_tiles(M, N, 128), s);
}

template <int ACT>
hipError_t fc1(const bf16_t* x, const bf16_t* w_gu, int64_t T, int64_t d,
               int64_t f, bf16_t* ab, bf16_t* s_out, hipStream_t s) {
  if (T <= kThinRows) {
    ThinParams P{};
    P.W = w_gu; P.X = x;
    P.T = static_cast<int>(T); P.N = static_cast<int>(f);
    P.K = static_cast<int>(d);
    P.C = ab; P.S = s_out;
    return thin<kAct, ACT>(P, s);
  }
  TileParams P{};
  P.A = x; P.lda = d;
  P.B = w_gu; P.ldb = d; P.b_rows = 2 * f;
  P.M = static_cast<int>(T); P.N = static_cast<int>(f);
  P.K = static_cast<int>(d);
  P.kchunk = (P.K + kBK - 1) / kBK * kBK;
  P.C = ab; P.ldc = 2 * f; P.S = s_out;
  return tile<true, true, kAct, ACT>(P, 1, wide_tiles(T, f, 64), s);
}

template <int ACT>
hipError_t dact(const bf16_t* dy, const bf16_t* w2, const bf16_t* ab,
                int64_t T, int64_t d, int64_t f, bf16_t* dab,
                hipStream_t s) {
  TileParams P{};
  P.A = dy; P.lda = d;
  P.B = w2; P.ldb = f; P.b_rows = d;
  P.M = static_cast<int>(T); P.N = static_cast<int>(f);
  P.K = static_cast<int>(d);
  P.kchunk = (P.K + kBK - 1) / kBK * kBK;
  P.C = dab; P.ldc = 2 * f; P.AB = ab;
  return tile<true, false, kDAct, ACT>(P, 1, wide_tiles(T, f, 128), s);
}

// Workspaces.  Forward: S (when the caller keeps none), then the fp32
// planes of y.  Backward: dAB, then the planes of dx.
int64_t plane_bytes(int64_t T, int64_t N, int64_t K) {
  const RowPlan r = row_plan(T, N, K);
  return r.splits > 1 ? r.splits * T * N * 4 : 0;
}

}  // namespace

size_t ffn_fwd_workspace(int64_t T, int64_t d, int64_t f) {
  return up256(T * f * 2) +
         (T <= kThinRows ? 0 : up256(plane_bytes(T, d, f)));
}

size_t ffn_bwd_workspace(int64_t T, int64_t d, int64_t f) {
  return up256(T * 2 * f * 2) + up256(plane_bytes(T, d, 2 * f));
}

hipError_t launch_ffn_fwd(int act, const bf16_t* x, const bf16_t* w_gu,
                          const bf16_t* w2, const bf16_t* y_add, int64_t T,
                          int64_t d, int64_t f, bf16_t* ab, bf16_t* s_saved,
                          bf16_t* y, void* ws, hipStream_t s) {
  bf16_t* sb = s_saved ? s_saved : static_cast<bf16_t*>(ws);
  float* planes = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                           up256(T * f * 2));
  hipError_t e =
      act == kActSilu
          ? fc1<kActSilu>(x, w_gu, T, d, f, ab, sb, s)
          : fc1<kActGeluTanh>(x, w_gu, T, d, f, ab, sb, s);
  if (e != hipSuccess) return e;
  if (T <= kThinRows) {
    ThinParams P{};
    P.W = w2; P.X = sb;
    P.T = static_cast<int>(T); P.N = static_cast<int>(d);
    P.K = static_cast<int>(f);
    P.C = y; P.add = y_add;
    return thin<kRow, kActSilu>(P, s);
  }
  return row_product<true>(sb, w2, f, T, d, f, y_add, y, planes, s);
}

hipError_t launch_ffn_bwd(int act, const bf16_t* dy, const bf16_t* x,
                          const bf16_t* w_gu, const bf16_t* w2,
                          const bf16_t* ab, const bf16_t* s_saved,
                          const bf16_t* dx_add, int64_t T, int64_t d,
                          int64_t f, bf16_t* dx, bf16_t* dw_gu, bf16_t* dw2,
                          void* ws, hipStream_t s) {
  bf16_t* dab = static_cast<bf16_t*>(ws);
  float* planes = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                           up256(T * 2 * f * 2));
  hipError_t e = act == kActSilu
                     ? dact<kActSilu>(dy, w2, ab, T, d, f, dab, s)
                     : dact<kActGeluTanh>(dy, w2, ab, T, d, f, dab, s);
  if (e != hipSuccess) return e;
  if (dw2) {
    e = weight_product(dy, s_saved, T, d, f, dw2, s);
    if (e != hipSuccess) return e;
  }
  if (dw_gu) {
    e = weight_product(dab, x, T, 2 * f, d, dw_gu, s);
    if (e != hipSuccess) return e;
  }
  if (!dx) return hipSuccess;
  return row_product<false>(dab, w_gu, d, T, d, 2 * f, dx_add, dx, planes, s);
}

}  // namespace moe
