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
//    tile.  ffn_tile_kernel, 128 x 128, 128 x 64 or 64 x 64 output tiles,
//    optionally with the reduction split over workgroups.
//  * large: bound by the matrix cores.  The grouped GEMM's 256 x 256 kernel
//    without its routing plan (gemm.hip, gemm_dense_*).
// On MI355X, a pass among others: 1 token through d 4096, f 14336 forward 66
// us (5.3 TB/s of weights); 24 through 2048 x 1408 10.3 us; 777 through 2048 x
// 2816 49 us (550 TFLOP/s); 2000 through it forward and backward 248 to 252 us
// (820 to 840 TFLOP/s); 8192 through 4096 x 14336 6.8 to 7.0 ms (1240 to 1280
// TFLOP/s).
//
// What is rounded to bf16, and why: S and [dA dU], since they are operands of
// bf16 matrix products (their fp32 form would need the products in two parts
// or at the fp32 rate, a sixteenth); AB as saved for the backward, since it is
// the largest tensor of the block (fp32 would double it), as in the expert
// layer; y, dx and the weight gradients once, from fp32 sums.  S is computed
// from the fp32 sums, not from the saved AB.  Against 64 bits y is off by
// 0.0018 to 0.0023 of its norm and the gradients by 0.0030, where the last
// rounding alone is 0.0017; without AB's the gradients would be at 0.0024.

#include "common.cuh"
#include "ffn_plan.h"
#include "internal.h"

namespace moe {
namespace {

static_assert(kMaxOperandBytes == kMaxResourceBytes, "one limit");

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

// tiles in flight from global memory, in 128 x 128 and in smaller tiles
constexpr int kDepthWide = 2;
constexpr int kDepthNarrow = 4;

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

// NG groups of 256 threads; a group is 2 x 2 waves, each (WM / 2) x (WN / 2)
// of a WM x WN tile.  With two groups each runs half of the reduction out of
// its own LDS stages and the second group's sums are added to the first's:
// what a CU with a single tile needs to keep its matrix cores busy.
//
// The LDS of a tile: two stages of both operands a group, or the fp32 tile
// of the epilogue (rows of WN + 4).
template <int WM, int WN, int NG>
constexpr int tile_smem() {
  constexpr int k = NG * 2 * (WM + WN) * kBK * 2, e = WM * (WN + 4) * 4;
  return k > e ? k : e;
}

// tile: index in the product's mtn x ntn tiles, already in XCD order.
template <int WM, int WN, int NG, bool AKC, bool BKC, int EPI, int ACT>
__device__ __forceinline__ void tile_product(const TileParams& P,
                                             uint8_t* smem_all, int tile,
                                             int split) {
  constexpr int BM = WM / 64, BN = WN / 64;       // 32-blocks a wave and side
  constexpr int kTileA = WM * kBK * 2;            // bytes of an operand's tile
  constexpr int kTileB = WN * kBK * 2;
  constexpr int kLd = WN + 4;                     // fp32 stage stride
  constexpr bool kDual = EPI == kAct;
  const int grp = NG == 1 ? 0
                          : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int tid = threadIdx.x & 255, lane = tid & 63, wave = tid >> 6;
  uint8_t* const smem = smem_all + grp * 2 * (kTileA + kTileB);
  const int wm = wave >> 1, wn = wave & 1;
  // blocks of 8 m-tiles, m fastest: the consecutive tiles that an XCD gets
  // share B columns and A rows in its L2
  const int per = 8 * P.ntn;
  const int mb = tile / per;
  const int mh = min(8, P.mtn - mb * 8);
  const int rem = tile - mb * per;
  const int mt = mb * 8 + rem % mh, nt = rem / mh;
  const int m0 = mt * WM;
  const int n0 = nt * (kDual ? WN / 2 : WN);
  // the workgroup's range of the reduction, then the group's; groups take
  // equally many steps (barriers are shared), empty past the range's end
  const int kb0 = split * P.kchunk;
  const int kend0 = min(P.K, kb0 + P.kchunk);
  const int nk = ((kend0 - kb0 + kBK - 1) / kBK + NG - 1) / NG;
  const int kbeg = kb0 + grp * nk * kBK;
  const int kend = min(kend0, kbeg + nk * kBK);

  TileMover<WM, AKC> ma;
  TileMover<WN, BKC> mb_;
  ma.init(tid, P.A, P.lda, m0, P.M, false, 0);
  mb_.init(tid, P.B, P.ldb, n0, BKC ? P.b_rows : P.N, kDual, P.N);
  TileFrag<WM, AKC> fa;
  TileFrag<WN, BKC> fb;
  fa.init(lane);
  fb.init(lane);

  f32x16 acc[BM][BN];
#pragma unroll
  for (int i = 0; i < BM; ++i)
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[i][j] = f32x16{};

  // LDS: [A 0][A 1][B 0][B 1], tile kt in stage kt & 1.  The registers hold
  // the next kDepth tiles from global memory and two sets of fragments:
  // while the products of one group of kG k-slices run from one set, the
  // next group is read into the other.  Step kt sends tile kt + 1 to its
  // stage (whose fragments every wave held before the previous barrier),
  // refills the freed registers with tile kt + 1 + kDepth, and before its
  // last group's products passes the barrier that completes tile kt + 1 and
  // reads the first group of it.
  constexpr int kDepth = WM + WN > 192 ? kDepthWide : kDepthNarrow;
  static_assert(kDepth % 2 == 0, "the LDS stage is a compile-time constant");
  i32x4 va[kDepth][TileMover<WM, AKC>::NP], vb[kDepth][TileMover<WN, BKC>::NP];
  {
    i32x4 fa0[TileMover<WM, AKC>::NP], fb0[TileMover<WN, BKC>::NP];
    ma.load(fa0, kbeg, kend);
    mb_.load(fb0, kbeg, kend);
#pragma unroll
    for (int q = 0; q < kDepth; ++q) {
      // in order, so that the loop's waits need not assume the worst
      __builtin_amdgcn_sched_barrier(0);
      ma.load(va[q], kbeg + (q + 1) * kBK, kend);
      mb_.load(vb[q], kbeg + (q + 1) * kBK, kend);
    }
    __builtin_amdgcn_sched_barrier(0);
    ma.store(fa0, smem);
    mb_.store(fb0, smem + 2 * kTileA);
  }
  __syncthreads();
  constexpr int kG = WM + WN > 128 ? 2 : 4;      // k-slices a group
  constexpr int kGroups = 4 / kG;
  bf16x8_v fra[2][kG][BM], frb[2][kG][BN];
  auto read_group = [&](int set, int stage, int group) {
    const uint8_t* ta = smem + stage * kTileA;
    const uint8_t* tb = smem + 2 * kTileA + stage * kTileB;
#pragma unroll
    for (int k = 0; k < kG; ++k) {
#pragma unroll
      for (int i = 0; i < BM; ++i)
        fra[set][k][i] = fa.read(ta, wm * BM + i, group * kG + k);
#pragma unroll
      for (int j = 0; j < BN; ++j)
        frb[set][k][j] = fb.read(tb, wn * BN + j, group * kG + k);
    }
  };
  auto products = [&](int set, int k0, int k1) {
#pragma unroll
    for (int k = k0; k < k1; ++k)
#pragma unroll
      for (int i = 0; i < BM; ++i)
#pragma unroll
        for (int j = 0; j < BN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              fra[set][k][i], frb[set][k][j], acc[i][j], 0, 0, 0);
  };
  // Instruction order: the next group's fragment reads, the LDS stores and
  // the global loads a few after each product, the reads first, so that they
  // land while later products run from registers (reads all behind the
  // first product: 5% slower in 128-wide tiles).
  constexpr int kRd = kG * (BM * (AKC ? 1 : 2) + BN * (BKC ? 1 : 2));
  constexpr int kMv = TileMover<WM, AKC>::NP + TileMover<WN, BKC>::NP;
  constexpr int kMf = 2 * BM * BN;               // products a section
  constexpr int kSgMfma = 0x008, kSgVmem = 0x020, kSgRead = 0x100,
                kSgWrite = 0x200;
  constexpr int kPer = (kMv + kMf - 1) / kMf;    // moves a product
  constexpr int kSpread = kMf < 4 ? kMf : 4;     // products with reads
  constexpr int kRdPer = (kRd + kSpread - 1) / kSpread;
  read_group(0, 0, 0);
  // step kt with kt % kDepth == q, a compile-time constant
  auto step = [&](int q, int kt) {
    const int cs = q & 1, ns = cs ^ 1;
    const int s1 = kGroups == 1 ? cs : 0;      // set before the barrier
    const int s2 = kGroups == 1 ? cs : 1;      // and after it
    __builtin_amdgcn_sched_barrier(0);
    if (kGroups > 1) read_group(1, cs, 1);
    ma.store(va[q], smem + ns * kTileA);
    mb_.store(vb[q], smem + 2 * kTileA + ns * kTileB);
    const int k2 = kbeg + (kt + 1 + kDepth) * kBK;
    ma.load(va[q], k2, kend);
    mb_.load(vb[q], k2, kend);
    products(s1, 0, 2);
#pragma unroll
    for (int i = 0; i < kMf; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
      if (kGroups > 1 && i < kSpread)
        __builtin_amdgcn_sched_group_barrier(kSgRead, kRdPer, 0);
      __builtin_amdgcn_sched_group_barrier(kSgWrite, kPer, 0);
      __builtin_amdgcn_sched_group_barrier(kSgVmem, kPer, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    read_group(s2 ^ 1, ns, 0);
    products(s2, kGroups == 1 ? 2 : 0, kGroups == 1 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kMf; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
      if (i < kSpread)
        __builtin_amdgcn_sched_group_barrier(kSgRead, kRdPer, 0);
    }
  };
  int kt0 = 0;
  for (; kt0 + kDepth <= nk; kt0 += kDepth)
#pragma unroll
    for (int q = 0; q < kDepth; ++q) step(q, kt0 + q);
#pragma unroll
  for (int q = 0; q < kDepth - 1; ++q)
    if (kt0 + q < nk) step(q, kt0 + q);

  // The whole tile goes through LDS as fp32 (after the K-loop's last barrier
  // only fragments that no product uses are read there), then each thread
  // takes 8 columns of a row at a time.
  float* st = reinterpret_cast<float*>(smem_all);
#pragma unroll
  for (int h = NG - 1; h >= 0; --h) {
    if (grp == h)
#pragma unroll
      for (int i = 0; i < BM; ++i)
#pragma unroll
        for (int j = 0; j < BN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int r = (wm * BM + i) * 32 + (v >> 2) * 8 +
                          (lane >> 5) * 4 + (v & 3);
            float* p = st + r * kLd + (wn * BN + j) * 32 + (lane & 31);
            *p = h == NG - 1 ? acc[i][j][v] : acc[i][j][v] + *p;
          }
    __syncthreads();
  }
  constexpr int kCols = kDual ? WN / 2 : WN;
  constexpr int kCh = kCols / 8;                  // chunks a row
  constexpr int kThr = 256 * NG;
#pragma unroll
  for (int it = 0; it < (WM * kCh + kThr - 1) / kThr; ++it) {
    const int idx = static_cast<int>(threadIdx.x) + kThr * it;
    if (WM * kCh < kThr && idx >= WM * kCh) continue;
    const int r = idx / kCh, c = (idx % kCh) * 8;
    const int row = m0 + r, col = n0 + c;
    if (row >= P.M || col >= P.N) continue;
    float x[8];
    lds8(st + r * kLd + c, x);
    const int64_t ro = static_cast<int64_t>(row);
    if constexpr (EPI == kAct) {
      float u[8], s[8];
      lds8(st + r * kLd + WN / 2 + c, u);
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
      float* o = P.Cf + (split * static_cast<int64_t>(P.M) + ro) * P.N + col;
      *reinterpret_cast<f32x4*>(o) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
  }
}

template <int WM, int WN, int NG, bool AKC, bool BKC, int EPI, int ACT>
__global__ __launch_bounds__(256 * NG, NG == 1 ? 2 : 1) void ffn_tile_kernel(
    TileParams P) {
  __shared__ __attribute__((aligned(16))) uint8_t
      smem[tile_smem<WM, WN, NG>()];
  tile_product<WM, WN, NG, AKC, BKC, EPI, ACT>(
      P, smem, xcd_remap(blockIdx.x, P.mtn * P.ntn), blockIdx.y);
}

// Two independent products of the backward in one launch: a row product `a`
// (dS with its activation, or dx) and a weight gradient `b`.  One's last
// round of tiles runs beside the other's, and the gap of a launch is saved.
struct PairParams {
  TileParams a, b;
  int splits_a;
  int b_first;         // the product with the longer tiles goes first
};

template <int W, int EPI, int ACT>
__global__ __launch_bounds__(256, 2) void ffn_pair_kernel(PairParams P) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[tile_smem<W, W, 1>()];
  const int ta = P.a.mtn * P.a.ntn, na = ta * P.splits_a;
  const int nb = P.b.mtn * P.b.ntn;
  const int id = blockIdx.x;
  const int ia = P.b_first ? id - nb : id, ib = P.b_first ? id : id - na;
  if (ia >= 0 && ia < na) {
    const int split = ia / ta;
    tile_product<W, W, 1, true, false, EPI, ACT>(
        P.a, smem, xcd_remap(ia - split * ta, ta), split);
  } else {
    tile_product<W, W, 1, false, false, kRow, kActSilu>(P.b, smem,
                                                     xcd_remap(ib, nb), 0);
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
// in wave order through LDS.  Past a few tokens (kStageX) a wave loads its
// chunk of x as whole 256-byte rows and turns it into fragments through its
// own piece of LDS, in place of 16 rows x 64 bytes a load (2048 x 1408, whole
// forwards in a captured sequence over data that leaves the caches: 64 tokens
// 20.0 -> 14.9 us, 24 tokens 12.5 -> 10.7, 16 tokens 10.6 -> 9.1, 5 tokens 8.7
// -> 9.0; one token, where the turn only adds its latency, 8.2 -> 8.9).
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

template <int NTB, bool kStageX, int RT, int EPI, int ACT>
__global__ __launch_bounds__(512) void ffn_thin_kernel(ThinParams P) {
  constexpr int NWV = 8;
  constexpr int NWT = (EPI == kAct && RT == 16) ? 2 : 1;   // weight tiles
  constexpr int kRedBytes = NWV * NWT * NTB * 1024;
  constexpr int kXBytes = kStageX ? NWV * NTB * 4096 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t
      smem[kRedBytes > kXBytes ? kRedBytes : kXBytes];
  auto red = reinterpret_cast<float (*)[NWT][NTB][256]>(smem);
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
  const auto rx = make_rsrc(P.X, static_cast<uint32_t>(P.T) * ld2);
  uint8_t* const xs = smem + wave * NTB * 4096;
  const int xp = lane & 15;                      // staged: 16-byte piece
  uint32_t xv[kStageX ? NTB * 4 : NTB];
#pragma unroll
  for (int i = 0; i < (kStageX ? NTB * 4 : NTB); ++i) {
    const int t = kStageX ? 4 * i + g : 16 * i + fr;
    xv[i] = t < P.T ? static_cast<uint32_t>(t) * ld2 : kOob;
  }

  // x: fragment b of k-slice s (4 b + s), or staged the rows 4 i + lane / 16
  struct Chunk {
    i32x4 w[NWT][4], x[NTB * 4];
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
      if constexpr (!kStageX)
#pragma unroll
        for (int b = 0; b < NTB; ++b)
          c.x[4 * b + s] =
              buf_load16(rx, ok && xv[b] != kOob ? xv[b] + kb : kOob);
    }
    if constexpr (kStageX) {
      const int k = kc * 128 + xp * 8;
#pragma unroll
      for (int i = 0; i < NTB * 4; ++i)
        c.x[i] = buf_load16(rx, k < P.K && xv[i] != kOob
                                    ? xv[i] + static_cast<uint32_t>(k) * 2
                                    : kOob);
    }
  };
  // orders a wave's LDS writes before its own reads, and the reverse
  auto wave_sync = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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
    if constexpr (kStageX) {
      // piece p of row t in slot p ^ (t % 16): both the row-wise stores and
      // the fragment reads (one piece of 16 rows) meet every bank once
#pragma unroll
      for (int i = 0; i < NTB * 4; ++i) {
        const int t = 4 * i + g;
        *reinterpret_cast<i32x4*>(xs + t * 256 + ((xp ^ (t & 15)) << 4)) =
            cur.x[i];
      }
      wave_sync();
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int b = 0; b < NTB; ++b) {
        const i32x4 xf =
            kStageX ? *reinterpret_cast<const i32x4*>(
                          xs + (16 * b + fr) * 256 + (((4 * s + g) ^ fr) << 4))
                    : cur.x[4 * b + s];
#pragma unroll
        for (int i = 0; i < NWT; ++i)
          acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_v, cur.w[i][s]),
              __builtin_bit_cast(bf16x8_v, xf), acc[i][b], 0, 0, 0);
      }
    if constexpr (kStageX) wave_sync();
    cur = nxt;
  }
  if constexpr (kStageX) __syncthreads();   // red takes the stages' place
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

template <int NTB, bool kStageX, int RT, int EPI, int ACT>
hipError_t thin_rt(const ThinParams& P, hipStream_t s) {
  hipLaunchKernelGGL((ffn_thin_kernel<NTB, kStageX, RT, EPI, ACT>),
                     dim3((P.N + RT - 1) / RT), dim3(512), 0, s, P);
  return hipGetLastError();
}

template <int EPI, int ACT>
hipError_t thin(const ThinParams& P, hipStream_t s) {
  const ThinPlan r = thin_plan(P.T, P.N);
  const bool narrow = r.rows == 8;
  if (!r.staged)
    return narrow ? thin_rt<1, false, 8, EPI, ACT>(P, s)
                  : thin_rt<1, false, 16, EPI, ACT>(P, s);
  if (r.blocks == 1)
    return narrow ? thin_rt<1, true, 8, EPI, ACT>(P, s)
                  : thin_rt<1, true, 16, EPI, ACT>(P, s);
  if (r.blocks == 2)
    return narrow ? thin_rt<2, true, 8, EPI, ACT>(P, s)
                  : thin_rt<2, true, 16, EPI, ACT>(P, s);
  return thin_rt<4, true, 8, EPI, ACT>(P, s);
}

// ---------------------------------------------------------- tile launches
template <int WM, int WN, int NG, bool AKC, bool BKC, int EPI, int ACT>
hipError_t tile_w(TileParams P, int splits, hipStream_t s) {
  constexpr int wn = EPI == kAct ? WN / 2 : WN;
  P.mtn = (P.M + WM - 1) / WM;
  P.ntn = (P.N + wn - 1) / wn;
  hipLaunchKernelGGL((ffn_tile_kernel<WM, WN, NG, AKC, BKC, EPI, ACT>),
                     dim3(static_cast<uint32_t>(P.mtn) * P.ntn, splits),
                     dim3(256 * NG), 0, s, P);
  return hipGetLastError();
}

template <bool AKC, bool BKC, int EPI, int ACT>
hipError_t tile(TileParams P, const Plan& r, hipStream_t s) {
  P.kchunk = r.kchunk;
  if (r.width == 64 && r.height == 64)
    return r.groups == 1
               ? tile_w<64, 64, 1, AKC, BKC, EPI, ACT>(P, r.splits, s)
               : tile_w<64, 64, 2, AKC, BKC, EPI, ACT>(P, r.splits, s);
  if (r.width == 64)
    return r.groups == 1
               ? tile_w<128, 64, 1, AKC, BKC, EPI, ACT>(P, r.splits, s)
               : tile_w<128, 64, 2, AKC, BKC, EPI, ACT>(P, r.splits, s);
  return r.groups == 1
             ? tile_w<128, 128, 1, AKC, BKC, EPI, ACT>(P, r.splits, s)
             : tile_w<128, 128, 2, AKC, BKC, EPI, ACT>(P, r.splits, s);
}

template <int W, int EPI, int ACT>
hipError_t pair_w(PairParams P, hipStream_t s) {
  for (TileParams* t : {&P.a, &P.b}) {
    t->mtn = (t->M + W - 1) / W;
    t->ntn = (t->N + W - 1) / W;
  }
  P.b_first = P.b.kchunk > P.a.kchunk;
  const uint32_t grid = static_cast<uint32_t>(P.a.mtn) * P.a.ntn *
                            P.splits_a +
                        static_cast<uint32_t>(P.b.mtn) * P.b.ntn;
  hipLaunchKernelGGL((ffn_pair_kernel<W, EPI, ACT>), dim3(grid), dim3(256), 0,
                     s, P);
  return hipGetLastError();
}

template <int EPI, int ACT>
hipError_t pair(const TileParams& a, const TileParams& b, const Plan& r,
                hipStream_t s) {
  PairParams P{a, b, r.splits, 0};
  P.a.kchunk = r.kchunk;
  return r.width == 64 ? pair_w<64, EPI, ACT>(P, s)
                       : pair_w<128, EPI, ACT>(P, s);
}

hipError_t finish_rows(const float* planes, int n_planes, int64_t n,
                       const bf16_t* add, bf16_t* out, hipStream_t s) {
  int64_t nb = (n / 8 + 255) / 256;
  if (nb > 4096) nb = 4096;
  hipLaunchKernelGGL(ffn_rows_kernel, dim3(static_cast<uint32_t>(nb)),
                     dim3(256), 0, s, planes, n_planes, n, add, out);
  return hipGetLastError();
}

size_t up256(int64_t v) {
  return (static_cast<size_t>(v) + 255) & ~static_cast<size_t>(255);
}

TileParams row_params(const bf16_t* A, const bf16_t* B, int64_t ldb,
                      int64_t T, int64_t N, int64_t K) {
  TileParams P{};
  P.A = A; P.lda = K;
  P.B = B; P.ldb = ldb; P.b_rows = N;
  P.M = static_cast<int>(T); P.N = static_cast<int>(N);
  P.K = static_cast<int>(K);
  return P;
}

// out[T][N] = add + A . B (B K-contiguous or not).
template <bool BKC>
hipError_t row_product(const bf16_t* A, const bf16_t* B, int64_t ldb,
                       int64_t T, int64_t N, int64_t K, const bf16_t* add,
                       bf16_t* out, float* planes, hipStream_t s) {
  const Plan r = row_plan(T, N, K);
  if (r.width == 256)
    return gemm_dense_rows(A, B, BKC, T, N, K, add, out, s);
  TileParams P = row_params(A, B, ldb, T, N, K);
  if (r.splits == 1) {
    P.C = out; P.ldc = N; P.AB = add;
    return tile<true, BKC, kRow, kActSilu>(P, r, s);
  }
  P.Cf = planes;
  hipError_t e = tile<true, BKC, kPlane, kActSilu>(P, r, s);
  if (e != hipSuccess) return e;
  return finish_rows(planes, r.splits, T * N, add, out, s);
}

// c[M][N] = sum_t a[t][m] b[t][n]
TileParams weight_params(const bf16_t* a, const bf16_t* b, int64_t T,
                         int64_t M, int64_t N, bf16_t* c) {
  TileParams P{};
  P.A = a; P.lda = M;
  P.B = b; P.ldb = N;
  P.M = static_cast<int>(M); P.N = static_cast<int>(N);
  P.K = static_cast<int>(T);
  P.kchunk = (P.K + kBK - 1) / kBK * kBK;
  P.C = c; P.ldc = N;
  return P;
}
hipError_t weight_product(const bf16_t* a, const bf16_t* b, int64_t T,
                          int64_t M, int64_t N, bf16_t* c, hipStream_t s) {
  const Plan r = weight_plan(T, M, N);
  if (r.width == 256) return gemm_dense_wgrad(a, b, T, M, N, c, s);
  return tile<false, false, kRow, kActSilu>(
      weight_params(a, b, T, M, N, c), r, s);
}

template <int ACT>
hipError_t fc1(const bf16_t* x, const bf16_t* w_gu, int64_t T, int64_t d,
               int64_t f, bf16_t* ab, bf16_t* s_out, hipStream_t s) {
  if (thin_form(T, d, f)) {
    ThinParams P{};
    P.W = w_gu; P.X = x;
    P.T = static_cast<int>(T); P.N = static_cast<int>(f);
    P.K = static_cast<int>(d);
    P.C = ab; P.S = s_out;
    return thin<kAct, ACT>(P, s);
  }
  const Plan r = fc1_plan(T, d, f);
  if (r.width == 256)
    return gemm_dense_fc1_fwd(x, w_gu, T, d, f, ACT, ab, s_out, s);
  TileParams P{};
  P.A = x; P.lda = d;
  P.B = w_gu; P.ldb = d; P.b_rows = 2 * f;
  P.M = static_cast<int>(T); P.N = static_cast<int>(f);
  P.K = static_cast<int>(d);
  P.C = ab; P.ldc = 2 * f; P.S = s_out;
  return tile<true, true, kAct, ACT>(P, r, s);
}

// dAB, and dW2 unless it is null.
template <int ACT>
hipError_t dact_dw2(const bf16_t* dy, const bf16_t* w2, const bf16_t* ab,
                    const bf16_t* s_saved, int64_t T, int64_t d, int64_t f,
                    bf16_t* dab, bf16_t* dw2, hipStream_t s) {
  TileParams P = row_params(dy, w2, f, T, f, d);
  P.C = dab; P.ldc = 2 * f; P.AB = ab;
  if (dw2) {
    const Plan both = dact_pair(T, d, f);
    if (both.width)
      return pair<kDAct, ACT>(P, weight_params(dy, s_saved, T, d, f, dw2),
                              both, s);
    hipError_t e = weight_product(dy, s_saved, T, d, f, dw2, s);
    if (e != hipSuccess) return e;
  }
  const Plan r = dact_plan(T, d, f);
  if (r.width == 256)
    return gemm_dense_fc2_dgrad(dy, w2, T, d, f, ACT, ab, dab, s);
  return tile<true, false, kDAct, ACT>(P, r, s);
}

// dx and dW_gu, either of them null to skip it.
hipError_t dx_dw_gu(const bf16_t* dab, const bf16_t* x, const bf16_t* w_gu,
                    const bf16_t* dx_add, int64_t T, int64_t d, int64_t f,
                    bf16_t* dx, bf16_t* dw_gu, float* planes,
                    hipStream_t s) {
  if (dx && dw_gu) {
    const Plan r = dx_pair(T, d, f);
    if (r.width) {
      TileParams P = row_params(dab, w_gu, d, T, d, 2 * f);
      const TileParams Q = weight_params(dab, x, T, 2 * f, d, dw_gu);
      if (r.splits == 1) {
        P.C = dx; P.ldc = d; P.AB = dx_add;
        return pair<kRow, kActSilu>(P, Q, r, s);
      }
      P.Cf = planes;
      hipError_t e = pair<kPlane, kActSilu>(P, Q, r, s);
      if (e != hipSuccess) return e;
      return finish_rows(planes, r.splits, T * d, dx_add, dx, s);
    }
  }
  if (dw_gu) {
    hipError_t e = weight_product(dab, x, T, 2 * f, d, dw_gu, s);
    if (e != hipSuccess || !dx) return e;
  }
  if (!dx) return hipSuccess;
  return row_product<false>(dab, w_gu, d, T, d, 2 * f, dx_add, dx, planes, s);
}

// Workspaces.  Forward: S (when the caller keeps none), then the fp32
// planes of y.  Backward: dAB, then the planes of dx.
int64_t plane_bytes(int64_t T, int64_t N, int64_t K) {
  const Plan r = row_plan(T, N, K);
  return r.splits > 1 ? r.splits * T * N * 4 : 0;
}

}  // namespace

size_t ffn_fwd_workspace(int64_t T, int64_t d, int64_t f) {
  return up256(T * f * 2) +
         (thin_form(T, d, f) ? 0 : up256(plane_bytes(T, d, f)));
}

size_t ffn_bwd_workspace(int64_t T, int64_t d, int64_t f) {
  const Plan r = dx_pair(T, d, f);
  const int64_t alone = plane_bytes(T, d, 2 * f);
  const int64_t both = r.width && r.splits > 1 ? r.splits * T * d * 4 : 0;
  return up256(T * 2 * f * 2) + up256(alone > both ? alone : both);
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
  if (thin_form(T, d, f)) {
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
  if (!dx && !dw_gu) return weight_product(dy, s_saved, T, d, f, dw2, s);
  bf16_t* dab = static_cast<bf16_t*>(ws);
  float* planes = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                           up256(T * 2 * f * 2));
  hipError_t e =
      act == kActSilu
          ? dact_dw2<kActSilu>(dy, w2, ab, s_saved, T, d, f, dab, dw2, s)
          : dact_dw2<kActGeluTanh>(dy, w2, ab, s_saved, T, d, f, dab, dw2, s);
  if (e != hipSuccess) return e;
  return dx_dw_gu(dab, x, w_gu, dx_add, T, d, f, dx, dw_gu, planes, s);
}

}  // namespace moe
