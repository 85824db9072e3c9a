// Which form each product of the dense gated feed-forward block takes
// (ffn.hip launches them).  Host code without HIP, so that a test can ask for
// the forms of a size.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kBK = 64;      // reduction length of a k-step
// bytes of a buffer resource (kMaxResourceBytes of internal.h)
constexpr int64_t kMaxOperandBytes = 0xffffff00;

// The form of one product: output tiles of `height` x `width` (256 x 256 for
// the grouped GEMM's kernel), `groups` of 256 threads a tile, the reduction in
// `splits` ranges of kchunk.
struct Plan {
  int height, width, groups, splits, kchunk;
  double us;           // estimated time
};

// Workgroups of 256 threads that one launch holds (2^32 threads).
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;

// A form's output tile, and the microseconds that a CU with n such tiles
// takes: a + b n for a k-step of all of them, c n for what no k-step covers
// (see plan).
struct TileCost {
  int height, width;
  double a, b, c;
};
constexpr TileCost kTiles[] = {{64, 64, 0.15, 0.16, 0.6},
                               {128, 64, 0.05, 0.31, 1.25},
                               {128, 128, 0.08, 0.43, 2.5},
                               {256, 256, 0.0, 1.3, 6.0}};

// Microseconds of moving the operands and the result of a product once.
inline double move_us(int64_t M, int64_t N, int64_t K) {
  const double m = static_cast<double>(M), n = static_cast<double>(N),
               k = static_cast<double>(K);
  return 2 * (m * k + n * k + m * n) / 4.5e6;
}

// Microseconds of summing `splits` fp32 planes of M x N.
inline double planes_us(int64_t splits, int64_t M, int64_t N) {
  return splits < 2 ? 0.0
                    : 4 + static_cast<double>(splits * M) *
                              static_cast<double>(N) * 8 / 4e6;
}

// The form with the least estimated time.  cols: output columns of a
// width-256 tile (128 where a tile holds gate and up).  split: the reduction
// may be cut over workgroups (row outputs, through fp32 planes).
//
// A CU with n tiles of a form takes a + b n microseconds for a k-step of all
// of them, and c n to fill the pipeline and to write the results (about 3.4
// TB/s, hardly overlapped); n lies between the mean and the fullest CU's
// tiles.  kTiles holds the values measured on MI355X over T = 65..4096, d =
// 2048 and 4096, f = 1408..14336.  Per output the 128-wide tile costs half
// of the 64-wide one, but 88 tiles of 256 leave two thirds of the CUs idle
// (dS of 2000 x 2816 over 2048: 43, 38 and 49 us at 64, 128 and 256).  128 x
// 64 stands between where its tiles just fill the CUs: 777 x 2048 over 2816,
// of 416, 224 and 112 tiles, 21.4, 18.8 and 22.9 us; 128 x 14336 over 4096
// 44, 36 and 44 us (64 x 128 is within 3% of it).  Two groups act as twice
// the tiles for half the steps (45 128-wide tiles: 23.7 -> 20.2 us).
// Cutting the reduction adds a pass over the planes at about 4 TB/s and a
// launch; it pays where few tiles meet a long reduction (128 x 4096 over
// 14336: 70 -> 47 us) and costs where the tiles fill the CUs (2000 x 2048
// over 2816: 27 -> 37 us).
inline Plan plan(int64_t M, int64_t N, int64_t K, int64_t cols, bool split,
          bool allow256 = true) {
  const int64_t steps = (K + kBK - 1) / kBK;
  const double least = move_us(M, N * (256 / cols), K);
  Plan best{};
  double best_us = 1e30;
  for (const TileCost& t : kTiles) {
    const bool large = t.width == 256;
    if (large && !allow256) break;
    const int64_t h = t.height, c = cols * t.width / 256;
    const int64_t tiles = ((M + h - 1) / h) * ((N + c - 1) / c);
    for (int64_t sp = 1; sp <= (split && !large ? 8 : 1); sp *= 2) {
      if (sp > 1 && sp * 4 > steps) break;       // at least 4 steps a split
      if (tiles * sp > kMaxGroups / 2) break;
      const int64_t per = (steps + sp - 1) / sp;
      const int64_t full = (tiles * sp + 255) / 256;
      const double n = full == 1 ? 1.0
                                 : 0.5 * static_cast<double>(full) +
                                       static_cast<double>(tiles * sp) / 512;
      for (int g = 1; g <= 2; ++g) {
        if (g == 2 && (large || full > 1)) break;
        double us = (t.a + t.b * g * n) *
                        static_cast<double>((per + g - 1) / g) +
                    t.c * n + 1 + g + planes_us(sp, M, N);
        if (us < best_us) {
          best_us = us;
          best = Plan{t.height, t.width, g,
                      static_cast<int>((steps + per - 1) / per),
                      static_cast<int>(per * kBK), us};
        }
      }
    }
  }
  if (best.us < least) best.us = least;
  return best;
}

// The same for a row product a (M x Na over Ka; split: its reduction may be
// cut) and a weight gradient b (Mb x Nb over M rows) in one launch of
// `width`-wide tiles, which fill the CUs together: all k-steps at the full
// CU's rate, half of the longest tile for the ragged end, and a quarter of
// the writes (the rest overlaps other tiles' k-steps).  Width 0: not better
// than the two launches, which take `apart`; also where the pair would be
// bound by memory (within a quarter of it), since interleaving two such
// streams costs more than a launch.  (Backward of 64 x 2048 x 1408: 37 us
// apart, 31 us in pairs; of 2000 x 2048 x 1408: 104 and 97 us; of 64 x 4096
// x 14336, bound by memory: 209 and 233 us.)
inline Plan pair_plan(int64_t M, int64_t Na, int64_t Ka, bool split, int64_t Mb,
               int64_t Nb, double apart) {
  const double least = move_us(M, Na, Ka) + move_us(Mb, Nb, M);
  Plan best{0, 0, 1, 1, 0, apart};
  const int64_t sa = (Ka + kBK - 1) / kBK, sb = (M + kBK - 1) / kBK;
  for (const TileCost& t : kTiles) {
    if (t.width != t.height || t.width == 256) continue;
    const int64_t w = t.width;
    const double ta = static_cast<double>((M + w - 1) / w) *
                      static_cast<double>((Na + w - 1) / w);
    const double tb = static_cast<double>((Mb + w - 1) / w) *
                      static_cast<double>((Nb + w - 1) / w);
    for (int64_t sp = 1; sp <= (split ? 8 : 1); sp *= 2) {
      if (sp > 1 && sp * 4 > sa) break;
      if (ta * static_cast<double>(sp) + tb > kMaxGroups) break;
      const int64_t per = (sa + sp - 1) / sp;
      const double work = (ta * static_cast<double>(sa) +
                           tb * static_cast<double>(sb)) * t.b / 256;
      const double one = static_cast<double>(per > sb ? per : sb) *
                         (t.a + t.b);
      const double us = (work > one ? work : one) + 0.5 * one + 2 +
                        t.c * (ta * static_cast<double>(sp) + tb) / 1024 +
                        planes_us(sp, M, Na);
      if (us > 1.25 * least && us < best.us)
        best = Plan{static_cast<int>(w), static_cast<int>(w), 1,
                    static_cast<int>((sa + per - 1) / per),
                    static_cast<int>(per * kBK), us};
    }
  }
  return best;
}

// The first product [gate up] = x . w_gu^T with its activation; tiles of half
// the width in gate columns.
inline Plan fc1_plan(int64_t T, int64_t d, int64_t f) {
  return plan(T, f, d, 128, false);
}

// A row product [T][N] = [T][K] . B: y and dx.
inline Plan row_plan(int64_t T, int64_t N, int64_t K) {
  return plan(T, N, K, 256, true);
}

// dS = dy . w2 with the activation's slope, [dA dU].
inline Plan dact_plan(int64_t T, int64_t d, int64_t f) {
  return plan(T, f, d, 256, false);
}

// A weight gradient [M][N], a sum over T.
inline Plan weight_plan(int64_t T, int64_t M, int64_t N) {
  // the 256-wide kernel addresses an operand's rows with 32 bits
  const bool fits = T * (M > N ? M : N) * 2 <= kMaxOperandBytes;
  return plan(M, N, T, 256, false, fits);
}
// A second launch costs about this much more than its kernel.
constexpr double kLaunchUs = 2;

// The launch of [dA dU] together with dW2 (width 0: apart).
inline Plan dact_pair(int64_t T, int64_t d, int64_t f) {
  const double apart = dact_plan(T, d, f).us + weight_plan(T, d, f).us +
                       kLaunchUs;
  return pair_plan(T, f, d, false, d, f, apart);
}

// The launch of dx together with dW_gu (width 0: apart).
inline Plan dx_pair(int64_t T, int64_t d, int64_t f) {
  const double apart = row_plan(T, d, 2 * f).us +
                       weight_plan(T, 2 * f, d).us + kLaunchUs;
  return pair_plan(T, d, 2 * f, true, 2 * f, d, apart);
}

// Whether the weight-streaming form runs.  Its time grows with the tokens
// (every workgroup reads all of them), the tiles' hardly does up to 64, but
// tiles of narrow blocks leave CUs idle.  Forward on MI355X in a captured
// sequence over data that leaves the caches, thin and tiles, us: 16 tokens 9
// and 16 (d 2048, f 1408), 15 and 20 (2048, 2816), 27 and 32 (4096, 4096), 80
// and 78 (4096, 14336); 24 tokens 11 and 17, 20 and 20, 31 and 33, 97 and 76;
// 64 tokens 15 and 18, 28 and 23, 58 and 39, 176 and 85.
inline bool thin_form(int64_t T, int64_t d, int64_t f) {
  const int64_t bytes = 6 * d * f;
  return T <= 16 || (T <= 32 && bytes <= (int64_t{128} << 20)) ||
         (T <= 64 && bytes <= (int64_t{24} << 20));
}

// The instance of the weight-streaming form for T <= 64 tokens and N outputs
// (gate columns): token blocks of 16, whether x is staged through LDS, and
// outputs a workgroup.
struct ThinPlan {
  int blocks;
  bool staged;
  int rows;
};

// Tokens whose fragments are loaded straight from x.
constexpr int kDirectTokens = 4;

inline ThinPlan thin_plan(int64_t T, int64_t N) {
  // 8 rows where 16 would leave CUs without a workgroup; four token blocks
  // leave no registers for a second weight tile
  const int rows = N < 16 * 256 || T > 32 ? 8 : 16;
  return {T <= 16 ? 1 : T <= 32 ? 2 : 4, T > kDirectTokens, rows};
}

}  // namespace moe
