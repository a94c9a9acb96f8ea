// Which kernel runs an 8-bit product or input gradient, and in what tiles: the
// cheapest by estimates of their times.  Host code alone, without HIP, so that a
// test can ask it on the CPU which path a size takes.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace lbq {

constexpr int I8K = 64;  // codes in a slice of K

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Few short tokens are quantized by the product's own launch, k_i8_decode: one
// launch and no workspace where the others take a quantizer's launch first.  Called
// one after another, that and one launch, in us (m x k through n):
//   1 x 1024, 4096: 8.0, 5.5    1 x 4096, 4096: 9.2, 8.5    1 x 16384, 4096: 20.6, 19.3
//   1 x 8192, 14336: 31.2, 26.8  1 x 16384, 14336: 58.2, 50.0  4 x 4096, 4096: 10.3, 10.2
// and, where there are many workgroups or several longer tokens, each workgroup's
// quantizing costs more than the launch it saves:
//   1 x 1024, 14336: 8.6, 10.0  4 x 4096, 14336: 18.8, 21.2    2 x 8192, 4096: 12.4, 13.5
// The limit is what leaves two workgroups on a CU (48 KiB of rings and the codes):
// with twice as many codes 1 x 4096 through 14336 takes 26.8 instead of 18.2, and 1 x
// 28672 through 4096 30.2 where two launches take 31.2.
constexpr int kI8DecodeCodes = 16384;
inline bool i8_decode_fits(int64_t m, int64_t k) { return m <= 4 && m * k <= kI8DecodeCodes; }

// Tiles of one launch: 256 x 256 outputs each, numbered over all the weights'
// row tiles; the first `whole` of them by one workgroup each, the others cut
// into `cut` pieces (2: 128 x 256, 4: 128 x 128).  With whole = 0 the pieces
// themselves are numbered, nx x ny of them: workgroups that find their piece
// past the end would leave the others to a part of the chip, since workgroups
// go round the shader engines in turn (m = 128, n = 18965, k = 2624: 42.1 us
// against 25.2).  With ks > 1 (only where nothing is whole) K is split into ks
// ranges of `per` slices, gridDim.y of them, whose integer sums k_i8_reduce adds.
struct I8Plan {
  int nx, ny;
  int whole, cut;
  int ks, per;
};

// How a product of count weights of ns channels runs: by k_i8_skinny with tiles
// of 16 tn channels and 16 tm tokens, or (tn 0) by k_i8_gemm as `plan` says.
struct I8Choice {
  int tn, tm;
  I8Plan plan;
};

constexpr int64_t kMostGridY = 65535;

// Tiles of k_i8_skinny and what they cost (us): `base`, and a round of `room`
// workgroups `start`, and for a 128-byte line of a wave `line` and, where all of the
// room is taken, `share`; `read` for a byte of the weights.  All of them are what
// fitted the times best, none below 0 and `room` of 256, 512 and 768: no count of
// what a CU holds (LDS has room for two workgroups of 16 x 16, 64 x 16 and 32 x 32
// tiles and for three of 32 x 16, which share what comes to the CU).
struct I8Skinny {
  int tn, tm, room;
  double base, start, line, share, read;
};
constexpr I8Skinny kI8Skinny[] = {
    {1, 1, 256, 2.38, 0.21, 0.401, 0.104, 0.110e-6}, {2, 1, 512, 2.33, 0.00, 0.615, 1.141, 0.122e-6},
    {4, 1, 256, 2.20, 0.00, 1.234, 0.344, 0.147e-6}, {2, 2, 256, 2.40, 0.00, 0.832, 0.356, 0.110e-6},
    {4, 2, 256, 1.51, 0.89, 1.288, 0.733, 0.131e-6}, {4, 4, 256, 1.28, 1.94, 1.599, 1.025, 0.109e-6}};

// The cheapest by an estimate in microseconds, fitted to the times of all of
// them on 1400 products (m 1 to 3000, n 256 to 28672, k 256 to 28672, weights not in
// cache): on these the choice is 2.3% off the best one on average.
//  * k_i8_skinny: rounds of workgroups, each at a rate for a 128-byte line of a wave
//    that grows with the CUs at work.  (Its tokens are the grid's second dimension,
//    which has 65535 workgroups.)
//  * k_i8_gemm: the same with a rate for 64 of k: in 256 x 256 tiles whose last
//    round is cut where it would leave half of the chip idle (128 x 256 pieces) or
//    three quarters (128 x 128), or all in tiles or pieces of one size; 128 x 128
//    pieces may split K, which costs a second launch and the traffic of the sums.
inline I8Choice i8_choose(const int64_t* ns, int count, int64_t k, int64_t m, bool split) {
  // us of `groups` workgroups, `room` of them at a time: each costs `steps` steps
  // of `step` and `share` where all of the room is taken
  const auto rounds = [](double groups, int room, double start, double step, double share, double steps) {
    const double r = groups / room, full = std::floor(r);
    double us = full * (start + steps * (step + share));
    if (r > full) us += start + steps * (step + share * (r - full));
    return us;
  };
  I8Choice best{};
  double least = 1e30;
  int64_t n = 0, tiles = 0;
  for (int i = 0; i < count; ++i) n += ns[i], tiles += ceil_div(ns[i], 256) * ceil_div(m, 256);
  for (const I8Skinny& c : kI8Skinny) {
    int64_t groups = 0;
    if (ceil_div(m, 16 * c.tm) > kMostGridY) continue;
    for (int j = 0; j < count; ++j) groups += ceil_div(ns[j], 16 * c.tn);
    groups *= ceil_div(m, 16 * c.tm);
    const double us = c.base + rounds((double)groups, c.room, c.start, c.line, c.share, (double)ceil_div(k, 1024)) +
                      c.read * (double)n * k;
    if (us < least) least = us, best.tn = c.tn, best.tm = c.tm;
  }
  const int slices = (int)(k / I8K);
  const auto plan = [&](int64_t whole, int cut) {
    I8Plan p{};
    const int tn = whole > 0 ? 256 : 128;
    for (int i = 0; i < count; ++i) p.nx += (int)ceil_div(ns[i], tn);
    p.ny = (int)ceil_div(m, whole > 0 || cut == 2 ? 256 : 128);
    p.whole = (int)whole, p.cut = cut, p.ks = 1, p.per = slices;
    return p;
  };
  const auto consider = [&](I8Plan p) {
    const int64_t pieces = p.whole > 0 ? (tiles - p.whole) * p.cut : (int64_t)p.nx * p.ny;
    double us = 3.1 + (double)(n + m) * k * 0.070e-6 + rounds(p.whole, 256, 8.19, 0.357, 0.349, slices);
    us += p.cut == 2 ? rounds((double)pieces, 256, 3.69, 0.309, 0.124, slices)
                     : rounds((double)pieces * p.ks, 256, 1.96, 0.183, 0.078, p.per);
    if (p.ks > 1) us += 3.4 + 0.44e-6 * 4 * p.ks * m * n;
    if (us < least) least = us, best = {0, 0, p};
  };
  const int64_t rest = tiles % 256;
  if (tiles > 256 && rest > 0 && rest <= 128) consider(plan(tiles - rest, rest <= 64 ? 4 : 2));
  consider(plan(tiles, 2));
  consider(plan(0, 2));
  for (int ks = 1; ks <= 8; ++ks) {
    if (ks > 1 && (!split || tiles > 64 || slices < 4 * ks)) break;
    I8Plan p = plan(0, 4);
    p.per = (int)ceil_div(slices, ks);
    p.ks = (int)ceil_div(slices, p.per);
    consider(p);
  }
  return best;
}

// How an input gradient runs: by k_i8_dx with 16 tm tokens and ks ranges of `per`
// slices, or (tm 0) by k_bwd_dx's bk x bm tiles.
struct I8DxChoice {
  int tm, ks, per;
  int bk, bm;
};
constexpr double kI8DxMostPart = 256e6;  // bytes of sums of a split reduction

// The cheapest by an estimate in microseconds, fitted to the times of all of
// them on 300 input gradients (m 1 to 3000, n 256 to 28672, k 256 to 28672, weights
// not in cache): on these the choice is 2% off the best one on average.
//  * k_i8_dx: a round is one workgroup a CU (their rings fill its LDS), and costs
//    its slices at a rate that grows with the CUs at work; a split adds a second
//    launch and the traffic of the sums.  (An estimate that went on linearly past
//    one round chose 384 workgroups for 256 CUs: m = 40, n = 14336, k = 4096 34.8 us
//    against 27.7 with four ranges.)
//  * k_bwd_dx, per 64 rows: 0.713 a round of 128 x 128 tiles and 0.302, 1.20 a round
//    of 256 x 128, 1.78 a round of 256 x 256.
inline I8DxChoice i8_dx_choose(const int64_t* ns, int count, int64_t k, int64_t m, bool split) {
  static constexpr double kBase[3] = {2.27, 2.25, 2.43}, kRound[3] = {1.31, 1.45, 1.84}, kSlice[3] = {0.0675, 0.075, 0.0955},
                          kShare[3] = {0.0192, 0.0215, 0.0366}, kRead[3] = {0.138e-6, 0.119e-6, 0.080e-6},
                          kSums[3] = {2.77e-6, 2.38e-6, 2.10e-6};
  int64_t slices = 0, n = 0;
  for (int i = 0; i < count; ++i) slices += ceil_div(ns[i], 32), n += ns[i];
  I8DxChoice best{};
  double least = 1e30;
  for (int t = 0; t < 3; ++t) {
    const int tm = 1 << t;
    for (int want : {1, 2, 3, 4, 6, 8}) {
      const int per = (int)ceil_div(slices, want), ks = (int)ceil_div(slices, per);
      if (ks > 1 && (!split || 4.0 * ks * m * k > kI8DxMostPart)) break;
      const double r = (double)(k / 64 * ceil_div(m, 16 * tm)) * ks / 256, full = std::floor(r);
      double us = kBase[t] + full * (kRound[t] + per * (kSlice[t] + kShare[t])) + kRead[t] * (double)n * k;
      if (r > full) us += kRound[t] + per * (kSlice[t] + kShare[t] * (r - full));
      if (ks > 1) us += 2.0 + kSums[t] * ks * m * k;
      if (us < least) least = us, best = {tm, ks, per, 0, 0};
    }
  }
  const double stages = std::ceil(n / 64.0);
  const double t128 = 3.3 + stages * (0.713 * std::ceil(ceil_div(k, 128) * ceil_div(m, 128) / 256.0) + 0.302);
  const double t256x128 = 4.2 + stages * 1.20 * std::ceil(ceil_div(k, 256) * ceil_div(m, 128) / 256.0);
  const double t256 = 5.2 + stages * 1.78 * std::ceil(ceil_div(k, 256) * ceil_div(m, 256) / 256.0);
  if (t128 < least) least = t128, best = {0, 1, 0, 128, 128};
  if (t256x128 < least) least = t256x128, best = {0, 1, 0, 256, 128};
  if (t256 < least) least = t256, best = {0, 1, 0, 256, 256};
  return best;
}

}  // namespace lbq
