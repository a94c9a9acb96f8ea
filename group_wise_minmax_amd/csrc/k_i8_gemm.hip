// Products of 8-bit integers with one scale for each token and each output
// channel (the INT8 weight format):
//   Y[i][j] = bf16( fl(fl(fl(acc) * sx[i]) * sw[j]) ),  acc = sum_k Xq[i][k] Wq[j][k]
// on v_mfma_i32_16x16x64_i8.  acc is exact in 32-bit integers (k <= 2^17:
// 127 * 127 * 2^17 < 2^31), so the result does not depend on the order of the
// sum, on the tile or on how K is split: every kernel here gives the same bits.
//
// A workgroup (one a CU, eight waves) computes 256 x 256 outputs, or a piece of
// that where the tiles leave CUs idle; K goes through four LDS stages of 64 codes,
// loaded straight to LDS three steps ahead.  What bounds it:
//  * large products the card's power: the MFMAs alone run at 4.9 POP/s on zeros
//    and at 4.0 on random codes (32 x 32 x 32 shapes: 3.45, they take more power);
//    m = 4096, n = 14336, k = 4096 200 us (2.4 POP/s; the library's product 217 to
//    235), m = n = k = 8192 415 us, and 320 us with all codes 0.  Each wave takes
//    128 x 64, so that its LDS reads (12 KiB for 32 MFMAs) fit under them (four
//    waves of 128 x 128: 249 us where these took 247); loads are spread between
//    the MFMAs (issued together 259 and 247).
//  * pieces the operands: 80 to 92 bytes a ns come to a CU from L2 (m = 333, n = k
//    = 8192 40.6 us).  Fewer LDS reads (64 x 64 a wave, two groups of waves that
//    take a slice each) and operands read a whole step ahead gained nothing: 41.3
//    and 45.5 us.
#pragma clang fp contract(off)

#include "lbq_device.h"

#include <algorithm>

namespace lbq {

namespace {

// 64 codes of K of a tile in LDS: BN rows of W and BM rows of X, 64 bytes each, in
// the order of i8_key (no bank conflicts; rows in plain order have 2.2e7 conflict
// cycles in m = 4096, n = 14336, k = 4096).
template <int BN, int BM>
struct I8Stage {
  int8_t w[BN * 64];
  int8_t x[BM * 64];
};

// Channels of a token's partial sums: 16 bytes at a time for any n.
__host__ __device__ constexpr int padded(int n) { return (n + 3) & ~3; }

// Order of a half step's instructions: R LDS reads and L loads, one after each
// MFMA, then the rest of the M MFMAs.
template <int R, int L, int M>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
  __builtin_amdgcn_sched_barrier(0);
}

constexpr int kGemmThreads = 512;
constexpr int kGemmLds = 1 << 17;  // bytes of LDS for the stages
constexpr int kGemmOut = 1 << 15;  // and for the outputs on their way to memory
constexpr int kStages = 4;
// A K step of a tile, one stage in LDS, is KS slices of 64 codes: the barrier
// of a step costs some 300 cycles, so a step holds at least 512 cycles of a
// SIMD's MFMAs (128 x 128 pieces: 2 slices; m = 130, n = k = 4096 22.6 -> 20.2 us,
// m = 333, n = k = 8192 50.7 -> 42.0).
template <int BN, int BM>
constexpr int i8_slices() {
  return kStages * 2 * (int)sizeof(I8Stage<BN, BM>) <= kGemmLds ? 2 : 1;
}

// The BN x BM outputs from channel n0 of weight wi and token m0 on, by WGN x
// WGM waves, summed over `slices` slices of K from s0 on.  With PART the integer
// sums go to part, [m][padded(n)], where that is not null.
template <int BN, int BM, int WGN, int WGM, bool LORA, bool PART>
__device__ __forceinline__ void i8_tile(const I8Set& set, const int8_t* __restrict__ Xq, const float* __restrict__ xs,
                                        int m, int k, const LoraEpi& lora, int wi, int n0, int m0, int s0, int slices,
                                        int* __restrict__ part, int8_t* lds) {
  constexpr int NW = WGN * WGM;
  constexpr int TN = BN / WGN / 16, TM = BM / WGM / 16, TH = TN / 2;
  constexpr int LW = BN / 16 / NW, LX = BM / 16 / NW;  // 1-KiB pieces (16 rows) a wave loads of each operand
  static_assert(NW * 64 == kGemmThreads && LW * NW * 16 == BN && LX * NW * 16 == BM, "whole pieces");
  constexpr int S = kStages, KS = i8_slices<BN, BM>();
  auto& st = *reinterpret_cast<I8Stage<BN, BM>(*)[S][KS]>(lds);
  static_assert(sizeof(st) <= kGemmLds, "stages fit");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // the same in the wave: scalar load offsets
  const int wn = wave % WGN, wm = wave / WGN;
  const int n = set.n[wi];

  // Global loads go straight to LDS: a wave's load fills 16 rows, lane l the
  // 16 bytes at position l % 4 of row l / 4, which hold chunk (l % 4) ^ key(row).
  // Rows past the end load the last row instead (their outputs are not stored).
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(set.w[wi], (int64_t)n * k);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)m * k);
  const int lr = lane >> 2, lc = ((lane & 3) ^ i8_key(lr)) * 16;
  int ow[LW], ox[LX];
#pragma unroll
  for (int i = 0; i < LW; ++i) ow[i] = min(n0 + 16 * (wave * LW + i) + lr, n - 1) * k + lc;
#pragma unroll
  for (int i = 0; i < LX; ++i) ox[i] = min(m0 + 16 * (wave * LX + i) + lr, m - 1) * k + lc;
  // The loads of step t; slices past the last one repeat it (they are not
  // multiplied), so that the count of loads in flight stays what the wait says.
  auto at = [&](int t, int c) { return I8K * (s0 + min(KS * t + c, slices - 1)); };
  auto load_w = [&](int t) {
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int i = 0; i < LW; ++i) load_to_lds(rw, st[t % S][c].w + 1024 * (wave * LW + i), ow[i], at(t, c));
  };
  auto load_x = [&](int t) {
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int i = 0; i < LX; ++i) load_to_lds(rx, st[t % S][c].x + 1024 * (wave * LX + i), ox[i], at(t, c));
  };

  i32x4_t acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};

  // Operands of the MFMAs of a step: lane l holds chunk l / 16 of row l % 16
  // of a 16-row block.  The wave's W rows are multiplied in two halves.
  const int li = lane & 15, lg = lane >> 4;
  const uint32_t fc = li * 64 + 16 * (lg ^ i8_key(li));
  const uint32_t fw = wn * TN * 1024 + fc, fx = wm * TM * 1024 + fc;
  i32x4_t w0[TH], w1[TH], x0[TM], x1[TM];
  auto read_w = [&](const I8Stage<BN, BM>& st, int half, i32x4_t (&w)[TH]) {
#pragma unroll
    for (int a = 0; a < TH; ++a) w[a] = *reinterpret_cast<const i32x4_t*>(st.w + fw + (half * TH + a) * 1024);
  };
  auto read_x = [&](const I8Stage<BN, BM>& st, i32x4_t (&x)[TM]) {
#pragma unroll
    for (int b = 0; b < TM; ++b) x[b] = *reinterpret_cast<const i32x4_t*>(st.x + fx + b * 1024);
  };
  auto mma = [&](int half, const i32x4_t (&w)[TH], const i32x4_t (&x)[TM]) {
#pragma unroll
    for (int a = 0; a < TH; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[half * TH + a][b] = mfma_i8(w[a], x[b], acc[half * TH + a][b]);
  };

  // Step t lies in stage t % S.  While it is multiplied, steps t + 1 to t + S - 2
  // are on their way and the loads of step t + S - 1 are issued, spread between
  // the MFMAs (issued together they fill the load queue and hold up the wave's
  // MFMAs behind them).  The first operands of a step are read before the last
  // MFMAs of the one before it.
  //
  // In step t: step t + 1 is there, by this wave's loads (all but those of the
  // steps after it: vmcnt) and by the barrier every wave's; and every wave has
  // read step t.
  constexpr int kLater = KS * ((S - 3) * (LW + LX) + LW);
  static_assert(kLater < 16, "vmcnt's low four bits");
  auto arrive = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | kLater);  // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int steps = slices / KS;
#pragma unroll
  for (int t = 0; t < S - 1; ++t) {
    load_w(t);
    load_x(t);
  }
  arrive();
  read_w(st[0][0], 0, w0);
  read_x(st[0][0], x0);
  // xa: the tokens of this step's first slice, xb: those of the next slice
  auto step = [&](int t, i32x4_t (&xa)[TM], i32x4_t (&xb)[TM]) {
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      const I8Stage<BN, BM>& cur = st[t % S][c];
      const I8Stage<BN, BM>& next = c + 1 < KS ? st[t % S][c + 1] : st[(t + 1) % S][0];
      i32x4_t(&x)[TM] = (c & 1) ? xb : xa;
      i32x4_t(&y)[TM] = (c & 1) ? xa : xb;
      read_w(cur, 1, w1);
      if (c == 0) load_w(t + S - 1);
      mma(0, w0, x);
      interleave<TH, (KS == 1 ? LW : 0), TH * TM>();
      if (c + 1 == KS) arrive();
      read_w(next, 0, w0);
      read_x(next, y);
      if (c + 1 == KS) load_x(t + S - 1);
      mma(1, w1, x);
      interleave<TH + TM, (KS == 1 ? LX : 0), TH * TM>();
    }
  };
  int t = 0;
  for (; t + 1 < steps; t += 2) {
    step(t, x0, x1);
    if constexpr (KS == 1) step(t + 1, x1, x0);
    else step(t + 1, x0, x1);
  }
  if (t < steps) step(t, x0, x1);
  if (KS == 2 && slices % 2 != 0) {  // half a step
    read_w(st[steps % S][0], 1, w1);
    mma(0, w0, x0);
    mma(1, w1, x0);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // no load to LDS is left behind

  // Epilogue: lane l holds channels n = 4 (l / 16) + i of token m = l % 16.
  if (PART && part != nullptr) {
    const int n4 = padded(n);
#pragma unroll
    for (int b = 0; b < TM; ++b) {
      const int mr = m0 + (wm * TM + b) * 16 + li;
      if (mr >= m) continue;
      int* prow = part + (int64_t)mr * n4;
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        const int nb = n0 + (wn * TN + a) * 16 + 4 * lg;
        if (nb < n4) *reinterpret_cast<i32x4_t*>(prow + nb) = acc[a][b];
      }
    }
    return;
  }
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(set.ws[wi], (int64_t)n * 4);
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(xs, (int64_t)m * 4);
  f32x4_t out[TN][TM];
  float sx[TM];
#pragma unroll
  for (int b = 0; b < TM; ++b)
    sx[b] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsx, (m0 + (wm * TM + b) * 16 + li) * 4, 0, 0));
#pragma unroll
  for (int a = 0; a < TN; ++a) {
    const f32x4_t sw = __builtin_bit_cast(
        f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsw, (n0 + (wn * TN + a) * 16 + 4 * lg) * 4, 0, 0));
#pragma unroll
    for (int b = 0; b < TM; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) out[a][b][i] = (float)acc[a][b][i] * sx[b] * sw[i];
  }
  if constexpr (LORA) {
    // the adapter term on bf16 MFMA: B [n][r] . T [m][rp], r zero-padded to rp
    const bool whole = lora_whole(lora);
    for (int ks = 0; ks < lora.rp; ks += 32) {
      u32x4_t bf[TN], tf[TM];
#pragma unroll
      for (int a = 0; a < TN; ++a) bf[a] = lora_b(lora, whole, n0 + (wn * TN + a) * 16 + li, n, ks + 8 * lg);
#pragma unroll
      for (int b = 0; b < TM; ++b) tf[b] = lora_t(lora, m0 + (wm * TM + b) * 16 + li, m, ks + 8 * lg);
#pragma unroll
      for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) out[a][b] = mfma16x16x32(bf[a], tf[b], out[a][b]);
    }
  }
  uint16_t* Y = set.y[wi];
  const int32_t* rows = set.rows[wi];
  const int64_t ldy = set.ldy[wi];
  // A lane's values lie in one token each, four channels of it: stored from here
  // they are 32-byte runs.  Through LDS (16 tokens at a time, in the wave's own
  // part) a token's TN * 16 channels of the wave follow one another, 16 bytes a
  // lane.  Chunk c of token r lies at position c ^ (r & (TN * 2 - 1)).
  constexpr int C = TN * 2, R = 64 / C;  // 16-byte chunks of a token, tokens of a store
  int8_t* buf = lds + kGemmLds + wave * (16 * C * 16);
  const int nb = n0 + wn * TN * 16 + 8 * (lane % C);
#pragma unroll
  for (int b = 0; b < TM; ++b) {
#pragma unroll
    for (int a = 0; a < TN; ++a) {
      uint2 o;
      o.x = cvt_pk_bf16(out[a][b][0], out[a][b][1]);
      o.y = cvt_pk_bf16(out[a][b][2], out[a][b][3]);
      *reinterpret_cast<uint2*>(buf + li * C * 16 + 16 * ((2 * a + (lg >> 1)) ^ (li & (C - 1))) + 8 * (lg & 1)) = o;
    }
    u32x4_t v[16 / R];
#pragma unroll
    for (int i = 0; i < 16 / R; ++i) {
      const int r = i * R + lane / C, c = lane % C;
      v[i] = *reinterpret_cast<const u32x4_t*>(buf + r * C * 16 + 16 * (c ^ (r & (C - 1))));
    }
    const int mr = m0 + (wm * TM + b) * 16 + lane / C;
    uint16_t* y = Y + (int64_t)mr * ldy;
    if (rows == nullptr && nb + 8 <= n) {
#pragma unroll
      for (int i = 0; i < 16 / R; ++i)
        if (mr + i * R < m) *reinterpret_cast<u32x4_any_t*>(y + (int64_t)i * R * ldy + nb) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16 / R; ++i)
        if (mr + i * R < m)
          for (int e = 0; e < 8 && nb + e < n; ++e) {
            const uint32_t d = e < 4 ? (e < 2 ? v[i][0] : v[i][1]) : (e < 6 ? v[i][2] : v[i][3]);
            y[(int64_t)i * R * ldy + (rows != nullptr ? rows[nb + e] : nb + e)] = (uint16_t)(d >> (16 * (e & 1)));
          }
    }
  }
}

template <bool LORA>
__global__ __launch_bounds__(kGemmThreads, 1) void k_i8_gemm(I8Set set, I8Plan plan, const int8_t* __restrict__ Xq,
                                                            const float* __restrict__ xs, int m, int k, LoraEpi lora,
                                                            int* __restrict__ part) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[kGemmLds + kGemmOut];
  const int bid = blockIdx.x;
  const bool whole = bid < plan.whole;
  const int t = whole ? xcd_order(bid, plan.whole) : xcd_order(bid - plan.whole, gridDim.x - plan.whole);
  const bool pieces = plan.whole == 0;
  const int piece = whole || pieces ? 0 : t % plan.cut;
  int tx, ty;
  tile_at(whole || pieces ? t : plan.whole + t / plan.cut, plan.nx, plan.ny, tx, ty);
  int wi = 0;
#pragma unroll
  for (int i = 1; i < kGemvMaxGroup; ++i)
    if (i < set.count && tx >= set.tile_end[i - 1]) wi = i;
  if (wi > 0) tx -= set.tile_end[wi - 1];
  const int n0 = tx * (pieces ? 128 : 256) + 128 * (piece & 1);
  const int m0 = ty * (pieces && plan.cut == 4 ? 128 : 256) + 128 * (piece >> 1);
  if (n0 >= set.n[wi] || m0 >= m) return;
  const int s0 = blockIdx.y * plan.per, steps = min(k / I8K - s0, plan.per);
  if (part != nullptr) part += (int64_t)m * ((int64_t)blockIdx.y * set.n_end[set.count - 1] + (wi == 0 ? 0 : set.n_end[wi - 1]));
  if (whole) i8_tile<256, 256, 2, 4, LORA, false>(set, Xq, xs, m, k, lora, wi, n0, m0, 0, steps, nullptr, lds);
  else if (plan.cut == 2) i8_tile<128, 256, 2, 4, LORA, false>(set, Xq, xs, m, k, lora, wi, n0, m0, 0, steps, nullptr, lds);
  else i8_tile<128, 128, 2, 4, LORA, !LORA>(set, Xq, xs, m, k, lora, wi, n0, m0, s0, steps, part, lds);
}

// Outputs from the integer sums of ks K ranges: 16 channels of 16 tokens a wave.
__global__ __launch_bounds__(256) void k_i8_reduce(I8Set set, const int* __restrict__ part, int ks,
                                                  const float* __restrict__ xs, int m, LoraEpi lora) {
  const int wi = blockIdx.z;
  const int n = set.n[wi];
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int n0 = 64 * blockIdx.x + 16 * (threadIdx.x >> 6), nb = n0 + 4 * lg;
  const int mr = 16 * blockIdx.y + li;
  if (n0 >= n) return;
  const int64_t stride = (int64_t)m * set.n_end[set.count - 1];
  const int* p = part + (int64_t)m * (wi == 0 ? 0 : set.n_end[wi - 1]) + (int64_t)mr * padded(n) + nb;
  i32x4_t v = {0, 0, 0, 0};
  if (mr < m && nb < n) {
#pragma unroll 4
    for (int j = 0; j < ks; ++j) v += *reinterpret_cast<const i32x4_t*>(p + j * stride);
  }
  i8_store(set, wi, mr < m ? xs[mr] : 0.f, v, mr, m, n0, lora);
}

}  // namespace

static size_t part_bytes(const I8Choice& c, const int64_t* ns, int count, int64_t m) {
  if (c.tn != 0 || c.plan.ks == 1) return 0;
  int64_t n = 0;
  for (int i = 0; i < count; ++i) n += padded((int)ns[i]);
  return (size_t)c.plan.ks * (size_t)m * (size_t)n * sizeof(int);
}

size_t i8_fwd_workspace_bytes(const int64_t* ns, int count, int64_t k, int64_t m) {
  return part_bytes(i8_choose(ns, count, k, m, true), ns, count, m);
}

I8Set i8_set(const WView* ws, uint16_t* const* ys, const int64_t* ldys, const int32_t* const* out_rows, int count) {
  I8Set set{};
  set.count = count;
  int64_t n = 0;
  for (int i = 0; i < count; ++i) {
    set.w[i] = reinterpret_cast<const int8_t*>(ws[i].packed);
    set.ws[i] = ws[i].scales;
    set.y[i] = ys[i];
    set.rows[i] = out_rows[i];
    set.ldy[i] = ldys[i];
    set.n[i] = (int)ws[i].n;
    n += padded((int)ws[i].n);
    set.n_end[i] = n;
  }
  return set;
}

hipError_t launch_i8_fwd(const I8Set& weights, const int8_t* Xq, const float* xs, int64_t m, int64_t k,
                         const LoraEpi& lora, void* work, size_t work_bytes, hipStream_t s) {
  I8Set set = weights;
  int64_t ns[kGemvMaxGroup];
  int end = 0, most = 0;
  for (int i = 0; i < set.count; ++i) {
    ns[i] = set.n[i];
    most = std::max(most, set.n[i]);
  }
  I8Choice c = i8_choose(ns, set.count, k, m, true);
  if (part_bytes(c, ns, set.count, m) > work_bytes) c = i8_choose(ns, set.count, k, m, false);
  if (c.tn != 0) return launch_i8_skinny(set, c.tn, c.tm, Xq, xs, m, k, lora, s);
  const I8Plan& plan = c.plan;
  for (int i = 0; i < set.count; ++i) set.tile_end[i] = end += (int)ceil_div(set.n[i], plan.whole > 0 ? 256 : 128);
  int* part = plan.ks > 1 ? static_cast<int*>(work) : nullptr;
  const int tiles = plan.nx * plan.ny;
  const dim3 grid((unsigned)(plan.whole > 0 ? plan.whole + (tiles - plan.whole) * plan.cut : tiles), (unsigned)plan.ks);
  if (lora.t != nullptr && plan.ks == 1)
    hipLaunchKernelGGL(k_i8_gemm<true>, grid, dim3(kGemmThreads), 0, s, set, plan, Xq, xs, (int)m, (int)k, lora, part);
  else
    hipLaunchKernelGGL(k_i8_gemm<false>, grid, dim3(kGemmThreads), 0, s, set, plan, Xq, xs, (int)m, (int)k, lora, part);
  if (part != nullptr)
    hipLaunchKernelGGL(k_i8_reduce, dim3((unsigned)ceil_div(most, 64), (unsigned)ceil_div(m, 16), (unsigned)set.count), dim3(256), 0, s,
                       set, part, plan.ks, xs, (int)m, lora);
  return hipGetLastError();
}

}  // namespace lbq
