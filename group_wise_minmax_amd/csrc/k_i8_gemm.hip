// Products of 8-bit integers with one scale for each token and each output
// channel (the INT8 weight format):
//   Y[i][j] = bf16( fl(fl(fl(acc) * sx[i]) * sw[j]) ),  acc = sum_k Xq[i][k] Wq[j][k]
// on v_mfma_i32_16x16x64_i8.  acc is exact in 32-bit integers (k <= 2^17:
// 127 * 127 * 2^17 < 2^31), so the result does not depend on the order of the
// sum, on the tile or on how K is split: every kernel here gives the same bits.
#pragma clang fp contract(off)

#include "lbq_device.h"

namespace lbq {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mfma_i8(const i32x4_t& a, const i32x4_t& b, const i32x4_t& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}


// 16 bytes a lane from r (byte offset voff of the lane plus soff) to LDS: lane
// l's at `lds` + 16 l, `lds` the same in the whole wave.  (The host pass knows
// no 16-byte form of the builtin.)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, int8_t* lds, int voff, int soff) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
#endif
}

// One K step of a tile in LDS: BN rows of W and BM rows of X, 64 bytes each.
// Chunk c (16 bytes) of row r lies at position c ^ key(r): the 16 lanes that a
// 16-byte LDS read serves together (0-3, 12-15, 20-23 and 24-27 of a half wave,
// or the other 16) then read 16 different sixteenths of the 64 banks, where
// lane l reads chunk l / 16 of row l % 16.
template <int BN, int BM>
struct I8Stage {
  int8_t w[BN * 64];
  int8_t x[BM * 64];
};
__device__ __forceinline__ int i8_key(int r) { return -(r >> 2) & 3; }

constexpr int I8K = 64;      // K step
constexpr int kStages = 4;   // stages in LDS

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

template <int BN, int BM, int WGN, int WGM, bool LORA>
__global__ __launch_bounds__(64 * WGN * WGM, 1) void k_i8_gemm(I8Set set, const int8_t* __restrict__ Xq,
                                                              const float* __restrict__ xs, int m, int k, LoraEpi lora) {
  constexpr int NW = WGN * WGM;
  constexpr int TN = BN / WGN / 16, TM = BM / WGM / 16, TH = TN / 2;
  constexpr int LW = BN / 16 / NW, LX = BM / 16 / NW;  // 1-KiB pieces (16 rows) a wave loads of each operand
  static_assert(LW * NW * 16 == BN && LX * NW * 16 == BM, "whole pieces");
  __shared__ __attribute__((aligned(16))) I8Stage<BN, BM> st[kStages];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave % WGN, wm = wave / WGN;
  const int nx = set.tile_end[set.count - 1], ny = (m + BM - 1) / BM;
  int tx, ty;
  tile_of(blockIdx.x, nx, ny, tx, ty);
  int wi = 0;
#pragma unroll
  for (int i = 1; i < kGemvMaxGroup; ++i)
    if (i < set.count && tx >= set.tile_end[i - 1]) wi = i;
  if (wi > 0) tx -= set.tile_end[wi - 1];
  const int n = set.n[wi];
  const int n0 = tx * BN, m0 = ty * BM;

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
  auto load_w = [&](int8_t* w, int kt) {
#pragma unroll
    for (int i = 0; i < LW; ++i) load_to_lds(rw, w + 1024 * (wave * LW + i), ow[i], kt);
  };
  auto load_x = [&](int8_t* x, int kt) {
#pragma unroll
    for (int i = 0; i < LX; ++i) load_to_lds(rx, x + 1024 * (wave * LX + i), ox[i], kt);
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

  // Step t lies in stage t % 4.  While it is multiplied, steps t + 1 and t + 2
  // are on their way and the loads of step t + 3 are issued, spread between
  // the MFMAs (issued together they fill the load queue and hold up the wave's
  // MFMAs behind them).  The first slice of a step is read before the last
  // MFMAs of the one before it.  Past the last step the loads repeat it, so
  // that the count of loads in flight stays what the wait says.
  const int steps = k / I8K;
  auto at = [&](int t) { return I8K * min(t, steps - 1); };
  // Steps up to t + 1 are there: this wave's loads but the last two steps'
  // (vmcnt), and by the barrier every wave's; every wave has read step t.
  auto arrive = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LW + LW + LX));  // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  for (int t = 0; t < 3; ++t) {
    load_w(st[t].w, at(t));
    load_x(st[t].x, at(t));
  }
  arrive();
  read_w(st[0], 0, w0);
  read_x(st[0], x0);
  // xa: this step's tokens, xb: the next one's
  auto step = [&](int t, const i32x4_t (&xa)[TM], i32x4_t (&xb)[TM]) {
    I8Stage<BN, BM>& cur = st[t % kStages];
    I8Stage<BN, BM>& next = st[(t + 1) % kStages];
    I8Stage<BN, BM>& far = st[(t + 3) % kStages];
    read_w(cur, 1, w1);
    load_w(far.w, at(t + 3));
    mma(0, w0, xa);
    interleave<TH, LW, TH * TM>();
    arrive();
    read_w(next, 0, w0);
    read_x(next, xb);
    load_x(far.x, at(t + 3));
    mma(1, w1, xa);
    interleave<TH + TM, LX, TH * TM>();
  };
  int t = 0;
  for (; t + 1 < steps; t += 2) {
    step(t, x0, x1);
    step(t + 1, x1, x0);
  }
  if (t < steps) step(t, x0, x1);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // no load to LDS is left behind

  // Epilogue: lane l holds channels n = 4 (l / 16) + i of token m = l % 16.
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
    for (int ks = 0; ks < lora.rp; ks += 32) {
      u32x4_t bf[TN], tf[TM];
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        const int64_t nr = n0 + (wn * TN + a) * 16 + li;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c0 = ks + 8 * lg + 2 * j;
          uint32_t lo = 0, hi = 0;
          if (nr < n && c0 < lora.r) lo = lora.b[nr * lora.r + c0];
          if (nr < n && c0 + 1 < lora.r) hi = lora.b[nr * lora.r + c0 + 1];
          v[j] = lo | (hi << 16);
        }
        bf[a] = u32x4_t{v[0], v[1], v[2], v[3]};
      }
#pragma unroll
      for (int b = 0; b < TM; ++b) {
        const int64_t mr = m0 + (wm * TM + b) * 16 + li;
        tf[b] = mr < m ? *reinterpret_cast<const u32x4_t*>(lora.t + mr * lora.rp + ks + 8 * lg) : u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) out[a][b] = mfma16x16x32(bf[a], tf[b], out[a][b]);
    }
  }
  uint16_t* Y = set.y[wi];
  const int32_t* rows = set.rows[wi];
  const int64_t ldy = set.ldy[wi];
  const bool vec = rows == nullptr && (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(Y) & 7) == 0;
#pragma unroll
  for (int b = 0; b < TM; ++b) {
    const int mr = m0 + (wm * TM + b) * 16 + li;
    if (mr >= m) continue;
    uint16_t* yrow = Y + (int64_t)mr * ldy;
#pragma unroll
    for (int a = 0; a < TN; ++a) {
      const int nb = n0 + (wn * TN + a) * 16 + 4 * lg;
      uint2 o;
      o.x = cvt_pk_bf16(out[a][b][0], out[a][b][1]);
      o.y = cvt_pk_bf16(out[a][b][2], out[a][b][3]);
      if (vec && nb + 3 < n) {
        *reinterpret_cast<uint2*>(yrow + nb) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (nb + i < n)
            yrow[rows != nullptr ? rows[nb + i] : nb + i] = (uint16_t)((i < 2 ? o.x : o.y) >> (16 * (i & 1)));
      }
    }
  }
}

template <int BN, int BM, int WGN, int WGM>
hipError_t launch_gemm(I8Set set, const int8_t* Xq, const float* xs, int64_t m, int64_t k, const LoraEpi& lora,
                       hipStream_t s) {
  int end = 0;
  for (int i = 0; i < set.count; ++i) {
    end += (set.n[i] + BN - 1) / BN;
    set.tile_end[i] = end;
  }
  const dim3 grid((unsigned)(end * ((m + BM - 1) / BM)));
  if (lora.t != nullptr)
    hipLaunchKernelGGL((k_i8_gemm<BN, BM, WGN, WGM, true>), grid, dim3(64 * WGN * WGM), 0, s, set, Xq, xs, (int)m, (int)k, lora);
  else
    hipLaunchKernelGGL((k_i8_gemm<BN, BM, WGN, WGM, false>), grid, dim3(64 * WGN * WGM), 0, s, set, Xq, xs, (int)m, (int)k, lora);
  return hipGetLastError();
}

}  // namespace

size_t i8_fwd_workspace_bytes(const int64_t*, int, int64_t, int64_t) { return 0; }

hipError_t launch_i8_fwd(const WView* ws, uint16_t* const* ys, const int64_t* ldys, const int32_t* const* out_rows,
                         int count, const int8_t* Xq, const float* xs, int64_t m, const LoraEpi& lora, void*,
                         hipStream_t s) {
  I8Set set{};
  set.count = count;
  int64_t t256 = 0;
  for (int i = 0; i < count; ++i) {
    set.w[i] = reinterpret_cast<const int8_t*>(ws[i].packed);
    set.ws[i] = ws[i].scales;
    set.y[i] = ys[i];
    set.rows[i] = out_rows[i];
    set.ldy[i] = ldys[i];
    set.n[i] = (int)ws[i].n;
    t256 += (ws[i].n + 255) / 256 * ((m + 255) / 256);
  }
  const int64_t k = ws[0].k;
  if (t256 >= 128) return launch_gemm<256, 256, 2, 4>(set, Xq, xs, m, k, lora, s);
  return launch_gemm<128, 128, 2, 2>(set, Xq, xs, m, k, lora, s);
}

}  // namespace lbq
