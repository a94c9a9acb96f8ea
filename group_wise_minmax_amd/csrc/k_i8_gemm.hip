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

typedef float f32x16_t __attribute__((ext_vector_type(16)));

typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x16_t mfma_i8_32(const i32x4_t& a, const i32x4_t& b, const i32x16_t& c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// 16 bytes a lane from r (byte offset voff of the lane plus soff) to LDS: lane
// l's at `lds` + 16 l, `lds` the same in the whole wave.  (The host pass knows
// no 16-byte form of the builtin.)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, int8_t* lds, int voff, int soff) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
#endif
}

// One K step of a tile in LDS: BN rows of W and BM rows of X, 128 bytes each,
// the 16-byte chunks of a row swizzled as swz() places them.
template <int BN, int BM>
struct I8Stage {
  int8_t w[BN * 128];
  int8_t x[BM * 128];
};

constexpr int I8K = 128;  // K step

template <int BN, int BM, int WGN, int WGM, bool LORA>
__global__ __launch_bounds__(64 * WGN * WGM, 1) void k_i8_gemm(I8Set set, const int8_t* __restrict__ Xq,
                                                              const float* __restrict__ xs, int m, int k, LoraEpi lora) {
  constexpr int NW = WGN * WGM;
  constexpr int TN = BN / WGN / 32, TM = BM / WGM / 32;
  constexpr int LW = BN / 8 / NW, LX = BM / 8 / NW;  // 1-KiB pieces (8 rows) a wave loads of each operand
  __shared__ __attribute__((aligned(16))) I8Stage<BN, BM> st[2];

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

  // Global loads go straight to LDS: a wave's load fills 8 rows, lane l the
  // 16 bytes at position l % 8 of row l / 8, which hold chunk (l % 8) ^ (row % 8).
  // Rows past the end load the last row instead (their outputs are not
  // stored); bytes past the end of the operand read as zeros.
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(set.w[wi], (int64_t)n * k);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)m * k);
  const int lr = lane >> 3, lc = ((lane & 7) ^ lr) * 16;
  int ow[LW], ox[LX];
#pragma unroll
  for (int i = 0; i < LW; ++i) ow[i] = min(n0 + 8 * (wave * LW + i) + lr, n - 1) * k + lc;
#pragma unroll
  for (int i = 0; i < LX; ++i) ox[i] = min(m0 + 8 * (wave * LX + i) + lr, m - 1) * k + lc;
  auto load = [&](I8Stage<BN, BM>& st, int kt) {
#pragma unroll
    for (int i = 0; i < LW; ++i)
      load_to_lds(rw, st.w + 1024 * (wave * LW + i), ow[i], kt);
#pragma unroll
    for (int i = 0; i < LX; ++i)
      load_to_lds(rx, st.x + 1024 * (wave * LX + i), ox[i], kt);
  };

  i32x16_t acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0;

  // Operand fragments of one 32-wide slice of a stage: lane l holds 16 bytes
  // of row l % 32, chunk 2 * s + l / 32.
  struct Frag {
    i32x4_t w[TN], x[TM];
  };
  const int fr = lane & 31, fc = lane >> 5;
  const uint32_t fw = (wn * TN * 32 + fr) * 128, fx = (wm * TM * 32 + fr) * 128;
  auto frags = [&](const I8Stage<BN, BM>& st, int s) {
    const uint32_t c = 16u * ((2 * s + fc) ^ (fr & 7));
    Frag f;
#pragma unroll
    for (int a = 0; a < TN; ++a) f.w[a] = *reinterpret_cast<const i32x4_t*>(st.w + fw + c + a * 32 * 128);
#pragma unroll
    for (int b = 0; b < TM; ++b) f.x[b] = *reinterpret_cast<const i32x4_t*>(st.x + fx + c + b * 32 * 128);
    return f;
  };
  auto mma = [&](const Frag& f) {
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] = mfma_i8_32(f.w[a], f.x[b], acc[a][b]);
  };

  // Whole steps of 128, then one of 64 where k ends in the middle of one.
  // Step t lies in stage t % 2; while it is multiplied, step t + 1 arrives.
  // The first slice of a step is read before the last MFMAs of the one before
  // it.
  const int steps = k / I8K, loads = (k + I8K - 1) / I8K;
  // A wave's own loads to LDS are in (vmcnt 0), then every wave's.
  auto arrive = [&]() {
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
  };
  load(st[0], 0);
  arrive();
  if (loads > 1) load(st[1], I8K);
  Frag f = frags(st[0], 0);
  for (int t = 0; t < steps; ++t) {
    I8Stage<BN, BM>& cur = st[t & 1];
    I8Stage<BN, BM>& next = st[(t & 1) ^ 1];
    Frag g = frags(cur, 1);
    mma(f);
    f = frags(cur, 2);
    mma(g);
    g = frags(cur, 3);
    mma(f);
    arrive();  // step t + 1 is there, and every wave has read step t
    if (t + 2 < loads) load(cur, I8K * (t + 2));
    f = frags(next, 0);
    mma(g);
  }
  if (loads > steps) {
    const Frag g = frags(st[steps & 1], 1);
    mma(f);
    mma(g);
  }

  // Epilogue: lane l holds channels n = 8 g + 4 (l / 32) + i of token m = l % 32.
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(set.ws[wi], (int64_t)n * 4);
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(xs, (int64_t)m * 4);
  f32x16_t out[TN][TM];
  float sx[TM];
#pragma unroll
  for (int b = 0; b < TM; ++b)
    sx[b] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsx, (m0 + (wm * TM + b) * 32 + fr) * 4, 0, 0));
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4_t sw = __builtin_bit_cast(
          f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsw, (n0 + (wn * TN + a) * 32 + 8 * g + 4 * fc) * 4, 0, 0));
#pragma unroll
      for (int b = 0; b < TM; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) out[a][b][4 * g + i] = (float)acc[a][b][4 * g + i] * sx[b] * sw[i];
    }
  if constexpr (LORA) {
    // the adapter term on bf16 MFMA: B [n][r] . T [m][rp], r zero-padded to rp
    for (int ks = 0; ks < lora.rp; ks += 16) {
      u32x4_t bf[TN], tf[TM];
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        const int64_t nr = n0 + (wn * TN + a) * 32 + fr;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c0 = ks + 8 * fc + 2 * j;
          uint32_t lo = 0, hi = 0;
          if (nr < n && c0 < lora.r) lo = lora.b[nr * lora.r + c0];
          if (nr < n && c0 + 1 < lora.r) hi = lora.b[nr * lora.r + c0 + 1];
          v[j] = lo | (hi << 16);
        }
        bf[a] = u32x4_t{v[0], v[1], v[2], v[3]};
      }
#pragma unroll
      for (int b = 0; b < TM; ++b) {
        const int64_t mr = m0 + (wm * TM + b) * 32 + fr;
        tf[b] = mr < m ? *reinterpret_cast<const u32x4_t*>(lora.t + mr * lora.rp + ks + 8 * fc) : u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b)
          out[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, bf[a]),
                                                              __builtin_bit_cast(bf16x8_t, tf[b]), out[a][b], 0, 0, 0);
    }
  }
  uint16_t* Y = set.y[wi];
  const int32_t* rows = set.rows[wi];
  const int64_t ldy = set.ldy[wi];
  const bool vec = rows == nullptr && (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(Y) & 7) == 0;
#pragma unroll
  for (int b = 0; b < TM; ++b) {
    const int mr = m0 + (wm * TM + b) * 32 + fr;
    if (mr >= m) continue;
    uint16_t* yrow = Y + (int64_t)mr * ldy;
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int nb = n0 + (wn * TN + a) * 32 + 8 * g + 4 * fc;
        uint2 o;
        o.x = cvt_pk_bf16(out[a][b][4 * g], out[a][b][4 * g + 1]);
        o.y = cvt_pk_bf16(out[a][b][4 * g + 2], out[a][b][4 * g + 3]);
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
