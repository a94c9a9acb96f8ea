// Products of 8-bit tokens with 8-bit weights for few outputs: short batches
// (the weight is streamed from memory once and bounds the time) and small
// weights at longer ones (too few 256 x 256 tiles to fill the chip).
//
// A workgroup computes 16 TN channels of 16 TM tokens (1, 2 or 4; more channels than
// tokens where the tokens are few and would be fetched for every 16 channels again:
// m = 24, n = 14336, k = 4096 16.8 us with 64 x 32, 18.6 with 32 x 32; m = 39, n =
// 5079, k = 5952 16.1 with 64 x 16, 17.3 with 32 x 32, 18.8 with 32 x 16).  Its eight
// waves split K among them, a 128-byte line of every row by turns; each wave
// loads its share straight to LDS into a ring of its own, so that it waits
// for its own loads only and no barrier is needed, and multiplies it on
// v_mfma_i32_16x16x64_i8.  (Loaded straight to registers in the MFMA's layout,
// neighbouring lanes are in different rows, and the L1 serves a third as much:
// m = 512, n = k = 4096 37.5 -> 29.3 us through LDS; with lines of 64 bytes the
// two halves of a line are fetched by two waves: m = 3, n = 8192, k = 28672
// 54.8 -> 49.1 us with whole lines.  Given a workspace that size goes to k_i8_gemm
// with K split over workgroups, 48.8 us with the launch that adds the sums against
// 49.8 here.)  The waves' integer sums are added at the end: exact, so no split
// changes a bit, and no second launch is needed.  Bound by memory where the weight
// is large (m = 24, n = 14336, k = 4096: 60 MB in 13.4 us, 4.5 TB/s), by latency
// where it is small (m = 130, n = 1001, k = 4160: 7.6 us).
//
// k_i8_decode is the same for up to 4 tokens that are short enough to be
// quantized by every workgroup for itself while its first weights are on
// their way: one launch from bf16 tokens to outputs (m = 1, n = k = 4096: 6.5 us).
#pragma clang fp contract(off)

#include "lbq_device.h"

namespace lbq {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// Weight of row tile `tile` of the set, and the tile's place in it.
__device__ __forceinline__ int weight_of(const I8Set& set, int& tile) {
  int wi = 0;
#pragma unroll
  for (int i = 1; i < kGemvMaxGroup; ++i)
    if (i < set.count && tile >= set.tile_end[i - 1]) wi = i;
  if (wi > 0) tile -= set.tile_end[wi - 1];
  return wi;
}

// Slices of 64 codes that a wave multiplies: both of lines wave, wave + 8, ...
// of 128, where k may end in the middle of the last line.
__device__ __forceinline__ int slices_of(int wave, int k) {
  const int lines = (k + 127) / 128;
  const int mine = (lines - wave + kWaves - 1) / kWaves;
  return 2 * mine - ((k & 64) && mine > 0 && wave + kWaves * (mine - 1) == lines - 1 ? 1 : 0);
}
__device__ __forceinline__ int slice_at(int wave, int j) { return 128 * (wave + kWaves * (j >> 1)) + 64 * (j & 1); }

// Barrier for LDS alone: loads of weights stay on their way.
__device__ __forceinline__ void barrier_lds() {
  asm volatile("" ::: "memory");
  lds_barrier();
  asm volatile("" ::: "memory");
}

// U slots of a ring: with two for 32 x 32 a CU has room for two workgroups (m = 24, n
// = 14336, k = 4096 in these tiles, 448 workgroups: four slots 19.9 us, two 18.9);
// 16 x 16 gains nothing from fewer (m = 5, the same weight: 16.2 and 16.5).
template <int TN, int TM, int U>
__global__ __launch_bounds__(kThreads) void k_i8_skinny(I8Set set, const int8_t* __restrict__ Xq,
                                                       const float* __restrict__ xs, int m, int k, LoraEpi lora) {
  static_assert(U * (TN + TM) >= TN * TM, "a wave's sums fit its ring");
  __shared__ __attribute__((aligned(1024))) int8_t ring[kWaves][U][(TN + TM) * 1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // the same in the wave: scalar load offsets
  const int li = lane & 15, lg = lane >> 4;
  int tile = blockIdx.x;
  const int wi = weight_of(set, tile);
  const int n = set.n[wi];
  const int n0 = tile * 16 * TN, m0 = blockIdx.y * 16 * TM;

  // A load fills 16 rows of 64 bytes: lane l the 16 bytes at position l % 4 of
  // row l / 4.  Rows past the end load the last row instead (their outputs are
  // not stored).
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(set.w[wi], (int64_t)n * k);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)m * k);
  const int lr = lane >> 2, lc = 16 * ((lane & 3) ^ i8_key(lr));
  int ow[TN], ox[TM];
#pragma unroll
  for (int a = 0; a < TN; ++a) ow[a] = min(n0 + 16 * a + lr, n - 1) * k + lc;
#pragma unroll
  for (int b = 0; b < TM; ++b) ox[b] = min(m0 + 16 * b + lr, m - 1) * k + lc;
  auto load = [&](int u, int j) {
    const int kt = slice_at(wave, j);
#pragma unroll
    for (int a = 0; a < TN; ++a) load_to_lds(rw, &ring[wave][u][1024 * a], ow[a], kt);
#pragma unroll
    for (int b = 0; b < TM; ++b) load_to_lds(rx, &ring[wave][u][1024 * (TN + b)], ox[b], kt);
  };
  const int cnt = slices_of(wave, k);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < cnt) load(u, u);

  i32x4_t acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};
  const int f = li * 64 + 16 * (lg ^ i8_key(li));
  run_ring<U, TN + TM>(cnt, load, [&](int u, int) {
    i32x4_t w[TN], x[TM];
#pragma unroll
    for (int a = 0; a < TN; ++a) w[a] = *reinterpret_cast<const i32x4_t*>(&ring[wave][u][1024 * a + f]);
#pragma unroll
    for (int b = 0; b < TM; ++b) x[b] = *reinterpret_cast<const i32x4_t*>(&ring[wave][u][1024 * (TN + b) + f]);
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] = mfma_i8(w[a], x[b], acc[a][b]);
  });

  // The waves' sums, each in its own ring, then added.
  i32x4_t* const sums = reinterpret_cast<i32x4_t*>(&ring[wave][0][0]);
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) sums[(a * TM + b) * 64 + lane] = acc[a][b];
  __syncthreads();
  // Channels n = 4 (lane / 16) + i of token lane % 16, a block a wave by turns.
  for (int blk = wave; blk < TN * TM; blk += kWaves) {
    i32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const i32x4_t*>(&ring[w][0][0])[blk * 64 + lane];
    const int mr = m0 + (blk % TM) * 16 + li;
    i8_store(set, wi, mr < m ? xs[mr] : 0.f, v, mr, m, n0 + (blk / TM) * 16, lora);
  }
}

constexpr int kDecodeU = 6;      // slots of a wave's ring (1 KiB each)
constexpr int kDecodeChunks = 6;  // 8-value chunks of a token a thread holds

// Up to 4 tokens X (bf16, rows of k) of at most kI8DecodeCodes codes in all.  With
// an adapter every workgroup also finishes the tokens' T from its partial sums
// (t; lora.t is not read): one launch less (m = 1, n = k = 4096, rank 16 15.6 -> 13.5 us).
__global__ __launch_bounds__(kThreads) void k_i8_decode(I8Set set, const uint16_t* __restrict__ X, int m, int k,
                                                       LoraEpi lora, XaSums t) {
  __shared__ __attribute__((aligned(16))) uint16_t T[4 * 64];  // [m][rp]
  __shared__ __attribute__((aligned(1024))) int8_t ring[kWaves][kDecodeU][1024];
  __shared__ __attribute__((aligned(16))) int8_t codes[kI8DecodeCodes];
  __shared__ uint32_t top[kWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  int tile = blockIdx.x;
  const int wi = weight_of(set, tile);
  const int n = set.n[wi];
  const int n0 = tile * 16;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(set.w[wi], (int64_t)n * k);
  const int lr = lane >> 2;
  const int ow = min(n0 + lr, n - 1) * k + 16 * ((lane & 3) ^ i8_key(lr));
  auto load = [&](int u, int j) { load_to_lds(rw, &ring[wave][u][0], ow, slice_at(wave, j)); };
  const int cnt = slices_of(wave, k);

  // Each token by 8 / m of the waves: loaded before the weights, its largest
  // magnitude by shuffles and through LDS, its codes to LDS.
  const int per = kWaves / m, row = wave / per;
  const bool on = row < m;
  const int first = (wave - row * per) * 64 + lane, stride = per * 64, chunks = on ? k / 8 : 0;
  const uint16_t* x = X + (int64_t)row * k;
  u32x4_t c[kDecodeChunks];
#pragma unroll
  for (int i = 0; i < kDecodeChunks; ++i)
    if (first + i * stride < chunks) c[i] = *reinterpret_cast<const u32x4_t*>(x + 8 * (first + i * stride));
#pragma unroll
  for (int u = 0; u < kDecodeU; ++u)
    if (u < cnt) load(u, u);
  if (t.part != nullptr && tid < m * t.rp) {
    const int r = tid / t.rp, j = tid % t.rp;
    float v = 0.f;
    if (j < t.r) v = t.sigma * sum_splits16(t.part, t.splits, t.m * t.rb, (int64_t)r * t.rb + j);
    T[tid] = (uint16_t)bf16_rne(v);
  }
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < kDecodeChunks; ++i)
    if (first + i * stride < chunks) mx = max(mx, i8_top_bf16(c[i]));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) mx = max(mx, (uint32_t)__shfl_xor(mx, o));
  if (lane == 0) top[wave] = mx;
  barrier_lds();
  // the scale of this wave's token, and of lane li's token for the outputs
  auto top_of = [&](int r) {
    uint32_t t = 0;
    for (int i = 0; i < per; ++i) t = max(t, top[min(r * per + i, kWaves - 1)]);
    return t;
  };
  bool finite;
  const float s = i8_scale(top_of(row), finite), rs = 1.f / s;
#pragma unroll
  for (int i = 0; i < kDecodeChunks; ++i)
    if (first + i * stride < chunks)
      *reinterpret_cast<uint2*>(codes + row * k + 8 * (first + i * stride)) = i8_codes_bf16(c[i], s, rs, finite);
  barrier_lds();

  i32x4_t acc = {0, 0, 0, 0};
  const int f = li * 64 + 16 * (lg ^ i8_key(li));
  run_ring<kDecodeU, 1>(cnt, load, [&](int u, int j) {
    const i32x4_t w = *reinterpret_cast<const i32x4_t*>(&ring[wave][u][f]);
    i32x4_t t = {0, 0, 0, 0};
    if (li < m) t = *reinterpret_cast<const i32x4_t*>(codes + li * k + slice_at(wave, j) + 16 * lg);
    acc = mfma_i8(w, t, acc);
  });
  reinterpret_cast<i32x4_t*>(&ring[wave][0][0])[lane] = acc;
  __syncthreads();
  if (wave == 0) {
    i32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const i32x4_t*>(&ring[w][0][0])[lane];
    if (t.part != nullptr) lora.t = T;
    i8_store(set, wi, i8_scale(top_of(li), finite), v, li, m, n0, lora);
  }
}

// Row tiles of 16 t channels over the weights of a set.
unsigned tile_rows(I8Set& set, int t) {
  int end = 0;
  for (int i = 0; i < set.count; ++i) {
    end += (set.n[i] + 16 * t - 1) / (16 * t);
    set.tile_end[i] = end;
  }
  return (unsigned)end;
}

template <int TN, int TM, int U>
hipError_t launch(I8Set set, const int8_t* Xq, const float* xs, int64_t m, int64_t k, const LoraEpi& lora, hipStream_t s) {
  const unsigned rows = tile_rows(set, TN);
  hipLaunchKernelGGL((k_i8_skinny<TN, TM, U>), dim3(rows, (unsigned)((m + 16 * TM - 1) / (16 * TM))), dim3(kThreads), 0, s,
                     set, Xq, xs, (int)m, (int)k, lora);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_skinny(const I8Set& set, int tn, int tm, const int8_t* Xq, const float* xs, int64_t m, int64_t k,
                            const LoraEpi& lora, hipStream_t s) {
  switch (8 * tn + tm) {
    case 8 * 1 + 1: return launch<1, 1, 4>(set, Xq, xs, m, k, lora, s);
    case 8 * 2 + 1: return launch<2, 1, 2>(set, Xq, xs, m, k, lora, s);
    case 8 * 4 + 1: return launch<4, 1, 2>(set, Xq, xs, m, k, lora, s);
    case 8 * 2 + 2: return launch<2, 2, 2>(set, Xq, xs, m, k, lora, s);
    case 8 * 4 + 2: return launch<4, 2, 2>(set, Xq, xs, m, k, lora, s);
    case 8 * 4 + 4: return launch<4, 4, 2>(set, Xq, xs, m, k, lora, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_i8_decode(const I8Set& weights, const uint16_t* X, int64_t m, int64_t k, const LoraEpi& lora,
                            const XaSums& t, hipStream_t s) {
  I8Set set = weights;
  const unsigned rows = tile_rows(set, 1);
  hipLaunchKernelGGL(k_i8_decode, dim3(rows), dim3(kThreads), 0, s, set, X, (int)m, (int)k, lora, t);
  return hipGetLastError();
}

}  // namespace lbq
