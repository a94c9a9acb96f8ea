// Products of 8-bit tokens with 8-bit weights for few outputs: short batches
// (the weight is streamed from memory once and bounds the time) and small
// weights at longer ones (too few 256 x 256 tiles to fill the chip).
//
// A workgroup computes 16 TN channels of 16 TM tokens.  Its eight waves split K
// among them, 64 codes at a time by turns, so a row of W is read in runs of 512
// bytes; each wave multiplies its share on v_mfma_i32_16x16x64_i8 with both
// operands straight from memory in the MFMA's own layout (lane l: 16 bytes
// of row l % 16; no value is used by two waves, so LDS would only add a
// copy), kept several steps ahead in registers.  The waves' integer sums are
// added in LDS: exact, so their order does not matter, and no second launch
// or global partial sums are needed.
#pragma clang fp contract(off)

#include "lbq_device.h"

namespace lbq {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// TN x TM blocks of 16 x 16 outputs, U steps of 64 in flight.
template <int TN, int TM, int U>
__global__ __launch_bounds__(kThreads) void k_i8_skinny(I8Set set, const int8_t* __restrict__ Xq,
                                                       const float* __restrict__ xs, int m, int k, LoraEpi lora) {
  __shared__ __attribute__((aligned(16))) int sum[TN * TM * 256];  // [block][i][lane]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int li = lane & 15, lg = lane >> 4;
  int wi = 0;
#pragma unroll
  for (int i = 1; i < kGemvMaxGroup; ++i)
    if (i < set.count && (int)blockIdx.x >= set.tile_end[i - 1]) wi = i;
  const int tx = blockIdx.x - (wi == 0 ? 0 : set.tile_end[wi - 1]);
  const int n = set.n[wi];
  const int n0 = tx * 16 * TN, m0 = blockIdx.y * 16 * TM;

  // Rows past the end read the last row instead (their outputs are not stored).
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(set.w[wi], (int64_t)n * k);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)m * k);
  int ow[TN], ox[TM];
#pragma unroll
  for (int a = 0; a < TN; ++a) ow[a] = min(n0 + 16 * a + li, n - 1) * k + 16 * lg;
#pragma unroll
  for (int b = 0; b < TM; ++b) ox[b] = min(m0 + 16 * b + li, m - 1) * k + 16 * lg;

  i32x4_t acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};

  // This wave's steps: wave, wave + 8, ...
  const int steps = k / 64;
  const int mine = (steps - wave + kWaves - 1) / kWaves;
  i32x4_t w[U][TN], x[U][TM];
  auto load = [&](int u, int j) {
    if (j >= mine) return;
    const int kt = 64 * (wave + kWaves * j);
#pragma unroll
    for (int a = 0; a < TN; ++a)
      w[u][a] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, ow[a], kt, 0));
#pragma unroll
    for (int b = 0; b < TM; ++b)
      x[u][b] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, ox[b], kt, 0));
  };
  auto mma = [&](int u) {
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] = mfma_i8(w[u][a], x[u][b], acc[a][b]);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u);
  for (int i = tid; i < TN * TM * 64; i += kThreads) *reinterpret_cast<i32x4_t*>(sum + 4 * i) = i32x4_t{0, 0, 0, 0};
  int j = 0;
  for (; j + U <= mine; j += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mma(u);
      load(u, j + U + u);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (j + u < mine) mma(u);

  __syncthreads();
  if (mine > 0) {
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) atomicAdd(&sum[((a * TM + b) * 4 + i) * 64 + lane], acc[a][b][i]);
  }
  __syncthreads();

  // Channels n = 4 (lane / 16) + i of token lane % 16, a block a wave by turns.
  for (int blk = wave; blk < TN * TM; blk += kWaves) {
    const int mr = m0 + (blk % TM) * 16 + li, nb = n0 + (blk / TM) * 16 + 4 * lg;
    if (mr >= m || nb >= n) continue;
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = sum[(blk * 4 + i) * 64 + lane];
    i8_store(set, wi, xs[mr], v, mr, nb, lora);
  }
}

template <int TN, int TM, int U>
hipError_t launch(I8Set set, const int8_t* Xq, const float* xs, int64_t m, int64_t k, const LoraEpi& lora, hipStream_t s) {
  int end = 0;
  for (int i = 0; i < set.count; ++i) {
    end += (set.n[i] + 16 * TN - 1) / (16 * TN);
    set.tile_end[i] = end;
  }
  hipLaunchKernelGGL((k_i8_skinny<TN, TM, U>), dim3((unsigned)end, (unsigned)((m + 16 * TM - 1) / (16 * TM))),
                     dim3(kThreads), 0, s, set, Xq, xs, (int)m, (int)k, lora);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_skinny(const I8Set& set, int tn, int tm, const int8_t* Xq, const float* xs, int64_t m, int64_t k,
                            const LoraEpi& lora, hipStream_t s) {
  switch (tn * 8 + tm) {
    case 8 + 1: return launch<1, 1, 8>(set, Xq, xs, m, k, lora, s);
    case 8 + 2: return launch<1, 2, 8>(set, Xq, xs, m, k, lora, s);
    case 8 + 4: return launch<1, 4, 4>(set, Xq, xs, m, k, lora, s);
    case 16 + 1: return launch<2, 1, 8>(set, Xq, xs, m, k, lora, s);
    case 16 + 2: return launch<2, 2, 4>(set, Xq, xs, m, k, lora, s);
    case 16 + 4: return launch<2, 4, 4>(set, Xq, xs, m, k, lora, s);
    case 32 + 1: return launch<4, 1, 4>(set, Xq, xs, m, k, lora, s);
    case 32 + 2: return launch<4, 2, 4>(set, Xq, xs, m, k, lora, s);
    case 32 + 4: return launch<4, 4, 4>(set, Xq, xs, m, k, lora, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace lbq
