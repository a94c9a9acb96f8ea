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

// Adapter term of outputs (row mr, channels nb .. nb + 3) in fp32: T[mr] . B[n].
__device__ __forceinline__ float lora_dot(const LoraEpi& lora, int64_t mr, int64_t n) {
  float v = 0.f;
  const uint16_t* t = lora.t + mr * lora.rp;
  const uint16_t* b = lora.b + n * lora.r;
  for (int j = 0; j < lora.r; ++j)
    v = fmaf(__uint_as_float((uint32_t)t[j] << 16), __uint_as_float((uint32_t)b[j] << 16), v);
  return v;
}

// 128 x 128 output tiles, four waves of 64 x 64, K in steps of 64 through LDS.
__global__ __launch_bounds__(256) void k_i8_gemm(I8Set set, const int8_t* __restrict__ Xq,
                                                const float* __restrict__ xs, int m, int k, LoraEpi lora) {
  constexpr int LD = 80;  // bytes of an LDS row: 64 and a pad that spreads the banks
  __shared__ __attribute__((aligned(16))) int8_t Ws[128 * LD];
  __shared__ __attribute__((aligned(16))) int8_t Xs[128 * LD];
  int wi = 0;
  for (int i = 1; i < set.count; ++i)
    if ((int)blockIdx.x >= set.tile_end[i - 1]) wi = i;
  const int tx = blockIdx.x - (wi == 0 ? 0 : set.tile_end[wi - 1]);
  const int8_t* W = set.w[wi];
  const int n = set.n[wi];
  const int n0 = tx * 128, m0 = blockIdx.y * 128;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wm = wave >> 1;
  const int li = lane & 15, lg = lane >> 4;
  i32x4_t acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};
  for (int kt = 0; kt < k; kt += 64) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = tid + 256 * i, row = c >> 2, col = (c & 3) * 16;
      const int64_t nr = min(n0 + row, n - 1), mr = min(m0 + row, m - 1);
      *reinterpret_cast<i32x4_t*>(Ws + row * LD + col) = *reinterpret_cast<const i32x4_t*>(W + nr * k + kt + col);
      *reinterpret_cast<i32x4_t*>(Xs + row * LD + col) = *reinterpret_cast<const i32x4_t*>(Xq + mr * k + kt + col);
    }
    __syncthreads();
    i32x4_t af[4], bf[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) af[a] = *reinterpret_cast<const i32x4_t*>(Ws + (64 * wn + 16 * a + li) * LD + 16 * lg);
#pragma unroll
    for (int b = 0; b < 4; ++b) bf[b] = *reinterpret_cast<const i32x4_t*>(Xs + (64 * wm + 16 * b + li) * LD + 16 * lg);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = mfma_i8(af[a], bf[b], acc[a][b]);
    __syncthreads();
  }
  const float* sw = set.ws[wi];
  uint16_t* Y = set.y[wi];
  const int32_t* rows = set.rows[wi];
  const int64_t ldy = set.ldy[wi];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int mr = m0 + 64 * wm + 16 * b + li;
    if (mr >= m) continue;
    const float sx = xs[mr];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int nr = n0 + 64 * wn + 16 * a + 4 * lg + i;
        if (nr >= n) continue;
        float v = (float)acc[a][b][i] * sx * sw[nr];
        if (lora.t != nullptr) v += lora_dot(lora, mr, nr);
        Y[(int64_t)mr * ldy + (rows != nullptr ? rows[nr] : nr)] = i8_bf16(v);
      }
  }
}

}  // namespace

size_t i8_fwd_workspace_bytes(const int64_t*, int, int64_t, int64_t) { return 0; }

hipError_t launch_i8_fwd(const WView* ws, uint16_t* const* ys, const int64_t* ldys, const int32_t* const* out_rows,
                         int count, const int8_t* Xq, const float* xs, int64_t m, const LoraEpi& lora, void*,
                         hipStream_t s) {
  I8Set set{};
  set.count = count;
  int end = 0;
  for (int i = 0; i < count; ++i) {
    set.w[i] = reinterpret_cast<const int8_t*>(ws[i].packed);
    set.ws[i] = ws[i].scales;
    set.y[i] = ys[i];
    set.rows[i] = out_rows[i];
    set.ldy[i] = ldys[i];
    set.n[i] = (int)ws[i].n;
    end += (int)((ws[i].n + 127) / 128);
    set.tile_end[i] = end;
  }
  hipLaunchKernelGGL(k_i8_gemm, dim3((unsigned)end, (unsigned)((m + 127) / 128)), dim3(256), 0, s, set, Xq, xs, (int)m,
                     (int)ws[0].k, lora);
  return hipGetLastError();
}

}  // namespace lbq
