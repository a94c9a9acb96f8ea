// Symmetric 8-bit quantization of rows, and the standalone dequantize of
// 8-bit weights.
//
// A row (an output channel of a weight, or a token of an activation) has one
// scale s = fl(max|x| / 127), 1 when that is 0, and codes
// q = clamp(rne(fl(x / s)), -127, 127).  Every fp32 step is one IEEE operation
// rounded to nearest-even (contraction is off for this file here and on its
// compile line).  The magnitudes are compared as integers (the bits without
// the sign order like the values, infinities and NaN above every finite one),
// so a row that holds an infinity or a NaN is seen as such: it gets the scale
// NaN and codes 0, and only that token's outputs are NaN.
//
// Bound by memory: a row of up to 32768 values is read once and kept in registers
// between the search for its largest magnitude and the codes; a longer row is
// read again, from L2.  m = k = 4096: 10.2 us (4.9 TB/s); a few rows are bound by
// their latency (3 rows of 28672: 5.5 us).
#pragma clang fp contract(off)

#include "lbq_device.h"

#include <algorithm>

namespace lbq {

namespace {

constexpr int kThreads = 256;

// Eight consecutive values of a row as they are stored.
template <typename T>
struct Chunk8;
template <>
struct Chunk8<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4_t*>(p);
    b = *(reinterpret_cast<const f32x4_t*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(__float_as_uint(a[i]) & 0x7FFFFFFFu, __float_as_uint(b[i]) & 0x7FFFFFFFu));
    return m;
  }
  __device__ __forceinline__ uint2 codes(float s, float rs, bool finite) const {
    return i8_codes([&](int i) { return i < 4 ? a[i] : b[i - 4]; }, s, rs, finite);
  }
};
template <>
struct Chunk8<uint16_t> {
  u32x4_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ uint32_t top() const { return i8_top_bf16(v); }
  __device__ __forceinline__ uint2 codes(float s, float rs, bool finite) const { return i8_codes_bf16(v, s, rs, finite); }
};

// One workgroup of NT threads a row.  NC: chunks of 8 values a thread keeps
// (k <= 8 * NT * NC).  The row's adapter product comes along (NT >= rp): its
// partial sums are loaded behind the row, which saves their own launch (m =
// 2048, n = k = 4096, rank 16 63.8 -> 60.9 us; m = 64, rank 64 29.9 -> 23.9; the
// whole product X A^T in this kernel, from the same registers, was slower: 65.8).
// T is rounded to bf16, which the adapter term's MFMA takes: off by at most 2^-8 of T,
// as Y is by its own rounding.
// row0: the first row's place in t.
template <typename T, int NT, int NC, bool KEEP>
__global__ __launch_bounds__(NT) void k_i8_quant_rows(const T* __restrict__ X, int64_t ldx, int64_t k,
                                                     int8_t* __restrict__ Q, float* __restrict__ scales, XaSums t,
                                                     int64_t row0) {
  __shared__ uint32_t red[NT / 64];
  const int64_t row = blockIdx.x;
  const T* x = X + row * ldx;
  int8_t* q = Q + row * k;
  const int tid = threadIdx.x;
  const int chunks = (int)(k / 8);
  Chunk8<T> c[NC];
  uint32_t m = 0;
  auto adapter = [&]() {
    if (t.part == nullptr || tid >= t.rp) return;
    const int64_t tr = row0 + row;
    float v = 0.f;
    if (tid < t.r) v = t.sigma * sum_splits16(t.part, t.splits, t.m * t.rb, tr * t.rb + tid);
    t.T[tr * t.rp + tid] = (uint16_t)bf16_rne(v);
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (tid + i * NT < chunks) c[i].load(x + 8 * (tid + i * NT));
    adapter();
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (tid + i * NT < chunks) m = max(m, c[i].top());
  } else {
    adapter();
    for (int i = tid; i < chunks; i += NT) {
      c[0].load(x + 8 * i);
      m = max(m, c[0].top());
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    m = max(m, (uint32_t)__shfl_xor(m, o));
  }
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) m = max(m, red[i]);
  bool finite;
  const float s = i8_scale(m, finite), rs = 1.f / s;
  if (tid == 0) scales[row] = s;
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (tid + i * NT < chunks)
        *reinterpret_cast<uint2*>(q + 8 * (tid + i * NT)) = c[i].codes(s, rs, finite);
  } else {
    for (int i = tid; i < chunks; i += NT) {
      c[0].load(x + 8 * i);
      *reinterpret_cast<uint2*>(q + 8 * i) = c[0].codes(s, rs, finite);
    }
  }
}

// Rows of one launch: a grid has fewer than 2^32 threads, and a row up to 1024.
constexpr int64_t kMostRows = int64_t(1) << 21;

template <int NT, int NC, bool KEEP, typename T>
hipError_t launch_rows(const T* X, int64_t rows, int64_t k, int64_t ldx, int8_t* Q, float* scales, const XaSums& t,
                       hipStream_t s) {
  for (int64_t r = 0; r < rows; r += kMostRows)
    hipLaunchKernelGGL((k_i8_quant_rows<T, NT, NC, KEEP>), dim3((unsigned)std::min(rows - r, kMostRows)), dim3(NT), 0, s,
                       X + r * ldx, ldx, k, Q + r * k, scales + r, t, r);
  return hipGetLastError();
}

// At most two chunks a thread where the workgroup can be that large: a row's
// time is its latency (3 rows of 28672: 256 threads that read the row twice
// 14.8 us).
template <typename T>
hipError_t launch_quant(const T* X, int64_t rows, int64_t k, int64_t ldx, int8_t* Q, float* scales, const XaSums& t,
                        hipStream_t s) {
  if (k <= 2048) return launch_rows<256, 1, true>(X, rows, k, ldx, Q, scales, t, s);
  if (k <= 4096) return launch_rows<256, 2, true>(X, rows, k, ldx, Q, scales, t, s);
  if (k <= 8192) return launch_rows<512, 2, true>(X, rows, k, ldx, Q, scales, t, s);
  if (k <= 16384) return launch_rows<1024, 2, true>(X, rows, k, ldx, Q, scales, t, s);
  if (k <= 32768) return launch_rows<1024, 4, true>(X, rows, k, ldx, Q, scales, t, s);
  return launch_rows<1024, 1, false>(X, rows, k, ldx, Q, scales, t, s);
}

__global__ __launch_bounds__(kThreads) void k_i8_dequant(const int8_t* __restrict__ Q,
                                                        const float* __restrict__ scales, int k,
                                                        uint16_t* __restrict__ out) {
  const int64_t row = blockIdx.x;
  const float s = scales[row];
  const int8_t* q = Q + row * k;
  uint16_t* o = out + row * k;
  for (int i = 8 * threadIdx.x; i < k; i += 8 * kThreads) {
    const uint2 v = *reinterpret_cast<const uint2*>(q + i);
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = (j < 2 ? v.x : v.y) >> (16 * (j & 1));
      d[j] = cvt_pk_bf16((float)(int8_t)(uint8_t)w * s, (float)(int8_t)(uint8_t)(w >> 8) * s);
    }
    *reinterpret_cast<u32x4_t*>(o + i) = u32x4_t{d[0], d[1], d[2], d[3]};
  }
}

}  // namespace

hipError_t launch_i8_quant_f32(const float* W, int64_t n, int64_t k, int8_t* Q, float* scales, hipStream_t s) {
  return launch_quant(W, n, k, k, Q, scales, XaSums{}, s);
}

hipError_t launch_i8_quant_bf16(const uint16_t* X, int64_t m, int64_t k, int64_t ldx, int8_t* Q, float* scales,
                                const XaSums& t, hipStream_t s) {
  return launch_quant(X, m, k, ldx, Q, scales, t, s);
}

hipError_t launch_i8_dequant(const WView& w, uint16_t* out, hipStream_t s) {
  for (int64_t r = 0; r < w.n; r += kMostRows)
    hipLaunchKernelGGL(k_i8_dequant, dim3((unsigned)std::min(w.n - r, kMostRows)), dim3(kThreads), 0, s,
                       reinterpret_cast<const int8_t*>(w.packed) + r * w.k, w.scales + r, (int)w.k, out + r * w.k);
  return hipGetLastError();
}

}  // namespace lbq
