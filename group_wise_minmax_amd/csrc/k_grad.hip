// Global norm of a training step's gradients and their scaling to a largest
// norm, over many tensors at once:
//   norm = (sum over all tensors of x^2)^(1/2), or max |x|;
//   c = min(1, max_norm / (norm + 1e-6));  out = g * c.
//
// Two launches for each group of tensors (their table travels in the kernel's
// arguments, so nothing is copied to the device and a captured launch keeps
// it): the first sums, the second scales.  Bound by memory: the gradients are
// read twice and written once; a set within the 256 MB Infinity Cache is read
// the second time from there.
//
// The squares are summed in fp64 (a square of any finite fp32 value is
// finite there, and 10^9 of them lose nothing that fp32 could show).  Each
// workgroup owns a fixed run of 16-KiB pieces of the tensors laid end to end,
// and every workgroup of the second launch adds the partial sums in the same
// fixed order: the result does not change from run to run.
#include "lbq_device.h"

namespace lbq {

namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 16384;  // bytes of one tensor that a workgroup takes at a time

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == LBQ_F32) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == LBQ_BF16 ? __uint_as_float(b << 16) : f16_bits_to_f32(b);
}

__device__ __forceinline__ uint32_t f16_rne(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}

// bf16 bits of f, round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ uint32_t bf16_rne_nan(float f) { return f != f ? 0x7FC0u : bf16_rne(f); }

// Combines the threads' values in a fixed order; the result in every thread.
template <bool INF>
__device__ __forceinline__ double block_combine(double v) {
  __shared__ double red[kThreads / 64];
  if constexpr (INF) {
    // magnitudes are not negative: their bits order like the values, NaN last
    uint64_t u = __builtin_bit_cast(uint64_t, v);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t t = __shfl_xor((unsigned long long)u, o);
      u = t > u ? t : u;
    }
    v = __builtin_bit_cast(double, u);
  } else {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = red[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) {
    if constexpr (INF) {
      const uint64_t a = __builtin_bit_cast(uint64_t, r), b = __builtin_bit_cast(uint64_t, red[i]);
      r = __builtin_bit_cast(double, b > a ? b : a);
    } else {
      r += red[i];
    }
  }
  return r;
}

template <bool INF>
__device__ __forceinline__ double take(double acc, float x) {
  if constexpr (INF) {
    const double d = (double)__uint_as_float(__float_as_uint(x) & 0x7FFFFFFFu);
    const uint64_t a = __builtin_bit_cast(uint64_t, acc), b = __builtin_bit_cast(uint64_t, d) & ~(uint64_t(1) << 63);
    return __builtin_bit_cast(double, b > a ? b : a);
  } else {
    return fma((double)x, (double)x, acc);
  }
}

// The pieces [lo, hi) of this workgroup, one call of f(tensor, first element, end) each.
template <typename F>
__device__ __forceinline__ void for_pieces(const GradTable& t, F f) {
  const int64_t total = t.piece_end[t.count - 1];
  const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  int i = 0;
  for (int64_t p = lo; p < hi; ++p) {
    while (p >= t.piece_end[i]) ++i;
    const int64_t per = kPiece / (t.dtype[i] == LBQ_F32 ? 4 : 2);
    const int64_t first = (p - (i == 0 ? 0 : t.piece_end[i - 1])) * per;
    f(i, first, min(first + per, (int64_t)t.numel[i]));
  }
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void k_grad_norm(GradTable t, double* __restrict__ part) {
  double acc = 0.0;
  for_pieces(t, [&](int i, int64_t first, int64_t end) {
    for (int64_t e = first + threadIdx.x; e < end; e += kThreads) acc = take<INF>(acc, load_as_f32(t.grad[i], e, t.dtype[i]));
  });
  acc = block_combine<INF>(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm from all the partial values, in every thread.
template <bool INF>
__device__ __forceinline__ float norm_of(const double* __restrict__ part, int parts) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    if constexpr (INF) {
      const uint64_t a = __builtin_bit_cast(uint64_t, acc), b = __builtin_bit_cast(uint64_t, part[i]);
      acc = __builtin_bit_cast(double, b > a ? b : a);
    } else {
      acc += part[i];
    }
  }
  acc = block_combine<INF>(acc);
  return (float)(INF ? acc : sqrt(acc));
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void k_grad_norm_out(const double* __restrict__ part, int parts,
                                                           float* __restrict__ norm) {
  const float n = norm_of<INF>(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void k_grad_scale(GradTable t, const double* __restrict__ part, int parts,
                                                        float max_norm, float* __restrict__ norm) {
  const float n = norm_of<INF>(part, parts);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  float c = max_norm / (n + 1e-6f);
  if (c > 1.f) c = 1.f;  // a NaN norm keeps c a NaN
  for_pieces(t, [&](int i, int64_t first, int64_t end) {
    const int dt = t.dtype[i];
    if (c == 1.f && t.out[i] == t.grad[i]) return;
    for (int64_t e = first + threadIdx.x; e < end; e += kThreads) {
      const float v = load_as_f32(t.grad[i], e, dt) * c;
      if (dt == LBQ_F32) static_cast<float*>(t.out[i])[e] = v;
      else static_cast<uint16_t*>(t.out[i])[e] = (uint16_t)(dt == LBQ_BF16 ? bf16_rne_nan(v) : f16_rne(v));
    }
  });
}

int64_t pieces_of(const lbq_grad& g) {
  return (g.numel * (g.dtype == LBQ_F32 ? 4 : 2) + kPiece - 1) / kPiece;
}

// The next table of tensors from `at` on (empty ones left out); false when none is left.
bool next_table(const lbq_grad* g, int count, int& at, GradTable& t) {
  t.count = 0;
  int64_t end = 0;
  for (; at < count && t.count < kGradTable; ++at) {
    if (g[at].numel == 0) continue;
    end += pieces_of(g[at]);
    t.grad[t.count] = g[at].grad;
    t.out[t.count] = g[at].out;
    t.numel[t.count] = g[at].numel;
    t.dtype[t.count] = (uint8_t)g[at].dtype;
    t.piece_end[t.count++] = (int)end;
  }
  return t.count > 0;
}

// Workgroups of a table with p of all the total pieces: the chip holds eight a CU.
int groups_of(int64_t p, int64_t total) {
  if (total <= kGradGroups) return (int)p;
  const int64_t g = kGradGroups * p / total;
  return (int)(g < 1 ? 1 : g);
}

}  // namespace

int64_t grad_pieces(const lbq_grad* g, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += pieces_of(g[i]);
  return total;
}

int grad_parts(const lbq_grad* g, int count) {
  const int64_t total = grad_pieces(g, count);
  GradTable t;
  int parts = 0;
  for (int at = 0; next_table(g, count, at, t);) parts += groups_of(t.piece_end[t.count - 1], total);
  return parts;
}

hipError_t launch_grad_norm(const lbq_grad* g, int count, bool inf, double* part, hipStream_t s) {
  const int64_t total = grad_pieces(g, count);
  GradTable t;
  int parts = 0;
  for (int at = 0; next_table(g, count, at, t);) {
    const int groups = groups_of(t.piece_end[t.count - 1], total);
    if (inf) hipLaunchKernelGGL(k_grad_norm<true>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part + parts);
    else hipLaunchKernelGGL(k_grad_norm<false>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part + parts);
    parts += groups;
  }
  return hipGetLastError();
}

hipError_t launch_grad_norm_out(bool inf, const double* part, int parts, float* norm, hipStream_t s) {
  if (inf) hipLaunchKernelGGL(k_grad_norm_out<true>, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
  else hipLaunchKernelGGL(k_grad_norm_out<false>, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const lbq_grad* g, int count, bool inf, const double* part, int parts, float max_norm,
                             float* norm, hipStream_t s) {
  const int64_t total = grad_pieces(g, count);
  GradTable t;
  bool first = true;
  for (int at = 0; next_table(g, count, at, t); first = false) {
    const int groups = groups_of(t.piece_end[t.count - 1], total);
    float* out = first ? norm : nullptr;
    if (inf) hipLaunchKernelGGL(k_grad_scale<true>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part, parts, max_norm, out);
    else hipLaunchKernelGGL(k_grad_scale<false>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part, parts, max_norm, out);
  }
  return hipGetLastError();
}

}  // namespace lbq
