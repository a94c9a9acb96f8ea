// Global norm of a training step's gradients and their scaling to a largest
// norm, over many tensors at once:
//   norm = (sum over all tensors of x^2)^(1/2), or max |x|;
//   c = min(1, max_norm / (norm + 1e-6));  out = g * c.
//
// Two launches for each table of up to 120 tensors (the table travels in the
// kernel's arguments, so nothing is copied to the device and a captured launch
// keeps it): one sums, one scales; with several tables one more launch adds up
// all the partial sums.  Bound by memory: the gradients are read twice and
// written once.  448 adapter gradients of rank 64 (671 MB): 400 us, of them 130 the
// sums, 5.2 TB/s, and 259 the scaling, 5.2 TB/s read and written (a copy runs at
// 5.05).  The scaling walks back from what the sums read last, which is still in the
// 256 MB Infinity Cache (that table 42 us, the others 72).  Few small tensors are
// bound by the two launches (4 of rank 16, 0.9 MB: 12 us a call, 8.6 of them the
// kernels and the rest the host).
//
// The squares are summed in fp64 (a square of any finite fp32 value is
// finite there, and 10^9 of them lose nothing that fp32 could show).  Each
// workgroup owns a fixed run of 16-KiB pieces of the tensors laid end to end,
// and whoever adds the partial sums does it in one fixed order: the result does
// not change from run to run.
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
template <bool INF, int NT>
__device__ __forceinline__ double block_combine(double v) {
  __shared__ double red[NT / 64];
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
  for (int i = 1; i < NT / 64; ++i) {
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

// The pieces of this workgroup, one call of f(tensor, first element, end)
// each: [lo, hi) of the tensors laid end to end, from the first to the last, or
// from the last to the first.
template <bool BACK, int N, typename F>
__device__ __forceinline__ void for_pieces(const GradTable<N>& t, F f) {
  const int64_t total = t.piece_end[t.count - 1];
  const int lo = (int)(total * blockIdx.x / gridDim.x), hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
  if (lo >= hi) return;
  // the tensor of the piece to start with: the first whose end lies behind it
  int a = 0, b = t.count - 1;
  while (a < b) {
    const int mid = (a + b) >> 1;
    if (t.piece_end[mid] > (BACK ? hi - 1 : lo)) b = mid;
    else a = mid + 1;
  }
  int begin = a == 0 ? 0 : t.piece_end[a - 1], end = t.piece_end[a];
  for (int n = 0; n < hi - lo; ++n) {
    const int p = BACK ? hi - 1 - n : lo + n;
    if constexpr (BACK) {
      while (p < begin) end = begin, --a, begin = a == 0 ? 0 : t.piece_end[a - 1];
    } else {
      while (p >= end) begin = end, ++a, end = t.piece_end[a];
    }
    const int64_t per = kPiece / (t.dtype[a] == LBQ_F32 ? 4 : 2);
    const int64_t first = (int64_t)(p - begin) * per;
    f(a, first, min(first + per, t.numel[a]));
  }
}

constexpr int kLoads = kPiece / (kThreads * 16);  // 16-byte loads of a thread and piece

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Value i of a 16-byte chunk.
template <int DT>
__device__ __forceinline__ float value_of(const u32x4_t& v, int i) {
  if constexpr (DT == LBQ_F32) return __uint_as_float(v[i]);
  const uint32_t b = (i & 1) ? v[i >> 1] >> 16 : v[i >> 1] & 0xFFFFu;
  return DT == LBQ_BF16 ? __uint_as_float(b << 16) : f16_bits_to_f32(b);
}

template <bool INF, int DT>
__device__ __forceinline__ double take_piece(double acc, const void* g, int64_t first, int64_t end) {
  constexpr int V = DT == LBQ_F32 ? 4 : 8;  // values of a chunk
  if (aligned16(g)) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(g) + first / V;
    const int chunks = (int)((end - first) / V);
    u32x4_t v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int c = threadIdx.x + kThreads * j;
      v[j] = c < chunks ? p[c] : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) acc = take<INF>(acc, value_of<DT>(v[j], i));
    first += (int64_t)chunks * V;
  }
  for (int64_t e = first + threadIdx.x; e < end; e += kThreads) acc = take<INF>(acc, load_as_f32(g, e, DT));
  return acc;
}

template <bool INF, int N>
__global__ __launch_bounds__(kThreads) void k_grad_norm(GradTable<N> t, double* __restrict__ part) {
  double acc = 0.0;
  for_pieces<false>(t, [&](int i, int64_t first, int64_t end) {
    const int dt = t.dtype[i];
    if (dt == LBQ_F32) acc = take_piece<INF, LBQ_F32>(acc, t.grad[i], first, end);
    else if (dt == LBQ_BF16) acc = take_piece<INF, LBQ_BF16>(acc, t.grad[i], first, end);
    else acc = take_piece<INF, LBQ_F16>(acc, t.grad[i], first, end);
  });
  acc = block_combine<INF, kThreads>(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

template <int DT>
__device__ __forceinline__ uint32_t bits_of(float f) {
  if constexpr (DT == LBQ_F32) return __float_as_uint(f);
  return DT == LBQ_BF16 ? bf16_rne_nan(f) : f16_rne(f);
}

template <int DT>
__device__ __forceinline__ void scale_piece(const void* g, void* out, float c, int64_t first, int64_t end) {
  constexpr int V = DT == LBQ_F32 ? 4 : 8;
  if (aligned16(g) && aligned16(out)) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(g) + first / V;
    u32x4_t* o = reinterpret_cast<u32x4_t*>(out) + first / V;
    const int chunks = (int)((end - first) / V);
    u32x4_t v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int n = threadIdx.x + kThreads * j;
      if (n < chunks) v[j] = p[n];
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int n = threadIdx.x + kThreads * j;
      if (n >= chunks) continue;
      u32x4_t r;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (DT == LBQ_F32) {
          r[d] = __float_as_uint(value_of<DT>(v[j], d) * c);
        } else {
          r[d] = bits_of<DT>(value_of<DT>(v[j], 2 * d) * c) | bits_of<DT>(value_of<DT>(v[j], 2 * d + 1) * c) << 16;
        }
      }
      __builtin_nontemporal_store(r, o + n);
    }
    first += (int64_t)chunks * V;
  }
  for (int64_t e = first + threadIdx.x; e < end; e += kThreads) {
    const float v = load_as_f32(g, e, DT) * c;
    if constexpr (DT == LBQ_F32) static_cast<float*>(out)[e] = v;
    else static_cast<uint16_t*>(out)[e] = (uint16_t)bits_of<DT>(v);
  }
}

// The norm from all the partial values, in every thread.
template <bool INF, int NT>
__device__ __forceinline__ float norm_of(const double* __restrict__ part, int parts) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += 8 * NT) {  // eight loads in flight
    double v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j * NT < parts ? part[i + j * NT] : 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (INF) {
        const uint64_t a = __builtin_bit_cast(uint64_t, acc), b = __builtin_bit_cast(uint64_t, v[j]);
        acc = __builtin_bit_cast(double, b > a ? b : a);
      } else {
        acc += v[j];
      }
    }
  }
  acc = block_combine<INF, NT>(acc);
  return (float)(INF ? acc : sqrt(acc));
}

template <bool INF>
__global__ __launch_bounds__(1024) void k_grad_norm_out(const double* __restrict__ part, int parts,
                                                       float* __restrict__ norm) {
  const float n = norm_of<INF, 1024>(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

// Scales the tensors of a table; the norm from `parts` partial values, or from
// *norm itself (parts == 0) where a launch before this one has summed them.
template <bool INF, int N>
__global__ __launch_bounds__(kThreads) void k_grad_scale(GradTable<N> t, const double* __restrict__ part, int parts,
                                                        float max_norm, float* __restrict__ norm) {
  float n;
  if (parts > 0) {
    n = norm_of<INF, kThreads>(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  } else {
    n = *norm;
  }
  float c = max_norm / (n + 1e-6f);
  if (c > 1.f) c = 1.f;  // a NaN norm keeps c a NaN
  for_pieces<true>(t, [&](int i, int64_t first, int64_t end) {
    const int dt = t.dtype[i];
    const void* g = t.grad[i];
    void* out = t.out[i];
    if (c == 1.f && out == g) return;
    if (dt == LBQ_F32) scale_piece<LBQ_F32>(g, out, c, first, end);
    else if (dt == LBQ_BF16) scale_piece<LBQ_BF16>(g, out, c, first, end);
    else scale_piece<LBQ_F16>(g, out, c, first, end);
  });
}

int64_t pieces_of(const lbq_grad& g) {
  return (g.numel * (g.dtype == LBQ_F32 ? 4 : 2) + kPiece - 1) / kPiece;
}

// The next table of tensors from `at` on (empty ones left out); false when none is left.
bool next_table(const lbq_grad* g, int count, int& at, GradTable<kGradTable>& t) {
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

// f(table) with the table cut to kGradFew where they suffice: the arguments of a
// launch are written to it (4 tensors, norm and scaling 12.3 us a call against
// 11.6).
template <typename F>
void with_table(const GradTable<kGradTable>& t, F f) {
  if (t.count > kGradFew) return f(t);
  GradTable<kGradFew> few;
  for (int i = 0; i < t.count; ++i) {
    few.grad[i] = t.grad[i], few.out[i] = t.out[i], few.numel[i] = t.numel[i];
    few.piece_end[i] = t.piece_end[i], few.dtype[i] = t.dtype[i];
  }
  few.count = t.count;
  f(few);
}

// Workgroups of a table of p pieces: eight a CU where there are that many.
int groups_of(int64_t p) { return (int)(p < kGradGroups ? p : kGradGroups); }

template <bool INF>
hipError_t norm_launches(const lbq_grad* g, int count, double* part, hipStream_t s) {
  GradTable<kGradTable> all;
  for (int at = 0; next_table(g, count, at, all);) {
    const int groups = groups_of(all.piece_end[all.count - 1]);
    with_table(all, [&](const auto& t) {
      hipLaunchKernelGGL(k_grad_norm<INF>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part);
    });
    part += groups;
  }
  return hipGetLastError();
}

template <bool INF>
hipError_t scale_launches(const lbq_grad* g, int count, const double* part, int parts, float max_norm, float* norm,
                          hipStream_t s) {
  // One table: its workgroups sum the partial values themselves (at most 2048,
  // from L2).  More: one launch sums them once.
  if (count > kGradTable) {
    hipLaunchKernelGGL(k_grad_norm_out<INF>, dim3(1), dim3(1024), 0, s, part, parts, norm);
    parts = 0;
  }
  // The last table first, and each from its end (for_pieces): what the sums
  // read last is still in the Infinity Cache.
  int full = 0;
  for (int i = 0; i < count; ++i) full += g[i].numel > 0;
  for (int first = full > 0 ? (full - 1) / kGradTable * kGradTable : -1; first >= 0; first -= kGradTable) {
    GradTable<kGradTable> all;
    int at = 0;
    for (int skip = first; skip > 0 || g[at].numel == 0; ++at) skip -= g[at].numel > 0;
    next_table(g, count, at, all);
    const int groups = groups_of(all.piece_end[all.count - 1]);
    with_table(all, [&](const auto& t) {
      hipLaunchKernelGGL(k_grad_scale<INF>, dim3((unsigned)groups), dim3(kThreads), 0, s, t, part, parts, max_norm, norm);
    });
  }
  return hipGetLastError();
}

}  // namespace

int grad_parts(const lbq_grad* g, int count) {
  int parts = 0;
  int64_t pieces = 0;
  for (int i = 0, n = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    pieces += pieces_of(g[i]);
    if (++n % kGradTable == 0) parts += groups_of(pieces), pieces = 0;
  }
  return parts + groups_of(pieces);
}

hipError_t launch_grad_norm(const lbq_grad* g, int count, bool inf, double* part, hipStream_t s) {
  return inf ? norm_launches<true>(g, count, part, s) : norm_launches<false>(g, count, part, s);
}

hipError_t launch_grad_norm_out(bool inf, const double* part, int parts, float* norm, hipStream_t s) {
  if (inf) hipLaunchKernelGGL(k_grad_norm_out<true>, dim3(1), dim3(1024), 0, s, part, parts, norm);
  else hipLaunchKernelGGL(k_grad_norm_out<false>, dim3(1), dim3(1024), 0, s, part, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const lbq_grad* g, int count, bool inf, const double* part, int parts, float max_norm,
                             float* norm, hipStream_t s) {
  return inf ? scale_launches<true>(g, count, part, parts, max_norm, norm, s)
             : scale_launches<false>(g, count, part, parts, max_norm, norm, s);
}

}  // namespace lbq
