// Input gradient through 8-bit weights for few outputs, dX = sum_i dY_i . deq(W_i)
// with deq(W) = bf16(fl(q * s)) (m * k too small for k_bwd_dx's tiles to fill the
// chip; that kernel, in k_bwd.hip, does the larger ones).  The weight is rounded to
// bf16 for the MFMA, and is the weight that lbq_dequant writes, as for the other
// formats: dX is off by 0.0023 of its norm, where fp32 weights would leave the 0.0017
// of its own rounding; a second bf16 part of each weight would cost as many MFMAs
// again.
//
// A workgroup computes 64 columns of dX (k) of 16 TM tokens; its eight waves
// split the reduction over n among them, 32 rows of W at a time by turns, each
// through an LDS ring of its own (as in k_i8_skinny.hip: no barrier, and whole
// 64-byte runs for the L1), and the waves' fp32 sums are added at the end in a
// fixed order.  Given a workspace, the rows are also split over workgroups,
// whose sums k_i8_dx_reduce adds: a CU keeps some 0.25 cache lines a ns coming,
// so a weight needs all of them (m = 40, n = k = 4096: 64 workgroups 24.7 us, split
// into four ranges 13.9; by k_bwd_dx's 128 x 128 tiles 108).  Bound by latency:
// 17 MB at 5 TB/s are 3.4 us, and a launch, a wave's few loads and the second
// launch follow one another.
//
// The reduction runs along W's rows, so an MFMA (v_mfma_f32_16x16x32_bf16) wants
// 8 rows of one column from a lane, while memory has a row's columns side by
// side.  The columns of a workgroup are therefore numbered so that no value has
// to change lanes: row r of MFMA block a is column 4 r + a, so that the dword at
// column 4 (l % 16) of a row, which lane l reads at once, is that lane's values
// in the four blocks.
#pragma clang fp contract(off)

#include "lbq_device.h"

namespace lbq {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int TK = 4;  // MFMA blocks of 16 columns

struct DxSet {
  const int8_t* w[kGemvMaxGroup];
  const float* s[kGemvMaxGroup];
  const uint16_t* dy[kGemvMaxGroup];
  int n[kGemvMaxGroup];
  int end[kGemvMaxGroup];  // slices of 32 rows of weights 0 .. i
  int count;
};

// dX at o from 4 N sums.
template <int N>
__device__ __forceinline__ void store_dx(const float (&v)[4 * N], uint16_t* __restrict__ o) {
#pragma unroll
  for (int h = 0; h < N; ++h)
    reinterpret_cast<uint2*>(o)[h] = make_uint2(cvt_pk_bf16(v[4 * h], v[4 * h + 1]), cvt_pk_bf16(v[4 * h + 2], v[4 * h + 3]));
}

// Slices [per * blockIdx.y, + per) of the reduction.  `part`: [gridDim.y][m][k]
// sums instead of dX.
template <int TM, int U>
__global__ __launch_bounds__(kThreads) void k_i8_dx(DxSet set, int m, int k, int per, uint16_t* __restrict__ dX,
                                                   float* __restrict__ part, LoraDx lora) {
  constexpr int L = 2 + TM;  // KiB of a slice: 32 rows of 64 codes, TM blocks of 16 tokens of 32 gradients
  static_assert(U * L >= TK * TM, "a wave's sums fit its ring");
  __shared__ __attribute__((aligned(1024))) int8_t ring[kWaves][U][L * 1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int nx = k / 64;
  const int t = xcd_order(blockIdx.x, gridDim.x);  // neighbouring columns share lines of W: one XCD
  const int k0 = (t % nx) * 64, m0 = (t / nx) * 16 * TM;

  // The weight that the loads are in; a wave's slices come in order.
  int wi = 0, n = set.n[0], begin = 0, end = set.end[0];
  __amdgpu_buffer_rsrc_t rw, rs, rd;
  int od[TM];  // (of up to 32 bits)
  // Loads of 16 x 64 bytes.  W: the row q + 8 g of a slice lies in slot 4 q + g, so
  // that the four rows that a read takes together are in different banks.  dY: 32
  // gradients of a token a row, in the order of i8_key.
  const int slot = lane >> 2;
  int ow[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) ow[h] = (8 * (slot & 3) + 4 * h + (slot >> 2)) * k + k0 + 16 * (lane & 3);
  auto bind = [&]() {
    rw = make_rsrc(set.w[wi], (int64_t)n * k);
    rs = make_rsrc(set.s[wi], (int64_t)n * 4);
    rd = make_rsrc(set.dy[wi], (int64_t)m * n * 2);
#pragma unroll
    for (int b = 0; b < TM; ++b)
      od[b] = (int)((uint32_t)min(m0 + 16 * b + slot, m - 1) * (uint32_t)n * 2u) + 16 * ((lane & 3) ^ i8_key(slot));
  };
  bind();
  f32x4_t s[U][2];  // scales of this lane's 8 rows
  int left[U];      // rows of the weight from the slice on
  // Rows of W past n read as zeros, and their scales; dY past a token's end is the
  // next token's and is left out when it is multiplied (n % 8 == 0).
  auto load = [&](int u, int j) {
    while (j >= end) {
      begin = end;
      ++wi;
      n = set.n[wi], end = set.end[wi];
      bind();
    }
    const int r0 = 32 * (j - begin);
    left[u] = n - r0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s[u][h] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 32 * lg + 16 * h, 4 * r0, 0));
#pragma unroll
    for (int h = 0; h < 2; ++h) load_to_lds(rw, &ring[wave][u][1024 * h], ow[h], r0 * k);
#pragma unroll
    for (int b = 0; b < TM; ++b) load_to_lds(rd, &ring[wave][u][1024 * (2 + b)], od[b], 2 * r0);
  };
  f32x4_t acc[TK][TM];
#pragma unroll
  for (int a = 0; a < TK; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int fd = li * 64 + 16 * (lg ^ i8_key(li)), fw = lg * 64 + li * 4;
  auto mma = [&](int u) {
    uint32_t c[8];  // four columns of row 8 lg + q
    u32x4_t d[TM], w[TK];
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = *reinterpret_cast<const uint32_t*>(&ring[wave][u][fw + 256 * q]);
#pragma unroll
    for (int b = 0; b < TM; ++b) d[b] = *reinterpret_cast<const u32x4_t*>(&ring[wave][u][1024 * (2 + b) + fd]);
    if (left[u] < 32) {
#pragma unroll
      for (int b = 0; b < TM; ++b)
        if (8 * lg >= left[u]) d[b] = u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      const float s0 = s[u][q >> 2][q & 3], s1 = s[u][q >> 2][(q & 3) + 1];
#pragma unroll
      for (int a = 0; a < TK; ++a)
        w[a][q >> 1] = cvt_pk_bf16((float)(int8_t)(uint8_t)(c[q] >> (8 * a)) * s0,
                                   (float)(int8_t)(uint8_t)(c[q + 1] >> (8 * a)) * s1);
    }
#pragma unroll
    for (int a = 0; a < TK; ++a)
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] = mfma16x16x32(w[a], d[b], acc[a][b]);
  };
  // Slices first, first + 8, ..., U of them on their way.
  const int first = per * blockIdx.y + wave, last = min(per * ((int)blockIdx.y + 1), set.end[set.count - 1]);
  const int cnt = first < last ? (last - first + kWaves - 1) / kWaves : 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < cnt) load(u, first + kWaves * u);
  // The adapter's G . A, 32 of the rank by each of the first waves (of the first
  // range), in the columns' order of the weight.  (Added to each output where it
  // is stored, with scalar sums: m = 300, n = k = 4096, rank 64, all of lbq_lora_bwd 103 us against 67.)
  if (lora.g != nullptr && blockIdx.y == 0 && 32 * wave < lora.rp) {
    const int j0 = 32 * wave + 8 * lg;
    uint2 c[8];  // four columns of row j0 + q
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      c[q] = make_uint2(0u, 0u);
      if (j0 + q < lora.r) c[q] = *reinterpret_cast<const uint2*>(lora.a + (int64_t)(j0 + q) * k + k0 + 4 * li);
    }
    u32x4_t d[TM];
#pragma unroll
    for (int b = 0; b < TM; ++b) {
      const int64_t mr = min(m0 + 16 * b + li, m - 1);
      d[b] = *reinterpret_cast<const u32x4_t*>(lora.g + mr * lora.rp + j0);
    }
#pragma unroll
    for (int a = 0; a < TK; ++a) {
      u32x4_t w;
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        const uint32_t lo = (a < 2 ? c[q].x : c[q].y) >> (16 * (a & 1)), hi = (a < 2 ? c[q + 1].x : c[q + 1].y) >> (16 * (a & 1));
        w[q >> 1] = (lo & 0xFFFFu) | hi << 16;
      }
#pragma unroll
      for (int b = 0; b < TM; ++b) acc[a][b] = mfma16x16x32(w, d[b], acc[a][b]);
    }
  }
  run_ring<U, 2 + L>(cnt, [&](int u, int j) { load(u, first + kWaves * j); }, [&](int u, int) { mma(u); });

  f32x4_t* const sums = reinterpret_cast<f32x4_t*>(&ring[wave][0][0]);
#pragma unroll
  for (int a = 0; a < TK; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) sums[(b * TK + a) * 64 + lane] = acc[a][b];
  __syncthreads();
  // Lane l: token l % 16, columns 16 (l / 16) + 4 i + a.
  if (wave >= TM) return;
  const int mr = m0 + 16 * wave + li, kb = k0 + 16 * lg;
  if (mr >= m) return;
  float v[16];
#pragma unroll
  for (int a = 0; a < TK; ++a) {
    f32x4_t r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) r += reinterpret_cast<const f32x4_t*>(&ring[w][0][0])[(wave * TK + a) * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * i + a] = r[i];
  }
  if (part != nullptr) {
    f32x4_t* o = reinterpret_cast<f32x4_t*>(part + ((int64_t)blockIdx.y * m + mr) * k + kb);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    return;
  }
  store_dx<4>(v, dX + (int64_t)mr * k + kb);
}

// dX from the sums of ks ranges: one thread for four columns of a token.
__global__ __launch_bounds__(256) void k_i8_dx_reduce(const float* __restrict__ part, int ks, int m, int k,
                                                     uint16_t* __restrict__ dX) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = k / 4;
  if (i >= (int64_t)m * per) return;
  const int64_t stride = (int64_t)m * per;
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(part) + i;
  f32x4_t r = p[0];
#pragma unroll 3
  for (int j = 1; j < ks; ++j) r += p[j * stride];
  const float v[4] = {r[0], r[1], r[2], r[3]};
  store_dx<1>(v, dX + 4 * i);
}

template <int TM, int U>
void launch(const DxSet& set, int64_t m, int64_t k, int ks, int per, uint16_t* dX, float* part, const LoraDx& lora, hipStream_t s) {
  const int64_t groups = k / 64 * ((m + 16 * TM - 1) / (16 * TM));
  hipLaunchKernelGGL((k_i8_dx<TM, U>), dim3((unsigned)groups, (unsigned)ks), dim3(kThreads), 0, s, set, (int)m, (int)k, per,
                     dX, part, lora);
}

}  // namespace

size_t i8_dx_workspace_bytes(const int64_t* ns, int count, int64_t k, int64_t m) {
  const I8DxChoice c = i8_dx_choose(ns, count, k, m, true);
  return c.tm != 0 && c.ks > 1 ? (size_t)c.ks * (size_t)m * (size_t)k * sizeof(float) : 0;
}

hipError_t launch_i8_dx(const WView* ws, const uint16_t* const* dys, int count, int64_t m, uint16_t* dX,
                        const LoraDx& lora, float* part, size_t part_bytes, hipStream_t s) {
  DxSet set{};
  set.count = count;
  int64_t ns[kGemvMaxGroup];
  int end = 0;
  for (int i = 0; i < count; ++i) {
    set.w[i] = reinterpret_cast<const int8_t*>(ws[i].packed);
    set.s[i] = ws[i].scales;
    set.dy[i] = dys[i];
    set.n[i] = (int)ws[i].n;
    ns[i] = ws[i].n;
    end += (int)((ws[i].n + 31) / 32);
    set.end[i] = end;
  }
  const int64_t k = ws[0].k;
  const size_t need = i8_dx_workspace_bytes(ns, count, k, m);
  const bool split = need > 0 && part != nullptr && part_bytes >= need;
  const I8DxChoice c = i8_dx_choose(ns, count, k, m, split || need == 0);
  if (c.tm == 0) return launch_bwd_dx_i8_tiles(ws, dys, count, c.bk, c.bm, m, dX, lora, s);
  if (c.ks > 1 && !split) return hipErrorInvalidValue;
  if (c.ks == 1) part = nullptr;
  if (c.tm == 1) launch<1, 4>(set, m, k, c.ks, c.per, dX, part, lora, s);
  else if (c.tm == 2) launch<2, 3>(set, m, k, c.ks, c.per, dX, part, lora, s);
  else launch<4, 3>(set, m, k, c.ks, c.per, dX, part, lora, s);
  if (part != nullptr)
    hipLaunchKernelGGL(k_i8_dx_reduce, dim3((unsigned)((m * (k / 4) + 255) / 256)), dim3(256), 0, s, part, c.ks, (int)m,
                       (int)k, dX);
  return hipGetLastError();
}

}  // namespace lbq
