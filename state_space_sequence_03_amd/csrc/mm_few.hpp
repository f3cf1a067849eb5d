// Products of few rows (generation steps): bound by reading Q once.
//
// A block owns 16 rows of Q (gated: 16 of each half) and its eight waves
// split k in runs of U steps of 64 bytes: one 16-byte load per lane and
// operand straight into the fragment layout of the 16 x 16 products (lane l:
// row l mod 16, 16 bytes l / 16), no LDS on the way.  A run's loads are issued
// before its products, so that a wave has U KB (gated 2U) of Q in flight.  The
// waves' sums are joined in LDS in order.  One row through 2048 -> 2 x 5632
// takes 10.2 us (46 MB: 4.5 TB/s), 16 rows 13.1: every block reads all of P,
// from its L2.
// (Sixteen waves, for calls with fewer blocks than CUs, measured the same: 7.1
// us for one row of 4096 -> 2048.)
// Rows of P past the last and rows of Q past N repeat the last row; their
// outputs are not written.
#pragma once

#include "act.hpp"
#include "m3_launch.hpp"
#include "m3_rows.hpp"

namespace m3 {

template <typename T>
__device__ __forceinline__ f32x4 mma16(const u32x4& p, const u32x4& q, f32x4 acc) {
  if constexpr (io<T>::BYTES == 2) {
    return mfma_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), acc);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mfma_f32(__uint_as_float(p[j]), __uint_as_float(q[j]), acc);
    return acc;
  }
}

// 16 bytes of a row at byte b of `bytes`; what lies past the row's end is 0
template <typename T>
__device__ __forceinline__ u32x4 few_load(const char* row, int b, int bytes) {
  if (b + 16 <= bytes) return *(const u32x4_any*)(row + b);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16 / io<T>::BYTES; ++j)
    if (b + (j + 1) * io<T>::BYTES <= bytes) {
      if constexpr (io<T>::BYTES == 2) v[j >> 1] |= (uint32_t)*(const u16*)(row + b + 2 * j) << (16 * (j & 1));
      else v[j] = *(const uint32_t*)(row + b + 4 * j);
    }
  return v;
}

template <typename T, int EPI, int ACT, int MT>
__global__ __launch_bounds__(512) void mm_few_kernel(MmArgs a) {
  constexpr int ES = io<T>::BYTES;
  constexpr bool G = EPI == MM_GATED;
  constexpr int NW = 8, QT = G ? 2 : 1, U = MT == 1 ? 8 : 4;
  __shared__ f32x4 sh[NW][QT * MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int r = lane & 15, c16 = (lane >> 4) * 16;
  const int bytes = (int)(a.K * ES);
  const char* q[QT];
  const char* p[MT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int64_t n = n0 + r < a.N ? n0 + r : a.N - 1;
    q[i] = (const char*)a.Q + (i * a.N + n) * a.ldq * ES;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = j * 16 + r < a.M ? j * 16 + r : a.M - 1;
    p[j] = (const char*)a.P + m * a.ldp * ES;
  }
  f32x4 acc[QT][MT];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // whole runs of U steps per wave
  int k0 = 0;
  for (; k0 + NW * U * 64 <= bytes; k0 += NW * U * 64) {
    const int b = k0 + wave * U * 64 + c16;
    u32x4 fq[U][QT], fp[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < QT; ++i) fq[u][i] = *(const u32x4_any*)(q[i] + b + u * 64);
#pragma unroll
      for (int j = 0; j < MT; ++j) fp[u][j] = *(const u32x4_any*)(p[j] + b + u * 64);
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them before the first product
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = mma16<T>(fq[u][i], fp[u][j], acc[i][j]);
  }
  for (int b = k0 + wave * 64 + c16; b - c16 < bytes; b += NW * 64) {
    u32x4 fq[QT], fp[MT];
#pragma unroll
    for (int i = 0; i < QT; ++i) fq[i] = few_load<T>(q[i], b, bytes);
#pragma unroll
    for (int j = 0; j < MT; ++j) fp[j] = few_load<T>(p[j], b, bytes);
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = mma16<T>(fq[i], fp[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) sh[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  // thread e: column e mod 16 of row e / 16; its sum sits in lane
  // row + 16 (column / 4), word column mod 4
  constexpr bool FINE = ES == 4;
  for (int e = threadIdx.x; e < MT * 256; e += 64 * NW) {
    const int j = e >> 8, row = (e >> 4) & 15, col = e & 15, l = row + 16 * (col >> 2), w = col & 3;
    const int64_t m = j * 16 + row, n = n0 + col;
    if (m >= a.M || n >= a.N) continue;
    float z = 0.0f, u = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      z += sh[k][j][l][w];
      if constexpr (G) u += sh[k][MT + j][l][w];
    }
    if (a.bias) z += a.bias[n];
    if constexpr (G) {
      if (a.bias) u += a.bias[a.N + n];
      if (a.pre) {
        io<T>::store1(a.pre, m * 2 * a.N + n, z);
        io<T>::store1(a.pre, m * 2 * a.N + a.N + n, u);
      }
      z = act_fwd<ACT, FINE>(z) * u;
    } else {
      if (a.pre) io<T>::store1(a.pre, m * a.N + n, z);
      z = act_fwd<ACT, FINE>(z);
      if (a.res) z += io<T>::load1(a.res, m * a.ldr + n);
    }
    io<T>::store1(a.out, m * a.ldo + n, z);
  }
}

template <typename T, int EPI, int ACT>
hipError_t mm_few_run(const MmArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), blk(512);
  if (a.M <= 16) hipLaunchKernelGGL((mm_few_kernel<T, EPI, ACT, 1>), grid, blk, 0, s, a);
  else if (a.M <= 32) hipLaunchKernelGGL((mm_few_kernel<T, EPI, ACT, 2>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((mm_few_kernel<T, EPI, ACT, 4>), grid, blk, 0, s, a);
  return hipGetLastError();
}

}  // namespace m3
