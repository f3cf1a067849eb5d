// Matrix products of the linear and gated feed-forward operators:
//   out[m][n] = epilogue(sum_k P(m, k) Q(n, k)).
#include "mm_tile.hpp"
#include "mm_parts.hpp"

namespace m3 {

namespace {

template <typename T>
__device__ __forceinline__ void move1(void* dst, int64_t i, const void* src, int64_t j, bool in) {
  if constexpr (io<T>::BYTES == 2) ((u16*)dst)[i] = in ? ((const u16*)src)[j] : (u16)0;
  else ((float*)dst)[i] = in ? ((const float*)src)[j] : 0.0f;
}

// 64 x 64 outputs per block, four waves of 32 x 32, k in steps of 32
// elements; operands element by element through LDS, so that any stride,
// alignment and size is right.
template <typename T, int LAYOUT, int EPI, int ACT>
__global__ __launch_bounds__(256) void mm_kernel(MmArgs a) {
  constexpr int ES = io<T>::BYTES;
  constexpr int BK = 32, PITCH = BK + 16 / ES;
  constexpr bool PK = LAYOUT != MM_NONE_K, QK = LAYOUT == MM_PQ_K;
  constexpr int BN = EPI == MM_GATED ? 32 : 64;
  __shared__ __attribute__((aligned(16))) char Ps[64 * PITCH * ES];
  __shared__ __attribute__((aligned(16))) char Qs[64 * PITCH * ES];
  __shared__ float Cs[64][65];
  const int64_t nb = (a.N + BN - 1) / BN;
  const int64_t m0 = (blockIdx.x / nb) * 64, n0 = (blockIdx.x % nb) * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  for (int64_t k0 = 0; k0 < a.K; k0 += BK) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = i * 256 + tid;
      {
        const int r = PK ? e / BK : e % 64, k = PK ? e % BK : e / 64;
        const int64_t m = m0 + r, kk = k0 + k;
        move1<T>(Ps, r * PITCH + k, a.P, PK ? m * a.ldp + kk : kk * a.ldp + m, m < a.M && kk < a.K);
      }
      {
        const int r = QK ? e / BK : e % 64, k = QK ? e % BK : e / 64;
        const int64_t f = n0 + (EPI == MM_GATED ? r % 32 : r), kk = k0 + k;
        const int64_t n = EPI == MM_GATED && r >= 32 ? a.N + f : f;
        move1<T>(Qs, r * PITCH + k, a.Q, QK ? n * a.ldq + kk : kk * a.ldq + n, f < a.N && kk < a.K);
      }
    }
    __syncthreads();
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int s = 0; s < BK * ES / 32; ++s) {
      const uint4 p = *(const uint4*)(Ps + ((wave & 1) * 32 + r) * PITCH * ES + (2 * s + h) * 16);
      const uint4 q = *(const uint4*)(Qs + ((wave >> 1) * 32 + r) * PITCH * ES + (2 * s + h) * 16);
      acc = mma32<T>(q, p, acc);
    }
  }
  // lane l holds output row l mod 32 and columns 8(v / 4) + 4(l / 32) + v mod 4
#pragma unroll
  for (int v = 0; v < 16; ++v)
    Cs[(wave & 1) * 32 + (lane & 31)][(wave >> 1) * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)] = acc[v];
  __syncthreads();
  constexpr bool FINE = ES == 4;
  for (int e = tid; e < 64 * BN; e += 256) {
    const int r = e / BN, c = e % BN;
    const int64_t m = m0 + r, n = n0 + c;
    if (m >= a.M || n >= a.N) continue;
    float z = Cs[r][c];
    if constexpr (EPI != MM_STORE) z += a.bias ? a.bias[n] : 0.0f;
    if constexpr (EPI == MM_LINEAR) {
      if (a.pre) io<T>::store1(a.pre, m * a.N + n, z);
      z = act_fwd<ACT, FINE>(z);
      if (a.res) z += io<T>::load1(a.res, m * a.ldr + n);
    }
    if constexpr (EPI == MM_GATED) {
      const float u = Cs[r][32 + c] + (a.bias ? a.bias[a.N + n] : 0.0f);
      if (a.pre) {
        io<T>::store1(a.pre, m * 2 * a.N + n, z);
        io<T>::store1(a.pre, m * 2 * a.N + a.N + n, u);
      }
      z = act_fwd<ACT, FINE>(z) * u;
    }
    io<T>::store1(a.out, m * a.ldo + n, z);
  }
}

template <typename T>
hipError_t mm_run(MmLayout layout, MmEpilogue epi, const MmArgs& a, hipStream_t s) {
  const int64_t bn = epi == MM_GATED ? 32 : 64;
  const dim3 grid((unsigned)(((a.M + 63) / 64) * ((a.N + bn - 1) / bn))), blk(256);
  if (epi == MM_STORE) {
    if (layout == MM_P_K) hipLaunchKernelGGL((mm_kernel<T, MM_P_K, MM_STORE, 0>), grid, blk, 0, s, a);
    else if (layout == MM_NONE_K) hipLaunchKernelGGL((mm_kernel<T, MM_NONE_K, MM_STORE, 0>), grid, blk, 0, s, a);
    else return hipErrorInvalidValue;
  } else {
    if (layout != MM_PQ_K) return hipErrorInvalidValue;
    with_act(a.act, [&](auto act) {
      if (epi == MM_LINEAR) hipLaunchKernelGGL((mm_kernel<T, MM_PQ_K, MM_LINEAR, act.value>), grid, blk, 0, s, a);
      else hipLaunchKernelGGL((mm_kernel<T, MM_PQ_K, MM_GATED, act.value>), grid, blk, 0, s, a);
    });
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm(int io_bf16, MmLayout layout, MmEpilogue epi, const MmArgs& a, hipStream_t s) {
  const int es = io_bf16 ? 2 : 4;
  auto on16 = [&](const void* p, int64_t ld, int64_t width) {
    return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0 && width * es % 16 == 0;
  };
  if (on16(a.P, a.ldp, layout == MM_NONE_K ? a.M : a.K) && on16(a.Q, a.ldq, layout == MM_PQ_K ? a.K : a.N)) {
    if (epi == MM_STORE) return io_bf16 ? mm_store_bf16(layout, a, s) : mm_store_f32(layout, a, s);
    if (epi == MM_LINEAR) return io_bf16 ? mm_linear_bf16(a, s) : mm_linear_f32(a, s);
    return io_bf16 ? mm_gated_bf16(a, s) : mm_gated_f32(a, s);
  }
  return io_bf16 ? mm_run<bf16_t>(layout, epi, a, s) : mm_run<float>(layout, epi, a, s);
}

}  // namespace m3
