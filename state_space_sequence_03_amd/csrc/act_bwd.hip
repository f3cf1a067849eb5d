// The elementwise part of the backward of the linear and gated feed-forward
// operators, in one pass over dy and the stored pre-activations:
//   linear: dP = dy act'(pre);   gated: dP = [dy u act'(g), dy act(g)],
// rounded once to the io type, and the column sums of the unrounded dP (the
// bias' gradient).  The products that follow take their operands in the io
// type, and the bf16 matrix cores nothing wider: for bf16 io that rounding and
// the output's, 1.7e-3 relative each, leave dx and dW 2.3e-3 off; dP as a sum
// of two bf16 operands would double the products' time.  fp32 io keeps it whole.
// Bound by HBM: 3 reads and 2 writes of rows x cols run at 5.1-5.5 TB/s (32768 x
// 5632 bf16, 0.34-0.36 ms), one row per thread at a time: unrolled by 2 or 4 the
// loop holds fewer waves, and a call of it and a short product takes 616 and
// 583 us against 545.  A block owns 32 vectors of columns and a slab of rows,
// eight rows at a time; each thread sums its columns over its rows, the eight
// row groups are added in LDS and the slabs by launch_reduce_parts, all in a
// fixed order.
#include "act.hpp"
#include "m3_launch.hpp"
#include "m3_rows.hpp"

namespace m3 {

namespace {

template <typename T, int ACT, bool GATED>
__global__ __launch_bounds__(256) void act_bwd_kernel(ActBwdArgs a, int64_t slab) {
  constexpr int V = io<T>::VEC;
  constexpr bool FINE = io<T>::BYTES == 4;
  constexpr int W = GATED ? 2 : 1;
  __shared__ float sh[7][32][W * V + 1];
  const int cv = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int64_t c = ((int64_t)blockIdx.x * 32 + cv) * V, C = a.cols, ld = W * C;
  const int64_t r0 = (int64_t)blockIdx.y * slab, r1 = r0 + slab < a.rows ? r0 + slab : a.rows;
  float s[W][V];
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int j = 0; j < V; ++j) s[w][j] = 0.0f;
  if (c < C)
#pragma unroll 1
    for (int64_t r = r0 + rg; r < r1; r += 8) {
      float d[V], z[V], u[V];
      row_load<T>((const char*)a.dy + r * a.ldy * io<T>::BYTES, c, C, d);
      const char* pre = (const char*)a.pre + r * ld * io<T>::BYTES;
      if constexpr (GATED || ACT != ACT_NONE) row_load<T>(pre, c, C, z);
      if constexpr (GATED) row_load<T>(pre + C * io<T>::BYTES, c, C, u);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float f, df;
        if constexpr (GATED || ACT != ACT_NONE) act_both<ACT, FINE>(z[j], f, df);
        if constexpr (GATED) {
          z[j] = d[j] * f;
          d[j] = d[j] * u[j] * df;
          s[1][j] += z[j];
        } else if constexpr (ACT != ACT_NONE) {
          d[j] *= df;
        }
        s[0][j] += d[j];
      }
      if (a.dp) {
        char* dp = (char*)a.dp + r * a.ldp * io<T>::BYTES;
        row_stream<T>(dp, c, C, d);
        if constexpr (GATED) row_stream<T>(dp + C * io<T>::BYTES, c, C, z);
        if (c + V >= C)
          for (int64_t k = ld; k < a.ldp; ++k) io<T>::store1(dp, k, 0.0f);
      }
    }
  if (!a.dbias) return;
  if (rg > 0)
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int j = 0; j < V; ++j) sh[rg - 1][cv][w * V + j] = s[w][j];
  __syncthreads();
  if (rg > 0 || c >= C) return;
  float* part = gridDim.y == 1 ? a.dbias : a.part + (int64_t)blockIdx.y * ld;
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      for (int g = 0; g < 7; ++g) s[w][j] += sh[g][cv][w * V + j];
      if (c + j < C) part[w * C + c + j] = s[w][j];
    }
}

template <typename T>
hipError_t act_bwd_run(const ActBwdArgs& a, hipStream_t s) {
  const int64_t parts = act_bwd_parts(a.rows, a.cols), per = 32 * io<T>::VEC;
  const int64_t slab = (a.rows + parts - 1) / parts;
  const dim3 grid((unsigned)((a.cols + per - 1) / per), (unsigned)parts), blk(256);
  with_act(a.act, [&](auto act) {
    if (a.gated) hipLaunchKernelGGL((act_bwd_kernel<T, act.value, true>), grid, blk, 0, s, a, slab);
    else hipLaunchKernelGGL((act_bwd_kernel<T, act.value, false>), grid, blk, 0, s, a, slab);
  });
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void zero_kernel(u16* dst, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) dst[i] = 0;
}

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a) {
  constexpr int V = io<T>::VEC;
  const auto& m = a.m[blockIdx.y];
  const int64_t vecs = m.ld / V, n = m.rows * vecs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / vecs, c = (i - r * vecs) * V;
    float f[V];
    row_load<T>((const char*)m.src + r * m.src_ld * io<T>::BYTES, c, m.width, f);
    stg16<T>(m.dst, r * m.ld + c, io<T>::pack(f));
  }
}

}  // namespace

hipError_t launch_pack(int io_bf16, const PackArgs& a, hipStream_t s) {
  if (a.count == 0) return hipSuccess;
  int64_t most = 1;
  for (int i = 0; i < a.count; ++i) {
    const int64_t blocks = (a.m[i].rows * (a.m[i].ld / (io_bf16 ? 8 : 4)) + 255) / 256;
    if (blocks > most) most = blocks;
  }
  const dim3 grid((unsigned)(most < 4096 ? most : 4096), (unsigned)a.count);
  if (io_bf16) hipLaunchKernelGGL((pack_kernel<bf16_t>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((pack_kernel<float>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_zero(void* dst, int64_t bytes, hipStream_t s) {
  const int64_t blocks = (bytes / 2 + 255) / 256;
  hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, (u16*)dst,
                     bytes / 2);
  return hipGetLastError();
}

// Slabs of rows: eight rows each until there are 64, or as many as make 1024
// blocks where the columns are few (32768 rows bf16, with the sums of the
// slabs: of 128 columns 40 us with 64 slabs, 15 so; of 1024 columns 62 and 24);
// up to 64 rows one slab, which needs no second kernel for its sums.
int64_t act_bwd_parts(int64_t rows, int64_t cols) {
  const int64_t p = (rows + 7) / 8, across = (cols + 255) / 256;
  const int64_t most = across >= 16 ? 64 : 1024 / across;
  return rows <= 64 ? 1 : p < most ? p : most;
}

hipError_t launch_act_bwd(int io_bf16, const ActBwdArgs& a, hipStream_t s) {
  const hipError_t e = io_bf16 ? act_bwd_run<bf16_t>(a, s) : act_bwd_run<float>(a, s);
  const int64_t parts = act_bwd_parts(a.rows, a.cols), n = a.gated ? 2 * a.cols : a.cols;
  if (e != hipSuccess || !a.dbias || parts == 1) return e;
  return launch_reduce_parts(a.part, parts, n, n, a.dbias, n, nullptr, s);
}

}  // namespace m3
