// Layer norm over the model width, forward and backward.
//   forward:  mean = sum x / D, rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
//             y = (x - mean) rstd gain + bias
//   backward: xh = (x - mean) rstd, a = dy gain,
//             dx = rstd (a - mean_D(a) - xh mean_D(a xh)) + dskip,
//             dgain = sum_rows dy xh, dbias = sum_rows dy.
// Both are bound by HBM: every row is read once into registers, the row sums
// are taken there (the variance about the mean, not as a difference of
// moments), and the result is written once.  A row belongs to one wave (TPR =
// 64) or one block (TPR = 256, 1024); NV is the number of 16-byte vectors a
// thread holds of each operand.  32768 x 2048 bf16: forward with statistics
// 45 us from a warm cache, 59 (4.6 TB/s) cold; backward with dskip 108 us (5.0
// TB/s) and 5 for the column sums, a block per row: a wave per row spilled (227).
// Rows too wide for that are re-read from the caches (the *_wide kernels).  The
// backward walks many rows per block and keeps the column sums of its rows in
// registers; one partial row per block and a second kernel that adds the partial
// rows in order give dgain and dbias (no atomics: the result does not depend on
// timing).
#include "m3_lanes.hpp"
#include "m3_launch.hpp"
#include "m3_rows.hpp"

namespace m3 {

namespace {

// Sum over the TPR threads of a row, received by all of them.  sh: one float
// per wave, its own for every call between two barriers of the block.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = lane_sum<1, 64>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += sh[w];
  }
  return v;
}

template <typename T, int NV, int TPR>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a) {
  constexpr int V = io<T>::VEC;
  __shared__ float sh[2][4];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;  // whole waves (TPR = 64) or whole blocks leave
  const int64_t D = a.width;
  const char* x = (const char*)a.x + row * a.x_stride * io<T>::BYTES;
  float f[NV][V];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) row_load<T>(x, (int64_t)(i * TPR + t) * V, D, f[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s += f[i][j];
  const float n = (float)D;
  const float mean = row_sum<TPR>(s, sh[0]) / n;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f[i][j] -= mean;
      q += (int64_t)(i * TPR + t) * V + j < D ? f[i][j] * f[i][j] : 0.0f;
    }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, sh[1]) / n + a.eps);
  if (t == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  char* y = (char*)a.y + row * a.y_stride * io<T>::BYTES;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(i * TPR + t) * V;
    if (c >= D) break;
    float g[V], b[V];
    col_load<V>(a.gain, c, D, 1.0f, g);
    col_load<V>(a.bias, c, D, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = f[i][j] * rstd * g[j] + b[j];
    row_store<T>(y, c, D, g);
  }
}

// One block per row, the row re-read for each of the three passes.
template <typename T>
__global__ __launch_bounds__(256) void norm_fwd_wide_kernel(NormArgs a) {
  constexpr int V = io<T>::VEC;
  __shared__ float sh[2][4];
  const int64_t row = blockIdx.x, D = a.width;
  const char* x = (const char*)a.x + row * a.x_stride * io<T>::BYTES;
  char* y = (char*)a.y + row * a.y_stride * io<T>::BYTES;
  float f[V], s = 0.0f, q = 0.0f;
  for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
    row_load<T>(x, c, D, f);
#pragma unroll
    for (int j = 0; j < V; ++j) s += f[j];
  }
  const float n = (float)D;
  const float mean = row_sum<256>(s, sh[0]) / n;
  for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
    row_load<T>(x, c, D, f);
#pragma unroll
    for (int j = 0; j < V; ++j) q += c + j < D ? (f[j] - mean) * (f[j] - mean) : 0.0f;
  }
  const float rstd = 1.0f / sqrtf(row_sum<256>(q, sh[1]) / n + a.eps);
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
    float g[V], b[V];
    row_load<T>(x, c, D, f);
    col_load<V>(a.gain, c, D, 1.0f, g);
    col_load<V>(a.bias, c, D, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = (f[j] - mean) * rstd * g[j] + b[j];
    row_store<T>(y, c, D, g);
  }
}

// Rows blockIdx, blockIdx + gridDim, ... (in groups of 256 / TPR), and the
// column sums of the block's rows.
template <typename T, int NV, int TPR, bool SKIP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int V = io<T>::VEC;
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float sh[2][2][TPR / 64];
  __shared__ float comb[RPB > 1 ? (RPB - 1) * 64 * V : 1];
  const int t = threadIdx.x % TPR, rr = threadIdx.x / TPR;
  const int64_t D = a.width;
  const float n = (float)D;
  float g[NV][V], sg[NV][V], sb[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col_load<V>(a.gain, (int64_t)(i * TPR + t) * V, D, 1.0f, g[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) sg[i][j] = sb[i][j] = 0.0f;
  }
  // the next row is requested while this one is worked on
  u32x4 nx[NV], nd[NV], ns[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto request = [&](int64_t row) {
    const char* x = (const char*)a.x + row * a.x_stride * io<T>::BYTES;
    const char* dy = (const char*)a.dy + row * a.y_stride * io<T>::BYTES;
    const char* sk = (const char*)a.dskip + row * a.skip_stride * io<T>::BYTES;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(i * TPR + t) * V;
      nx[i] = row_raw<T>(x, c, D);
      nd[i] = row_raw<T>(dy, c, D);
      if (SKIP) ns[i] = row_raw<T>(sk, c, D);
    }
    nmean = a.mean[row];
    nrstd = a.rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + rr;
  if (row < a.rows) request(row);
  for (int par = 0; row < a.rows; row += step, par ^= 1) {  // uniform per wave, and per block where a row is a block's
    const float mean = nmean, rstd = nrstd;
    float f[NV][V], d[NV][V];
    u32x4 sk[NV];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack_raw<T>(nx[i], f[i]);
      unpack_raw<T>(nd[i], d[i]);
      if (SKIP) sk[i] = ns[i];
    }
    if (row + step < a.rows) request(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[i][j] = (f[i][j] - mean) * rstd;  // past the row's end dy is 0: no share in any sum
        sg[i][j] += d[i][j] * f[i][j];
        sb[i][j] += d[i][j];
        d[i][j] *= g[i][j];
        c1 += d[i][j];
        c2 += d[i][j] * f[i][j];
      }
    if (!a.dx) continue;
    c1 = row_sum<TPR>(c1, sh[par][0]) / n;
    c2 = row_sum<TPR>(c2, sh[par][1]) / n;
    char* dx = (char*)a.dx + row * a.skip_stride * io<T>::BYTES;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(i * TPR + t) * V;
      if (c >= D) break;
      float o[V];
      if (SKIP) unpack_raw<T>(sk[i], o);
      else
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] += rstd * (d[i][j] - c1 - f[i][j] * c2);
      row_store<T>(dx, c, D, o);
    }
  }
  if (!a.dgain && !a.dbias) return;
  float* out[2] = {a.dgain, a.dbias};  // a lone block's sums are the result
  if (gridDim.x > 1) {
    out[0] = a.part + (int64_t)blockIdx.x * 2 * D;
    out[1] = out[0] + D;
  }
  // the block's waves, in order
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float* s = which ? sb[i] : sg[i];
      if constexpr (RPB > 1) {
        __syncthreads();
        if (rr > 0)
#pragma unroll
          for (int j = 0; j < V; ++j) comb[((rr - 1) * V + j) * 64 + t] = s[j];
        __syncthreads();
        if (rr == 0)
#pragma unroll
          for (int j = 0; j < V; ++j)
#pragma unroll
            for (int w = 0; w < RPB - 1; ++w) s[j] += comb[(w * V + j) * 64 + t];
      }
      const int64_t c = (int64_t)(i * TPR + t) * V;
      if (rr == 0 && out[which])
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c + j < D) out[which][c + j] = s[j];
    }
}

// dx of wide rows: one block per row, two passes.
template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_wide_kernel(NormBwdArgs a) {
  constexpr int V = io<T>::VEC;
  __shared__ float sh[2][4];
  const int64_t row = blockIdx.x, D = a.width;
  const char* x = (const char*)a.x + row * a.x_stride * io<T>::BYTES;
  const char* dy = (const char*)a.dy + row * a.y_stride * io<T>::BYTES;
  const float mean = a.mean[row], rstd = a.rstd[row], n = (float)D;
  float f[V], d[V], g[V], c1 = 0.0f, c2 = 0.0f;
  for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
    row_load<T>(x, c, D, f);
    row_load<T>(dy, c, D, d);
    col_load<V>(a.gain, c, D, 1.0f, g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c1 += d[j] * g[j];
      c2 += d[j] * g[j] * ((f[j] - mean) * rstd);
    }
  }
  c1 = row_sum<256>(c1, sh[0]) / n;
  c2 = row_sum<256>(c2, sh[1]) / n;
  char* dx = (char*)a.dx + row * a.skip_stride * io<T>::BYTES;
  const char* sk = a.dskip ? (const char*)a.dskip + row * a.skip_stride * io<T>::BYTES : nullptr;
  for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
    float o[V];
    row_load<T>(x, c, D, f);
    row_load<T>(dy, c, D, d);
    col_load<V>(a.gain, c, D, 1.0f, g);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.0f;
    if (sk) row_load<T>(sk, c, D, o);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] += rstd * (d[j] * g[j] - c1 - (f[j] - mean) * rstd * c2);
    row_store<T>(dx, c, D, o);
  }
}

// Column sums of wide rows: block (x, y) takes 256 vectors of columns and the
// rows y, y + gridDim.y, ...
template <typename T>
__global__ __launch_bounds__(256) void norm_cols_wide_kernel(NormBwdArgs a) {
  constexpr int V = io<T>::VEC;
  const int64_t D = a.width, c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= D) return;
  float f[V], d[V], sg[V], sb[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sg[j] = sb[j] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    row_load<T>((const char*)a.x + row * a.x_stride * io<T>::BYTES, c, D, f);
    row_load<T>((const char*)a.dy + row * a.y_stride * io<T>::BYTES, c, D, d);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sg[j] += d[j] * ((f[j] - mean) * rstd);
      sb[j] += d[j];
    }
  }
  float* og = gridDim.y > 1 ? a.part + (int64_t)blockIdx.y * 2 * D : a.dgain;
  float* ob = gridDim.y > 1 ? og + D : a.dbias;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (c + j < D) {
      if (og) og[c + j] = sg[j];
      if (ob) ob[c + j] = sb[j];
    }
}

// out[c] = sum over p of part[p * stride + c], c < n0 to out0 and the rest to
// out1 (each nullable).  64 columns per block, the partial rows split over
// its 16 waves, which are then added in order.
__global__ __launch_bounds__(1024) void reduce_parts_kernel(const float* part, int64_t np, int64_t stride, int64_t n,
                                                            float* out0, int64_t n0, float* out1) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < n)
#pragma unroll 8
    for (int64_t p = w; p < np; p += 16) s += part[p * stride + c];
  sh[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += sh[k][lane];
    float* o = c < n0 ? out0 : out1;
    if (o) o[c < n0 ? c : c - n0] = s;
  }
}

// vectors a thread must hold of a row of `width` elements split over tpr
template <typename T>
int64_t vectors(int64_t width, int tpr) {
  const int64_t per = (int64_t)tpr * io<T>::VEC;
  return (width + per - 1) / per;
}

template <typename T>
hipError_t norm_fwd_run(const NormArgs& a, hipStream_t s) {
  const int64_t n64 = vectors<T>(a.width, 64), n256 = vectors<T>(a.width, 256);
  const dim3 rows((unsigned)a.rows), rows4((unsigned)((a.rows + 3) / 4)), blk(256);
  if (n64 == 1) hipLaunchKernelGGL((norm_fwd_kernel<T, 1, 64>), rows4, blk, 0, s, a);
  else if (n64 == 2) hipLaunchKernelGGL((norm_fwd_kernel<T, 2, 64>), rows4, blk, 0, s, a);
  else if (n64 <= 4) hipLaunchKernelGGL((norm_fwd_kernel<T, 4, 64>), rows4, blk, 0, s, a);
  else if (n256 <= 2) hipLaunchKernelGGL((norm_fwd_kernel<T, 2, 256>), rows, blk, 0, s, a);
  else if (n256 <= 4) hipLaunchKernelGGL((norm_fwd_kernel<T, 4, 256>), rows, blk, 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_wide_kernel<T>), rows, blk, 0, s, a);
  return hipGetLastError();
}

template <typename T, bool SKIP>
hipError_t norm_bwd_run(const NormBwdArgs& a, hipStream_t s) {
  const int64_t n64 = vectors<T>(a.width, 64), n256 = vectors<T>(a.width, 256);
  const dim3 parts((unsigned)norm_bwd_parts(io<T>::BYTES == 2, a.rows, a.width)), blk(256);
  if (n64 == 1) hipLaunchKernelGGL((norm_bwd_kernel<T, 1, 64, SKIP>), parts, blk, 0, s, a);
  else if (n64 == 2) hipLaunchKernelGGL((norm_bwd_kernel<T, 2, 64, SKIP>), parts, blk, 0, s, a);
  else if (n256 == 1) hipLaunchKernelGGL((norm_bwd_kernel<T, 1, 256, SKIP>), parts, blk, 0, s, a);
  else if (n256 == 2) hipLaunchKernelGGL((norm_bwd_kernel<T, 2, 256, SKIP>), parts, blk, 0, s, a);
  else if (n256 <= 4) hipLaunchKernelGGL((norm_bwd_kernel<T, 1, 1024, SKIP>), parts, dim3(1024), 0, s, a);
  else {
    if (a.dx) hipLaunchKernelGGL((norm_bwd_wide_kernel<T>), dim3((unsigned)a.rows), blk, 0, s, a);
    if (a.dgain || a.dbias)
      hipLaunchKernelGGL((norm_cols_wide_kernel<T>), dim3((unsigned)n256, parts.x), blk, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

// Blocks of the backward: up to four per CU, each with one pass over four rows
// (a wave each) at least, or with two rows of a block each; up to 8 rows one
// block, which needs no second kernel for its sums.  Where rows are re-read, a
// slab of rows is a row of blocks already, and as many slabs are taken as make
// 1024 blocks: their partial rows are 16 MB at most, whatever the width (2048 x
// 65536 bf16: 355 us, against 724 with 1024 slabs).
int64_t norm_bwd_parts(int io_bf16, int64_t rows, int64_t width) {
  const bool wave = (io_bf16 ? vectors<bf16_t>(width, 64) : vectors<float>(width, 64)) <= 2;
  const int64_t n256 = io_bf16 ? vectors<bf16_t>(width, 256) : vectors<float>(width, 256);
  const int64_t groups = wave ? (rows + 3) / 4 : (rows + 1) / 2;
  const int64_t most = n256 <= 4 ? 1024 : n256 < 1024 ? 1024 / n256 : 1;
  return rows <= 8 ? 1 : groups < most ? groups : most;
}

hipError_t launch_reduce_parts(const float* part, int64_t np, int64_t stride, int64_t n, float* out0, int64_t n0,
                               float* out1, hipStream_t s) {
  hipLaunchKernelGGL(reduce_parts_kernel, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, s, part, np, stride, n, out0,
                     n0, out1);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(int io_bf16, const NormArgs& a, hipStream_t s) {
  return io_bf16 ? norm_fwd_run<bf16_t>(a, s) : norm_fwd_run<float>(a, s);
}

hipError_t launch_norm_bwd(int io_bf16, const NormBwdArgs& a, hipStream_t s) {
  const hipError_t e = io_bf16 ? (a.dskip ? norm_bwd_run<bf16_t, true>(a, s) : norm_bwd_run<bf16_t, false>(a, s))
                               : (a.dskip ? norm_bwd_run<float, true>(a, s) : norm_bwd_run<float, false>(a, s));
  const int64_t parts = norm_bwd_parts(io_bf16, a.rows, a.width);
  if (e != hipSuccess || parts == 1 || (!a.dgain && !a.dbias)) return e;
  return launch_reduce_parts(a.part, parts, 2 * a.width, 2 * a.width, a.dgain, a.width, a.dbias, s);
}

}  // namespace m3
