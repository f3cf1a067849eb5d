// Norms of queries and keys for each head, with the position rotation in the
// same pass.
//   forward:  r = 1 / sqrt(sum x^2 / D + eps), z = x r gain, and the pairs of
//             z's first R entries turned by pos theta[pair];
//   backward: dz = dy turned back, a = dz gain, xh = x r,
//             dx = r (a - xh mean_D(a xh)), dgain = sum over vectors of dz xh.
// Both are bound by HBM: a vector (one head of one token) belongs to LPV lanes
// that hold it in registers, is read once and its result written once, queries
// and keys in one launch.  32768 tokens, 16 + 4 heads of 128, bf16: 63 us, 5.3 TB/s
// (71 with a division for each vector's place and root: the vector units were the
// bound); backward of 8 x 4096 tokens, 32 + 8 heads of 64: 112 us, 4.5 TB/s of what
// it needs (a lane's sums for the gains lie in scratch memory, whose traffic comes on
// top: 644 MB instead of 504; without it 102), and 5 for their reduction; fp32 200 us, 5.0 TB/s; 256
// tokens: 4.5 us, a launch.  The cosines and sines are taken once per token and
// pair, shared by the token's heads through LDS; the angle is a product in 64
// bits reduced to a fraction of a turn there, so that far positions lose
// nothing.
#include "m3_lanes.hpp"
#include "m3_launch.hpp"
#include "m3_rows.hpp"

namespace m3 {

namespace {

constexpr int kTable = 2048;  // (token, pair) entries a block holds

// Cosine and sine of each pair's angle for tokens [t0, t0 + n).
__device__ __forceinline__ void fill_table(const NormRopeArgs& a, int64_t t0, int n, float2* tab) {
  const int pairs = a.rope / 2;
  for (int i = threadIdx.x; i < n * pairs; i += 256) {
    const int t = i / pairs;
    const int64_t row = t0 + t;
    const int64_t pos = a.pos ? a.pos[row] : a.seqlen ? (int64_t)((uint32_t)row % (uint32_t)a.seqlen) : row;
    const double turn = (double)pos * (double)a.theta[i - t * pairs] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
    tab[i] = make_float2(c, s);
  }
}

// The lane's entries [c, c + V) of a vector turned by its token's angles (DIR
// = 1) or back (-1).  xs: LDS of the vector's own, for pairs half apart.
template <int V, bool HALVES, int DIR>
__device__ __forceinline__ void turn(const NormRopeArgs& a, const float2* tab, float* xs, int c, float* f) {
  const int R = a.rope;
  if constexpr (HALVES) {
    const int h = R / 2;
    // the lanes of a vector are of one wave: its LDS accesses go in order
#pragma unroll
    for (int j = 0; j < V; j += 4) *(f32x4*)(xs + c + j) = f32x4{f[j], f[j + 1], f[j + 2], f[j + 3]};
    asm volatile("" ::: "memory");
    if (h % V == 0) {  // the lane's partners are one lane's
      if (c < R) {
        const bool low = c < h;
        const int p = low ? c + h : c - h;
        const float sign = (low ? -1.0f : 1.0f) * DIR;
        const float2* t = tab + (low ? c : p);
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const f32x4 o = *(const f32x4*)(xs + p + j);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cs = t[j + e];
            f[j + e] = f[j + e] * cs.x + sign * o[e] * cs.y;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < R) {
          const bool low = c + j < h;
          const int p = low ? c + j + h : c + j - h;
          const float2 cs = tab[low ? c + j : p];
          f[j] = f[j] * cs.x + (low ? -1.0f : 1.0f) * DIR * xs[p] * cs.y;
        }
    }
    asm volatile("" ::: "memory");
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2)
      if (c + j < R) {
        const float2 cs = tab[(c + j) / 2];
        const float x = f[j], y = f[j + 1];
        f[j] = x * cs.x - DIR * y * cs.y;
        f[j + 1] = y * cs.x + DIR * x * cs.y;
      }
  }
}

// One of the vectors of a block's tokens, which are counted token by token, the
// token's heads in order (queries', then keys'); a step goes VPB vectors on.
template <int VPB>
struct Place {
  int token, head;
  __device__ __forceinline__ Place(const NormRopeArgs& a, int u) {
    const int H = a.q_heads + a.k_heads;
    token = u / H;
    head = u - token * H;
  }
  __device__ __forceinline__ void step(const NormRopeArgs& a) {
    const int H = a.q_heads + a.k_heads, over = VPB / H;  // of all threads alike
    token += over;
    head += VPB - over * H;
    if (head >= H) {
      head -= H;
      ++token;
    }
  }
  __device__ __forceinline__ bool key(const NormRopeArgs& a) const { return head >= a.q_heads; }
  // its place in a matrix of the two operands' row strides, from token t0's row
  // on: 64 tokens at most, of rows of 2^20 entries at most
  template <typename T>
  __device__ __forceinline__ char* at(const NormRopeArgs& a, const void* q, const void* k, int64_t sq, int64_t sk,
                                      int64_t t0) const {
    const bool kv = key(a);
    char* base = kv ? (char*)k + t0 * sk * io<T>::BYTES : (char*)q + t0 * sq * io<T>::BYTES;
    const int e = __mul24(token, kv ? (int)sk : (int)sq) + __mul24(kv ? head - a.q_heads : head, a.dim);
    return base + (uint32_t)e * (uint32_t)io<T>::BYTES;
  }
};

// 1 / sqrt(mean x^2 + eps) of a vector held by LPV lanes (entries past its
// width are 0).  For bf16 by v_rsq_f32, which is good to one unit in the last
// place (of numbers below the normal ones it takes no root), and with the width's
// reciprocal: 2^-15 of a result's rounding, and 40 instructions less a vector.
template <typename T, int V, int LPV>
__device__ __forceinline__ float rms(const float* f, int dim, float per, float eps) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) s += f[j] * f[j];
  s = lane_sum<1, LPV>(s);
  if constexpr (io<T>::BYTES == 2) {
    const float m = s * per + eps;
    if (m >= 0x1p-126f) return __builtin_amdgcn_rsqf(m);
  }
  return 1.0f / sqrtf(s / (float)dim + eps);
}

template <typename T, int LPV, bool HALVES>
__global__ __launch_bounds__(256) void norm_rope_fwd_kernel(NormRopeArgs a) {
  constexpr int V = io<T>::VEC, VPB = 256 / LPV;
  __shared__ float2 tab[kTable];
  __shared__ __attribute__((aligned(16))) float xs[HALVES ? 256 * V : 4];
  const int lane = threadIdx.x % LPV, slot = threadIdx.x / LPV, c = lane * V;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int n = a.rows - t0 < a.tokens ? (int)(a.rows - t0) : a.tokens;
  const int vectors = n * (a.q_heads + a.k_heads);
  const float per = 1.0f / (float)a.dim;
  u32x4 raw = {0u, 0u, 0u, 0u};
  Place<VPB> next(a, slot);
  auto load = [&] { raw = row_raw<T>(next.template at<T>(a, a.q, a.k, a.q_stride, a.k_stride, t0), c, a.dim); };
  if (slot < vectors) load();
  float g[2][V];
  col_load<V>(a.gain_q, c, a.dim, 1.0f, g[0]);
  col_load<V>(a.gain_k, c, a.dim, 1.0f, g[1]);
  fill_table(a, t0, n, tab);
  __syncthreads();
  for (int u = slot; u < vectors; u += VPB) {
    const Place<VPB> at = next;
    const bool key = at.key(a);
    float f[V];
    unpack_raw<T>(raw, f);
    next.step(a);
    if (u + VPB < vectors) load();
    const float r = rms<T, V, LPV>(f, a.dim, per, a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] *= r * (key ? g[1][j] : g[0][j]);
    turn<V, HALVES, 1>(a, tab + at.token * (a.rope / 2), xs + (HALVES ? slot * LPV * V : 0), c, f);
    row_store<T>(at.template at<T>(a, a.q_out, a.k_out, a.q_out_stride, a.k_out_stride, t0), c, a.dim, f);
  }
}

// Token groups blockIdx, blockIdx + gridDim, ..., and the sums over them that
// the gains' gradients take from a block.
template <typename T, int LPV, bool HALVES>
__global__ __launch_bounds__(256) void norm_rope_bwd_kernel(NormRopeArgs a) {
  constexpr int V = io<T>::VEC, VPB = 256 / LPV;
  __shared__ float2 tab[kTable];
  __shared__ __attribute__((aligned(16))) float xs[256 * V];
  const int lane = threadIdx.x % LPV, slot = threadIdx.x / LPV, c = lane * V;
  const float per = 1.0f / (float)a.dim;
  float g[2][V], sum[2][V];
  col_load<V>(a.gain_q, c, a.dim, 1.0f, g[0]);
  col_load<V>(a.gain_k, c, a.dim, 1.0f, g[1]);
#pragma unroll
  for (int j = 0; j < V; ++j) sum[0][j] = sum[1][j] = 0.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tokens; t0 < a.rows; t0 += (int64_t)gridDim.x * a.tokens) {
    const int n = a.rows - t0 < a.tokens ? (int)(a.rows - t0) : a.tokens;
    const int vectors = n * (a.q_heads + a.k_heads);
    u32x4 rx = {0u, 0u, 0u, 0u}, ry = rx;
    Place<VPB> next(a, slot);
    auto load = [&] {
      rx = row_raw<T>(next.template at<T>(a, a.q, a.k, a.q_stride, a.k_stride, t0), c, a.dim);
      ry = row_raw<T>(next.template at<T>(a, a.dq_out, a.dk_out, a.q_out_stride, a.k_out_stride, t0), c, a.dim);
    };
    if (slot < vectors) load();
    fill_table(a, t0, n, tab);
    __syncthreads();
    for (int u = slot; u < vectors; u += VPB) {
      const Place<VPB> at = next;
      const bool key = at.key(a);
      float x[V], d[V];
      unpack_raw<T>(rx, x);
      unpack_raw<T>(ry, d);
      next.step(a);
      if (u + VPB < vectors) load();
      const float r = rms<T, V, LPV>(x, a.dim, per, a.eps);
      turn<V, HALVES, -1>(a, tab + at.token * (a.rope / 2), xs + slot * LPV * V, c, d);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] *= r;
        const float w = d[j] * x[j];
        if (key) sum[1][j] += w;
        else sum[0][j] += w;
        d[j] *= key ? g[1][j] : g[0][j];
        s += d[j] * x[j];
      }
      s = io<T>::BYTES == 2 ? lane_sum<1, LPV>(s) * per : lane_sum<1, LPV>(s) / (float)a.dim;
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = r * (d[j] - x[j] * s);
      row_store<T>(at.template at<T>(a, a.q_out, a.k_out, a.dq_stride, a.dk_stride, t0), c, a.dim, d);
    }
    __syncthreads();  // the table is read
  }
  if (!a.part) return;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) xs[slot * LPV * V + c + j] = sum[o][j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.dim; e += 256) {
      float s = 0.0f;
      for (int i = 0; i < VPB; ++i) s += xs[i * LPV * V + e];
      a.part[((int64_t)blockIdx.x * 2 + o) * a.dim + e] = s;
    }
  }
}

template <typename T, int LPV, bool HALVES>
void launch(bool bwd, const NormRopeArgs& a, unsigned blocks, hipStream_t s) {
  if (bwd) hipLaunchKernelGGL((norm_rope_bwd_kernel<T, LPV, HALVES>), dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((norm_rope_fwd_kernel<T, LPV, HALVES>), dim3(blocks), dim3(256), 0, s, a);
}
template <typename T, bool HALVES>
void launch_lanes(bool bwd, const NormRopeArgs& a, unsigned blocks, hipStream_t s) {
  const int lanes = (a.dim + io<T>::VEC - 1) / io<T>::VEC;
  if (lanes <= 4) launch<T, 4, HALVES>(bwd, a, blocks, s);
  else if (lanes <= 8) launch<T, 8, HALVES>(bwd, a, blocks, s);
  else if (lanes <= 16) launch<T, 16, HALVES>(bwd, a, blocks, s);
  else if (lanes <= 32) launch<T, 32, HALVES>(bwd, a, blocks, s);
  else launch<T, 64, HALVES>(bwd, a, blocks, s);
}

// Tokens per block: enough vectors for a few passes of the block, while the
// grid still covers the chip twice over.  (Passes of 1024 lanes in all: forward of
// 32768 tokens of 20 heads of 128 63 us, backward of 40 heads of 64 111; of 640: 68
// and 121, of 2048: 68 and 114.)
int tokens_per_block(int io_bf16, int64_t rows, int64_t heads, int64_t dim, int64_t rope) {
  const int64_t per = heads * ((dim + (io_bf16 ? 7 : 3)) / (io_bf16 ? 8 : 4));  // lanes of a token
  int64_t t = (1024 + per - 1) / per;
  if (t > rows / 512) t = rows / 512;
  if (rope > 0 && t > kTable / (rope / 2)) t = kTable / (rope / 2);
  return t < 1 ? 1 : t > 64 ? 64 : (int)t;
}

}  // namespace

int64_t norm_rope_parts(int io_bf16, int64_t rows, int64_t heads, int64_t dim, int64_t rope) {
  const int64_t t = tokens_per_block(io_bf16, rows, heads, dim, rope), groups = (rows + t - 1) / t;
  return groups < 1024 ? groups : 1024;  // the backward above: with 512 136 us, 768 114, 2048 116
}

hipError_t launch_norm_rope(int io_bf16, bool bwd, NormRopeArgs a, hipStream_t s) {
  const int64_t heads = a.q_heads + a.k_heads;
  a.tokens = tokens_per_block(io_bf16, a.rows, heads, a.dim, a.rope);
  const int64_t groups = (a.rows + a.tokens - 1) / a.tokens;
  const unsigned blocks = (unsigned)(bwd ? norm_rope_parts(io_bf16, a.rows, heads, a.dim, a.rope) : groups);
  if (io_bf16) {
    if (a.halves) launch_lanes<bf16_t, true>(bwd, a, blocks, s);
    else launch_lanes<bf16_t, false>(bwd, a, blocks, s);
  } else {
    if (a.halves) launch_lanes<float, true>(bwd, a, blocks, s);
    else launch_lanes<float, false>(bwd, a, blocks, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !bwd || !a.part) return e;
  return launch_reduce_parts(a.part, blocks, 2 * (int64_t)a.dim, 2 * (int64_t)a.dim, a.dgain_q, a.dim, a.dgain_k, s);
}

}  // namespace m3
