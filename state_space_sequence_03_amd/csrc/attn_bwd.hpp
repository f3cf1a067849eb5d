// Windowed attention with sinks, backward.  With p = exp(scale q k - lse) for
// what is seen, dp = do v^T, delta = rowsum(do o):
//   ds = p (dp - delta),  dq = scale ds k,  dk = scale ds^T q,  dv = p^T do.
// One kernel sums over the queries (dk, dv), one over the keys (dq): each
// output has one writer and a fixed order of summation.
#pragma once

#include "attn.hpp"

namespace m3 {

// lse in powers of two and delta, (heads, rows) each, where no kernel of dq
// takes them on its way.  16 lanes per vector.
template <typename T>
__global__ __launch_bounds__(256) void attn_delta_kernel(AttnArgs a) {
  constexpr int V = io<T>::VEC;
  const int lane = threadIdx.x & 15;
  const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t row = id / a.q_heads, hq = id - row * a.q_heads;
  if (row >= a.rows) return;
  const char* o = (const char*)a.o + (row * a.o_stride + hq * a.dim) * io<T>::BYTES;
  const char* d = (const char*)a.dout + (row * a.do_stride + hq * a.dim) * io<T>::BYTES;
  float s = 0.0f;
  for (int c = lane * V; c < a.dim; c += 16 * V) {
    float x[V], y[V];
    row_load<T>(o, c, a.dim, x);
    row_load<T>(d, c, a.dim, y);
#pragma unroll
    for (int j = 0; j < V; ++j) s += x[j] * y[j];
  }
  s = lane_sum<1, 16>(s);
  if (lane == 0) {
    const float l = a.lse[row * a.q_heads + hq];
    a.lse2[hq * a.rows + row] = l == -INFINITY ? INFINITY : l * kLog2e;
    a.delta[hq * a.rows + row] = s;
  }
}

// The lse2 and delta of BQ queries in LDS, a load of 4 bytes per lane each.
template <int BQ>
__device__ __forceinline__ void load_stats(const AttnArgs& a, int64_t at, int rows, float* lds, int wave) {
  if (wave > 1) return;
  const float* src = (wave ? a.delta : a.lse2) + at;
  const int n = rows < BQ ? rows : BQ;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, 0, (uint32_t)(n * 4), 0x00020000);
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + wave * 64), 4, lane < BQ ? lane * 4 : kFar, 0, 0, 0);
}

// dk and dv of 128 keys: each wave holds 32 of them as the columns of its
// products (scores = Q k^T, dp = dO v^T; dv^T += dO^T p, dk^T += Q^T ds) and
// walks the queries that see them, of every head that shares them, in tiles of
// BQ rows that all four waves read.
//
// The sinks are seen from the whole sequence.  Where that is longer than
// a.piece queries, a sinks' tile is left to blocks of its own (the first
// `pieces`), each with a.piece queries, whose sums go to the workspace in fp32
// and are joined in order.
template <typename T, int DP, int BQ>
__global__ __launch_bounds__(256, 2) void attn_dkv_kernel(AttnArgs a, int64_t items, int64_t pieces) {
  using QD = Tile<T, DP, BQ, 4>;
  constexpr int ES = io<T>::BYTES, STEPS = 32 / QD::CK;
  constexpr int STAGE = 2 * QD::BYTES + 512;  // Q, dO, statistics
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  const int sunk = (a.sinks + 127) / 128;
  const bool cut = blockIdx.x < pieces;
  int64_t id = blockIdx.x;
  AttnSeq s;
  int t, piece = 0;
  int64_t hk;
  if (cut) {
    hk = id % a.kv_heads;
    id /= a.kv_heads;
    t = (int)(id % sunk);
    if (!attn_item<false>(a, id / sunk, a.piece, a.piece, s, piece)) return;
    if (t * 128 >= s.nk) return;
  } else {
    id = xcd_order(id - pieces, gridDim.x - pieces);
    hk = id / items;
    if (!attn_item<true>(a, id % items, 128, 0, s, t)) return;
    if (t < sunk && s.nq > a.piece) return;
  }
  const int past = s.past();
  const int j0 = t * 128, jw = j0 + wave * 32, j = jw + (lane & 31);
  const bool in = j < s.nk;
  // queries that see some of the block's keys
  int r0 = j0 - past < 0 ? 0 : j0 - past, r1 = s.nq - 1;
  if (a.window < kNoWindow && j0 >= a.sinks) {
    const int64_t last = (int64_t)j0 + 127 + a.window - 1 - past;
    if (last < r1) r1 = (int)last;
  }
  if (cut) {
    if (r0 < piece * a.piece) r0 = piece * a.piece;
    if (r1 > piece * a.piece + a.piece - 1) r1 = piece * a.piece + a.piece - 1;
  }
  r0 = r0 / BQ * BQ;  // whole tiles, so that a piece's last one ends with it
  const int per = r1 < r0 ? 0 : (r1 - r0) / BQ + 1, count = per * G;

  const int64_t row = s.k0 + (in ? j : s.nk - 1);
  RowRegs<T, DP> k, v;
  k.load((const char*)a.k + (row * a.k_stride + hk * a.dim) * ES, in, a.dim, h);
  v.load((const char*)a.v + (row * a.v_stride + hk * a.dim) * ES, in, a.dim, h);
  QD qt, dt;
  qt.init(a.q_stride, a.dim, lane, wave);
  dt.init(a.do_stride, a.dim, lane, wave);
  auto load = [&](int n, int buf) {
    const int64_t hq = hk * G + n / per;
    const int r = r0 + n % per * BQ;
    char* lds = smem + buf * STAGE;
    qt.load((const char*)a.q + ((s.q0 + r) * a.q_stride + hq * a.dim) * ES, s.nq - r, a.dim, lds, wave);
    dt.load((const char*)a.dout + ((s.q0 + r) * a.do_stride + hq * a.dim) * ES, s.nq - r, a.dim, lds + QD::BYTES, wave);
    load_stats<BQ>(a, hq * a.rows + s.q0 + r, s.nq - r, (float*)(lds + 2 * QD::BYTES), wave);
  };
  f32x16 dk[QD::CT], dv[QD::CT];
#pragma unroll
  for (int i = 0; i < QD::CT; ++i) dk[i] = dv[i] = f32x16{};
  const float c = a.scale * kLog2e;
  if (count > 0) load(0, 0);
  for (int n = 0; n < count; ++n) {
    attn_settle();
    if (n + 1 < count) load(n + 1, (n + 1) & 1);
    const char* ql = smem + (n & 1) * STAGE;
    const char* dl = ql + QD::BYTES;
    const float* stat = (const float*)(dl + QD::BYTES);
    const int r = r0 + n % per * BQ;
#pragma unroll 1
    for (int b = 0; b < BQ / 32; ++b) {
      const int p0 = past + r + 32 * b;
      if (sees_none(p0, p0 + 31, jw, jw + 31, a.window, a.sinks)) continue;
      // one product after the other: their operands together would not fit
      // the registers that two waves on a SIMD have each
      const bool all = sees_all(p0, p0 + 31, jw, jw + 31, a.window, a.sinks);
      float p[16], ds[16];
      {
        f32x16 z = f32x16{};
#pragma unroll
        for (int st = 0; st < QD::KS; ++st) z = mma32<T>(qt.row(ql, b, st), k.v[st], z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 l2 = __builtin_bit_cast(f32x4, read16((const u32x4*)(stat + 32 * b + 8 * i + 4 * h)));
#pragma unroll
          for (int e = 0; e < 4; ++e) p[4 * i + e] = __builtin_amdgcn_exp2f(fmaf(z[4 * i + e], c, -l2[e]));
        }
      }
      if (!all) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!sees(p0 + i / 4 * 8 + 4 * h + i % 4, j, a.window, a.sinks)) p[i] = 0.0f;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const uint4 w = result_step<T>(p, st);
#pragma unroll
        for (int d = 0; d < QD::CT; ++d) dv[d] = mma32<T>(dt.col(dl, d, b * STEPS + st), w, dv[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
      {
        f32x16 y = f32x16{};
#pragma unroll
        for (int st = 0; st < QD::KS; ++st) y = mma32<T>(dt.row(dl, b, st), v.v[st], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 de = __builtin_bit_cast(f32x4, read16((const u32x4*)(stat + 64 + 32 * b + 8 * i + 4 * h)));
#pragma unroll
          for (int e = 0; e < 4; ++e) ds[4 * i + e] = p[4 * i + e] * (y[4 * i + e] - de[e]);
        }
      }
      if (!all) {  // what is not seen may have met an infinity
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!sees(p0 + i / 4 * 8 + 4 * h + i % 4, j, a.window, a.sinks)) ds[i] = 0.0f;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const uint4 x = result_step<T>(ds, st);
#pragma unroll
        for (int d = 0; d < QD::CT; ++d) dk[d] = mma32<T>(qt.col(ql, d, b * STEPS + st), x, dk[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (cut) {
    // (2, 128 keys, dim) per piece
    float* part = a.part + (int64_t)blockIdx.x * 2 * 128 * a.dim + (int64_t)(wave * 32 + (lane & 31)) * a.dim;
#pragma unroll
    for (int d = 0; d < QD::CT; ++d) {
      if (d * 32 >= a.dim) break;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dk[d][i] * a.scale;
      tile_store<float, false>((char*)part, true, d * 32, a.dim, x, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dv[d][i];
      tile_store<float, false>((char*)(part + 128 * a.dim), true, d * 32, a.dim, x, h);
    }
  } else {
#pragma unroll
    for (int d = 0; d < QD::CT; ++d) {
      if (d * 32 >= a.dim) break;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dk[d][i] * a.scale;
      if (a.dk) tile_store<T, false>((char*)a.dk + (row * a.dk_stride + hk * a.dim) * ES, in, d * 32, a.dim, x, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dv[d][i];
      if (a.dv) tile_store<T, false>((char*)a.dv + (row * a.dv_stride + hk * a.dim) * ES, in, d * 32, a.dim, x, h);
    }
  }
}

// The pieces of a sinks' tile joined in order, four entries to a thread; the
// blocks of a tile's pieces share its entries.
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int sunk = (a.sinks + 127) / 128;
  const int64_t hk = blockIdx.x % a.kv_heads, id = blockIdx.x / a.kv_heads;
  const int t = (int)(id % sunk);
  AttnSeq s;
  int piece;
  if (!attn_item<false>(a, id / sunk, a.piece, a.piece, s, piece)) return;
  const int keys = s.nk - t * 128 < 128 ? s.nk - t * 128 : 128;
  if (keys <= 0) return;
  const int pieces = (s.nq + a.piece - 1) / a.piece;
  const int64_t step = (int64_t)sunk * a.kv_heads * 2 * 128 * a.dim;  // from piece to piece
  const float* part = a.part + (int64_t)blockIdx.x * 2 * 128 * a.dim - piece * step;
  const int n = keys * a.dim;
  const bool key = blockIdx.y == 0;
  void* out = key ? a.dk : a.dv;
  if (!out) return;
  if (!key) part += 128 * a.dim;
  for (int e = (piece * 256 + (int)threadIdx.x) * 4; e < n; e += pieces * 1024) {
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const f32x4 y = *(const f32x4*)(part + i * step + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += y[j];
    }
    const int j = e / a.dim;
    io<T>::store4(out, (s.k0 + t * 128 + j) * (key ? a.dk_stride : a.dv_stride) + hk * a.dim + e - j * a.dim, x);
  }
}

// dq of 128 queries: each wave holds 32 of them as the columns of its products
// (scores = K q^T, dp = V do^T, dq^T += K^T ds) and walks the keys they see as
// the forward does.  It comes first and leaves the queries' statistics to the
// other kernel.
template <typename T, int DP, int BN>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnArgs a, int64_t items) {
  using KV = Tile<T, DP, BN, 4>;
  constexpr int ES = io<T>::BYTES, NT = BN / 32, STEPS = 32 / KV::CK;
  __shared__ __attribute__((aligned(1024))) char smem[4 * KV::BYTES];  // K V K V
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  const int64_t i = xcd_order(blockIdx.x, gridDim.x);
  const int g = (int)(i % G);
  const int64_t hk = i / G / items;
  AttnSeq s;
  int t;
  if (!attn_item<false>(a, i / G % items, 128, 0, s, t)) return;
  t = (s.nq + 127) / 128 - 1 - t;
  const int64_t hq = hk * G + g;

  const int r = t * 128 + wave * 32 + (lane & 31);
  const bool in = r < s.nq;
  const int p = s.past() + r;
  const int p0 = s.past() + t * 128, p1 = s.past() + (s.nq - 1 < t * 128 + 127 ? s.nq - 1 : t * 128 + 127);
  const int w0 = p0 + wave * 32, w1 = w0 + 31 < p1 ? w0 + 31 : p1;
  const int64_t row = s.q0 + (in ? r : s.nq - 1);
  RowRegs<T, DP> q, y;
  q.load((const char*)a.q + (row * a.q_stride + hq * a.dim) * ES, in, a.dim, h);
  y.load((const char*)a.dout + (row * a.do_stride + hq * a.dim) * ES, in, a.dim, h);
  float delta = 0.0f;
  {
    RowRegs<T, DP> o;
    o.load((const char*)a.o + (row * a.o_stride + hq * a.dim) * ES, in, a.dim, h);
#pragma unroll
    for (int st = 0; st < RowRegs<T, DP>::KS; ++st) {
      constexpr int V = io<T>::VEC;
      float x[V], z[V];
      io<T>::unpack(__builtin_bit_cast(typename io<T>::vec, o.v[st]), x);
      io<T>::unpack(__builtin_bit_cast(typename io<T>::vec, y.v[st]), z);
#pragma unroll
      for (int e = 0; e < V; ++e) delta += x[e] * z[e];
    }
    delta = swap_sum32(delta);
  }
  const float lse = a.lse[row * a.q_heads + hq], l2 = lse == -INFINITY ? INFINITY : lse * kLog2e;
  if (in && h == 0) {
    a.lse2[hq * a.rows + row] = l2;
    a.delta[hq * a.rows + row] = delta;
  }

  KV kt, vt;
  kt.init(a.k_stride, a.dim, lane, wave);
  vt.init(a.v_stride, a.dim, lane, wave);
  const char* kb = (const char*)a.k + (s.k0 * a.k_stride + hk * a.dim) * ES;
  const char* vb = (const char*)a.v + (s.k0 * a.v_stride + hk * a.dim) * ES;
  int first = p0 - a.window + 1;
  first = first < 0 ? 0 : first / BN;
  const int sunk = (a.sinks + BN - 1) / BN, ns = sunk < first ? sunk : first;
  const int count = p1 < 0 ? 0 : ns + p1 / BN - first + 1;
  auto load = [&](int n, int buf) {
    const int64_t j0 = (int64_t)(n < ns ? n : first + n - ns) * BN;
    kt.load(kb + j0 * a.k_stride * ES, s.nk - (int)j0, a.dim, smem + buf * 2 * KV::BYTES, wave);
    vt.load(vb + j0 * a.v_stride * ES, s.nk - (int)j0, a.dim, smem + (buf * 2 + 1) * KV::BYTES, wave);
  };
  f32x16 acc[KV::CT];
#pragma unroll
  for (int i = 0; i < KV::CT; ++i) acc[i] = f32x16{};
  const float c = a.scale * kLog2e;
  if (count > 0) load(0, 0);
  for (int n = 0; n < count; ++n) {
    attn_settle();
    if (n + 1 < count) load(n + 1, (n + 1) & 1);
    const char* kl = smem + (n & 1) * 2 * KV::BYTES;
    const char* vl = kl + KV::BYTES;
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      const int j0 = (n < ns ? n : first + n - ns) * BN + 32 * b;
      if (sees_none(w0, w1, j0, j0 + 31, a.window, a.sinks)) continue;
      f32x16 z = f32x16{}, dp = f32x16{};
#pragma unroll
      for (int st = 0; st < KV::KS; ++st) z = mma32<T>(kt.row(kl, b, st), q.v[st], z);
#pragma unroll
      for (int st = 0; st < KV::KS; ++st) dp = mma32<T>(vt.row(vl, b, st), y.v[st], dp);
      float ds[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] = __builtin_amdgcn_exp2f(fmaf(z[i], c, -l2)) * (dp[i] - delta);
      if (!sees_all(w0, w1, j0, j0 + 31, a.window, a.sinks)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!sees(p, j0 + i / 4 * 8 + 4 * h + i % 4, a.window, a.sinks)) ds[i] = 0.0f;
      }
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const uint4 w = result_step<T>(ds, st);
#pragma unroll
        for (int d = 0; d < KV::CT; ++d) acc[d] = mma32<T>(kt.col(kl, d, b * STEPS + st), w, acc[d]);
      }
    }
  }
  char* out = (char*)a.dq + (row * a.dq_stride + hq * a.dim) * ES;
#pragma unroll
  for (int d = 0; d < KV::CT; ++d) {
    if (d * 32 >= a.dim) break;
    float x[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) x[v] = acc[d][v] * a.scale;
    tile_store<T, false>(out, in, d * 32, a.dim, x, h);
  }
}

template <typename T, int DP>
hipError_t attn_bwd_run(const AttnArgs& a, hipStream_t s) {
  constexpr int BN = io<T>::BYTES == 2 ? 64 : 32, BQ = BN;
  const dim3 block(256);
  const int64_t vectors = a.rows * a.q_heads, items = attn_items(a, false, 128), tiles = attn_items(a, true, 128);
  if (a.dq && items > 0)
    hipLaunchKernelGGL((attn_dq_kernel<T, DP, BN>), dim3((unsigned)(items * a.q_heads)), block, 0, s, a, items);
  else if (vectors > 0)
    hipLaunchKernelGGL((attn_delta_kernel<T>), dim3((unsigned)((vectors + 15) / 16)), block, 0, s, a);
  if ((a.dk || a.dv) && tiles > 0) {
    const int64_t pieces = attn_pieces(a) * ((a.sinks + 127) / 128) * a.kv_heads;
    hipLaunchKernelGGL((attn_dkv_kernel<T, DP, BQ>), dim3((unsigned)(pieces + tiles * a.kv_heads)), block, 0, s, a,
                       tiles, pieces);
    if (pieces > 0) hipLaunchKernelGGL((attn_join_kernel<T>), dim3((unsigned)pieces, 2), block, 0, s, a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  return a.dim <= 64 ? attn_bwd_run<T, 64>(a, s) : attn_bwd_run<T, 128>(a, s);
}

}  // namespace m3
