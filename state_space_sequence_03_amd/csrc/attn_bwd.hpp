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
#if defined(__HIP_DEVICE_COMPILE__)
  if (wave > 1) return;
  const int n = rows < BQ ? rows : BQ, lane = threadIdx.x & 63;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)((wave ? a.delta : a.lse2) + at), 0, (uint32_t)(n * 4), 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + wave * 64), 4, lane < BQ ? lane * 4 : kFar, 0, 0, 0);
#endif
}

// dk and dv of 128 keys: each wave holds 32 of them as the columns of its
// products (scores = Q k^T, dp = dO v^T; dv^T += dO^T p, dk^T += Q^T ds) and
// walks the queries that see them, of every head that shares them, in tiles of
// BQ rows that all four waves read.
//
// The sinks are seen from the whole sequence.  Where that is longer than
// a.piece queries, each 32 keys with sinks among them are left to blocks of
// their own (the last `pieces`), each with a.piece queries, of which each wave
// takes every fourth 32; the four sums go to the workspace in fp32 and are
// joined in order.
//
// Where the keys' tiles alone would leave the chip half empty, a.splits blocks
// share one, and a piece: each takes its part of the list of (head, queries) and
// its sums go to the workspace as well.
//
// Two waves share a SIMD, for which a width of 128 is four registers short in bf16
// (20 bytes of a lane in scratch memory).  With fragments three products ahead 510 to
// 600 us for 8 x 4096 queries, 16/4 heads of 128, window 1024, as the clock is; next
// to 620; six ahead with spills 740; one wave per SIMD 780.  There the matrix cores
// work in 47 % of the cycles and the vector units in 32 %.
template <typename T, int DP, int DU, int BQ>
__global__ __launch_bounds__(256, io<T>::BYTES == 2 || DP == 64 ? 2 : 1) void attn_dkv_kernel(
    AttnArgs a, int64_t items, int64_t pieces) {
  using QD = Tile<T, DP, DU, BQ, 4>;
  constexpr int ES = io<T>::BYTES, STEPS = 32 / QD::CK, AHEAD = 3;
  constexpr int STAGE = 2 * QD::BYTES + 512;  // Q, dO, statistics
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  const int sunk = (a.sinks + 31) / 32;
  const uint32_t tiles = gridDim.x - (uint32_t)pieces;
  const bool cut = blockIdx.x >= tiles;
  const uint32_t bx = cut ? blockIdx.x - tiles : blockIdx.x;
  AttnSeq s;
  int jw, piece = 0, split = 0;  // jw: the wave's first key
  int64_t hk;
  uint32_t item = 0;
  if (cut) {
    const uint32_t at = bx / (uint32_t)a.splits, id = at / (uint32_t)a.kv_heads;
    split = (int)(bx % (uint32_t)a.splits);
    hk = at % (uint32_t)a.kv_heads;
    jw = (int)(id % (uint32_t)sunk) * 32;
    if (!attn_item<false>(a, id / (uint32_t)sunk, a.piece, a.piece, s, piece)) return;
    if (jw >= s.nk) return;
  } else {
    const uint32_t id = xcd_order(bx, tiles);
    int t;
    item = id / (uint32_t)a.splits;
    split = (int)(id % (uint32_t)a.splits);
    hk = item / (uint32_t)items;
    if (!attn_item<true>(a, item % (uint32_t)items, 128, 0, s, t)) return;
    jw = t * 128 + wave * 32;
  }
  const bool apart = s.nq > a.piece;  // the sinks are summed in pieces
  const bool idle = !cut && apart && jw < sunk * 32;
  const int past = s.past();
  const int j0 = cut ? jw : jw - wave * 32, j = jw + (lane & 31);
  const bool in = j < s.nk;
  // queries that see some of the block's keys
  int r0 = j0 - past < 0 ? 0 : j0 - past, r1 = s.nq - 1;
  if (cut) {
    if (r0 < piece * a.piece) r0 = piece * a.piece;
    if (r1 > piece * a.piece + a.piece - 1) r1 = piece * a.piece + a.piece - 1;
  } else if (a.window < kNoWindow && (apart || j0 >= a.sinks)) {
    const int64_t last = (int64_t)j0 + 127 + a.window - 1 - past;
    if (last < r1) r1 = (int)last;
  }
  r0 = r0 / BQ * BQ;  // whole tiles, so that a piece's last one ends with it
  const int per = r1 < r0 ? 0 : (r1 - r0) / BQ + 1, all = per * G;
  const int begin = (int)((int64_t)all * split / a.splits);
  const int count = (int)((int64_t)all * (split + 1) / a.splits) - begin;

  const int64_t row = s.k0 + (in ? j : s.nk - 1);
  RowRegs<T, DU> k, v;
  k.load((const char*)a.k + (row * a.k_stride + hk * a.dim) * ES, in, a.dim, h);
  v.load((const char*)a.v + (row * a.v_stride + hk * a.dim) * ES, in, a.dim, h);
  QD qt, dt;
  qt.init(a.q_stride, a.dim, lane, wave);
  dt.init(a.do_stride, a.dim, lane, wave);
  auto load = [&](int head, int r, int buf) {
    const int64_t hq = hk * G + head;
    char* lds = smem + buf * STAGE;
    qt.load((const char*)a.q + ((s.q0 + r) * a.q_stride + hq * a.dim) * ES, s.nq - r, a.dim, lds, wave);
    dt.load((const char*)a.dout + ((s.q0 + r) * a.do_stride + hq * a.dim) * ES, s.nq - r, a.dim, lds + QD::BYTES, wave);
    load_stats<BQ>(a, hq * a.rows + s.q0 + r, s.nq - r, (float*)(lds + 2 * QD::BYTES), wave);
  };
  f32x16 dk[QD::CT], dv[QD::CT];
#pragma unroll
  for (int i = 0; i < QD::CT; ++i) dk[i] = dv[i] = f32x16{};
  const float c = a.scale * kLog2e;
  int head = per > 0 ? begin / per : 0, r = r0 + (begin - head * per) * BQ;
  if (count > 0) load(head, r, 0);
  for (int n = 0; n < count; ++n) {
    attn_settle();
    int next = r + BQ, other = head;
    if (next > r1) {
      next = r0;
      ++other;
    }
    if (n + 1 < count) load(other, next, (n + 1) & 1);
    const char* ql = smem + (n & 1) * STAGE;
    const char* dl = ql + QD::BYTES;
    const float* stat = (const float*)(dl + QD::BYTES);
#pragma unroll 1
    for (int b = 0; b < BQ / 32; ++b) {
      const int p0 = past + r + 32 * b;
      if (idle || sees_none(p0, p0 + 31, jw, jw + 31, a.window, a.sinks)) continue;
      if (cut && ((n * (BQ / 32) + b) & 3) != wave) continue;
      f32x16 x[2] = {f32x16{}, f32x16{}};  // scores, dp
      ahead<AHEAD, QD::KS * 2, 1, T>(
          [&](int i) { return i & 1 ? dt.row(dl, b, i / 2) : qt.row(ql, b, i / 2); },
          [&](int i, const uint4& f) { x[i & 1] = mma32<T>(f, i & 1 ? v.v[i / 2] : k.v[i / 2], x[i & 1]); });
      float p[16], ds[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 l2 = __builtin_bit_cast(f32x4, read16((const u32x4*)(stat + 32 * b + 8 * i + 4 * h)));
        const f32x4 de = __builtin_bit_cast(f32x4, read16((const u32x4*)(stat + 64 + 32 * b + 8 * i + 4 * h)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[4 * i + e] = __builtin_amdgcn_exp2f(fmaf(x[0][4 * i + e], c, -l2[e]));
          ds[4 * i + e] = p[4 * i + e] * (x[1][4 * i + e] - de[e]);
        }
      }
      if (!sees_all(p0, p0 + 31, jw, jw + 31, a.window, a.sinks)) {
        asm volatile("");  // a branch, not selects in every step
        const QueriesSeeing seen(a, p0 + 4 * h, j);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool in = seen(i / 4 * 8 + i % 4);
          p[i] = in ? p[i] : 0.0f;
          ds[i] = in ? ds[i] : 0.0f;
        }
      }
      uint4 w[2][STEPS];
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        w[0][st] = result_step<T>(p, st);
        w[1][st] = result_step<T>(ds, st);
      }
      ahead<AHEAD, 2 * STEPS * QD::CT, 2, T>(
          [&](int i) {
            const int d = i % QD::CT, st = i / QD::CT % STEPS;
            return i < STEPS * QD::CT ? dt.col(dl, d, b * STEPS + st) : qt.col(ql, d, b * STEPS + st);
          },
          [&](int i, const uint4& f) {
            const int d = i % QD::CT, st = i / QD::CT % STEPS;
            if (i < STEPS * QD::CT) dv[d] = mma32<T>(f, w[0][st], dv[d]);
            else dk[d] = mma32<T>(f, w[1][st], dk[d]);
          });
    }
    head = other;
    r = next;
  }
  if (cut || a.splits > 1) {
    // per split of a piece, and behind those of an item: (dk, dv; wave; 32 keys; dim)
    const int64_t at = cut ? bx : pieces + (int64_t)item * a.splits + split;
    float* part = a.part + (at * 8 + wave) * 32 * a.dim + (int64_t)(lane & 31) * a.dim;
#pragma unroll
    for (int d = 0; d < QD::CT; ++d) {
      if (d * 32 >= a.dim) break;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dk[d][i] * a.scale;
      tile_store<float, false>((char*)part, true, d * 32, a.dim, x, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = dv[d][i];
      tile_store<float, false>((char*)(part + 4 * 32 * a.dim), true, d * 32, a.dim, x, h);
    }
  } else if (!idle) {
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

// The sums of 32 keys' pieces joined in order: the blocks of the pieces (eight
// each, z) share the keys' entries, 128 at a time; eight groups of threads each
// add an eighth of the sums, four entries to a thread.  joined: blocks of all
// pieces, whose sums there are; starts that do not rise make up sequences with more
// pieces than that.
constexpr int kJoinZ = 8;
template <typename T>
__device__ __forceinline__ void join_pieces(const AttnArgs& a, uint32_t joined, int z) {
  __shared__ f32x4 sums[8][32];
  const int sunk = (a.sinks + 31) / 32;
  const uint32_t id = blockIdx.x / (uint32_t)a.kv_heads;  // of a piece, all its splits
  const int64_t hk = blockIdx.x % (uint32_t)a.kv_heads;
  const int j0 = (int)(id % (uint32_t)sunk) * 32;
  AttnSeq s;
  int piece;
  if (!attn_item<false>(a, id / (uint32_t)sunk, a.piece, a.piece, s, piece)) return;
  const int keys = s.nk - j0 < 32 ? s.nk - j0 : 32;
  if (keys <= 0) return;
  const int there = (int)(joined / (uint32_t)a.kv_heads / (uint32_t)sunk - id / (uint32_t)sunk) + piece;
  const int whole = (s.nq + a.piece - 1) / a.piece, pieces = whole < there ? whole : there;
  const bool key = blockIdx.y == 0;
  void* out = key ? a.dk : a.dv;
  if (!out) return;
  const int64_t half = 32 * a.dim, one = 8 * half;                   // of four waves, of a split
  const int64_t step = (int64_t)sunk * a.kv_heads * a.splits * one;  // from piece to piece
  const float* part = a.part + (int64_t)blockIdx.x * a.splits * one - piece * step + (key ? 0 : 4 * half);
  const int n = keys * a.dim, parts = a.splits * 4, g = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int c = (piece * kJoinZ + z) * 128; c < n; c += pieces * kJoinZ * 128) {
    const int e = c + lane * 4;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (e < n) {
#pragma unroll 4
      for (int w = g; w < pieces * parts; w += 8) {
        const int i = w / parts, u = w - i * parts;
        const f32x4 y = *(const f32x4*)(part + i * step + (u >> 2) * one + (u & 3) * half + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += y[j];
      }
    }
    __syncthreads();
    sums[g][lane] = x;
    __syncthreads();
    if (g == 0 && e < n) {
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] += sums[i][lane][j];
      const int j = e / a.dim;
      io<T>::store4(out, (s.k0 + j0 + j) * (key ? a.dk_stride : a.dv_stride) + hk * a.dim + e - j * a.dim, f);
    }
  }
}

// The splits of 128 keys joined in order (those of the sinks that are summed in
// pieces excepted): a block per item, dk and dv by blockIdx.y, a quarter of the
// keys by z.
constexpr int kJoinSplitsZ = 4;
template <typename T>
__device__ __forceinline__ void join_splits(const AttnArgs& a, int64_t items, int64_t pieces, int z) {
  const int64_t hk = blockIdx.x / (uint32_t)items;
  AttnSeq s;
  int t;
  if (!attn_item<true>(a, blockIdx.x % (uint32_t)items, 128, 0, s, t)) return;
  const int j0 = t * 128 + z * 32;
  if (s.nq > a.piece && j0 < (a.sinks + 31) / 32 * 32) return;
  const bool key = blockIdx.y == 0;
  void* out = key ? a.dk : a.dv;
  if (!out) return;
  const int keys = s.nk - j0 < 32 ? s.nk - j0 : 32, n = keys * a.dim;
  const int64_t wave = 32 * a.dim;
  const float* part = a.part + ((pieces + (int64_t)blockIdx.x * a.splits) * 8 + (key ? 0 : 4) + z) * wave;
  for (int e = (int)threadIdx.x * 4; e < n; e += 1024) {
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < a.splits; ++i) {
      const f32x4 y = *(const f32x4*)(part + i * 8 * wave + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += y[j];
    }
    const int j = e / a.dim;
    io<T>::store4(out, (s.k0 + j0 + j) * (key ? a.dk_stride : a.dv_stride) + hk * a.dim + e - j * a.dim, x);
  }
}

// Both in one launch (z from z0 on), or the one that there is: `joined` blocks
// of pieces, `split` of items.  (1 x 1500 queries, 8/2 heads of 128, window 200: dk
// and dv 42 us with two launches, 36 so.)
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int64_t items, int64_t pieces, int64_t joined,
                                                        int64_t split, int z0) {
  const int z = blockIdx.z + z0;
  if (z < kJoinZ) {
    if (blockIdx.x < joined) join_pieces<T>(a, (uint32_t)joined, z);
  } else if (blockIdx.x < split) {
    join_splits<T>(a, items, pieces, z - kJoinZ);
  }
}

// dq of 32 NW queries, 32 NW / HT positions of HT heads, by KW parties as in the
// forward: each wave holds 32 of them as the columns of its products
// (scores = K q^T, dp = V do^T, dq^T += K^T ds) and walks the tiles of keys that
// the block's queries see, but for halves that its own do not.  It comes first and
// leaves the queries' statistics to the other kernel.  8 x 4096 queries, 16/4 heads
// of 128, window 1024: 400 to 460 us, 0.8 to 0.9 PFLOP/s of three products.
template <typename T, int DP, int DU, int BN, int HT, int NW, int KW>
__global__ __launch_bounds__(64 * NW * KW, NW == 1 || (io<T>::BYTES == 4 && DP == 128) ? 1 : 2) void attn_dq_kernel(
    AttnArgs a, int64_t items) {
  using KV = Tile<T, DP, DU, BN, NW>;
  constexpr int ES = io<T>::BYTES, NT = BN / 32, STEPS = 32 / KV::CK, BM = 32 * NW / HT, HALF = 32 * KV::ROWB;
  // wide parties of one wave take the values into registers: LDS has room for four
  constexpr bool ALONE = NW == 1 && DP == 128;
  static_assert(!ALONE || NT == 1, "a run at a time");
  constexpr int PART = (ALONE ? 2 : 4) * KV::BYTES;  // K K or K V K V of each
  __shared__ __attribute__((aligned(1024))) char lds[KW * PART];
  const int lane = threadIdx.x & 63;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = all % NW, part = all / NW;
  char* smem = lds + part * PART;
  const int h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  const uint32_t id = xcd_order(blockIdx.x, gridDim.x), kg = id / (uint32_t)(G / HT);
  const int64_t hk = kg / (uint32_t)items;
  AttnSeq s;
  int t;
  if (!attn_item<false>(a, kg % (uint32_t)items, BM, 0, s, t)) return;
  t = (s.nq + BM - 1) / BM - 1 - t;
  const int64_t hq = hk * G + id % (uint32_t)(G / HT) * HT + wave % HT;

  const int r = t * BM + wave / HT * 32 + (lane & 31);
  const bool in = r < s.nq;
  const int p = s.past() + r;
  const int p0 = s.past() + t * BM, p1 = s.past() + (s.nq < t * BM + BM ? s.nq : t * BM + BM) - 1;
  const int w0 = p0 + wave / HT * 32, w1 = w0 + 31 < p1 ? w0 + 31 : p1;
  const int64_t row = s.q0 + (in ? r : s.nq - 1);
  RowRegs<T, DU> q, y;
  q.load((const char*)a.q + (row * a.q_stride + hq * a.dim) * ES, in, a.dim, h);
  y.load((const char*)a.dout + (row * a.do_stride + hq * a.dim) * ES, in, a.dim, h);
  float delta = 0.0f;
  {
    RowRegs<T, DU> o;
    o.load((const char*)a.o + (row * a.o_stride + hq * a.dim) * ES, in, a.dim, h);
#pragma unroll
    for (int st = 0; st < RowRegs<T, DU>::KS; ++st) {
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
  if (in && h == 0 && part == 0) {
    a.lse2[hq * a.rows + row] = l2;
    a.delta[hq * a.rows + row] = delta;
  }

  KV kt, vt;
  kt.init(a.k_stride, a.dim, lane, wave);
  RowStream<T, DU> vs;
  if constexpr (ALONE) vs.init(a.v_stride, a.dim, lane);
  else vt.init(a.v_stride, a.dim, lane, wave);
  const char* kb = (const char*)a.k + (s.k0 * a.k_stride + hk * a.dim) * ES;
  const char* vb = (const char*)a.v + (s.k0 * a.v_stride + hk * a.dim) * ES;
  int first = p0 - a.window + 1;
  first = first < 0 ? 0 : first / BN;
  const int sunk = (a.sinks + BN - 1) / BN, ns = sunk < first ? sunk : first;
  const int count = p1 < 0 ? 0 : ns + p1 / BN - first + 1;
  auto first_key = [&](int n) { return (n < ns ? n : first + n - ns) * BN; };
  auto load = [&](int n, int buf) {
    const int64_t j0 = first_key(n);
    const int rows = s.nk - (int)j0;
    char* to = smem + buf * (PART / 2);
    kt.load(kb + j0 * a.k_stride * ES, rows, a.dim, to, wave);
    if constexpr (ALONE) vs.load(vb + j0 * a.v_stride * ES, rows < 32 ? rows : 32, a.dim);
    else vt.load(vb + j0 * a.v_stride * ES, rows, a.dim, to + KV::BYTES, wave);
  };
  f32x16 acc[KV::CT];
#pragma unroll
  for (int i = 0; i < KV::CT; ++i) acc[i] = f32x16{};
  const float c = a.scale * kLog2e;
  if (part < count) load(part, 0);
  for (int i = 0; i * KW < count; ++i) {
    const int n = i * KW + part;
    if constexpr (ALONE) attn_settle_alone();
    else attn_settle();
    if (KW > 1 && n >= count) continue;
    uint4 v[ALONE ? KV::KS : 1];
    if constexpr (ALONE)
#pragma unroll
      for (int st = 0; st < KV::KS; ++st) v[st] = vs.v[st];
    if (n + KW < count) load(n + KW, (i + 1) & 1);
#pragma unroll 1
    for (int b = 0; b < NT; ++b) {
      const int j0 = first_key(n) + 32 * b;
      if (sees_none(w0, w1, j0, j0 + 31, a.window, a.sinks)) continue;
      const char* kl = smem + (i & 1) * (PART / 2) + b * HALF;
      const char* vl = kl + KV::BYTES;
      f32x16 x[2] = {f32x16{}, f32x16{}};  // scores, dp
      ahead<6, KV::KS * 2, 1, T>(
          [&](int i) {
            if constexpr (ALONE) return i & 1 ? v[i / 2] : kt.row(kl, 0, i / 2);
            else return i & 1 ? vt.row(vl, 0, i / 2) : kt.row(kl, 0, i / 2);
          },
          [&](int i, const uint4& f) { x[i & 1] = mma32<T>(f, i & 1 ? y.v[i / 2] : q.v[i / 2], x[i & 1]); });
      float ds[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] = __builtin_amdgcn_exp2f(fmaf(x[0][i], c, -l2)) * (x[1][i] - delta);
      if (!sees_all(w0, w1, j0, j0 + 31, a.window, a.sinks)) {
        asm volatile("");  // a branch, not selects in every step
        const KeysSeen seen(a, p, j0 + 4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = seen(i / 4 * 8 + i % 4) ? ds[i] : 0.0f;
      }
      uint4 w[STEPS];
#pragma unroll
      for (int st = 0; st < STEPS; ++st) w[st] = result_step<T>(ds, st);
      ahead<6, STEPS * KV::CT, 2, T>(
          [&](int i) { return kt.col(kl, i % KV::CT, i / KV::CT); },
          [&](int i, const uint4& f) { acc[i % KV::CT] = mma32<T>(f, w[i / KV::CT], acc[i % KV::CT]); });
    }
  }
  if constexpr (KW > 1) {
    float none = 0.0f;
    if (!join_parts<KW, NW, PART, false>(lds, acc, none, none, c, part, wave, lane)) return;
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

template <typename T, int DP, int DU, int HT, int NW, int KW>
void attn_dq_run(const AttnArgs& a, hipStream_t s) {
  const int64_t items = attn_items(a, false, 32 * NW / HT);
  if (items > 0)
    hipLaunchKernelGGL((attn_dq_kernel<T, DP, DU, io<T>::BYTES == 2 ? 64 : 32, HT, NW, KW>),
                       dim3((unsigned)(items * (a.q_heads / HT))), dim3(64 * NW * KW), 0, s, a, items);
}

template <typename T, int DP, int DU>
void attn_bwd_run(const AttnArgs& a, hipStream_t s) {
  const int64_t vectors = a.rows * a.q_heads;
  const dim3 block(256);
  if (a.dq)
    attn_by_size<T>(a, [&](auto ht, auto nw, auto kw) {
      attn_dq_run<T, DP, DU, decltype(ht)::value, decltype(nw)::value, decltype(kw)::value>(a, s);
    });
  else if (vectors > 0)
    hipLaunchKernelGGL((attn_delta_kernel<T>), dim3((unsigned)((vectors + 15) / 16)), block, 0, s, a);
  const int64_t tiles = attn_items(a, true, 128), pieces = attn_piece_blocks(a) * a.splits, blocks = tiles * a.kv_heads;
  if ((!a.dk && !a.dv) || tiles == 0) return;
  hipLaunchKernelGGL((attn_dkv_kernel<T, DP, DU, io<T>::BYTES == 2 ? 64 : 32>),
                     dim3((unsigned)(pieces + blocks * a.splits)), block, 0, s, a, tiles, pieces);
  const int64_t joined = pieces / a.splits, split = a.splits > 1 ? blocks : 0;
  if (joined == 0 && split == 0) return;
  const int z0 = joined > 0 ? 0 : kJoinZ, z1 = split > 0 ? kJoinZ + kJoinSplitsZ : kJoinZ;
  hipLaunchKernelGGL((attn_join_kernel<T>), dim3((unsigned)(joined > split ? joined : split), 2, z1 - z0), block, 0, s, a,
                     tiles, pieces, joined, split, z0);
}

template <typename T>
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  with_width(a.dim, [&](auto dp, auto du) { attn_bwd_run<T, decltype(dp)::value, decltype(du)::value>(a, s); });
  return hipGetLastError();
}

}  // namespace m3
