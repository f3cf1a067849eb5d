// Windowed attention with sinks of new tokens over a cache that wraps.
#pragma once

#include "attn.hpp"

namespace m3 {

constexpr int kMaxSplits = 256;

// The slots of a sequence's cache that its new tokens see, as two runs, and
// the position that each holds.  Positions are taken relative to the first new
// token's, n: those that matter lie within the cache's length of it.
struct CacheView {
  int end0, from1, end1;  // slots [0, end0) and [from1, end1)
  int slot_n;             // of the first new token; the others' follow, and go on behind the sinks at the cache's end
  int n;                  // tokens before the call, or 2^30 for more
  int ring, sinks, rem, newer;
  __device__ __forceinline__ void init(int64_t len, int tokens, int capacity, int sinks_, int window) {
    sinks = sinks_;
    ring = capacity - sinks;
    n = len < (1 << 30) ? (int)len : 1 << 30;
    const int64_t last = len + tokens - 1;
    slot_n = (int)(len < sinks ? len : sinks + (len - sinks) % ring);
    from1 = end1 = 0;
    rem = -1;
    newer = 0;
    if (last < sinks) {
      end0 = (int)(last + 1);
      return;
    }
    const int64_t turns = (last - sinks) / ring;
    rem = (int)(last - sinks - turns * ring);
    newer = (int)(sinks + turns * ring - len);
    int64_t lo = len - window + 1;
    if (lo < last - ring + 1) lo = last - ring + 1;
    if (lo < sinks) lo = sinks;
    const int count = (int)(last - lo + 1), at = (int)((lo - sinks) % ring);
    if (at + count <= ring) {
      end0 = sinks;
      from1 = sinks + at;
      end1 = from1 + count;
    } else {
      end0 = sinks + at + count - ring;
      from1 = sinks + at;
      end1 = capacity;
    }
    if (from1 == end0) {
      end0 = end1;
      from1 = end1 = 0;
    }
  }
  __device__ __forceinline__ int tiles0() const { return (end0 + 31) >> 5; }
  __device__ __forceinline__ int tiles() const { return tiles0() + ((end1 - from1 + 31) >> 5); }
  // slots [x, e) of tile i, 32 at most
  __device__ __forceinline__ void tile(int i, int& x, int& e) const {
    const int n0 = tiles0();
    x = i < n0 ? i * 32 : from1 + (i - n0) * 32;
    e = i < n0 ? end0 : end1;
    if (e > x + 32) e = x + 32;
  }
  // whether every new token sees the 32 slots from x on (e: the tile's end)
  __device__ __forceinline__ bool all_seen(int x, int e, int tokens, int window) const {
    if (e - x < 32) return false;
    if (e <= sinks) return e - 1 <= n;
    const int r = x - sinks, rel = r <= rem ? newer + r : newer + r - ring;
    return r >= 0 && (r <= rem) == (r + 31 <= rem) && rel + 31 <= 0 && tokens - 1 - rel < window;
  }
  // whether new token t sees what slot x holds
  __device__ __forceinline__ bool seen(int x, int t, int window) const {
    const int r = x - sinks, rel = newer + (r <= rem ? r : r - ring);
    return r < 0 ? x - n <= t : (rel <= t) & (t - rel < window);
  }
};

// A block takes the heads and tokens that share a head's keys, 32 at a time,
// as the columns of its products, and a share of the slots they see; each wave
// walks 32 slots at a time of its own, keys from memory into registers and
// values straight into its part of LDS, the next ones' while this one's products
// run, and needs no other wave until the end, when the waves' results are joined.  The new tokens' keys and
// values are written to the cache by the wave that then reads their slots.
//
// Bound by HBM: the slots seen are read once per 32 columns.  Batch 256, 16/4
// heads of 128, 1028 slots: 104 us, 5.2 TB/s, what a copy reaches.  Where each wave
// has a tile or two, by the time that one takes from its lengths to its result:
// 32768 slots of one sequence 16 us and 4 for the join, 3.5 TB/s; 8 new tokens of 32
// sequences, 32/8 heads of 64, up to 2059 slots: 20.5 and 4 us (8 of 1035 slots each:
// 25 in all for 32 sequences, 40 for 64, 72 for 128, 4.5 TB/s of what is added).
// (Without the branch around the masks, whose 250 instructions every tile then takes:
// 109, 18.5 and 23.7.)
template <typename T, int DP, int DU>
__global__ __launch_bounds__(256, (io<T>::BYTES == 2 ? 2 : 1) * (DP == 64 ? 2 : 1)) void attn_decode_kernel(
    AttnDecodeArgs a) {
  using KV = Tile<T, DP, DU, 32, 1>;
  constexpr int NW = 4, ES = io<T>::BYTES, STEPS = 32 / KV::CK, PART = 2 * KV::BYTES;
  static_assert(32 * DP * 4 <= PART, "a wave's result fits its part");
  __shared__ __attribute__((aligned(1024))) char smem[NW * PART];
  __shared__ float stat[NW][2][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int G = a.q_heads / a.kv_heads, cols = G * a.tokens;
  const int groups = (cols + 31) / 32;
  uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const int split = (int)(id % (uint32_t)a.splits);
  id /= (uint32_t)a.splits;
  const int group = (int)(id % (uint32_t)groups);
  id /= (uint32_t)groups;
  const int64_t hk = id % (uint32_t)a.kv_heads, b = id / (uint32_t)a.kv_heads;
  const int c0 = group * 32;
  const bool in = c0 + col < cols;
  const int tok = in ? (c0 + col) / G : 0;
  const int64_t hq = hk * G + (in ? (c0 + col) - tok * G : 0);
  RowRegs<T, DU> q;
  q.load((const char*)a.q + ((b * a.tokens + tok) * a.q_stride + hq * a.dim) * ES, in, a.dim, h);

  CacheView view;
  const int64_t len = a.lens[b];
  int begin = 0, end = 0;
  if (len >= 0) {
    view.init(len, a.tokens, (int)a.capacity, a.sinks, a.window);
    const int share = NW * a.splits, per = (view.tiles() + share - 1) / share;
    begin = (split * NW + wave) * per;
    end = begin + per < view.tiles() ? begin + per : view.tiles();
  }
  KV vt;
  RowStream<T, DU> kt;
  kt.init(a.kc_stride, a.dim, lane);
  vt.init(a.vc_stride, a.dim, lane, 0);
  char* kc = (char*)a.k_cache + (b * a.capacity * a.kc_stride + hk * a.dim) * ES;
  char* vc = (char*)a.v_cache + (b * a.capacity * a.vc_stride + hk * a.dim) * ES;
  char* mine = smem + wave * PART;
  auto load = [&](int i, int buf) {
    int x, e;
    view.tile(i, x, e);
    // new tokens that fall into the tile
    int at = view.slot_n + lane;
    if (at >= a.capacity) at -= view.ring;
    uint64_t fresh = __ballot(lane < a.tokens && at >= x && at < e);
    if (fresh) {
      while (fresh) {
        const int t = __builtin_ctzll(fresh);
        fresh &= fresh - 1;
        const int64_t slot = __builtin_amdgcn_readlane(at, t), row = b * a.tokens + t;
        const char* src = h ? (const char*)a.v + (row * a.v_stride + hk * a.dim) * ES
                            : (const char*)a.k + (row * a.k_stride + hk * a.dim) * ES;
        char* dst = h ? vc + slot * a.vc_stride * ES : kc + slot * a.kc_stride * ES;
        if (col * 16 < a.dim * ES) *(uint4*)(dst + col * 16) = *(const uint4*)(src + col * 16);
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0f70);  // the stores are done
      asm volatile("" ::: "memory");
    }
    kt.load(kc + (int64_t)x * a.kc_stride * ES, e - x, a.dim);
    vt.load(vc + (int64_t)x * a.vc_stride * ES, e - x, a.dim, mine + buf * KV::BYTES, 0);
  };
  f32x16 acc[KV::CT];
#pragma unroll
  for (int i = 0; i < KV::CT; ++i) acc[i] = f32x16{};
  Softmax<KV::CT> soft;
  soft.init();
  const float c = a.scale * kLog2e;
  if (begin < end) load(begin, 0);
  for (int i = begin; i < end; ++i) {
    const int buf = (i - begin) & 1;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    uint4 k[KV::KS];
#pragma unroll
    for (int st = 0; st < KV::KS; ++st) k[st] = kt.v[st];
    if (i + 1 < end) load(i + 1, buf ^ 1);
    const char* vl = mine + buf * KV::BYTES;
    int x, e;
    view.tile(i, x, e);
    f32x16 sc = f32x16{};
#pragma unroll
    for (int st = 0; st < KV::KS; ++st) sc = mma32<T>(k[st], q.v[st], sc);
    float z[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) z[v] = sc[v];
    if (!view.all_seen(x, e, a.tokens, a.window)) {
      asm volatile("");  // a branch, not selects in every step
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int j = x + v / 4 * 8 + 4 * h + v % 4;
        z[v] = (j < e) & view.seen(j, tok, a.window) ? z[v] : -INFINITY;
      }
    }
    float p[16];
    soft.template step<16>(z, c, acc, p);
#pragma unroll
    for (int n = 0; n < STEPS; ++n) {
      const uint4 w = result_step<T>(p, n);
#pragma unroll
      for (int d = 0; d < KV::CT; ++d) acc[d] = mma32<T>(vt.col(vl, d, n), w, acc[d]);
    }
  }
  // the waves' results: maximum, sum and unscaled output of each column
  const float l = swap_sum32(soft.l);
  float* res = (float*)mine;
  __syncthreads();
  if (h == 0) {
    stat[wave][0][col] = soft.m;
    stat[wave][1][col] = l;
  }
#pragma unroll
  for (int d = 0; d < KV::CT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f32x4*)(res + col * DP + (((d * 8 + 2 * i + h) ^ (col & 15)) << 2)) =
          f32x4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
  __syncthreads();
  const int width = a.dim / 4, valid = cols - c0 < 32 ? cols - c0 : 32;
  for (int e = threadIdx.x; e < valid * width; e += 64 * NW) {
    const int k = e / width, d = (e - k * width) * 4, t = (c0 + k) / G;
    float m = stat[0][0][k];
#pragma unroll
    for (int w = 1; w < NW; ++w) m = fmaxf(m, stat[w][0][k]);
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((stat[w][0][k] - m) * c);
      sum += f * stat[w][1][k];
      const f32x4 x = *(const f32x4*)((const float*)(smem + w * PART) + k * DP + (((d >> 2) ^ (k & 15)) << 2));
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += f * x[j];
    }
    const int64_t row = b * a.tokens + t, head = hk * G + (c0 + k - t * G);
    if (a.splits == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float f[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
      io<T>::store4(a.o, row * a.o_stride + head * a.dim + d, f);
    } else {
      // (row, head, split): output, then maximum and sum of all of them
      const int64_t at = (row * a.q_heads + head) * a.splits + split;
      *(f32x4*)(a.part + at * a.dim + d) = o;
      if (d == 0) {
        float* s = a.part + a.batch * a.tokens * a.q_heads * a.splits * a.dim + 2 * at;
        s[0] = m;
        s[1] = sum;
      }
    }
  }
}

// The splits joined in order: a block per row and head.  Lane i of every wave
// takes the statistics of splits i, i + 64, ...; then eight groups of threads
// each sum an eighth of the splits, four entries to a thread.
template <typename T>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(AttnDecodeArgs a) {
  __shared__ float weight[kMaxSplits];
  __shared__ f32x4 sums[8][32];
  const int lane = threadIdx.x & 63;
  const int64_t all = a.batch * a.tokens * a.q_heads, id = blockIdx.x;
  const float* stat = a.part + all * a.splits * a.dim + 2 * id * a.splits;
  const float c = a.scale * kLog2e;
  float m = -INFINITY;
  for (int i = lane; i < a.splits; i += 64) m = fmaxf(m, stat[2 * i]);
#pragma unroll
  for (int o = 1; o < 64; o *= 2) m = fmaxf(m, __shfl_xor(m, o, 64));
  float sum = 0.0f;
  for (int i = lane; i < a.splits; i += 64) {
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((stat[2 * i] - m) * c);
    sum += f * stat[2 * i + 1];
    if (threadIdx.x < 64) weight[i] = f;
  }
  sum = lane_sum<1, 64>(sum);
  __syncthreads();
  const int g = threadIdx.x >> 5, d = (threadIdx.x & 31) * 4;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (d < a.dim) {
    const float* part = a.part + id * a.splits * a.dim + d;
#pragma unroll 8
    for (int i = g; i < a.splits; i += 8) {
      const f32x4 x = *(const f32x4*)(part + (int64_t)i * a.dim);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += weight[i] * x[j];
    }
  }
  sums[g][threadIdx.x & 31] = o;
  __syncthreads();
  if (g != 0 || d >= a.dim) return;
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] += sums[i][threadIdx.x & 31][j];
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] *= inv;
  const int64_t row = id / a.q_heads;
  io<T>::store4(a.o, row * a.o_stride + (id - row * a.q_heads) * a.dim + d, f);
}

// The same for up to 4 splits: 32 threads per row and head, thread i with split
// i's statistics.  (With 16 of them its row after row of partial sums takes 3 us
// longer than the other kernel; with 2 and 8192 rows, 8 rows to a block save 7.)
template <typename T>
__global__ __launch_bounds__(256) void attn_decode_join_few_kernel(AttnDecodeArgs a) {
  const int64_t all = a.batch * a.tokens * a.q_heads, mine = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t id = mine < all ? mine : all - 1;  // a wave's threads all take part in the sums
  const int i0 = threadIdx.x & 31, d = i0 * 4;
  const float* stat = a.part + all * a.splits * a.dim + 2 * id * a.splits;
  const float* part = a.part + id * a.splits * a.dim + (d < a.dim ? d : 0);
  const float own = i0 < a.splits ? stat[2 * i0] : -INFINITY;
  float m = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) m = fmaxf(m, __shfl_xor(m, o, 64));
  const float weight = own == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((own - m) * (a.scale * kLog2e));
  const float sum = lane_sum<1, 32>(i0 < a.splits ? weight * stat[2 * i0 + 1] : 0.0f);
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = 0; i < a.splits; ++i) {
    const float w = __shfl(weight, i, 32);
    const f32x4 x = *(const f32x4*)(part + (int64_t)i * a.dim);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] += w * x[j];
  }
  if (mine >= all || d >= a.dim) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] *= inv;
  const int64_t row = id / a.q_heads;
  io<T>::store4(a.o, row * a.o_stride + (id - row * a.q_heads) * a.dim + d, f);
}

template <typename T>
hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t s) {
  const int64_t groups = ((int64_t)a.q_heads / a.kv_heads * a.tokens + 31) / 32;
  const dim3 grid((unsigned)(a.batch * a.kv_heads * groups * a.splits)), block(256);
  with_width(a.dim, [&](auto dp, auto du) {
    hipLaunchKernelGGL((attn_decode_kernel<T, decltype(dp)::value, decltype(du)::value>), grid, block, 0, s, a);
  });
  const int64_t rows = a.batch * a.tokens * a.q_heads;
  if (a.splits > 4) hipLaunchKernelGGL((attn_decode_join_kernel<T>), dim3((unsigned)rows), block, 0, s, a);
  else if (a.splits > 1)
    hipLaunchKernelGGL((attn_decode_join_few_kernel<T>), dim3((unsigned)((rows + 7) / 8)), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace m3
