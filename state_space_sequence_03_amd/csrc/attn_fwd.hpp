// Windowed attention with sinks, forward.
#pragma once

#include "attn.hpp"

namespace m3 {

// NW waves take 32 NW queries, 32 NW / HT positions of HT heads that share a head
// of keys, each wave 32 of one head as the columns of its products:
// scores = K q^T, o^T += V^T p.  (As many heads as there are, up to 4: the fewer
// positions, the fewer keys that only some of the block's queries see.)  They
// walk the runs of 32 keys that their queries see, the sinks' first, then the
// window's, BN / 32 at a time; with KW > 1 the block has as many such parties,
// each with every KW-th of these tiles.  Keys and values come straight from memory
// into LDS, the next tile's while this one's products run.
//
// Bound by the vector units next to the matrix cores: two waves per SIMD (three to
// a width of 64), so that one's softmax runs under another's products, overlap in
// part only: at a width of 128 products alone would take 0.53 of the time, the
// softmax 0.65.  1 x 32768 queries, 16/4 heads of 128, window 4096: 950 to 1030 us,
// 1.01 to 1.09 PFLOP/s; 8 x 4096, window 1024: 274 to 283, 0.87; packed documents,
// 16384 rows, 32/8 heads of 64, window 512: 96.  Runs of 32 that need not be
// neighbours save the rest of the sinks' tile and of the first of the window's: 103
// -> 96 us in the last of these, 29 -> 31 where there are few blocks and no window.
template <typename T, int DP, int DU, int BN, int HT, int NW, int KW>
__global__ __launch_bounds__(64 * NW * KW, NW == 1 ? 1 : 2) void attn_fwd_kernel(AttnArgs a, int64_t items) {
  using KV = Tile<T, DP, DU, BN, NW>;
  constexpr int ES = io<T>::BYTES, NT = BN / 32, STEPS = 32 / KV::CK, BM = 32 * NW / HT;
  // wide parties of one wave take the keys into registers: LDS has room for four
  constexpr bool ALONE = NW == 1 && DP == 128;
  static_assert(!ALONE || NT == 1, "a run at a time");
  constexpr int PART = (ALONE ? 2 : 4) * KV::BYTES;  // V V or K V K V of each
  __shared__ __attribute__((aligned(1024))) char lds[KW * PART];
  const int lane = threadIdx.x & 63;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = all % NW, part = all / NW;
  char* smem = lds + part * PART;
  const int h = lane >> 5;
  const int G = a.q_heads / a.kv_heads;
  // heads that share keys are neighbours, then the tiles of a sequence, the
  // longest first
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
  RowRegs<T, DU> q;
  q.load((const char*)a.q + (row * a.q_stride + hq * a.dim) * ES, in, a.dim, h);

  KV kt, vt;
  RowStream<T, DU> ks;
  if constexpr (ALONE) ks.init(a.k_stride, a.dim, lane);
  else kt.init(a.k_stride, a.dim, lane, wave);
  vt.init(a.v_stride, a.dim, lane, wave);
  const char* kb = (const char*)a.k + (s.k0 * a.k_stride + hk * a.dim) * ES;
  const char* vb = (const char*)a.v + (s.k0 * a.v_stride + hk * a.dim) * ES;
  int first = p0 - a.window + 1;
  first = first < 0 ? 0 : first / 32;
  const int sunk = (a.sinks + 31) / 32, ns = sunk < first ? sunk : first;
  const int units = p1 < 0 ? 0 : ns + p1 / 32 - first + 1, count = (units + NT - 1) / NT;
  // first keys of tile n's runs (past every position: there is none), which are
  // loaded
  auto load = [&](int n, int (&at)[NT], int buf) {
    char* to = smem + buf * (PART / 2);
    const int next = (first + n * NT - ns) * 32;
    if constexpr (ALONE) {
      const int64_t j = n < ns ? n * 32 : next;
      const int rows = s.nk - (int)j < 32 ? s.nk - (int)j : 32;
      at[0] = (int)j;
      ks.load(kb + j * a.k_stride * ES, rows, a.dim);
      vt.load(vb + j * a.v_stride * ES, rows, a.dim, to, wave);
    } else if (n * NT >= ns && next + BN <= s.nk) {  // one after the other, as most are
#pragma unroll
      for (int b = 0; b < NT; ++b) at[b] = next + 32 * b;
      kt.load(kb + (int64_t)next * a.k_stride * ES, BN, a.dim, to, wave);
      vt.load(vb + (int64_t)next * a.v_stride * ES, BN, a.dim, to + KV::BYTES, wave);
    } else {
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const int u = n * NT + b;
        const int64_t j = u < ns ? u * 32 : u < units ? next + 32 * b : 0;
        at[b] = u < units ? (int)j : 1 << 28;
        kt.load32(kb + j * a.k_stride * ES, s.nk - at[b], a.dim, to, wave, b);
        vt.load32(vb + j * a.v_stride * ES, s.nk - at[b], a.dim, to + KV::BYTES, wave, b);
      }
    }
  };

  f32x16 acc[KV::CT];
#pragma unroll
  for (int i = 0; i < KV::CT; ++i) acc[i] = f32x16{};
  Softmax<KV::CT> soft;
  soft.init();
  const float c = a.scale * kLog2e;
  int at[NT], ahead_at[NT];
  if (part < count) load(part, ahead_at, 0);
  for (int i = 0; i * KW < count; ++i) {
    const int n = i * KW + part;
    if constexpr (ALONE) attn_settle_alone();
    else attn_settle();
    if (KW > 1 && n >= count) continue;
    uint4 k[ALONE ? KV::KS : 1];
    if constexpr (ALONE)
#pragma unroll
      for (int st = 0; st < KV::KS; ++st) k[st] = ks.v[st];
#pragma unroll
    for (int b = 0; b < NT; ++b) at[b] = ahead_at[b];
    if (n + KW < count) load(n + KW, ahead_at, (i + 1) & 1);
    const char* kl = smem + (i & 1) * (PART / 2);
    const char* vl = ALONE ? kl : kl + KV::BYTES;
    f32x16 sc[NT];
    ahead<6, KV::KS * NT, 1, T>(
        [&](int i) {
          if constexpr (ALONE) return k[i];
          else return kt.row(kl, i % NT, i / NT);
        },
        [&](int i, const uint4& f) { sc[i % NT] = mma32<T>(f, q.v[i / NT], i < NT ? f32x16{} : sc[i % NT]); });
    float z[NT * 16], e[NT * 16];
#pragma unroll
    for (int v = 0; v < NT * 16; ++v) z[v] = sc[v / 16][v % 16];
    if (at[NT - 1] + 31 > w0 || (at[0] <= w1 - a.window && at[NT - 1] + 31 >= a.sinks)) {
      asm volatile("");  // a branch, not selects in every step
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const KeysSeen seen(a, p, at[b] + 4 * h);
#pragma unroll
        for (int v = 0; v < 16; ++v) z[16 * b + v] = seen(v / 4 * 8 + v % 4) ? z[16 * b + v] : -INFINITY;
      }
    }
    soft.template step<NT * 16>(z, c, acc, e);
    uint4 w[NT * STEPS];
#pragma unroll
    for (int k = 0; k < NT * STEPS; ++k) w[k] = result_step<T>(e, k);
    ahead<6, NT * STEPS * KV::CT, 2, T>(
        [&](int i) { return vt.col(vl, i % KV::CT, i / KV::CT); },
        [&](int i, const uint4& f) { acc[i % KV::CT] = mma32<T>(f, w[i / KV::CT], acc[i % KV::CT]); });
  }
  if constexpr (KW > 1)
    if (!join_parts<KW, NW, PART, true>(lds, acc, soft.m, soft.l, c, part, wave, lane)) return;
  const float l = swap_sum32(soft.l);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing: 0
  if (a.lse && in && h == 0) a.lse[row * a.q_heads + hq] = l == 0.0f ? -INFINITY : soft.m * a.scale + logf(l);
  char* out = (char*)a.o + (row * a.o_stride + hq * a.dim) * ES;
#pragma unroll
  for (int d = 0; d < KV::CT; ++d) {
    if (d * 32 >= a.dim) break;
    float z[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) z[v] = acc[d][v] * inv;
    tile_store<T, false>(out, in, d * 32, a.dim, z, h);
  }
}

template <typename T, int HT, int NW, int KW>
void attn_fwd_run(const AttnArgs& a, hipStream_t s) {
  const int64_t items = attn_items(a, false, 32 * NW / HT);
  const dim3 grid((unsigned)(items * (a.q_heads / HT)));
  with_width(a.dim, [&](auto dp, auto du) {
    constexpr int DP = decltype(dp)::value, BN = io<T>::BYTES == 2 ? 64 : 32;
    hipLaunchKernelGGL((attn_fwd_kernel<T, DP, decltype(du)::value, BN, HT, NW, KW>), grid, dim3(64 * NW * KW), 0, s, a,
                       items);
  });
}

template <typename T>
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) {
  attn_by_size<T>(a, [&](auto ht, auto nw, auto kw) {
    attn_fwd_run<T, decltype(ht)::value, decltype(nw)::value, decltype(kw)::value>(a, s);
  });
  return hipGetLastError();
}

}  // namespace m3
