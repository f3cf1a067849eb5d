// The 256 x 256 tile of the matrix products (mm_tile.hpp has the smaller one,
// the epilogue and the order of the work).
//
// Four waves, one per SIMD, each 128 x 128 of the tile: 16 products of 32 x 32
// with 256 accumulators, fed by 128 bytes of k per stage.  What bounds the
// loop is keeping the matrix core of a lone wave busy: a stage's 64 KB take
// about half a stage to come through the CU's 64-byte path, after a latency
// of about as long, so loads have to be in flight the whole time.  Hence a
// stage is cut into four pieces of 16 KB (of each operand, the first and the
// second half of every wave's rows) and four phases of one quadrant each:
//   phase 0: P0 Q0, reads Q1         phase 2: P1 Q1, reads the next P0
//   phase 1: P0 Q1, reads P1         phase 3: P1 Q0, reads the next Q0
// where a "read" takes the piece from LDS into registers, for the phase after.
// A piece's place in LDS is free one phase after its read and gets the piece
// of the stage after next at once: a load has six phases (3,000 cycles) to
// land, and every phase issues four loads per wave, reads one piece and ends
// in one barrier that waits for the loads of six phases before.
// 32768 x 11264 -> 2048 bf16 (dx): 1.10 ms, 1.37 PFLOP/s, the matrix cores busy
// in 80 % of the cycles at 1.64 GHz; two whole stages in LDS with all loads in
// a stage's last quarter took 1.36 ms, 52-55 % busy.  The epilogue goes through
// LDS so that rows leave in 128 bytes: 32768 x 2048 -> 2 x 5632 with stored
// pre-activations 1.31 -> 1.23 ms.
#pragma once

#include "mm_tile.hpp"

namespace m3 {

// A 16 KB piece of an operand: half `H` of the rows of the two wave groups
// (rows 128 g + 64 H .. + 63; in a gated block's second operand, all 128 rows
// of the half's own matrix).
// KC: 128 rows of 128 bytes; chunk c of row r at chunk c ^ fsw(r).
// Otherwise: 128 / ES rows of k, each 128 elements; bf16: chunk c of row k at
// c ^ 4 (k mod 4), for the transpose reads.
template <typename T, bool KC, bool APART>
struct Piece {
  static constexpr int ES = io<T>::BYTES;
  static constexpr int BK = 128 / ES;
  static constexpr int LPR = KC ? 8 : 8 * ES;  // lanes per row of LDS
  static constexpr int RPI = 64 / LPR;         // rows per load
  int voff, kpos, ldb;
  int at[KC ? 4 : 2];

  __device__ __forceinline__ void init(int64_t ld, int lane, int wave, int group) {
    ldb = (int)(ld * ES);
    const int row = wave * RPI + lane / LPR, slot = lane % LPR;
    if constexpr (KC) {
      const int c = slot ^ fsw<8>(row);
      kpos = c * 16;
      voff = row * ldb + kpos;
      const int r = group * 64 + (lane & 31);
#pragma unroll
      for (int s = 0; s < 4; ++s) at[s] = r * 128 + (((2 * s + (lane >> 5)) ^ fsw<8>(r)) << 4);
    } else {
      const int c = ES == 2 ? slot ^ ((row & 3) << 2) : slot;
      kpos = 0;
      voff = row * ldb + c / (LPR / 2) * 128 * ES + c % (LPR / 2) * 16;
      if constexpr (ES == 2) {
        const int g = lane >> 4, i = lane & 15, q = i >> 2;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          at[t] = (8 * (g >> 1) + q) * 256 +
                  (((((group * 2 + t) ^ q) * 4) + (g & 1) * 2 + ((i & 3) >> 1)) << 4) + (i & 1) * 8;
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) at[t] = 4 * (lane >> 5) * 512 + (group * 64 + t * 32 + (lane & 31)) * 4;
      }
    }
  }
  // base: the tile's first element at k = 0 (APART: the half's); rows: rows
  // of the tile that exist.  What lies past them or past K reads as zero (a
  // partial last 16 bytes exists in memory and holds zeros past K).
  template <int H>
  __device__ __forceinline__ void load(const char* base, int64_t rows, int64_t K, int kb, char* lds, int wave) const {
    if constexpr (KC) {
      const int most = APART ? 128 : 256;
      const int n = rows < most ? (int)rows : most;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)base, 0, (uint32_t)((n - 1) * ldb + (int)((K * ES + 15) & ~(int64_t)15)), 0x00020000);
      const int vo = kpos < (int)(K * ES) - kb * 128 ? voff : 0x7ff00000;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (lds_void*)(lds + (i * 4 + wave) * 1024), 16, vo,
            (APART ? i * 32 : (i >> 1) * 128 + H * 64 + (i & 1) * 32) * ldb + kb * 128, 0, 0);
    } else {
      const int64_t all = (int64_t)kb * BK, k0 = all < K ? all : K;
      const int left = K - k0 < BK ? (int)(K - k0) : BK;
      const int bytes = (left - 1) * ldb + (int)((rows * ES + 15) & ~(int64_t)15);
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(base + k0 * ldb), 0, bytes > 0 ? bytes : 0, 0x00020000);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + (i * 4 + wave) * 1024), 16, voff,
                                                 i * 4 * RPI * ldb + H * 64 * ES, 0, 0);
    }
  }
  // fragment of tile t (0, 1) of the wave's half, k-step s
  __device__ __forceinline__ uint4 read(const char* lds, int t, int s) const {
    if constexpr (KC) {
      return __builtin_bit_cast(uint4, read16((const u32x4*)(lds + at[s] + t * 4096)));
    } else if constexpr (ES == 2) {
      const char* p = lds + at[t] + s * 4096;
      const uint2 a = read_tr(p), b = read_tr(p + 1024);
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      const char* p = lds + at[t] + s * 4096;
      return make_uint4(read4((const uint32_t*)p), read4((const uint32_t*)(p + 512)),
                        read4((const uint32_t*)(p + 1024)), read4((const uint32_t*)(p + 1536)));
    }
  }
};

// 32 rows x 64 columns of bf16 between the accumulators' layout (lane l: row l
// mod 32, columns 8 q + 4 (l / 32) .. + 3 of each 32) and whole 128-byte rows
// (lane l: rows l / 8 + 8 k, columns 8 (l mod 8) .. + 7), through 4 KB of LDS
// of the wave's own: 16-byte chunk c of row r at chunk c ^ (r mod 8).  Stored
// straight from the accumulators' layout, an output row goes out in pieces of
// 32 bytes, at half the rate.
__device__ __forceinline__ void write8(uint2* __restrict p, uint2 v) { *p = v; }
__device__ __forceinline__ void write16(u32x4* __restrict p, u32x4 v) { *p = v; }
__device__ __forceinline__ uint2 read8(const uint2* __restrict p) { return *p; }
struct Rows64 {
  char* lds;
  int lane;
  __device__ __forceinline__ char* piece(int tile, int q) const {
    const int r = lane & 31;
    return lds + r * 128 + (((tile * 4 + q) ^ (r & 7)) << 4) + (lane >> 5) * 8;
  }
  __device__ __forceinline__ char* line(int k) const {
    const int r = 8 * k + (lane >> 3);
    return lds + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
  }
  // tile t's values in, from the accumulators' layout
  __device__ __forceinline__ void put(int t, const float (&z)[16]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      write8((uint2*)piece(t, q),
             make_uint2(pack_bf2(z[4 * q], z[4 * q + 1]), pack_bf2(z[4 * q + 2], z[4 * q + 3])));
  }
  // what is there for tile t added to z
  __device__ __forceinline__ void add(int t, float (&z)[16]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint2 w = read8((const uint2*)piece(t, q));
      z[4 * q] += bf_lo(w.x);
      z[4 * q + 1] += bf_hi(w.x);
      z[4 * q + 2] += bf_lo(w.y);
      z[4 * q + 3] += bf_hi(w.y);
    }
  }
  // whole rows out to memory (dst: row 0, column 0), and in
  __device__ __forceinline__ void store(char* dst, int64_t ld) const {
    asm volatile("" ::: "memory");
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = read16((const u32x4*)line(k));
#pragma unroll
    for (int k = 0; k < 4; ++k) *(u32x4_any*)(dst + ((8 * k + (lane >> 3)) * ld + 8 * (lane & 7)) * 2) = v[k];
    asm volatile("" ::: "memory");
  }
  __device__ __forceinline__ void load(const char* src, int64_t ld, u32x4 (&v)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *(const u32x4_any*)(src + ((8 * k + (lane >> 3)) * ld + 8 * (lane & 7)) * 2);
  }
  __device__ __forceinline__ void fill(const u32x4 (&v)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) write16((u32x4*)line(k), v[k]);
    asm volatile("" ::: "memory");
  }
};

// The epilogue of a whole tile inside the matrix, bf16 io.  bias: the tile's
// in LDS (gated: the first half's 128 columns, then the other's).
template <int EPI, int ACT>
__device__ __forceinline__ void wide_epilogue(const MmArgs& a, const MmItem& it, f32x16 (&acc)[4][4], char* lds,
                                              const float* bias, int lane, int wave) {
  constexpr bool G = EPI == MM_GATED;
  const int h = lane >> 5;
  const int64_t m = it.m0 + (wave & 1) * 128;
  const Rows64 rows{lds, lane};
  // acc[i][j] (+ bias) of the tile i from column c of the block on
  auto value = [&](int i, int j, int c, float (&z)[16]) {
    acc_values<true>(acc[i][j], z);
    if constexpr (EPI != MM_STORE)
      if (a.bias) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 b = *(const f32x4*)(bias + c + 8 * q + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[4 * q + e] += b[e];
        }
      }
  };
#pragma unroll
  for (int i = 0; i < (G ? 2 : 4); i += 2) {
    const int c = (wave >> 1) * (G ? 64 : 128) + i * 32;
    const int64_t n = it.n0 + c;
    u32x4 res[4];
    const char* rs = (const char*)a.res + (m * a.ldr + n) * 2;
    if constexpr (EPI == MM_LINEAR)
      if (a.res) rows.load(rs, a.ldr, res);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m + 32 * j;
      float z[16], u[16];
      if constexpr (EPI != MM_STORE)
        if (a.pre) {
          char* pre = (char*)a.pre + (r * (G ? 2 : 1) * a.N + n) * 2;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            value(i + t, j, c + 32 * t, z);
            rows.put(t, z);
          }
          rows.store(pre, (G ? 2 : 1) * a.N);
          if constexpr (G) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              value(2 + t, j, 128 + c + 32 * t, u);
              rows.put(t, u);
            }
            rows.store(pre + a.N * 2, 2 * a.N);
          }
        }
      if constexpr (EPI == MM_LINEAR)
        if (a.res) {
          rows.fill(res);
          if (j < 3) rows.load(rs + 32 * (j + 1) * a.ldr * 2, a.ldr, res);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        value(i + t, j, c + 32 * t, z);
        if constexpr (EPI != MM_STORE) {
#pragma unroll
          for (int v = 0; v < 16; ++v) z[v] = act_fwd<ACT, false>(z[v]);
        }
        if constexpr (EPI == MM_LINEAR)
          if (a.res) rows.add(t, z);
        if constexpr (G) {
          value(2 + t, j, 128 + c + 32 * t, u);
#pragma unroll
          for (int v = 0; v < 16; ++v) z[v] *= u[v];
        }
        rows.put(t, z);
      }
      rows.store((char*)a.out + (r * a.ldo + n) * 2, a.ldo);
    }
  }
}

template <typename T, int LAYOUT, int EPI, int ACT>
__global__ __launch_bounds__(256, 1) void mm_wide_kernel(MmArgs a, MmPlan pl) {
  constexpr bool PK = LAYOUT != MM_NONE_K, QK = LAYOUT == MM_PQ_K;
  constexpr int ES = io<T>::BYTES;
  constexpr bool G = EPI == MM_GATED;
  constexpr int BC = G ? 128 : 256;  // columns of out per tile
  constexpr int PIECE = 16384, BUF = 4 * PIECE;  // P0 P1 Q0 Q1
  // One array for all of it: with several, the compiler tracks which one a
  // load into LDS still in flight writes, and holds every fragment read back
  // until all of them have landed.
  constexpr int ROWS = 2 * BUF, BIAS = ROWS + (ES == 2 ? 4 * 4096 : 0);
  __shared__ __attribute__((aligned(1024))) char smem[BIAS + (ES == 2 ? 1024 : 0)];
  float* const bias = (float*)(smem + BIAS);

  const MmWalk walk(pl, blockIdx.x, gridDim.x);
  int id = walk.id;
  if (id >= walk.end) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Piece<T, PK, false> op;
  Piece<T, QK, G> oq;
  op.init(a.ldp, lane, wave, wave & 1);
  oq.init(a.ldq, lane, wave, wave >> 1);
  const int past = (int)((a.K + op.BK - 1) / op.BK);  // a stage that reads zeros

  auto load_p = [&](auto half, const MmItem& it, int kb, int buf) {
    constexpr int H = decltype(half)::value;
    const char* b = (const char*)a.P + (PK ? it.m0 * a.ldp : it.m0) * ES;
    op.template load<H>(b, a.M - it.m0, a.K, kb, smem + buf * BUF + H * PIECE, wave);
  };
  auto load_q = [&](auto half, const MmItem& it, int kb, int buf) {
    constexpr int H = decltype(half)::value;
    const int64_t n = it.n0 + (G && H ? a.N : 0);
    const char* b = (const char*)a.Q + (QK ? n * a.ldq : n) * ES;
    oq.template load<H>(b, a.N - it.n0, a.K, kb, smem + buf * BUF + (2 + H) * PIECE, wave);
  };
  // fragments of the pieces: P0, P1; Q0 and Q1 change places every stage,
  // since the next Q0 is read while this stage's is in use
  uint4 p[2][2][4], q[2][2][4];
  auto read_p = [&](int half, int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t) p[half][t][s] = op.read(smem + buf * BUF + half * PIECE, t, s);
  };
  auto read_q = [&](int half, int buf, int to) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t) q[to][t][s] = oq.read(smem + buf * BUF + (2 + half) * PIECE, t, s);
  };
  f32x16 acc[4][4];  // [tile of Q][tile of P]
  auto multiply = [&](int ph, int qh, int qat, auto fresh) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x16& c = acc[qh * 2 + i][ph * 2 + j];
          if (decltype(fresh)::value && s == 0) c = mma32<T>(q[qat][i][s], p[ph][j][s], f32x16{});
          else c = mma32<T>(q[qat][i][s], p[ph][j][s], c);
        }
  };
  constexpr int NM = 16 * (ES == 2 ? 1 : 4);
  constexpr int NP = PK ? 8 : ES == 2 ? 16 : 32, NQ = QK ? 8 : ES == 2 ? 16 : 32;  // LDS reads of a piece
  // All but the last 24 loads of this wave have landed (the six latest
  // phases'), its reads are done, and so it is with every wave.
  auto settle = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x4078);  // vmcnt(24) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  std::integral_constant<int, 0> c0;
  std::integral_constant<int, 1> c1;
  std::integral_constant<bool, true> yes;
  std::integral_constant<bool, false> no;
  // Stage in buffer B; n2, k2 and n3, k3: the stages two and three later.
  auto stage = [&](auto cur, auto fresh, const MmItem& n2, int k2, const MmItem& n3, int k3) {
    constexpr int B = decltype(cur)::value;
    read_q(1, B, B ^ 1);
    load_q(c0, n2, k2, B);
    multiply(0, 0, B, fresh);
    mix_k_step<NM, NQ, 4>();
    settle();
    read_p(1, B);
    load_q(c1, n2, k2, B);
    multiply(0, 1, B ^ 1, fresh);
    mix_k_step<NM, NP, 4>();
    settle();
    read_p(0, B ^ 1);
    load_p(c1, n2, k2, B);
    multiply(1, 1, B ^ 1, fresh);
    mix_k_step<NM, NP, 4>();
    settle();
    read_q(0, B ^ 1, B ^ 1);
    load_p(c0, n3, k3, B ^ 1);
    multiply(1, 0, B, fresh);
    mix_k_step<NM, NQ, 4>();
    settle();
  };

  MmItem it = walk.item<256, BC>(pl, id);
  load_p(c0, it, it.kb, 0);
  load_q(c0, it, it.kb, 0);
  load_q(c1, it, it.kb, 0);
  load_p(c1, it, it.kb, 0);
  load_p(c0, it, it.kb + 1, 1);
  load_q(c0, it, it.kb + 1, 1);
  load_q(c1, it, it.kb + 1, 1);
  load_p(c1, it, it.kb + 1, 1);
  settle();  // P0 and Q0 are there
  read_p(0, 0);
  read_q(0, 0, 0);
  settle();  // ... and read
  load_p(c0, it, it.kb + 2, 0);
  settle();  // Q1 is there
  for (;;) {
    id += walk.step;
    const bool last = id >= walk.end;
    MmItem nx = walk.item<256, BC>(pl, last ? 0 : id);
    if (last) nx.kb = past;
    const int nk = it.part < 0 ? pl.whole : pl.stages;  // even, at least 4
    float b = 0.0f;  // of column it.n0 + tid, for the epilogue
    if constexpr (ES == 2 && EPI != MM_STORE)
      if (a.bias) {
        const int64_t n = it.n0 + (threadIdx.x & (BC - 1));
        b = a.bias[(n < a.N ? n : a.N - 1) + (threadIdx.x >= BC ? a.N : 0)];
      }
    stage(c0, yes, it, it.kb + 2, it, it.kb + 3);
    stage(c1, no, it, it.kb + 3, nk == 4 ? nx : it, nk == 4 ? nx.kb : it.kb + 4);
    for (int t = 2; t < nk; t += 2) {
      const bool over = t + 2 >= nk, near = t + 4 >= nk;
      const int k2 = over ? nx.kb - nk : it.kb, k4 = near ? nx.kb - nk : it.kb;
      stage(c0, no, over ? nx : it, k2 + t + 2, over ? nx : it, k2 + t + 3);
      stage(c1, no, over ? nx : it, k2 + t + 3, near ? nx : it, k4 + t + 4);
    }
    // opaque, so that the epilogue's addresses are not kept in registers
    // across the products
    int el = lane, ew = wave;
    asm volatile("" : "+v"(el), "+s"(ew));
    mm_drain();
    bool done = false;
    if constexpr (ES == 2)
      if (it.part < 0 && it.m0 + 256 <= a.M && it.n0 + BC <= a.N) {
        if constexpr (EPI != MM_STORE)
          if (a.bias) {
            bias[threadIdx.x] = b;
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
          }
        wide_epilogue<EPI, ACT>(a, it, acc, smem + ROWS + ew * 4096, bias, el, ew);
        done = true;
      }
    if (!done) mm_finish<T, EPI, ACT, 256, 256>(a, it, acc, el, ew);
    if (last) break;
    it = nx;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the loads past the last item (zeros) have landed
}

}  // namespace m3
