// Tiled matrix products out[m][n] = epilogue(sum_k P(m, k) Q(n, k)) for
// operands whose rows lie on 16 bytes.
#pragma once

#include "act.hpp"
#include "m3_launch.hpp"
#include "m3_rows.hpp"

namespace m3 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef __attribute__((address_space(3))) void lds_void;

// acc += the product over the 32 bytes of k that a fragment pair holds: lane
// l carries row l mod 32 of its operand and 16 of those bytes, chunk l / 32.
// For fp32 the four words of a lane go to four products, whose k are those of
// both halves' same word: any order of k is right when both operands share it.
template <typename T>
__device__ __forceinline__ f32x16 mma32(const uint4& p, const uint4& q, f32x16 acc) {
  if constexpr (io<T>::BYTES == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(p), as_bf16x8(q), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p.x), __uint_as_float(q.x), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p.y), __uint_as_float(q.y), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p.z), __uint_as_float(q.z), acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p.w), __uint_as_float(q.w), acc, 0, 0, 0);
  }
}

// Fragment reads.  The pointers are restrict-qualified so that the compiler
// does not hold these reads back until every load into LDS still in flight
// has landed: which stage they read has been published by the kernel's own
// wait and barrier.
__device__ __forceinline__ u32x4 read16(const u32x4* __restrict p) { return *p; }
__device__ __forceinline__ uint32_t read4(const uint32_t* __restrict p) { return *p; }
__device__ __forceinline__ uint2 read_tr(const void* __restrict p) { return lds_tr16(p); }

// One operand's tile of ROWS rows (of m or n) and 128 bytes of k per stage:
// where its pieces lie in memory, in LDS and in a wave's fragments.
//
// KC (rows run along k): LDS holds ROWS rows of 128 bytes, 16-byte chunk c of
// row r at chunk c ^ fsw(r), so that the 32 rows of a fragment read fall into
// distinct bank groups.
// Otherwise (rows of memory run along m or n): LDS holds 128 / ES rows of k,
// each ROWS elements wide.  bf16 fragments come out of the transpose read,
// chunk c of row k stored at c ^ 4 turn(k), so that the four rows a 16-lane
// group addresses fall into distinct banks; fp32 fragments are four words.
template <typename T, bool KC, int ROWS>
struct Operand {
  static constexpr int ES = io<T>::BYTES;
  static constexpr int BK = 128 / ES;          // k per stage
  static constexpr int BYTES = ROWS * 128;     // per stage
  static constexpr int NI = BYTES / 4096;      // 1 KB loads per wave and stage
  static constexpr int LPR = KC ? 8 : ROWS * ES / 16;  // lanes per row of LDS
  static constexpr int RPI = 64 / LPR;         // rows per 1 KB load

  // bf16, not KC: chunk c of row k lies at c ^ 4 turn(k)
  __device__ __forceinline__ static int turn(int k) { return ROWS == 64 ? (k >> 1) & 1 : k & 3; }

  int voff;   // lane's byte offset within the tile
  int kpos;   // KC: lane's first byte of k within the stage
  int ldb;

  __device__ __forceinline__ void init(int64_t ld, int lane, int wave) {
    ldb = (int)(ld * ES);
    const int row = wave * RPI + lane / LPR, slot = lane % LPR;
    int chunk = slot;
    if constexpr (KC) chunk = slot ^ fsw<8>(row);  // rows 32 apart share it
    else if constexpr (ES == 2) chunk = slot ^ (turn(row) << 2);  // rows 4 RPI apart share it
    kpos = chunk * 16;
    voff = row * ldb + chunk * 16;
  }
  // Loads of stage kb into LDS, straight from memory (one wave instruction
  // fills 1 KB, lane l's 16 bytes at l * 16).  `base` is the tile's first
  // element: row 0 of the tile at k = 0 (KC), or the tile's first column at
  // k = 0.  `rows`: rows of the tile that exist; what lies past them or past
  // K reads as zero.  Instructions [I0, I1) of the stage.
  template <int I0, int I1>
  __device__ __forceinline__ void load(const char* base, int64_t rows, int64_t K, int kb, char* lds, int wave) const {
    if constexpr (KC) {
      const int64_t n = rows < (I1 - I0) * 4 * RPI ? rows : (I1 - I0) * 4 * RPI;
      // a last, partial 16 bytes of k exists in memory (the caller's rows end
      // on 16 bytes) and holds zeros past K
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)base, 0, (uint32_t)((n - 1) * ldb + ((K * ES + 15) & ~(int64_t)15)), 0x00020000);
      const int vo = kpos < (int)(K * ES) - kb * 128 ? voff : 0x7ff00000;
#pragma unroll
      for (int i = I0; i < I1; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + (i * 4 + wave) * 1024), 16, vo,
                                                 (i - I0) * 4 * RPI * ldb + kb * 128, 0, 0);
    } else {
      const int64_t all = (int64_t)kb * BK, k0 = all < K ? all : K;
      const int left = K - k0 < BK ? (int)(K - k0) : BK;
      // at most 0 where nothing is left; a partial last 16 bytes exists, as above
      const int bytes = (left - 1) * ldb + (int)((rows * ES + 15) & ~(int64_t)15);
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(base + k0 * ldb), 0, bytes > 0 ? bytes : 0, 0x00020000);
#pragma unroll
      for (int i = I0; i < I1; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + (i * 4 + wave) * 1024), 16, voff,
                                                 i * 4 * RPI * ldb, 0, 0);
    }
  }
};

// A wave's fragments of one operand: NT tiles of 32 rows from row r0 of the
// tile (tiles t >= NT / 2 lie GAP rows further, the second half of a gated
// block's rows).
template <typename T, bool KC, int ROWS, int NT, int GAP>
struct Fragments {
  static constexpr int ES = io<T>::BYTES;
  static constexpr int NB = KC ? 4 : (ES == 2 ? 4 : 1);
  int at[NB];  // KC: per k-step of 32 bytes; transposed: per tile position

  __device__ __forceinline__ void init(int r0, int lane) {
    if constexpr (KC) {
      const int r = lane & 31, h = lane >> 5, f = fsw<8>(r);
#pragma unroll
      for (int s = 0; s < 4; ++s) at[s] = (r0 + r) * 128 + (((2 * s + h) ^ f) << 4);
    } else if constexpr (ES == 2) {
      const int g = lane >> 4, i = lane & 15, q = i >> 2;
      const int row = 8 * (g >> 1) + q, c = (g & 1) * 2 + ((i & 3) >> 1);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        at[t] = row * ROWS * 2 + ((((r0 / 32 + t) ^ Operand<T, KC, ROWS>::turn(q)) * 4 + c) << 4) + (i & 1) * 8;
    } else {
      at[0] = (4 * (lane >> 5)) * ROWS * 4 + (r0 + (lane & 31)) * 4;
    }
  }
  // fragment of tile t, k-step s (32 bytes of k)
  __device__ __forceinline__ uint4 read(const char* lds, int t, int s) const {
    const int tt = t * 32 + (t >= NT / 2 ? GAP : 0);
    if constexpr (KC) {
      return __builtin_bit_cast(uint4, read16((const u32x4*)(lds + at[s] + tt * 128)));
    } else if constexpr (ES == 2) {
      const char* p = lds + at[t & 3] + s * 16 * ROWS * 2;
      const uint2 a = read_tr(p), b = read_tr(p + 4 * ROWS * 2);
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      const char* p = lds + at[0] + s * 8 * ROWS * 4 + tt * 4;
      return make_uint4(read4((const uint32_t*)p), read4((const uint32_t*)(p + ROWS * 4)),
                        read4((const uint32_t*)(p + 2 * ROWS * 4)), read4((const uint32_t*)(p + 3 * ROWS * 4)));
    }
  }
};

// ---------------------------------------------------------------------------
// Epilogue of one 32 x 32 tile: lane l holds row m = m0 + l mod 32 and, in
// v[4q + j], column n0 + 8q + 4 (l / 32) + j.  For bf16 the halves of the wave
// exchange every second quadruple, so that a lane stores 8 columns (16 bytes)
// at a time: columns 16p + 8 (l / 32) .. + 7.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = s[0];
  b = s[1];
}

// INNER: every row and column of the tile exists.
template <typename T, bool INNER>
__device__ __forceinline__ void tile_store(char* row, bool in, int64_t n0, int64_t N, const float* v, int h) {
  if constexpr (io<T>::BYTES == 2) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t a0 = pack_bf2(v[8 * p], v[8 * p + 1]), a1 = pack_bf2(v[8 * p + 2], v[8 * p + 3]);
      uint32_t b0 = pack_bf2(v[8 * p + 4], v[8 * p + 5]), b1 = pack_bf2(v[8 * p + 6], v[8 * p + 7]);
      swap_halves(a0, b0);
      swap_halves(a1, b1);
      const int64_t n = n0 + 16 * p + 8 * h;
      const u32x4 o = {a0, a1, b0, b1};
      if (INNER || (in && n + 8 <= N)) {
        *(u32x4_any*)(row + n * 2) = o;
      } else if (in) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n + j < N) ((u16*)row)[n + j] = (u16)(o[j >> 1] >> (16 * (j & 1)));
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t n = n0 + 8 * q + 4 * h;
      if (INNER || (in && n + 4 <= N)) {
        *(f32x4_any*)(row + n * 4) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      } else if (in) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) ((float*)row)[n + j] = v[4 * q + j];
      }
    }
  }
}

// The row's entries of a matrix of the io type, as loaded ...
template <typename T>
struct TileRow {
  static constexpr int NV = io<T>::BYTES == 2 ? 2 : 4;
  u32x4 o[NV];
  template <bool INNER>
  __device__ __forceinline__ void load(const char* row, bool in, int64_t n0, int64_t N, int h) {
    constexpr int ES = io<T>::BYTES, V = 16 / ES;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int64_t n = n0 + (32 / NV) * p + V * h;
      o[p] = u32x4{0u, 0u, 0u, 0u};
      if (INNER || (in && n + V <= N)) {
        o[p] = *(const u32x4_any*)(row + n * ES);
      } else if (in) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (n + j < N) {
            if constexpr (ES == 2) o[p][j >> 1] |= (uint32_t)((const u16*)row)[n + j] << (16 * (j & 1));
            else o[p][j] = ((const uint32_t*)row)[n + j];
          }
      }
    }
  }
  // ... and added to v
  __device__ __forceinline__ void add(float* v) const {
    if constexpr (io<T>::BYTES == 2) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t a0 = o[p][0], a1 = o[p][1], b0 = o[p][2], b1 = o[p][3];
        swap_halves(a0, b0);
        swap_halves(a1, b1);
        v[8 * p] += bf_lo(a0); v[8 * p + 1] += bf_hi(a0); v[8 * p + 2] += bf_lo(a1); v[8 * p + 3] += bf_hi(a1);
        v[8 * p + 4] += bf_lo(b0); v[8 * p + 5] += bf_hi(b0); v[8 * p + 6] += bf_lo(b1); v[8 * p + 7] += bf_hi(b1);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * q + j] += __uint_as_float(o[q][j]);
    }
  }
};

// The lane's 16 columns of a bias (the same for every row; 0 without one).
template <bool INNER>
__device__ __forceinline__ void tile_bias(const float* bias, int64_t n0, int64_t N, float* b, int h) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 8 * q + 4 * h;
    if (!bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[4 * q + j] = 0.0f;
    } else if (INNER) {
      const f32x4 x = *(const f32x4_any*)(bias + n);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[4 * q + j] = x[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[4 * q + j] = bias[n + j < N ? n + j : N - 1];
    }
  }
}

// The epilogue of COUNT tiles below each other (rows 32 apart from m on) in
// columns n0 .. n0 + 31; get(j, z, u) yields tile j's values (u: the second
// half's of a gated block).  What has to be loaded is requested first.
template <typename T, int EPI, int ACT, int COUNT, bool INNER, typename Get>
__device__ __forceinline__ void tile_column(const MmArgs& a, int64_t m, int64_t n0, int h, Get&& get) {
  constexpr int ES = io<T>::BYTES;
  constexpr bool FINE = ES == 4, G = EPI == MM_GATED;
  if (!INNER && n0 >= a.N) return;
  float b0[16], b1[16];
  TileRow<T> res[COUNT];
  asm volatile("" ::: "memory");  // this column's loads are not requested earlier: registers
  if constexpr (EPI != MM_STORE) tile_bias<INNER>(a.bias, n0, a.N, b0, h);
  if constexpr (G) tile_bias<INNER>(a.bias ? a.bias + a.N : nullptr, n0, a.N, b1, h);
  if constexpr (EPI == MM_LINEAR)
    if (a.res) {
#pragma unroll
      for (int j = 0; j < COUNT; ++j) {
        const int64_t r = m + 32 * j;
        res[j].template load<INNER>((const char*)a.res + (INNER || r < a.M ? r : a.M - 1) * a.ldr * ES, r < a.M, n0,
                                    a.N, h);
      }
    }
#pragma unroll
  for (int j = 0; j < COUNT; ++j) {
    const bool in = m + 32 * j < a.M;
    const int64_t r = INNER || in ? m + 32 * j : a.M - 1;
    float z[16], u[16];
    get(j, z, u);
    if constexpr (EPI == MM_LINEAR) {
#pragma unroll
      for (int v = 0; v < 16; ++v) z[v] += b0[v];
      if (a.pre) tile_store<T, INNER>((char*)a.pre + r * a.N * ES, in, n0, a.N, z, h);
#pragma unroll
      for (int v = 0; v < 16; ++v) z[v] = act_fwd<ACT, FINE>(z[v]);
      if (a.res) res[j].add(z);
    }
    if constexpr (G) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        z[v] += b0[v];
        u[v] += b1[v];
      }
      if (a.pre) {
        char* row = (char*)a.pre + r * 2 * a.N * ES;
        tile_store<T, INNER>(row, in, n0, a.N, z, h);
        tile_store<T, INNER>(row + a.N * ES, in, n0, a.N, u, h);
      }
#pragma unroll
      for (int v = 0; v < 16; ++v) z[v] = act_fwd<ACT, FINE>(z[v]) * u[v];
    }
    tile_store<T, INNER>((char*)a.out + r * a.ldo * ES, in, n0, a.N, z, h);
  }
}

// Instruction order of a k-step: the LDS reads for the next one spread over
// the first half of its matrix instructions (so that they have arrived by its
// end), the loads of a later stage over the second half.
template <int MASK, int STEPS, int COUNT, int I = 0>
__device__ __forceinline__ void mix() {  // COUNT instructions of the kind over STEPS products
  if constexpr (I < STEPS) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int N = (I + 1) * COUNT / STEPS - I * COUNT / STEPS;
    if constexpr (N > 0) __builtin_amdgcn_sched_group_barrier(MASK, N, 0);
    mix<MASK, STEPS, COUNT, I + 1>();
  }
}
template <int NM, int NR, int NL>
__device__ __forceinline__ void mix_k_step() {
  mix<0x100, NM / 2, NR>();
  mix<0x010, NM - NM / 2, NL>();
}

// ---------------------------------------------------------------------------
// The smaller tiles, BM x BN outputs (gated: BN / 2 columns of each half) of
// four waves, each BM / 2 x BN / 2 of them on 32 x 32 products: what has too
// few 256 x 256 tiles to fill the chip.
//
// k advances by 128 bytes per stage through NBUF stages of LDS.  A stage has
// four k-steps of 32 bytes; a wave reads the fragments of the next two k-steps
// while the products of these two run, across the stage's end too: half way through, every wave holds the second half's
// fragments in registers, so one barrier there frees this stage's LDS for the
// loads of NBUF stages later and publishes the next stage, whose first
// fragments are read under the second half's products.
//
// Blocks stay: each walks several items (a tile, or a tile's part of k), and
// the stage after an item's last is the next item's first, so that its loads
// are in flight during the epilogue.
//
// PER blocks share a CU: two where there are more items than CUs; where a
// block is alone on its CU, nobody covers its waits, and it takes all of the
// LDS for a pipeline twice as deep (dx and dW of 4096 x 1024 -> 4096, 128 x 128
// tiles, one per CU: 61 and 51 -> 41 us each, 0.83 PFLOP/s).  The matrix cores
// work about a third of the time there; the tiles' 537 MB of operands come in
// at 13 TB/s, 81 % of the requests met in the L2 and 101 MB from beyond it.
// ---------------------------------------------------------------------------
struct MmItem {
  int64_t m0, n0;  // first row and column of out
  int kb;          // first stage
  int part;        // index of the partial tile, -1: whole
};

template <int BM, int BC>
__device__ __forceinline__ MmItem mm_item(const MmPlan& pl, int id) {
  // tiles in groups of 4 rows of tiles, column after column
  int tile = id, part = -1, kb = 0;
  if (id >= pl.full) {
    const int r = id - pl.full, cut = pl.ntm * pl.ntn - pl.full;
    tile = pl.full + r % cut;
    part = r;
    kb = r / cut * pl.stages;
  }
  const int group = tile / (4 * pl.ntn), first = group * 4, rows = pl.ntm - first < 4 ? pl.ntm - first : 4;
  const int rest = tile - group * 4 * pl.ntn;
  return {(int64_t)(first + rest % rows) * BM, (int64_t)(rest / rows) * BC, kb, part};
}

// Workgroups go to the 8 XCDs in turn; each XCD gets a contiguous run of the
// whole tiles and one of the parts, so that its blocks in flight share operand
// tiles in its L2.
struct MmWalk {
  int id, step, f0, nf, p0, end;  // the block's items: id, id + step, ... below end
  // block of blocks; block 0 is on the first XCD of its eight
  __device__ __forceinline__ MmWalk(const MmPlan& pl, int block, int blocks) {
    const int xcd = block & 7;
    id = block >> 3;
    auto first = [&](int n) { return xcd * (n >> 3) + (xcd < (n & 7) ? xcd : (n & 7)); };
    auto count = [&](int n) { return (n >> 3) + (xcd < (n & 7) ? 1 : 0); };
    step = (blocks + 7 - xcd) >> 3;  // blocks of this XCD
    f0 = first(pl.full);
    nf = count(pl.full);
    p0 = pl.full + first(pl.items - pl.full);
    end = nf + count(pl.items - pl.full);
  }
  template <int BM, int BC>
  __device__ __forceinline__ MmItem item(const MmPlan& pl, int v) const {
    return mm_item<BM, BC>(pl, v < nf ? f0 + v : p0 + v - nf);
  }
};

// The values of an accumulator tile.  A 256 x 256 tile's leave the
// accumulation registers here and not before: left to the compiler, copies of
// all of them are made at the loop's end, and spilled.  (The caller has waited
// for the last product: mm_drain.)
template <bool WIDE>
__device__ __forceinline__ void acc_values(const f32x16& acc, float* z) {
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    if constexpr (WIDE) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(z[v]) : "a"(acc[v]));
    else z[v] = acc[v];
  }
}
// More wait states than any product's latency; the compiler does not know
// that acc_values reads what a product wrote.
__device__ __forceinline__ void mm_drain() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The end of an item: its epilogue, or its part's sums to the workspace.
template <typename T, int EPI, int ACT, int BM, int BN>
__device__ __forceinline__ void mm_finish(const MmArgs& a, const MmItem& it, f32x16 (&acc)[BN / 64][BM / 64], int lane,
                                          int wave) {
  constexpr bool G = EPI == MM_GATED;
  constexpr int MT = BM / 64, NT = BN / 64, BC = G ? BN / 2 : BN;
  const int h = lane >> 5, wm = wave & 1, wn = wave >> 1;
  if (it.part >= 0) {
    f32x4* part = (f32x4*)a.part + (int64_t)it.part * (BM * BN / 4) + wave * 64 + lane;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        float z[16];
        acc_values<BM == 256>(acc[i][j], z);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          part[((i * MT + j) * 4 + v) * 256] = f32x4{z[4 * v], z[4 * v + 1], z[4 * v + 2], z[4 * v + 3]};
      }
    return;
  }
  const int64_t m = it.m0 + wm * (BM / 2) + (lane & 31);
  auto columns = [&](auto inner) {
#pragma unroll
    for (int i = 0; i < (G ? NT / 2 : NT); ++i)
      tile_column<T, EPI, ACT, MT, decltype(inner)::value>(
          a, m, it.n0 + wn * (BC / 2) + i * 32, h, [&](int j, float* z, float* u) {
            acc_values<BM == 256>(acc[i][j], z);
            if constexpr (G) acc_values<BM == 256>(acc[i + NT / 2][j], u);
          });
  };
  if (it.m0 + BM <= a.M && it.n0 + BC <= a.N) columns(std::integral_constant<bool, true>{});
  else columns(std::integral_constant<bool, false>{});
}

template <typename T, int LAYOUT, int EPI, int ACT, int BM, int BN, int NBUF>
__device__ __forceinline__ void mm_tile_walk(const MmArgs& a, const MmPlan& pl, char* smem, int block, int blocks) {
  constexpr bool PK = LAYOUT != MM_NONE_K, QK = LAYOUT == MM_PQ_K;
  constexpr int ES = io<T>::BYTES;
  constexpr bool G = EPI == MM_GATED;
  constexpr int MT = BM / 64, NT = BN / 64;  // 32 x 32 tiles of a wave
  constexpr int BC = G ? BN / 2 : BN;        // columns of out per tile
  typedef Operand<T, PK, BM> OP;
  typedef Operand<T, QK, BN> OQ;
  constexpr int STAGE = OP::BYTES + OQ::BYTES;

  const MmWalk walk(pl, block, blocks);
  int id = walk.id;
  if (id >= walk.end) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  OP op;
  OQ oq;
  op.init(a.ldp, lane, wave);
  oq.init(a.ldq, lane, wave);
  auto load = [&](const MmItem& it, int kb, int at) {
    char* l = smem + at;
    const char* pb = (const char*)a.P + (PK ? it.m0 * a.ldp : it.m0) * ES;
    const char* qb = (const char*)a.Q + (QK ? it.n0 * a.ldq : it.n0) * ES;
    const int64_t pr = a.M - it.m0, qr = a.N - it.n0;
    op.template load<0, OP::NI>(pb, pr, a.K, kb, l, wave);
    if constexpr (G) {
      const char* qb2 = (const char*)a.Q + (a.N + it.n0) * a.ldq * ES;  // the second half's rows
      oq.template load<0, OQ::NI / 2>(qb, qr, a.K, kb, l + OP::BYTES, wave);
      oq.template load<OQ::NI / 2, OQ::NI>(qb2, qr, a.K, kb, l + OP::BYTES, wave);
    } else {
      oq.template load<0, OQ::NI>(qb, qr, a.K, kb, l + OP::BYTES, wave);
    }
  };
  Fragments<T, PK, BM, MT, 0> fp;
  Fragments<T, QK, BN, NT, G ? BN / 4 : 0> fq;
  fp.init(wm * (BM / 2), lane);
  fq.init(G ? wn * (BN / 4) : wn * (BN / 2), lane);

  f32x16 acc[NT][MT];
  // of two k-steps: matrix instructions and LDS reads
  constexpr int NM = 2 * MT * NT * (ES == 2 ? 1 : 4);
  constexpr int NR = 2 * (MT * (PK ? 1 : ES == 2 ? 2 : 4) + NT * (QK ? 1 : ES == 2 ? 2 : 4));
  uint4 p[2][2][MT], q[2][2][NT];
  auto read = [&](int at, int half) {  // k-steps 2 half, 2 half + 1
    const char* l = smem + at;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < MT; ++j) p[half][s][j] = fp.read(l, j, 2 * half + s);
#pragma unroll
      for (int i = 0; i < NT; ++i) q[half][s][i] = fq.read(l + OP::BYTES, i, 2 * half + s);
    }
  };
  auto multiply = [&](int half) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = mma32<T>(q[half][s][i], p[half][s][j], acc[i][j]);
  };
  // the loads run ahead of the products: the item and stage they are at
  int lid = id;
  MmItem lt = walk.item<BM, BC>(pl, id);
  int lk = 0, ln = lt.part < 0 ? pl.whole : pl.stages;
  auto advance = [&] {
    if (++lk < ln) return;
    lk = 0;
    lid += walk.step;
    if (lid < walk.end) {
      lt = walk.item<BM, BC>(pl, lid);
      ln = lt.part < 0 ? pl.whole : pl.stages;
    } else {  // nothing left: stages past K, which read zeros
      lt.kb = pl.whole;
      ln = 0x7fffffff;
    }
  };
  constexpr int NL = OP::NI + OQ::NI;    // loads of a stage
  constexpr int AHEAD = (NBUF - 2) * NL;  // in flight past the stage that comes next
  static_assert(AHEAD + NL < 64, "vmcnt");
  auto settle = [&](auto n) {
    constexpr int N = decltype(n)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < NBUF; ++i) {
    load(lt, lt.kb + lk, i * STAGE);
    advance();
  }
  settle(std::integral_constant<int, AHEAD + NL>{});
  read(0, 0);
  int at = 0;
  for (; id < walk.end; id += walk.step) {
    const MmItem it = walk.item<BM, BC>(pl, id);
    const int nk = it.part < 0 ? pl.whole : pl.stages;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    for (int kb = 0; kb < nk; ++kb) {
      const int nxt = at == (NBUF - 1) * STAGE ? 0 : at + STAGE;
      read(at, 1);
      multiply(0);
      mix_k_step<NM, NR, 0>();
      settle(std::integral_constant<int, AHEAD>{});
      read(nxt, 0);
      load(lt, lt.kb + lk, at);
      multiply(1);
      mix_k_step<NM, NR, NL>();
      __builtin_amdgcn_sched_barrier(0);
      advance();
      at = nxt;
    }
    // opaque, so that the epilogue's addresses are not kept in registers
    // across the products
    int el = lane, ew = wave;
    asm volatile("" : "+v"(el), "+s"(ew));
    mm_finish<T, EPI, ACT, BM, BN>(a, it, acc, el, ew);
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the loads past the last item (zeros) have landed
}

template <typename T, int LAYOUT, int EPI, int ACT, int BM, int BN, int NBUF, int PER>
__global__ __launch_bounds__(256, PER) void mm_tile_kernel(MmArgs a, MmPlan pl) {
  static_assert(PER * NBUF * (BM + BN) * 128 <= 163840, "blocks per CU");
  __shared__ __attribute__((aligned(1024))) char smem[NBUF * (BM + BN) * 128];
  mm_tile_walk<T, LAYOUT, EPI, ACT, BM, BN, NBUF>(a, pl, smem, blockIdx.x, gridDim.x);
}

// Both products of a small backward in one launch (each launch costs the host
// as long as such a product takes): the first `na` blocks do dx, the others
// dW.
template <typename T>
__global__ __launch_bounds__(256, 2) void mm_pair_kernel(MmArgs a, MmPlan pa, MmArgs b, MmPlan pb, int na) {
  __shared__ __attribute__((aligned(1024))) char smem[4 * 128 * 128];
  if ((int)blockIdx.x < na) mm_tile_walk<T, MM_P_K, MM_STORE, ACT_NONE, 64, 64, 4>(a, pa, smem, blockIdx.x, na);
  else mm_tile_walk<T, MM_NONE_K, MM_STORE, ACT_NONE, 64, 64, 4>(b, pb, smem, blockIdx.x - na, gridDim.x - na);
}

// Adds the parts of the split tiles in order and applies the epilogue: one
// block per tile and 32 x 32 piece of each wave.  Bound by the parts' traffic: 96
// tiles of 256 x 256 in 23 us, 312 fp32 tiles of 64 x 64 and less in 10.
template <typename T, int EPI, int ACT, int BM, int BN>
__global__ __launch_bounds__(256) void mm_join_kernel(MmArgs a, MmPlan pl) {
  constexpr bool G = EPI == MM_GATED;
  constexpr int MT = BM / 64, NT = BN / 64, BC = G ? BN / 2 : BN, PIECES = MT * (G ? NT / 2 : NT);
  const int r = blockIdx.x / PIECES, piece = blockIdx.x % PIECES, i = piece / MT, j = piece % MT;
  const int cut = pl.ntm * pl.ntn - pl.full;
  const MmItem it = mm_item<BM, BC>(pl, pl.full + r);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float z[16], u[16];
#pragma unroll
  for (int v = 0; v < 16; ++v) z[v] = u[v] = 0.0f;
#pragma unroll 8  // loads of several parts in flight: up to 64 parts of few tiles
  for (int s = 0; s < pl.split; ++s) {
    const f32x4* part = (const f32x4*)a.part + ((int64_t)s * cut + r) * (BM * BN / 4) + tid;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const f32x4 x = part[((i * MT + j) * 4 + v) * 256];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[4 * v + e] += x[e];
      if constexpr (G) {
        const f32x4 y = part[(((i + NT / 2) * MT + j) * 4 + v) * 256];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[4 * v + e] += y[e];
      }
    }
  }
  const int64_t m = it.m0 + (wave & 1) * (BM / 2) + j * 32 + (lane & 31);
  auto finish = [&](auto inner) {
    tile_column<T, EPI, ACT, 1, decltype(inner)::value>(a, m, it.n0 + (wave >> 1) * (BC / 2) + i * 32, lane >> 5,
                                                        [&](int, float* zz, float* uu) {
#pragma unroll
                                                          for (int v = 0; v < 16; ++v) {
                                                            zz[v] = z[v];
                                                            uu[v] = u[v];
                                                          }
                                                        });
  };
  if (it.m0 + BM <= a.M && it.n0 + BC <= a.N) finish(std::integral_constant<bool, true>{});
  else finish(std::integral_constant<bool, false>{});
}

}  // namespace m3
