// What the kernels of windowed attention share: which keys a query sees, the
// order of the work, and tiles of rows in LDS read as matrix operands both ways.
//
// All products are 32 x 32 tiles (mma32 of mm_tile.hpp).  A product's result
// has its columns over the lanes (lane l: column l mod 32) and its rows in
// registers (v[4 q + j]: row 8 q + 4 (l / 32) + j).  The first product is laid
// so that what the softmax runs over, and what the second product sums over,
// are the rows: the second product's operand is then the lane's own registers,
// without any exchange, when the other operand's rows come in that order too
// (Tile::col).
#pragma once

#include "m3_lanes.hpp"
#include "mm_tile.hpp"

namespace m3 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFar = 0x7ff00000;  // an offset past every buffer: reads as zero

// A sequence's rows.
struct AttnSeq {
  int64_t q0, k0;  // first row of its queries and keys
  int nq, nk;
  int64_t id;
  // position of its query r: past() + r; its keys' are 0 .. nk - 1
  __device__ __forceinline__ int past() const { return nk - nq; }
};

__device__ __forceinline__ int64_t start_of(const AttnArgs& a, int64_t i) {
  const int64_t s = a.starts[i];
  return s < 0 ? 0 : s > a.rows ? a.rows : s;
}

// Item `flat` (below 2^32) of all sequences' tiles of `tile` rows, longer than `over` rows
// (queries, or keys with KEYS): the sequence and the tile within it.  false:
// there are fewer.  Every lane of a wave calls it with the same arguments.
template <bool KEYS>
__device__ __forceinline__ bool attn_item(const AttnArgs& a, int64_t flat, int tile, int over, AttnSeq& s, int& t) {
  if (!a.starts) {
    const int n = KEYS ? a.kv_len : a.q_len;
    const int per = n > over ? (n + tile - 1) / tile : 0;
    if (per == 0) return false;
    s.id = (uint32_t)flat / (uint32_t)per;
    if (s.id >= a.batch) return false;
    t = (int)(flat - s.id * per);
    s.q0 = s.id * a.q_len;
    s.k0 = s.id * a.kv_rows;
    s.nq = a.q_len;
    s.nk = a.kv_len;
    return true;
  }
  const int lane = threadIdx.x & 63;
  for (int64_t b = 0; b < a.batch; b += 64) {
    int64_t lo = 0, n = 0;
    if (b + lane < a.batch) {
      lo = start_of(a, b + lane);
      n = start_of(a, b + lane + 1) - lo;
    }
    const int mine = n > over ? (int)((n + tile - 1) / tile) : 0;
    int sum = mine;  // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int x = __shfl_up(sum, o, 64);
      if (lane >= o) sum += x;
    }
    const uint64_t beyond = __ballot(flat < sum);
    if (beyond) {
      const int w = __builtin_ctzll(beyond);
      s.id = b + w;
      s.q0 = s.k0 = ((int64_t)__builtin_amdgcn_readlane((int)(lo >> 32), w) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)lo, w);
      s.nq = s.nk = __builtin_amdgcn_readlane((int)n, w);
      t = (int)flat - (__builtin_amdgcn_readlane(sum, w) - __builtin_amdgcn_readlane(mine, w));
      return true;
    }
    flat -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}
// At most as many items there are.
inline int64_t attn_items(const AttnArgs& a, bool keys, int tile) {
  if (!a.starts) return a.batch * (((keys ? a.kv_len : a.q_len) + tile - 1) / tile);
  return a.rows / tile + (a.batch < a.rows ? a.batch : a.rows);
}

// Which kernel of queries' blocks a call takes, by f(heads of a block, waves that
// share tiles of keys, parts of the keys).  Blocks of four waves, 128 queries of
// a head, that are no more than the chip's CUs leave half of each idle, or more.
// Their keys are then walked in parts by waves of their own (1 x 2048 queries, 16
// heads of 128, no window: forward 42.5 -> 36.5 us, dq 57 -> 49; with 512 keys or
// fewer for a query what the parts' join costs is not made up for: 300 queries
// 8.4 -> 8.8).  fp32 kernels, bound by their products, first take blocks of one
// wave (2 x 777 queries, 5 heads of 72, window 100: forward 35 -> 28 us, dq 53 ->
// 36), and of several parts while those leave CUs idle: in four parts 15 and 18; 1 x
// 1500, 8 heads of 64, no window, in two 68 and 90 instead of 110 and 159.
template <typename T, typename F>
void attn_by_size(const AttnArgs& a, F&& f) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, 4> four;
  const int G = a.q_heads / a.kv_heads;
  const int64_t blocks = attn_items(a, false, 128) * a.q_heads;
  if constexpr (io<T>::BYTES == 4) {
    if (blocks < 256) {
      const int64_t waves = attn_items(a, false, 32) * a.q_heads;
      if (waves <= 256) f(one, one, four);
      else if (waves <= 512) f(one, one, two);
      else f(one, one, one);
      return;
    }
  } else if (blocks <= 256 && (a.starts ? a.rows : (int64_t)a.kv_len) > 512 && a.window > 512) {
    if (G % 4 == 0) f(four, four, two);
    else if (G % 2 == 0) f(two, four, two);
    else f(one, four, two);
    return;
  }
  if (G % 4 == 0) f(four, four, one);
  else if (G % 2 == 0) f(two, four, one);
  else f(one, four, one);
}
// Pieces of the sequences that are longer than one, at most: every whole piece of
// all rows, and one that is not whole for each such sequence.
inline int64_t attn_pieces(const AttnArgs& a) {
  if (a.sinks == 0 || a.window >= kNoWindow) return 0;
  if (!a.starts) return a.q_len > a.piece ? a.batch * ((a.q_len + a.piece - 1) / a.piece) : 0;
  const int64_t whole = a.rows / a.piece;
  return whole + (a.batch < whole ? a.batch : whole);
}

inline int64_t attn_piece_blocks(const AttnArgs& a) { return attn_pieces(a) * ((a.sinks + 31) / 32) * a.kv_heads; }

// Blocks go to the 8 XCDs in turn, each with an L2 of its own: XCD x gets the
// x-th contiguous eighth of the work, whose neighbours share keys and values.
__device__ __forceinline__ uint32_t xcd_order(uint32_t i, uint32_t n) {
  const uint32_t x = i & 7, per = n >> 3, rem = n & 7;
  return x * per + (x < rem ? x : rem) + (i >> 3);
}

// Position p sees key j when j <= p and (j > p - window or j < sinks).  Which of
// a lane's rows of scores that is, with both taken from where the rows start
// (lengths stay below 2^24): three comparisons with a constant each.
struct KeysSeen {
  int last, out, sinks;
  __device__ __forceinline__ KeysSeen(const AttnArgs& a, int p, int j0)
      : last(p - j0), out(p - j0 - a.window), sinks(a.sinks - j0) {}
  __device__ __forceinline__ bool operator()(int k) const { return (k <= last) & ((k > out) | (k < sinks)); }
};
// ... where the rows are positions, from p0 on
struct QueriesSeeing {
  int first, end;
  __device__ __forceinline__ QueriesSeeing(const AttnArgs& a, int p0, int j)
      : first(j - p0), end(j < a.sinks ? 1 << 30 : j - p0 + a.window) {}
  __device__ __forceinline__ bool operator()(int k) const { return (k >= first) & (k < end); }
};
// Whether every key of [j0, j1] is seen from every position of [p0, p1].
__device__ __forceinline__ bool sees_all(int p0, int p1, int j0, int j1, int window, int sinks) {
  return j1 <= p0 && (p1 - j0 < window || j1 < sinks);
}
// ... none
__device__ __forceinline__ bool sees_none(int p0, int p1, int j0, int j1, int window, int sinks) {
  return j0 > p1 || (p0 - j1 >= window && j0 >= sinks);
}

// ROWS rows of DP entries in LDS, 16-byte chunk c of row r at chunk c ^ f(r):
// f spreads the 16 rows of a row read over all banks, and the 4 rows of a
// transposed read over the quarters of them.  Filled straight from memory by
// NW waves; entries past the width and rows past the last read as zero.  DU: the
// entries that products take, where fewer than DP do.
template <typename T, int DP, int DU, int ROWS, int NW>
struct Tile {
  static constexpr int ES = io<T>::BYTES;
  static constexpr int ROWB = DP * ES;
  static constexpr int BYTES = ROWS * ROWB;
  static constexpr int LPR = ROWB / 16;           // lanes per row
  static constexpr int RPI = 64 / LPR;            // rows per 1 KB load
  static constexpr int NI = BYTES / 1024 / NW;    // loads per wave
  static constexpr int KS = DU * ES / 32;         // steps of a product over a row
  static constexpr int CT = DU / 32;              // tiles of a product whose result's rows are the columns
  static constexpr int CK = ES == 2 ? 16 : 8;     // rows a step of such a product takes
  static constexpr int NV = RPI * NW % 16 == 0 ? 1 : 16 / (RPI * NW);  // loads until f repeats
  static_assert(BYTES % (1024 * NW) == 0 && LPR <= 64, "whole loads");

  __device__ __forceinline__ static int f(int r) {
    if constexpr (ES == 4) return (r & 7) << 1;
    else if constexpr (LPR == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return ((r & 3) << 2) | ((r >> 2) & 3);
  }

  int voff[NV];
  int ldb;
  int row_at, col_at[ES == 2 ? 2 : 4];
  int fx;

  // ld: entries from row to row in memory; width: entries a row has
  __device__ __forceinline__ void init(int64_t ld, int width, int lane, int wave) {
    ldb = (int)(ld * ES);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = (i * NW + wave) * RPI + lane / LPR, c = (lane % LPR) ^ f(row);
      voff[i] = c * 16 < width * ES ? (wave * RPI + lane / LPR) * ldb + c * 16 : kFar;
    }
    const int r = lane & 31, h = lane >> 5;
    row_at = r * ROWB + ((h ^ f(r)) << 4);  // step s: the chunk's other bits are flipped by 2 s
    if constexpr (ES == 2) {
      const int q = (lane & 15) >> 2, c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + 4 * h + q;
        col_at[i] = row * ROWB + ((c ^ f(row)) << 4) + (lane & 1) * 8;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * h + i;
        col_at[i] = row * ROWB + (((r >> 2) ^ f(row)) << 4) + (r & 3) * 4;
      }
    }
  }
  // base: the first row; rows: that exist, from 1.  Device code only: a second
  // kernel that calls this loses its host stub, without an error, where the
  // host's pass meets the builtins.
  __device__ __forceinline__ void load(const char* base, int rows, int width, char* lds, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)
    const int n = rows < ROWS ? rows : ROWS;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (uint32_t)((n - 1) * ldb + width * ES), 0x00020000);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + (i * NW + wave) * 1024), 16, voff[i % NV],
                                               i * NW * RPI * ldb, 0, 0);
#endif
  }
  // ... its rows [32 t, 32 t + 32) alone; rows: 0 or fewer read nothing
  __device__ __forceinline__ void load32(const char* base, int rows, int width, char* lds, int wave, int t) const {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int N = 32 / (NW * RPI);
    static_assert(N * NW * RPI == 32, "whole loads");
    const int n = rows < 32 ? rows : 32;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)base, 0, n > 0 ? (uint32_t)((n - 1) * ldb + width * ES) : 0u, 0x00020000);
#pragma unroll
    for (int i = 0; i < N; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + ((t * N + i) * NW + wave) * 1024), 16,
                                               voff[(t * N + i) % NV], i * NW * RPI * ldb, 0, 0);
#endif
  }
  // rows [32 t, 32 t + 32) as an operand whose sum runs over the columns, step s
  __device__ __forceinline__ uint4 row(const char* lds, int t, int s) const {
    return __builtin_bit_cast(uint4, read16((const u32x4*)(lds + ((row_at ^ (s << 5)) + t * 32 * ROWB))));
  }
  // columns [32 t, 32 t + 32) as an operand whose sum runs over the rows, step
  // ks: rows CK ks .. + CK - 1 in the order in which a product's result holds
  // its rows
  __device__ __forceinline__ uint4 col(const char* lds, int t, int ks) const {
    const char* p = lds + ks * CK * ROWB;
    if constexpr (ES == 2) {
      const uint2 a = read_tr(p + (col_at[0] ^ (t << 6))), b = read_tr(p + (col_at[1] ^ (t << 6)));
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      return make_uint4(read4((const uint32_t*)(p + (col_at[0] ^ (t << 7)))),
                        read4((const uint32_t*)(p + (col_at[1] ^ (t << 7)))),
                        read4((const uint32_t*)(p + (col_at[2] ^ (t << 7)))),
                        read4((const uint32_t*)(p + (col_at[3] ^ (t << 7)))));
    }
  }
};

// 32 rows from memory as the other operand of a product over their columns:
// lane l holds row l mod 32.  in: that row exists.
template <typename T, int DU>
struct RowRegs {
  static constexpr int KS = DU * io<T>::BYTES / 32;
  uint4 v[KS];
  __device__ __forceinline__ void load(const char* row, bool in, int width, int h) {
    constexpr int V = io<T>::VEC;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      v[s] = make_uint4(0u, 0u, 0u, 0u);
      if (in && (2 * s + h) * V < width) v[s] = *(const uint4*)(row + (2 * s + h) * 16);
    }
  }
};

// The same for consecutive rows, which may be requested ahead of their use.
template <typename T, int DU>
struct RowStream {
  static constexpr int KS = DU * io<T>::BYTES / 32;
  uint4 v[KS];
  int voff, ldb, last;  // last: chunks of a row past it do not exist
  __device__ __forceinline__ void init(int64_t ld, int width, int lane) {
    ldb = (int)(ld * io<T>::BYTES);
    voff = (lane & 31) * ldb + (lane >> 5) * 16;
    last = width * io<T>::BYTES / 16 - (lane >> 5);
  }
  // base: the first of `rows` rows (from 1, 32 at most); others read as zero
  __device__ __forceinline__ void load(const char* base, int rows, int width) {
#if defined(__HIP_DEVICE_COMPILE__)
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)base, 0, (uint32_t)((rows - 1) * ldb + width * io<T>::BYTES), 0x00020000);
#pragma unroll
    for (int s = 0; s < KS; ++s)
      v[s] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, 2 * s < last ? voff + s * 32 : kFar, 0, 0));
#endif
  }
};

// Step ks of a result (its rows 16 ks .. or 8 ks ..) as the operand that goes
// with Tile::col.  For bf16 operands the weights p and the gradients ds are rounded
// to bf16 here, once each, to the nearest: the matrix cores take fp32 at an eighth of
// the rate, and what goes with them holds no more bits either.  Outputs are then 2.0 to
// 2.6e-3 off the exact values, where their own rounding alone makes 1.5 to 1.8e-3.
template <typename T>
__device__ __forceinline__ uint4 result_step(const float* v, int ks) {
  if constexpr (io<T>::BYTES == 2) {
    const float* p = v + 8 * ks;
    return make_uint4(pack_bf2(p[0], p[1]), pack_bf2(p[2], p[3]), pack_bf2(p[4], p[5]), pack_bf2(p[6], p[7]));
  } else {
    const float* p = v + 4 * ks;
    return make_uint4(__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3]));
  }
}

// N products, the fragment of each read from LDS (READS instructions) AHEAD
// products before its use: left to itself the compiler reads it right before,
// and every product waits for LDS.
template <int AHEAD, int N, int READS, typename T, typename Read, typename Multiply>
__device__ __forceinline__ void ahead(Read&& read, Multiply&& multiply) {
  constexpr int RING = AHEAD + 1;
  uint4 f[RING];
#pragma unroll
  for (int i = 0; i < AHEAD && i < N; ++i) f[i % RING] = read(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + AHEAD < N) f[(i + AHEAD) % RING] = read(i + AHEAD);
    multiply(i, f[i % RING]);
  }
  if constexpr (io<T>::BYTES == 2) {
#pragma unroll
    for (int i = -AHEAD; i < N; ++i) {
      if (i >= 0) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      if (i + AHEAD < N) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    }
  }
}

// Calls f with DP and DU of a head's width: 32, 64, 96 or 128 entries in rows of
// 64 or 128.
template <typename F>
void with_width(int dim, F&& f) {
  const std::integral_constant<int, 32> c32;
  const std::integral_constant<int, 64> c64;
  const std::integral_constant<int, 96> c96;
  const std::integral_constant<int, 128> c128;
  if (dim <= 32) f(c64, c32);
  else if (dim <= 64) f(c64, c64);
  else if (dim <= 96) f(c128, c96);
  else f(c128, c128);
}

// Larger of lane l's and lane l ^ 32's.
__device__ __forceinline__ float max_halves(float v) {
  uint32_t a = __float_as_uint(v), b = a;
  asm volatile("" : "+v"(b));
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = s[0];
  b = s[1];
  asm volatile("" : "+v"(a), "+v"(b));
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

// This wave's loads into LDS have landed and its reads are done, and so it is
// with every wave of the block.
__device__ __forceinline__ void attn_settle() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// The same for loads and reads that no other wave has a part in.
__device__ __forceinline__ void attn_settle_alone() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// The softmax of 32 columns over rows that come in pieces: weights against a
// running reference m of each column, their sum, and the result's columns scaled
// along when m moves.
//
// m need not be the maximum: a weight may be as large as 2^12, where fp32
// sums and bf16 roundings are as exact as below 1.  So no maximum is taken while
// the sum of a piece's weights, which is needed anyway, stays below that; only
// when it does not is the piece weighed again, against its maximum.  (That moved
// 30 of 145 vector instructions out of a piece of 64 keys.)
template <int CT>
struct Softmax {
  float m, l;  // m of both halves of the wave, l of the lane's own rows
  __device__ __forceinline__ void init() {
    m = -INFINITY;
    l = 0.0f;
  }
  template <int NS>
  __device__ __forceinline__ static float weights(const float* s, float c, float mc, float* p) {
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // four chains: a lone wave waits for every dependent addition
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
      sum[i & 3] += p[i];
    }
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
  // p: weights of the NS scores s of the lane's column (-inf: not seen)
  template <int NS>
  __device__ __forceinline__ void step(const float* s, float c, f32x16 (&acc)[CT], float* p) {
    // before any score is met, m is as good as 0: what that yields is in order or too large
    float sum = weights<NS>(s, c, m == -INFINITY ? 0.0f : m * c, p);
    if (__any(sum > 0x1p12f || m == -INFINITY)) {
      float t = s[0];
#pragma unroll
      for (int i = 1; i < NS; ++i) t = fmaxf(t, s[i]);
      const float n = fmaxf(m, max_halves(t));
      const float scale = n == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - n) * c);
      m = n;
      l *= scale;
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] *= scale;
      sum = weights<NS>(s, c, m == -INFINITY ? 0.0f : m * c, p);
    }
    l += sum;
  }
};

// The results of a block's KW parts of the keys, joined in order by the first
// part's waves (true for them): sums acc, and for a softmax (SOFT) its reference
// m and sum l.  Each part leaves its sums in its own BYTES of LDS.
template <int KW, int NW, int BYTES, bool SOFT, int CT>
__device__ __forceinline__ bool join_parts(char* lds, f32x16 (&acc)[CT], float& m, float& l, float c, int part,
                                           int wave, int lane) {
  static_assert(NW * CT * 4096 <= BYTES, "a part's sums fit its LDS");
  __shared__ float stat[SOFT ? KW : 1][NW][2][64];
  attn_settle();  // the tiles are read
  if (part > 0) {
    f32x4* x = (f32x4*)(lds + part * BYTES + wave * CT * 4096) + lane;
#pragma unroll
    for (int i = 0; i < CT * 4; ++i) {
      const f32x16& o = acc[i / 4];
      const int e = i % 4 * 4;
      x[i * 64] = f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
    }
    if constexpr (SOFT) {
      stat[part][wave][0][lane] = m;
      stat[part][wave][1][lane] = l;
    }
  }
  __syncthreads();
  if (part > 0) return false;
  float f[KW];
  f[0] = 1.0f;
  if constexpr (SOFT) {
    float top = m;
#pragma unroll
    for (int k = 1; k < KW; ++k) top = fmaxf(top, stat[k][wave][0][lane]);
    f[0] = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * c);
    l *= f[0];
#pragma unroll
    for (int k = 1; k < KW; ++k) {
      const float other = stat[k][wave][0][lane];
      f[k] = other == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((other - top) * c);
      l += f[k] * stat[k][wave][1][lane];
    }
    m = top;
  }
#pragma unroll
  for (int i = 0; i < CT * 4; ++i) {
    f32x4 sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = acc[i / 4][i % 4 * 4 + e] * f[0];
#pragma unroll
    for (int k = 1; k < KW; ++k) {
      const f32x4 x = ((const f32x4*)(lds + k * BYTES + wave * CT * 4096))[i * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += SOFT ? f[k] * x[e] : x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i / 4][i % 4 * 4 + e] = sum[e];
  }
  return true;
}

}  // namespace m3
