// Windowed attention over a cache, both types, and the plans of the launches
// that the workspaces depend on.
#include "attn_decode.hpp"

namespace m3 {

template hipError_t launch_attn_decode<bf16_t>(const AttnDecodeArgs&, hipStream_t);
template hipError_t launch_attn_decode<float>(const AttnDecodeArgs&, hipStream_t);

// Enough blocks to occupy the chip, each wave with a tile of 32 slots at least;
// fewer than 16 tiles are one block's, which needs no second launch.  (One
// sequence, 4 heads of keys of 128: 512 slots in 4 splits 11.2 us, in 2 11.8, in 1
// 12.0; 384 in 3 10.9, in 1 10.6; 1024 in 8 10.9, in 4 12.7, in 1 17.9.  Twice as
// many blocks at a width of 64, as registers allow: 64 sequences of 1028 slots 37
// us instead of 32.)
int attn_decode_splits(int io_bf16, const AttnDecodeArgs& a) {
  const int64_t groups = ((int64_t)a.q_heads / a.kv_heads * a.tokens + 31) / 32;
  const int64_t blocks = a.batch * a.kv_heads * groups, room = io_bf16 || a.dim <= 64 ? 512 : 256;
  int64_t slots = a.capacity;
  if (a.window < kNoWindow && slots > (int64_t)a.sinks + a.window + a.tokens - 1)
    slots = (int64_t)a.sinks + a.window + a.tokens - 1;
  int64_t n = blocks > 0 ? (room + blocks - 1) / blocks : 1;
  const int64_t tiles = (slots + 31) / 32, most = tiles < 16 ? 1 : tiles / 4;
  n = n < most ? n : most;
  return n < 1 ? 1 : n < kMaxSplits ? (int)n : kMaxSplits;
}
size_t attn_decode_part_bytes(const AttnDecodeArgs& a) {
  return a.splits == 1 ? 0 : (size_t)a.batch * a.tokens * a.q_heads * a.splits * (a.dim + 2) * 4;
}

// Queries of a piece of 32 keys with sinks among them: a quarter of what sees a
// tile behind the sinks, so that the pieces, which come last, even out what the
// tiles leave (8 x 4096 queries, 16/4 heads of 128, window 1024: dk and dv 522 us,
// with halves 520, and first 541; 1 x 2048, window 512: 50, 55, 55), and so many that
// there are 8192 pieces at most.
int attn_bwd_piece(const AttnArgs& a) {
  int64_t n = ((a.window < (1 << 24) ? a.window : 1 << 24) + 128) / 4;
  const int64_t work = a.rows * ((a.sinks + 31) / 32) * a.kv_heads;
  if (n < 256) n = 256;
  if (n < work / 4096) n = work / 4096;
  n = (n + 127) / 128 * 128;
  return (int)(n < (1 << 25) ? n : 1 << 25);
}
// Blocks that share a tile of 128 keys (and a piece), where there are too few of
// those: two steps of queries for each at least.  (1 x 2048 queries, 16/4 heads of
// 64, no window: dk and dv 176 us with one, 47 with six; from 192 tiles on one each
// is faster: 4 x 2048, window 512, 103 us, 124 with two.  With the pieces counted
// 1 x 2048, 16/4 x 128, window 512, has 5 instead of 6: 61 -> 55 us.)  In fp32 a
// wide head's block has a CU to itself, so one round of the chip is best: 4 x 512
// queries, 2 heads of 128, window 64, with four 38 us, 60 with two; 2 x 777, 5 heads
// of 72, with two 47 us, 55 with four.  Of packed sequences every whole piece counts
// twice: what most leave of the chip is too little for more (8000 queries in one,
// 8/2 heads of 128, window 64: 64 us with the two that this gives, 76 with three).
int attn_bwd_splits(int io_bf16, const AttnArgs& a) {
  const int64_t blocks = attn_items(a, true, 128) * a.kv_heads;
  if (blocks == 0 || blocks >= 192) return 1;
  int64_t rows = a.starts ? a.rows : a.q_len;
  if (a.window < kNoWindow && rows > (int64_t)a.window + 128) rows = (int64_t)a.window + 128;
  const int64_t step = io_bf16 ? 64 : 32, most = (rows + step - 1) / step * (a.q_heads / a.kv_heads) / 2;
  int64_t pieces = attn_piece_blocks(a);
  if (a.starts && pieces > 0) pieces = a.rows / a.piece * 2 * ((a.sinks + 31) / 32) * a.kv_heads;
  const int64_t busy = blocks + pieces;
  int64_t n = io_bf16 ? (384 + busy - 1) / busy : (a.dim > 64 ? 256 : 512) / busy;
  n = n < most ? n : most;
  return n < 1 ? 1 : n < 16 ? (int)n : 16;
}
size_t attn_bwd_part_bytes(const AttnArgs& a) {
  const int64_t shared = a.splits > 1 ? attn_items(a, true, 128) * a.kv_heads : 0;
  return (size_t)(attn_piece_blocks(a) + shared) * a.splits * 8 * 32 * a.dim * 4;
}

}  // namespace m3
