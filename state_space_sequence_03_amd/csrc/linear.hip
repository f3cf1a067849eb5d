// Plans and dispatch of the matrix products of the linear and gated
// feed-forward operators.
#include "mm_parts.hpp"

namespace m3 {

MmPlan mm_plan(int io_bf16, MmEpilogue epi, int64_t M, int64_t N, int64_t K) {
  MmPlan p{};
  if (epi != MM_STORE && M <= MM_FEW_ROWS) return p;
  const int es = io_bf16 ? 2 : 4;
  const int total = (int)((K * es + 127) / 128);  // stages of 128 bytes
  auto even = [](int v) { return v + (v & 1); };
  const int gated = epi == MM_GATED ? 2 : 1;
  auto cut = [&](int tile) {
    const int bc = tile / gated;
    p.tile = tile;
    p.ntm = (int)((M + tile - 1) / tile);
    p.ntn = (int)((N + bc - 1) / bc);
    return (int64_t)p.ntm * p.ntn;
  };
  int64_t tiles = cut(256);
  if (tiles < 192) tiles = cut(128);
  const int room = mm_room(p.tile);
  p.whole = even(total);
  if (p.tile == 256 && p.whole < 4) p.whole = 4;
  p.stages = p.whole;
  p.split = 1;
  // The last, partial round of tiles: split over k so that its parts fill the
  // chip.  Cost in stages of one block: rounds of parts, plus what writing and
  // reading a part back takes.
  const int rest = (int)(tiles % room);
  p.full = (int)tiles;
  if (rest > 0) {
    const int join = p.tile == 256 ? 6 : 4;
    int best = p.whole;  // one more round of whole tiles
    for (int s = 2; s <= 64; ++s) {
      const int st = even((total + s - 1) / s), parts = (total + st - 1) / st;
      if (parts != s || st < 4) continue;
      const int cost = (int)(((int64_t)rest * s + room - 1) / room) * (st + join) + join;
      if (cost < best) {
        best = cost;
        p.split = s;
        p.stages = st;
      }
    }
    if (p.split > 1) p.full = (int)tiles - rest;
  }
  const int64_t parts = (tiles - p.full) * p.split;
  p.items = (int)(p.full + parts);
  p.part_bytes = (size_t)(parts * p.tile * p.tile) * 4;
  return p;
}

hipError_t launch_mm(int io_bf16, MmLayout layout, MmEpilogue epi, const MmArgs& a, const MmPlan& plan,
                     hipStream_t s) {
  if (epi == MM_STORE) return io_bf16 ? mm_store_bf16(layout, a, plan, s) : mm_store_f32(layout, a, plan, s);
  if (layout != MM_PQ_K) return hipErrorInvalidValue;
  if (epi == MM_LINEAR) return io_bf16 ? mm_linear_bf16(a, plan, s) : mm_linear_f32(a, plan, s);
  return io_bf16 ? mm_gated_bf16(a, plan, s) : mm_gated_f32(a, plan, s);
}

}  // namespace m3
