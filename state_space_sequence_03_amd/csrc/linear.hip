// Plans and dispatch of the matrix products of the linear and gated
// feed-forward operators.
#include "mm_parts.hpp"

namespace m3 {

namespace {

// What a product costs with a given tile, in microseconds, fitted to calls of
// 50 to 32768 rows on one MI355X (bf16 / fp32): a stage of one tile alone on
// its CU and with as many tiles as fit, the start and end of a tile, and the
// join of split tiles (a launch, and the parts written and read).
struct TileCost {
  int tile;
  double alone[2], shared[2], ends[2];
};
constexpr TileCost kTiles[] = {{256, {1.05, 7.2}, {1.05, 7.2}, {6.0, 6.0}},
                               {128, {0.60, 2.1}, {0.50, 2.1}, {2.0, 6.0}},
                               {64, {0.32, 0.62}, {0.26, 0.61}, {0.5, 0.5}}};
constexpr double kJoin = 6.0;
// parts that the caches hold are joined twice as fast
inline double join_time(double bytes) { return kJoin + bytes / (bytes < 4.0e7 ? 1.0e7 : 5.0e6); }

}  // namespace

MmPlan mm_plan(int io_bf16, MmEpilogue epi, int64_t M, int64_t N, int64_t K) {
  MmPlan best{};
  const int es = io_bf16 ? 2 : 4, ty = io_bf16 ? 0 : 1;
  const int gated = epi == MM_GATED ? 2 : 1;
  // the few-row kernel: every block reads all of P, so that more rows pay only
  // where Q is small too (64 rows through 256 -> 512: 3.7 us against 4.8
  // tiled; through 2048 -> 2 x 5632: 26.7 against 16.2)
  if (epi != MM_STORE && (M <= 32 || (M <= 64 && N * gated * K * es <= (int64_t(4) << 20)))) return best;
  const int total = (int)((K * es + 127) / 128);  // stages of 128 bytes
  double least = 0.0;
  for (const TileCost& c : kTiles) {
    MmPlan p{};
    p.tile = c.tile;
    const int64_t bm = c.tile, bn = c.tile == 64 ? 64 * gated : c.tile;
    p.ntm = (int)((M + bm - 1) / bm);
    p.ntn = (int)((N * gated + bn - 1) / bn);
    const int64_t tiles = (int64_t)p.ntm * p.ntn;
    const int room = mm_room(c.tile), per = mm_blocks(c.tile);
    // the 256 x 256 tile takes stages in pairs, at least four of them
    auto stages = [&](int n) { return c.tile != 256 ? n : n < 4 ? 4 : n + (n & 1); };
    auto time = [&](int64_t items, int st) {  // of one round of items of st stages
      const int64_t n = (items + 255) / 256;
      const double wide = c.tile == 64 && gated == 2 ? 1.8 : 1.0;  // 64 x 128 of W's rows there
      return n == 0 ? 0.0 : (n < per ? st * c.alone[ty] : n * st * c.shared[ty]) * wide + n * c.ends[ty];
    };
    p.whole = stages(total);
    const int64_t rest = tiles % room;
    const double rounds = time(tiles - rest, p.whole);
    // the last round's tiles whole, or split over k so that their parts fill
    // the chip
    for (int s = 1; s <= 64; ++s) {
      const int st = s == 1 ? p.whole : stages((total + s - 1) / s);
      if (s > 1 && (rest == 0 || st < 4 || rest * s > 4 * room)) break;
      if (s > 1 && (total + st - 1) / st != s) continue;
      const double bytes = s == 1 ? 0.0 : (double)(rest * s * bm * bn) * 8.0;
      const double t = rounds + time(rest * s, st) + (s == 1 ? 0.0 : join_time(bytes));
      if (best.tile != 0 && t >= least) continue;
      least = t;
      p.split = s;
      p.stages = st;
      p.full = (int)(s == 1 ? tiles : tiles - rest);
      p.items = (int)(p.full + (s == 1 ? 0 : rest * s));
      p.part_bytes = s == 1 ? 0 : (size_t)(rest * s * bm * bn) * 4;
      best = p;
    }
  }
  return best;
}

hipError_t launch_mm(int io_bf16, MmLayout layout, MmEpilogue epi, const MmArgs& a, const MmPlan& plan,
                     hipStream_t s) {
  if (epi == MM_STORE) return io_bf16 ? mm_store_bf16(layout, a, plan, s) : mm_store_f32(layout, a, plan, s);
  if (layout != MM_PQ_K) return hipErrorInvalidValue;
  if (epi == MM_LINEAR) return io_bf16 ? mm_linear_bf16(a, plan, s) : mm_linear_f32(a, plan, s);
  return io_bf16 ? mm_gated_bf16(a, plan, s) : mm_gated_f32(a, plan, s);
}

hipError_t launch_mm_pair(int io_bf16, const MmArgs& dx, const MmPlan& px, const MmArgs& dw, const MmPlan& pw,
                          hipStream_t s) {
  if (px.tile == 64 && pw.tile == 64 && px.split == 1 && pw.split == 1 && px.items + pw.items <= mm_room(64) - 8)
    return io_bf16 ? mm_pair_bf16(dx, px, dw, pw, s) : mm_pair_f32(dx, px, dw, pw, s);
  const hipError_t e = launch_mm(io_bf16, MM_P_K, MM_STORE, dx, px, s);
  return e != hipSuccess ? e : launch_mm(io_bf16, MM_NONE_K, MM_STORE, dw, pw, s);
}

}  // namespace m3

// How a product is cut, for the tests that mean to run a certain form: tile,
// tiles in all, whole ones of them, parts of each of the others (1: none).
// epilogue: an MmEpilogue.
extern "C" void m3_product_plan(int io_bf16, int epilogue, int64_t M, int64_t N, int64_t K, int64_t* out) {
  const m3::MmPlan p = m3::mm_plan(io_bf16, (m3::MmEpilogue)epilogue, M, N, K);
  out[0] = p.tile;
  out[1] = (int64_t)p.ntm * p.ntn;
  out[2] = p.full;
  out[3] = p.split;
}
