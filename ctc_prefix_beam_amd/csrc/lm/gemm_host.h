// How a product is cut into tiles, and its launches.
#pragma once
#include <algorithm>

#include "gemm.h"
#include "host.h"

namespace ctcpb_lm {

// How a product is cut up: tiles of BM (its m) x BN (its n), k in parts.
struct TileShape {
  int bm, bn, wn;   // wn: waves along n (dbias sums per token tile)
};
enum { kSmall = 0, kMiddle = 1, kLarge = 2 };
constexpr TileShape kShapes[3] = {{64, 64, 2}, {128, 128, 2}, {256, 256, 4}};
constexpr int kResident[3] = {4, 2, 1};   // workgroups that share a CU
constexpr int kCUs = 256;
// f32 sums in two levels, which leaves no registers for the large tiles.
constexpr int largest(int es) { return es == 4 ? kMiddle : kLarge; }

struct Cut {
  int shape;
  int32_t tiles_m, tiles_n, splits, part;
};

inline size_t up(size_t v, size_t n) { return (v + n - 1) / n * n; }

// Estimated time (us) of a cut.  What decides is how well the tiles feed the
// matrix units against how evenly the items fill the CUs.  Measured with bf16 and
// f32 on products of 10^8 to 10^12 multiplications, for each shape: the time that
// a k-tile of an item takes of its CU when CUs are full (`unit`; 256x256: 1430
// TFLOP/s with bf16, 145 with f32), and when the item is alone on it (`alone`: its
// fetches' latency), and a launch's beginning and end (`ends`).  int8 takes the figures of
// bf16, whose k-tiles are as many bytes: they were not measured for it.
inline double cut_time(int es, const Cut& c, int64_t m, int64_t n) {
  constexpr double unit[2][3] = {{0.26, 0.56, 1.5}, {0.56, 2.05, 0}};
  constexpr double alone[2][3] = {{0.5, 0.73, 1.5}, {0.73, 2.28, 0}};
  constexpr double ends[3] = {2.5, 5.0, 8.0};
  const int type = es == 4;
  const int64_t items = (int64_t)c.tiles_m * c.tiles_n * c.splits;
  const int64_t slots = kCUs * kResident[c.shape], rest = items % slots;
  const auto round = [&](int64_t shared) {   // one item each for `shared` workgroups of a CU
    const double full = (double)shared * unit[type][c.shape], one = alone[type][c.shape];
    return (full > one ? full : one) * (c.part * es / 128.0) + 2.5;
  };
  double time = ends[c.shape] + (double)(items / slots) * round(kResident[c.shape]);
  if (rest) time += round((rest + kCUs - 1) / kCUs);
  // planes are written, and read and added by a launch of its own
  if (c.splits > 1) time += 4.5 + (double)c.splits * m * n * 8 / 3.3e6;
  return time;
}

// The cut of an m x n x K product; only those with `split` may divide k (what
// they leave are sums that can be added).
inline Cut choose_cut(int es, int64_t m, int64_t n, int64_t K, bool split, double* time = nullptr) {
  const int64_t bk = 128 / es;
  Cut best{};
  double least = 0;
  for (int shape = kSmall; shape <= largest(es); ++shape) {
    const int32_t tm = ceil_div(m, kShapes[shape].bm), tn = ceil_div(n, kShapes[shape].bn);
    // parts of k fill a last round at most when there are many tiles
    const int most = !split ? 1 : (int64_t)tm * tn >= 1024 ? 2 : 16;
    for (int splits = 1; splits <= most; ++splits) {
      Cut c{shape, tm, tn, splits, 0};
      c.part = (int32_t)(ceil_div(ceil_div(K, splits), bk) * bk);
      if (c.part < bk) c.part = (int32_t)bk;   // K = 0: one empty part
      c.splits = K > 0 ? ceil_div(K, c.part) : 1;
      const double t = cut_time(es, c, m, n);
      if (best.part == 0 || t < least) {
        best = c;
        least = t;
      }
    }
  }
  if (time) *time = least;
  return best;
}

// A product in up to two launches: rows [0, n) of its n by `main`, the others by
// `rest`, which has no tiles where there are none.  Large tiles that fill whole
// rounds of the CUs, and smaller ones for what would be a last, mostly empty round:
// 20000 x 5000 x 1024 bf16 204 us in one launch, 193 in two.
struct Product {
  Cut main, rest;
  int32_t n;
  double time;
};
inline Product choose_product(int es, int64_t m, int64_t n, int64_t K, bool split, bool one = false) {
  Product p{};
  p.main = choose_cut(es, m, n, K, split, &p.time);
  p.n = (int32_t)n;
  for (int shape = kMiddle; shape <= largest(es) && !one; ++shape) {
    const TileShape& t = kShapes[shape];
    const int64_t tm = ceil_div(m, t.bm), tn = ceil_div(n, t.bn);
    const int64_t slots = kCUs * kResident[shape], rounds = tm * tn / slots;
    const int64_t columns = rounds * slots / tm;   // of whole rounds
    if (columns == 0 || columns * t.bn >= n) continue;
    const int32_t bk = 128 / es;
    const Cut c{shape, (int32_t)tm, (int32_t)columns, 1, std::max(ceil_div(K, bk), 1) * bk};
    double time;
    const Cut rest = choose_cut(es, m, n - columns * t.bn, K, split, &time);
    time += cut_time(es, c, m, columns * t.bn) + 2.0;
    if (time < p.time) p = Product{c, rest, (int32_t)(columns * t.bn), time};
  }
  return p;
}

template <typename T, int BM, int BN, int WM, int WN, bool AKC, bool BKC, typename Epilogue>
void launch_tiles(const GemmArgs& g, const Epilogue& ep, int resident, hipStream_t st) {
  const int64_t items = (int64_t)g.tiles_m * g.tiles_n * g.splits, slots = kCUs * resident;
  gemm_kernel<T, BM, BN, WM, WN, AKC, BKC, Epilogue>
      <<<(unsigned)(items < slots ? items : slots), 64 * WM * WN, 0, st>>>(g, ep);
}

// The product of a and b over K, cut as `c`; the epilogue's n begins at n0.
template <typename T, bool AKC, bool BKC, typename Epilogue>
void launch_cut(const Operand& a, const Operand& b, int32_t K, const Cut& c, int32_t n0,
                const Epilogue& ep, hipStream_t st) {
  const GemmArgs g{a, b, K, c.tiles_m, c.tiles_n, c.splits, c.part, n0};
  if constexpr (sizeof(T) <= 2)
    if (c.shape == kLarge)
      return launch_tiles<T, 256, 256, 2, 4, AKC, BKC>(g, ep, kResident[kLarge], st);
  if (c.shape == kMiddle)
    launch_tiles<T, 128, 128, 2, 2, AKC, BKC>(g, ep, kResident[kMiddle], st);
  else
    launch_tiles<T, 64, 64, 2, 2, AKC, BKC>(g, ep, kResident[kSmall], st);
}

// Rows [n0, n1) of an operand along n.
template <typename T, bool KC>
Operand rows_of(const Operand& b, int32_t n0, int32_t n1) {
  Operand r = b;
  r.data += KC ? n0 * b.ld : (int64_t)n0 * (int)sizeof(T);
  r.rows = n1 - n0;
  return r;
}

}  // namespace ctcpb_lm
