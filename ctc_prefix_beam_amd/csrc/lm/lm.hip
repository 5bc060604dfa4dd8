// Host side of libctcpb_lm.so: argument checks and launches (C ABI in
// include/ctcpb_lm.h).
#include "ctcpb_lm.h"

#include <algorithm>
#include <climits>
#include <exception>
#include <string>
#include <type_traits>

#include "attention.h"
#include "cache.h"
#include "ctcpb.h"
#include "loss.h"

using namespace ctcpb_lm;

namespace {

thread_local std::string g_err;

int ok() {
  g_err.clear();
  return CTCPB_OK;
}

int fail(int code, const char* msg) {
  g_err = msg;
  return code;
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return ok();
  g_err = std::string(what) + " launch failed: " + hipGetErrorString(e);
  return CTCPB_ERR_DEVICE;
}

// No C++ exception leaves a C entry point (the only ones possible here are
// allocation failures of the error text).
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return CTCPB_ERR_DEVICE;
  }
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int32_t ceil_div(int64_t a, int64_t b) { return (int32_t)((a + b - 1) / b); }

int log2_of(int32_t v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

bool page_size_ok(int32_t ps) { return ps >= 4 && ps <= 256 && (ps & (ps - 1)) == 0; }

int elem_size(int32_t dtype) {
  return dtype == CTCPB_LM_BF16 || dtype == CTCPB_LM_F16 ? 2 : dtype == CTCPB_LM_F32 ? 4 : 0;
}

constexpr const char* kBadPage = "page_size must be a power of two in 4..256";
constexpr const char* kBadType = "dtype must be CTCPB_LM_BF16, CTCPB_LM_F16 or CTCPB_LM_F32";
constexpr const char* kNull = "a required pointer is NULL";
constexpr const char* kNoArgs = "args is NULL";

int check_table(int32_t rows, int64_t stride, int32_t width, int32_t page_size) {
  if (rows < 0 || width < 0) return fail(CTCPB_ERR_INVALID, "rows and table_width must be >= 0");
  if (!page_size_ok(page_size)) return fail(CTCPB_ERR_INVALID, kBadPage);
  if (stride < width) return fail(CTCPB_ERR_INVALID, "table_stride must be >= table_width");
  if ((int64_t)width * page_size > (1 << 30))
    return fail(CTCPB_ERR_INVALID, "table_width * page_size must be at most 2^30");
  return CTCPB_OK;
}

int check_pages(int32_t num_pages, int32_t page_size) {
  if (!page_size_ok(page_size)) return fail(CTCPB_ERR_INVALID, kBadPage);
  if (num_pages < 1 || (int64_t)num_pages * page_size > INT_MAX)
    return fail(CTCPB_ERR_INVALID, "num_pages must be >= 1 and num_pages * page_size below 2^31");
  return CTCPB_OK;
}

int check_cache(const ctcpb_lm_cache& c) {
  if (!c.data) return fail(CTCPB_ERR_INVALID, kNull);
  if (c.stride_page < 0 || c.stride_token < 0 || c.stride_head < 0)
    return fail(CTCPB_ERR_INVALID, "cache strides must be >= 0");
  return CTCPB_OK;
}

CacheView view(const ctcpb_lm_cache& c, int es) {
  return CacheView{static_cast<char*>(c.data), c.stride_page * es, c.stride_token * es,
                   c.stride_head * es};
}

bool wide_cache(const CacheView& v) {
  return aligned(v.data, 16) && v.page % 16 == 0 && v.token % 16 == 0 && v.head % 16 == 0;
}

// ------------------------------------------------------------- attention --

// The launch plan of an attention call, a function of sizes only (the lengths
// stay on the device).
struct AttnPlan {
  int32_t head_tiles, max_len, waves, ranges;
  int64_t items;
  size_t o_part, bytes;   // workspace: the rows' prefix sums, then the parts
};

int32_t length_bound(const ctcpb_lm_attention_args& g) {
  const int32_t held = g.table_width * g.page_size;
  return g.max_len == 0 || g.max_len > held ? held : g.max_len;
}

AttnPlan plan_attention(const ctcpb_lm_attention_args& g) {
  AttnPlan p{};
  const int32_t tile = g.dtype == CTCPB_LM_F32 ? 16 : 32, group = g.q_heads / g.kv_heads;
  p.head_tiles = (group + 15) / 16;
  p.max_len = length_bound(g);
  // tokens a row can have in its range (a window starts at a tile's edge)
  int64_t span = p.max_len;
  if (g.window > 0) span = std::min<int64_t>(span, (int64_t)g.window + tile);
  const int64_t all = (int64_t)g.kv_heads * p.head_tiles;
  p.items = g.rows * all;
  // workgroups of a range kernel that fit on the card at once: by registers, a
  // head of up to 64 / 128 / 256 values leaves room for 4 / 3 (f32: 2) / 1 on a CU
  const int64_t slots =
      256 * (g.head_dim <= 64 ? 4 : g.head_dim > 128 ? 1 : g.dtype == CTCPB_LM_F32 ? 2 : 3);
  const int64_t steps = ceil_div(std::max<int64_t>(span, 1), kRangeWaves * tile);
  // Ranges cost some 4 to 6 us more than a workgroup to each item (the prefix sums, the
  // join), so they are for rows that would keep a workgroup's waves for more than a few
  // tiles each, where uneven lengths leave CUs idle (f32: fewer, its products take
  // longer).  Bytes alone decide once there are many items, and a wave to each then
  // saves joining waves.  Rows of random lengths up to a bound, in us (ranges / a
  // workgroup each / a wave each):
  //   bf16, 16 query and 4 key/value heads of 64: 64 rows up to 256 12.9 / 6.8 / 13.1, up
  //     to 2048 25.1 / 19.1 / 83, up to 4096 35.1 / 32.1 / 158; 256 rows up to 4096 122 /
  //     134 / 203; 1024 rows up to 256 38.9 / 40.1 / 30.9; 4096 rows up to 512 283 / 277 / 227
  //   bf16, 32 and 8 of 128: 16 rows up to 1024 18.9 / 15.6 / 54, up to 2048 27.1 / 26.8,
  //     up to 4096 35.8 / 43.9; 256 rows up to 512 62.7 / 67.0 / 56.1 (the workgroup is taken),
  //     1024 rows 254 / 286 / 223
  //   bf16, 8 and 4 of 256: 16 rows up to 1024 22.1 / 26.8 (the workgroup is taken), up to 2048
  //     32.7 / 48.1; 64 rows up to 128 12.2 / 8.5 / 16.6 (the wave is taken), up to 1024 33.2 /
  //     30.9 / 89; 1024 rows up to 512 231 / 248 / 225
  //   f32, 8 of 64: 16 rows up to 512 17.9 / 13.0 / 46, up to 1024 23.6 / 20.9, up to 2048
  //     27.7 / 39.0; 64 rows up to 1024 36.7 / 36.3; 256 rows up to 1024 133 / 119 / 145
  //   f32, 8 and 4 of 256: 16 rows up to 256 22.9 / 20.8, up to 512 31.9 / 37.8, up to 2048
  //     44 / 122
  // One short row in wide tables is dearer by ranges (f32, 8 heads of 64, up to 2048: 17.4
  // / 10.8): a max_len tells.
  // Wider heads leave a wave too few registers in workgroups of eight.
  const int32_t group_waves = g.head_dim <= 128 ? 8 : 4;
  const int64_t few = (int64_t)group_waves * tile * (g.dtype == CTCPB_LM_F32 ? 4 : 8);
  if (span <= few && p.items * 4 * tile >= slots * span) {
    p.waves = 1;
  } else if (span <= few) {
    p.waves = group_waves;
  } else {
    p.waves = 0;
    p.ranges = (int32_t)std::max<int64_t>(1, std::min(slots / all, g.rows * steps));
    p.o_part = ((size_t)(g.rows + 1) * sizeof(int32_t) + 255) / 256 * 256;
    p.bytes = p.o_part +
              (size_t)p.ranges * all * 2 * part_floats(group, g.head_dim) * sizeof(float);
  }
  return p;
}

int check_attention(const ctcpb_lm_attention_args& g) {
  if (!elem_size(g.dtype)) return fail(CTCPB_ERR_INVALID, kBadType);
  if (g.kv_heads < 1 || g.q_heads < g.kv_heads || g.q_heads % g.kv_heads)
    return fail(CTCPB_ERR_INVALID, "q_heads must be a multiple of kv_heads >= 1");
  if (g.head_dim < 8 || g.head_dim % 8)
    return fail(CTCPB_ERR_INVALID, "head_dim must be a multiple of 8");
  if (g.head_dim > 256) return fail(CTCPB_ERR_UNSUPPORTED, "head_dim above 256");
  if (g.max_len < 0 || g.window < 0)
    return fail(CTCPB_ERR_INVALID, "max_len and window must be >= 0");
  return check_table(g.rows, g.table_stride, g.table_width, g.page_size);
}

template <typename K>
void launch_with_lds(K kernel, unsigned blocks, int threads, size_t lds, const AttnArgs& a,
                     hipStream_t st) {
  if (lds > 65536)   // more dynamic LDS than a kernel has unasked
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  kernel<<<blocks, threads, lds, st>>>(a);
}

template <typename T, int DP>
void launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const size_t state = (size_t)std::min(16, a.group) * (DP + 6) * sizeof(float);
  if (p.waves == 1) {
    attn_kernel<T, DP, 1><<<(unsigned)((p.items + 3) / 4), 256, 0, st>>>(a);
  } else if (p.waves) {
    constexpr int NW = DP <= 128 ? 8 : 4;
    launch_with_lds(attn_kernel<T, DP, NW>, (unsigned)p.items, 64 * NW, NW * state, a, st);
  } else {
    launch_with_lds(attn_range_kernel<T, DP>,
                    (unsigned)((int64_t)p.ranges * a.kv_heads * a.head_tiles), 64 * kRangeWaves,
                    kRangeWaves * state, a, st);
    if (p.ranges == 1) return;   // no row is split
    constexpr int LANES = DP / 4, kGroups = 256 / LANES;
    const int64_t heads = (int64_t)a.rows * a.heads;
    // a workgroup to each head while that does not make more than a few to a CU
    const int ways = heads <= 1024 ? kGroups : 1, per = kGroups / ways;
    join_kernel<T, LANES><<<(unsigned)((heads + per - 1) / per), 256, 0, st>>>(a, ways);
  }
}

template <typename T>
void launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (a.D <= 64)
    launch_attention<T, 64>(a, p, st);
  else if (a.D <= 128)
    launch_attention<T, 128>(a, p, st);
  else
    launch_attention<T, 256>(a, p, st);
}

// ------------------------------------------------------------------ loss --

// Workspace for d at a time.  Larger pieces fill the CUs better and add to dx less often:
// 20000 x 30000 x 1024 bf16 4340 us with 128 MB, 3381 with 512, 3182 with 2 GB;
// 8192 x 50000 x 2048 4199 us with 512 MB (two pieces), 4035 in one.
constexpr size_t kPieceBytes = (size_t)1 << 30;
// Tokens, and multiplications of a product, up to which d has two rows for each token without
// being asked: for precision (see loss.h), where it costs little.  64 x 5000 x 512 bf16 20.3
// us with them, 21.5 without (another cut); 64 x 20000 x 2048 86 and 75; 128 x 20000 x 2048
// 108 and 89.  Small calls wait for their launches, of which bf16 has one less so, and take up to
// 2^26 0.95 to 1.0 times as long with them, f16 1.05 to 1.1 times (65 x 35 x 64 15.3 and 14.7
// us, f16 15.4 and 16.6; 256 x 500 x 512 21.5 and 21.0, f16 21.4 and 23.4); at twice that up to
// 1.1 and 1.2 (512 x 500 x 512 23.2 and 25.6, f16 23.3 and 27.9).
constexpr int32_t kPairRows = 64;
constexpr int64_t kPairWork = (int64_t)1 << 26;

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

size_t up(size_t v, size_t n) { return (v + n - 1) / n * n; }

// Estimated time (us) of a cut.  What decides is how well the tiles feed the
// matrix units against how evenly the items fill the CUs.  Measured with bf16 and
// f32 on products of 10^8 to 10^12 multiplications, for each shape: the time that
// a k-tile of an item takes of its CU when CUs are full (`unit`; 256x256: 1430
// TFLOP/s with bf16, 145 with f32), and when the item is alone on it (`alone`: its
// fetches' latency), and a launch's beginning and end (`ends`).
double cut_time(int es, const Cut& c, int64_t m, int64_t n) {
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
Cut choose_cut(int es, int64_t m, int64_t n, int64_t K, bool split, double* time = nullptr) {
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
Product choose_product(int es, int64_t m, int64_t n, int64_t K, bool split, bool one = false) {
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

// Sums per token tile and wave that a logits product leaves for dbias.
int32_t dbias_parts(const Cut& c) { return c.tiles_n * kShapes[c.shape].wn; }

// The products of a gradient for one piece of the vocabulary.
struct PieceCuts {
  Product logits, dx, dw;
  double time;
};
PieceCuts choose_piece(int es, int64_t rows, int64_t vocab, int64_t hidden, bool pairs = false) {
  const int64_t drows = pairs ? 2 * rows : rows;
  PieceCuts c;
  c.logits = choose_product(es, vocab, rows, hidden, false);
  c.dx = choose_product(es, hidden, drows, vocab, true, pairs);
  c.dw = choose_product(es, hidden, vocab, drows, true, pairs);
  // and the sums of dx between pieces
  c.time = c.logits.time + c.dx.time + c.dw.time + 8.0 * rows * hidden / 4e6;
  return c;
}

// Vocabulary rows of a piece, in whole tiles of any shape: all where d fits the
// workspace, else the size whose pieces fill the CUs best (of 24 from half of the
// largest up).
int32_t choose_piece_rows(int es, int64_t rows, int64_t vocab, int64_t hidden) {
  const int64_t unit = 256, all = ceil_div(vocab, unit);
  int64_t most = kPieceBytes / ((rows ? rows : 1) * es) / unit;
  if (most >= all) return (int32_t)(all * unit);
  if (most < 1) most = 1;
  int64_t best = most;
  double least = 0;
  for (int64_t k = 0; k < 24; ++k) {
    const int64_t u = most - k * most / 48, n = all / u;
    const int64_t tail = vocab - n * u * unit;
    double t = n * choose_piece(es, rows, u * unit, hidden).time;
    if (tail > 0) t += choose_piece(es, rows, tail, hidden).time;
    if (k == 0 || t < least) {
      best = u;
      least = t;
    }
  }
  return (int32_t)(best * unit);
}

// Sizes and workspace offsets of a loss or gradient call.
struct LossPlan {
  int es, padded;          // padded: hidden up to 16 bytes
  bool pad_x, pad_w;       // rows to be copied to aligned ones
  int32_t piece, pieces;   // gradient: vocabulary rows at a time
  bool pairs;              // d has two rows for each token
  Product logits;          // forward
  PieceCuts whole, tail;   // gradient: a whole piece, and the last one
  size_t o_x, o_w, o_part, o_hit, o_d, o_sums, o_planes, o_bias, o_scale, bytes;
};

// The element type, without what a gradient's dtype may carry besides.
int32_t type_of(const ctcpb_lm_loss_args& g) { return g.dtype; }
int32_t type_of(const ctcpb_lm_grad_args& g) { return g.dtype & ~CTCPB_LM_SPLIT_D; }

bool row_aligned(const void* p, int64_t stride, int es) {
  // within a tile, rows are addressed with 31 bits
  return aligned(p, 16) && stride * es % 16 == 0 && stride * es <= (1 << 23);
}

// Rows of a product's result, of `n`, that a launch of it makes.
int64_t rows_made(const Product& q, int64_t n, bool rest) {
  if (q.rest.tiles_n == 0) return rest ? 0 : n;
  return rest ? n - q.n : q.n;
}

// Floats that the parts of k of a product leave: the two launches use the same place.
size_t plane_floats(const Product& q, int64_t n, int32_t hidden) {
  size_t most = 0;
  for (int rest = 0; rest < 2; ++rest) {
    const int32_t splits = rest ? q.rest.splits : q.main.splits;
    if (splits > 1) most = std::max(most, (size_t)splits * rows_made(q, n, rest) * hidden);
  }
  return most;
}

// What only gradients have: partial sums for dbias, where it is asked for, and d as two
// values of a 16-bit type, where the caller or the number of rows says so.
bool wants_dbias(const ctcpb_lm_loss_args&) { return false; }
bool wants_dbias(const ctcpb_lm_grad_args& g) { return g.dbias != nullptr; }
bool wants_pairs(const ctcpb_lm_loss_args&) { return false; }
bool wants_pairs(const ctcpb_lm_grad_args& g) {
  if (elem_size(type_of(g)) != 2) return false;
  return g.rows <= kPairRows || (double)g.rows * g.vocab * g.hidden <= kPairWork ||
         (g.dtype & CTCPB_LM_SPLIT_D);
}

template <typename Args>
LossPlan plan_loss(const Args& g, bool grad) {
  const int32_t rows = g.rows, vocab = g.vocab, hidden = g.hidden;
  LossPlan p{};
  p.es = elem_size(type_of(g));
  p.padded = (int)up(hidden, 16 / p.es);
  // a row is read up to its last 16 bytes
  p.pad_x = p.padded != hidden || !row_aligned(g.x, g.stride_x, p.es);
  p.pad_w = p.padded != hidden || !row_aligned(g.w, g.stride_w, p.es);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  if (p.pad_x) p.o_x = take((size_t)rows * p.padded * p.es);
  if (p.pad_w) p.o_w = take((size_t)vocab * p.padded * p.es);
  if (!grad) {
    p.logits = choose_product(p.es, vocab, rows, p.padded, false);
    p.o_part = take((size_t)std::max(p.logits.main.tiles_m, p.logits.rest.tiles_m) * rows *
                    sizeof(float2));
    p.o_hit = take((size_t)rows * sizeof(float));
  } else {
    p.pairs = wants_pairs(g);
    p.piece = choose_piece_rows(p.es, p.pairs ? 2 * rows : rows, vocab, p.padded);
    p.pieces = ceil_div(vocab, p.piece);
    const int32_t first = p.pieces > 1 ? p.piece : vocab;
    const int32_t last = (int32_t)(vocab - (int64_t)(p.pieces - 1) * p.piece);
    p.whole = choose_piece(p.es, rows, first, p.padded, p.pairs);
    p.tail = choose_piece(p.es, rows, last, p.padded, p.pairs);
    p.o_d = take((size_t)rows * (p.pairs ? 2 : 1) * p.piece * p.es);
    if (p.pieces > 1) p.o_sums = take((size_t)rows * hidden * sizeof(float));
    size_t planes = 0, parts = 0;
    for (const PieceCuts* c : {&p.whole, &p.tail}) {
      const int32_t made = c == &p.whole ? first : last;   // vocabulary rows
      const Product& q = c->logits;
      planes = std::max(
          {planes, plane_floats(c->dx, rows, hidden), plane_floats(c->dw, made, hidden)});
      parts = std::max(parts, (size_t)(dbias_parts(q.main) + dbias_parts(q.rest)) * made);
    }
    p.o_planes = take(planes * sizeof(float));
    if (wants_dbias(g)) p.o_bias = take(parts * sizeof(float));
    p.o_scale = take(2 * sizeof(float));
  }
  p.bytes = at;
  return p;
}

template <typename Args>
int check_loss(const Args& g) {
  if (!elem_size(type_of(g))) return fail(CTCPB_ERR_INVALID, kBadType);
  if (g.rows < 0 || g.vocab < 1 || g.hidden < 1)
    return fail(CTCPB_ERR_INVALID, "need rows >= 0, vocab >= 1 and hidden >= 1");
  if (g.stride_x < g.hidden || g.stride_w < g.hidden)
    return fail(CTCPB_ERR_INVALID, "stride_x and stride_w must be >= hidden");
  if (g.hidden > 1 << 20 || g.vocab > 1 << 30 || g.rows > 1 << 30)
    return fail(CTCPB_ERR_UNSUPPORTED, "hidden above 2^20, or vocab or rows above 2^30");
  if (wants_pairs(g) && g.rows >= 1 << 30)
    return fail(CTCPB_ERR_UNSUPPORTED, "CTCPB_LM_SPLIT_D with 2^30 rows");
  if ((int64_t)ceil_div(g.vocab, 64) * ceil_div(g.rows, 64) > INT_MAX)
    return fail(CTCPB_ERR_UNSUPPORTED, "too many tiles for one launch");
  return CTCPB_OK;
}

// x or w as the kernels read it: in place, or its copy with aligned rows.
template <typename T>
Operand aligned_rows(const void* data, int64_t stride, int32_t rows, int32_t hidden,
                     const LossPlan& p, bool pad, char* copy, hipStream_t st) {
  if (!pad)
    return Operand{static_cast<const char*>(data), stride * (int)sizeof(T), rows, false};
  typedef typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type U;
  const int64_t all = (int64_t)rows * p.padded;
  if (all == 0) return Operand{copy, (int64_t)p.padded * (int)sizeof(T), rows, false};
  const int64_t blocks = (all + 255) / 256 < 8192 ? (all + 255) / 256 : 8192;
  pad_kernel<U><<<(unsigned)blocks, 256, 0, st>>>(static_cast<const U*>(data), stride,
                                                  reinterpret_cast<U*>(copy), rows, hidden,
                                                  p.padded);
  return Operand{copy, (int64_t)p.padded * (int)sizeof(T), rows, false};
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
  if constexpr (sizeof(T) == 2)
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

// Both launches of a product whose result is a matrix (OutEpilogue); parts of k are
// added by a launch of their own.
template <typename T, bool BKC>
void launch_out(const Operand& a, const Operand& b, int32_t K, const Product& p, OutEpilogue<T> ep,
                float* planes, const float* before, hipStream_t st) {
  const int32_t n = ep.pairs ? 2 * ep.N : ep.N;
  for (int second = 0; second < 2; ++second) {
    const Cut& c = second ? p.rest : p.main;
    if (c.tiles_n == 0) continue;
    const int32_t n0 = second ? p.n : 0, n1 = second ? n : p.n;
    const int32_t r0 = ep.pairs ? n0 / 2 : n0, r1 = ep.pairs ? n1 / 2 : n1;
    const int64_t from = (int64_t)r0 * ep.M, count = (int64_t)(r1 - r0) * ep.M;
    ep.planes = c.splits > 1 ? planes : nullptr;
    ep.from = from;
    ep.pitch = count;
    ep.add = before && c.splits == 1;
    launch_cut<T, false, BKC>(a, rows_of<T, BKC>(b, n0, n1), K, c, n0, ep, st);
    if (c.splits == 1) continue;
    const int64_t blocks = (count + 255) / 256;
    planes_kernel<T><<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(
        planes, c.splits, count, before ? before + from : nullptr,
        ep.last ? nullptr : ep.sums + from, ep.out + from, ep.scale);
  }
}

template <typename T>
void run_loss(const LossPlan& p, const ctcpb_lm_loss_args& g, char* ws, hipStream_t st) {
  const Operand x =
      aligned_rows<T>(g.x, g.stride_x, g.rows, g.hidden, p, p.pad_x, ws + p.o_x, st);
  const Operand w =
      aligned_rows<T>(g.w, g.stride_w, g.vocab, g.hidden, p, p.pad_w, ws + p.o_w, st);
  float2* part = reinterpret_cast<float2*>(ws + p.o_part);
  float* hit = reinterpret_cast<float*>(ws + p.o_hit);
  const ForwardEpilogue ep{Logits{g.bias, g.targets, g.rows, g.vocab, 0}, part, hit};
  const Product& q = p.logits;
  launch_cut<T, true, true>(w, rows_of<T, true>(x, 0, q.n), p.padded, q.main, 0, ep, st);
  if (q.rest.tiles_n)
    launch_cut<T, true, true>(w, rows_of<T, true>(x, q.n, g.rows), p.padded, q.rest, q.n, ep, st);
  // few tokens: more threads to each, for latency
  if (g.rows <= 2048)
    loss_join_kernel<4><<<(unsigned)ceil_div(g.rows, 4), 256, 0, st>>>(
        part, hit, g.targets, g.rows, g.vocab, q.n, q.main.tiles_m, q.rest.tiles_m, g.loss, g.lse);
  else
    loss_join_kernel<32><<<(unsigned)ceil_div(g.rows, 32), 256, 0, st>>>(
        part, hit, g.targets, g.rows, g.vocab, q.n, q.main.tiles_m, q.rest.tiles_m, g.loss, g.lse);
}

template <typename T>
void run_grad(const LossPlan& p, const ctcpb_lm_grad_args& g, char* ws, hipStream_t st) {
  const Operand x =
      aligned_rows<T>(g.x, g.stride_x, g.rows, g.hidden, p, p.pad_x, ws + p.o_x, st);
  const Operand w =
      aligned_rows<T>(g.w, g.stride_w, g.vocab, g.hidden, p, p.pad_w, ws + p.o_w, st);
  T* d = reinterpret_cast<T*>(ws + p.o_d);
  float* sums = reinterpret_cast<float*>(ws + p.o_sums);
  float* planes = reinterpret_cast<float*>(ws + p.o_planes);
  float* part = g.dbias ? reinterpret_cast<float*>(ws + p.o_bias) : nullptr;
  float* scale = nullptr;
  const bool f16 = std::is_same<T, _Float16>::value;
  if (sizeof(T) == 2 && (f16 || !p.pairs)) {
    scale = reinterpret_cast<float*>(ws + p.o_scale);
    // f16 holds 4096 times numbers down to 10^-11 of the largest
    scale_kernel<<<1, 1024, 0, st>>>(g.grad, g.targets, g.rows, g.vocab, f16 ? 4096.0f : 1.0f,
                                     scale);
  }
  const int32_t drows = p.pairs ? 2 * g.rows : g.rows;
  const int64_t ldd = (int64_t)p.piece * (int)sizeof(T);
  for (int32_t k = 0; k < p.pieces; ++k) {
    const int32_t v0 = k * p.piece;
    const int32_t nv = g.vocab - v0 < p.piece ? g.vocab - v0 : p.piece;
    const PieceCuts& cut = k == p.pieces - 1 ? p.tail : p.whole;
    const Operand wp{w.data + v0 * w.ld, w.ld, nv, false};
    const Product& q = cut.logits;
    const int32_t parts = dbias_parts(q.main);
    GradEpilogue<T> ge{Logits{g.bias, g.targets, g.rows, g.vocab, v0}, g.grad, g.lse, scale,
                       d, p.pairs, p.piece, part, nv, 0};
    if (g.rows)
      launch_cut<T, true, true>(wp, rows_of<T, true>(x, 0, q.n), p.padded, q.main, 0, ge, st);
    if (q.rest.tiles_n) {
      ge.first_part = parts;
      launch_cut<T, true, true>(wp, rows_of<T, true>(x, q.n, g.rows), p.padded, q.rest, q.n, ge,
                                st);
    }
    const Operand dk{reinterpret_cast<char*>(d), ldd, drows, false};
    if (g.dx && g.rows) {
      // out[token, h]: m = h, n = token, k = vocabulary
      const Operand a{wp.data, wp.ld, p.padded, false};
      const OutEpilogue<T> oe{static_cast<T*>(g.dx), sums, nullptr, 0, 0, scale, g.hidden, g.rows,
                              p.pairs, false, k == p.pieces - 1};
      launch_out<T, true>(a, dk, nv, cut.dx, oe, planes, k ? sums : nullptr, st);
    }
    if (g.dw) {
      // out[v, h]: m = h, n = v, k = token
      const Operand a{x.data, x.ld, p.padded, p.pairs}, b{dk.data, ldd, nv, false};
      const OutEpilogue<T> oe{static_cast<T*>(g.dw) + (int64_t)v0 * g.hidden, nullptr, nullptr,
                              0, 0, scale, g.hidden, nv, false, false, true};
      launch_out<T, false>(a, b, drows, cut.dw, oe, planes, nullptr, st);
    }
    if (g.dbias)
      dbias_kernel<<<(unsigned)((nv + 255) / 256), 256, 0, st>>>(
          part, g.rows ? parts + dbias_parts(q.rest) : 0, nv, g.dbias + v0);
  }
}

}  // namespace

extern "C" {

const char* ctcpb_lm_last_error(void) { return g_err.c_str(); }

int ctcpb_lm_cache_plan(const ctcpb_lm_plan_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_plan_args& g = *args;
    if (int rc = check_table(g.rows, g.table_stride, g.table_width, g.page_size)) return rc;
    if (g.pool_size < 0 || g.capacity < 0 || g.capacity > (1 << 30))
      return fail(CTCPB_ERR_INVALID, "need pool_size >= 0 and 0 <= capacity <= 2^30");
    if ((g.rows && (!g.lengths || !g.counts || !g.out_lengths || !g.status ||
                    (!g.tables && g.table_width))) ||
        (!g.pool && g.pool_size) || !g.taken || (g.capacity && (!g.slots || !g.positions)) ||
        !g.starts || !g.out_taken)
      return fail(CTCPB_ERR_INVALID, kNull);
    PlanArgs a{g.lengths,   g.counts, g.pool,        g.taken,     g.tables, g.slots,
               g.positions, g.starts, g.out_lengths, g.out_taken, g.status, g.table_stride,
               g.rows,      g.table_width, g.pool_size, log2_of(g.page_size), g.capacity, 0, false};
    const int threads = g.rows <= 256 ? 256 : kPlanThreads;
    // a workgroup's part of the slot map: no more workgroups than CUs (each scans all
    // rows) while that leaves every thread four tokens at least
    a.per_block = (int32_t)(ceil_div(ceil_div(g.capacity, 256), 4 * threads) * 4 * threads);
    if (a.per_block == 0) a.per_block = 4 * threads;
    a.wide = aligned(g.slots, 16) && aligned(g.positions, 16);
    const unsigned blocks = g.capacity ? ceil_div(g.capacity, a.per_block) : 1;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (g.rows <= kPlanThreads)
      plan_kernel<1><<<blocks, threads, 0, st>>>(a);
    else
      plan_kernel<4><<<blocks, threads, 0, st>>>(a);
    return launched("plan_kernel");
  });
}

int ctcpb_lm_cache_release(const ctcpb_lm_release_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_release_args& g = *args;
    if (int rc = check_table(g.rows, g.table_stride, g.table_width, g.page_size)) return rc;
    if (g.pool_size < 0) return fail(CTCPB_ERR_INVALID, "pool_size must be >= 0");
    if ((g.rows &&
         (!g.finished || !g.lengths || !g.out_lengths || (!g.tables && g.table_width))) ||
        (!g.pool && g.pool_size) || !g.taken || !g.out_taken)
      return fail(CTCPB_ERR_INVALID, kNull);
    // at least a row to each of a workgroup's waves, and at most a workgroup to a CU
    const int32_t per = std::max(ceil_div(g.rows, 256), kPlanThreads / 64);
    const ReleaseArgs a{g.finished,  g.lengths,      g.tables, g.taken,       g.pool,
                        g.out_lengths, g.out_taken, g.table_stride, g.rows, g.table_width,
                        g.pool_size, log2_of(g.page_size), per};
    release_kernel<<<(unsigned)std::max(ceil_div(g.rows, per), 1), kPlanThreads, 0,
                     static_cast<hipStream_t>(stream)>>>(a);
    return launched("release_kernel");
  });
}

int ctcpb_lm_cache_store(const ctcpb_lm_store_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_store_args& g = *args;
    const int es = elem_size(g.dtype);
    if (!es) return fail(CTCPB_ERR_INVALID, kBadType);
    if (int rc = check_pages(g.num_pages, g.page_size)) return rc;
    if (g.tokens < 0 || g.kv_heads < 1 || g.head_dim < 1)
      return fail(CTCPB_ERR_INVALID, "need tokens >= 0, kv_heads >= 1 and head_dim >= 1");
    if ((int64_t)g.kv_heads * g.head_dim > INT_MAX)
      return fail(CTCPB_ERR_INVALID, "kv_heads * head_dim must be below 2^31");
    if (g.k_stride_t < 0 || g.k_stride_h < 0 || g.v_stride_t < 0 || g.v_stride_h < 0)
      return fail(CTCPB_ERR_INVALID, "strides must be >= 0");
    if (int rc = check_cache(g.k_cache)) return rc;
    if (int rc = check_cache(g.v_cache)) return rc;
    if (g.tokens == 0) return ok();
    if (!g.k || !g.v || !g.slots) return fail(CTCPB_ERR_INVALID, kNull);
    StoreArgs a{};
    a.k = static_cast<const char*>(g.k);
    a.v = static_cast<const char*>(g.v);
    a.k_t = g.k_stride_t * es;
    a.k_h = g.k_stride_h * es;
    a.v_t = g.v_stride_t * es;
    a.v_h = g.v_stride_h * es;
    a.slots = g.slots;
    a.kc = view(g.k_cache, es);
    a.vc = view(g.v_cache, es);
    a.heads = g.kv_heads;
    a.page_log = log2_of(g.page_size);
    a.num_slots = g.num_pages * g.page_size;
    const bool wide = g.head_dim * es % 16 == 0 && aligned(g.k, 16) && aligned(g.v, 16) &&
                      a.k_t % 16 == 0 && a.k_h % 16 == 0 && a.v_t % 16 == 0 && a.v_h % 16 == 0 &&
                      wide_cache(a.kc) && wide_cache(a.vc);
    const int size = wide ? 16 : es;
    a.per_head = g.head_dim * es / size;
    a.pieces = (int64_t)g.tokens * g.kv_heads * a.per_head;
    int64_t blocks = (a.pieces + 255) / 256;
    if (blocks > 1 << 20) blocks = 1 << 20;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (wide)
      store_kernel<u32x4><<<(unsigned)blocks, 256, 0, st>>>(a);
    else if (es == 4)
      store_kernel<uint32_t><<<(unsigned)blocks, 256, 0, st>>>(a);
    else
      store_kernel<uint16_t><<<(unsigned)blocks, 256, 0, st>>>(a);
    return launched("store_kernel");
  });
}

int ctcpb_lm_attention_workspace(const ctcpb_lm_attention_args* args, size_t* out_bytes) {
  return guarded([&] {
    if (!args || !out_bytes) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_attention(*args)) return rc;
    *out_bytes = plan_attention(*args).bytes;
    return ok();
  });
}

int ctcpb_lm_attention(const ctcpb_lm_attention_args* args, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_attention_args& g = *args;
    if (int rc = check_attention(g)) return rc;
    if (int rc = check_pages(g.num_pages, g.page_size)) return rc;
    if (g.q_stride_r < 0 || g.q_stride_h < 0 || g.out_stride_r < 0 || g.out_stride_h < 0)
      return fail(CTCPB_ERR_INVALID, "strides must be >= 0");
    if (int rc = check_cache(g.k_cache)) return rc;
    if (int rc = check_cache(g.v_cache)) return rc;
    const int es = elem_size(g.dtype);
    AttnArgs a{};
    a.kc = view(g.k_cache, es);
    a.vc = view(g.v_cache, es);
    if (!wide_cache(a.kc) || !wide_cache(a.vc))
      return fail(CTCPB_ERR_INVALID,
                  "caches must be 16-byte aligned, with strides that are multiples of 16 bytes");
    if (g.rows == 0) return ok();
    if (!g.q || !g.out || !g.lengths || (!g.tables && g.table_width))
      return fail(CTCPB_ERR_INVALID, kNull);
    const AttnPlan p = plan_attention(g);
    if (p.bytes && (!workspace || !aligned(workspace, 16)))
      return fail(CTCPB_ERR_INVALID, "workspace must be 16-byte aligned and not NULL");
    if (workspace_bytes < p.bytes)
      return fail(CTCPB_ERR_TOO_SMALL, "workspace smaller than ctcpb_lm_attention_workspace");
    // steps of all rows are counted with 31 bits
    if (p.items > INT_MAX || (int64_t)g.rows * g.q_heads > INT_MAX ||
        (int64_t)g.rows * (p.max_len / 64 + 1) > INT_MAX)
      return fail(CTCPB_ERR_UNSUPPORTED, "too many rows for one launch");
    a.q = static_cast<const char*>(g.q);
    a.out = static_cast<char*>(g.out);
    a.lse = g.lse;
    a.prefix = static_cast<int32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.o_part);
    a.tables = g.tables;
    a.lengths = g.lengths;
    a.q_r = g.q_stride_r;
    a.q_h = g.q_stride_h;
    a.out_r = g.out_stride_r;
    a.out_h = g.out_stride_h;
    a.table_stride = g.table_stride;
    a.rows = g.rows;
    a.heads = g.q_heads;
    a.kv_heads = g.kv_heads;
    a.group = g.q_heads / g.kv_heads;
    a.head_tiles = p.head_tiles;
    a.D = g.head_dim;
    a.width = g.table_width;
    a.page_log = log2_of(g.page_size);
    a.num_pages = g.num_pages;
    a.max_len = p.max_len;
    a.window = g.window;
    a.items = (int32_t)p.items;
    a.ranges = p.ranges;
    a.wide_q = aligned(g.q, 16) && g.q_stride_r * es % 16 == 0 && g.q_stride_h * es % 16 == 0;
    a.wide_out =
        aligned(g.out, 16) && g.out_stride_r * es % 16 == 0 && g.out_stride_h * es % 16 == 0;
    a.scale = g.scale;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (g.dtype == CTCPB_LM_BF16)
      launch_attention<__bf16>(a, p, st);
    else if (g.dtype == CTCPB_LM_F16)
      launch_attention<_Float16>(a, p, st);
    else
      launch_attention<float>(a, p, st);
    return launched("attn_kernel");
  });
}

int ctcpb_lm_loss_workspace(const ctcpb_lm_loss_args* args, size_t* out_bytes) {
  return guarded([&] {
    if (!args || !out_bytes) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_loss(*args)) return rc;
    *out_bytes = plan_loss(*args, false).bytes;
    return ok();
  });
}

int ctcpb_lm_loss(const ctcpb_lm_loss_args* args, void* workspace, size_t workspace_bytes,
                  void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_loss_args& g = *args;
    if (int rc = check_loss(g)) return rc;
    if (g.rows == 0) return ok();
    if (!g.x || !g.w || !g.targets || !g.loss || !g.lse || !workspace)
      return fail(CTCPB_ERR_INVALID, kNull);
    if (!aligned(workspace, 256))
      return fail(CTCPB_ERR_INVALID, "workspace must be 256-byte aligned");
    const LossPlan p = plan_loss(g, false);
    if (workspace_bytes < p.bytes)
      return fail(CTCPB_ERR_TOO_SMALL, "workspace smaller than ctcpb_lm_loss_workspace");
    const auto f = g.dtype == CTCPB_LM_BF16  ? run_loss<__bf16>
                   : g.dtype == CTCPB_LM_F16 ? run_loss<_Float16>
                                             : run_loss<float>;
    f(p, g, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
    return launched("loss kernels");
  });
}

int ctcpb_lm_loss_grad_workspace(const ctcpb_lm_grad_args* args, size_t* out_bytes) {
  return guarded([&] {
    if (!args || !out_bytes) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_loss(*args)) return rc;
    *out_bytes = plan_loss(*args, true).bytes;
    return ok();
  });
}

int ctcpb_lm_loss_grad(const ctcpb_lm_grad_args* args, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_grad_args& g = *args;
    if (int rc = check_loss(g)) return rc;
    if (!g.dx && !g.dw && !g.dbias) return ok();
    if (!g.w || !workspace || (g.rows && (!g.grad || !g.x || !g.targets || !g.lse)))
      return fail(CTCPB_ERR_INVALID, kNull);
    if (!aligned(workspace, 256) || !aligned(g.dx, 16) || !aligned(g.dw, 16))
      return fail(CTCPB_ERR_INVALID, "workspace must be 256-byte aligned, dx and dw 16-byte");
    const LossPlan p = plan_loss(g, true);
    if (workspace_bytes < p.bytes)
      return fail(CTCPB_ERR_TOO_SMALL, "workspace smaller than ctcpb_lm_loss_grad_workspace");
    const int32_t type = type_of(g);
    const auto f = type == CTCPB_LM_BF16  ? run_grad<__bf16>
                   : type == CTCPB_LM_F16 ? run_grad<_Float16>
                                          : run_grad<float>;
    f(p, g, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
    return launched("loss gradient kernels");
  });
}

}  // extern "C"
