// Host side of libctcpb_lm.so for 8-bit operands: argument checks and launches (C ABI in
// include/ctcpb_lm.h).
#include <algorithm>

#include "attention8.h"
#include "attention_host.h"
#include "cache8.h"
#include "gemm_host.h"
#include "host.h"
#include "linear8.h"

using namespace ctcpb_lm;

namespace {

constexpr const char* kBadCode = "code must be CTCPB_LM_INT8 or CTCPB_LM_E4M3";

constexpr int64_t kMostBlocks = 1 << 24;   // of 256 threads: a launch has less than 2^32

bool code_ok(int32_t code) { return code == CTCPB_LM_INT8 || code == CTCPB_LM_E4M3; }

int check_scales(const ctcpb_lm_scales& s) {
  if (!s.data) return fail(CTCPB_ERR_INVALID, kNull);
  if (s.stride_page < 0 || s.stride_head < 0)
    return fail(CTCPB_ERR_INVALID, "strides of scales must be >= 0");
  return CTCPB_OK;
}

ScaleView view(const ctcpb_lm_scales& s) { return ScaleView{s.data, s.stride_page, s.stride_head}; }

// ----------------------------------------------------------- store, load --

int check_cache8(const ctcpb_lm_cache8_args& g) {
  if (!elem_size(g.dtype)) return fail(CTCPB_ERR_INVALID, kBadType);
  if (!code_ok(g.code)) return fail(CTCPB_ERR_INVALID, kBadCode);
  if (int rc = check_pages(g.num_pages, g.page_size)) return rc;
  if (g.tokens < 0 || g.kv_heads < 1 || g.head_dim < 1)
    return fail(CTCPB_ERR_INVALID, "need tokens >= 0, kv_heads >= 1 and head_dim >= 1");
  if ((int64_t)g.kv_heads * g.head_dim > 1 << 24)
    return fail(CTCPB_ERR_INVALID, "kv_heads * head_dim must be at most 2^24");
  if (g.k_stride_t < 0 || g.k_stride_h < 0 || g.v_stride_t < 0 || g.v_stride_h < 0)
    return fail(CTCPB_ERR_INVALID, "strides must be >= 0");
  if (int rc = check_cache(g.k_cache)) return rc;
  if (int rc = check_cache(g.v_cache)) return rc;
  if (int rc = check_scales(g.k_scale)) return rc;
  if (int rc = check_scales(g.v_scale)) return rc;
  if (g.tokens && (!g.k || !g.v || !g.slots)) return fail(CTCPB_ERR_INVALID, kNull);
  return CTCPB_OK;
}

bool view_aligned(const CacheView& v, int n) {
  return aligned(v.data, n) && v.page % n == 0 && v.token % n == 0 && v.head % n == 0;
}

// The kernels' arguments; `wide` says whether 16 bytes of k and v, and as many codes as they
// hold values, can be accessed at once.
Cache8Args cache8_args(const ctcpb_lm_cache8_args& g, bool& wide) {
  const int es = elem_size(g.dtype), n = 16 / es;
  Cache8Args a{};
  a.k = static_cast<char*>(g.k);
  a.v = static_cast<char*>(g.v);
  a.k_t = g.k_stride_t * es;
  a.k_h = g.k_stride_h * es;
  a.v_t = g.v_stride_t * es;
  a.v_h = g.v_stride_h * es;
  a.slots = g.slots;
  a.kc = ctcpb_lm::view(g.k_cache, 1);
  a.vc = ctcpb_lm::view(g.v_cache, 1);
  a.ks = view(g.k_scale);
  a.vs = view(g.v_scale);
  a.tokens = g.tokens;
  a.heads = g.kv_heads;
  a.dim = g.head_dim;
  a.page_log = log2_of(g.page_size);
  a.num_slots = g.num_pages * g.page_size;
  wide = g.head_dim % n == 0 && aligned(g.k, 16) && aligned(g.v, 16) && a.k_t % 16 == 0 &&
         a.k_h % 16 == 0 && a.v_t % 16 == 0 && a.v_h % 16 == 0 && view_aligned(a.kc, n) &&
         view_aligned(a.vc, n);
  a.per = wide ? g.head_dim / n : g.head_dim;
  return a;
}

// Runs f<T, C, N> for the call's types.
template <typename F>
void for_types(int32_t dtype, int32_t code, bool wide, F f) {
  const auto codes = [&](auto type, auto n) {
    typedef decltype(type) T;
    if (code == CTCPB_LM_INT8)
      f(T{}, Int8{}, n);
    else
      f(T{}, E4m3{}, n);
  };
  typedef std::integral_constant<int, 1> One;
  if (dtype == CTCPB_LM_F32) {
    if (wide)
      codes(float{}, std::integral_constant<int, 4>{});
    else
      codes(float{}, One{});
  } else {
    const auto half = [&](auto type) {
      if (wide)
        codes(type, std::integral_constant<int, 8>{});
      else
        codes(type, One{});
    };
    if (dtype == CTCPB_LM_BF16)
      half(__bf16{});
    else
      half(_Float16{});
  }
}

// ------------------------------------------------------------- attention --

AttnPlan plan_attention8(const ctcpb_lm_attention_args& g) {
  AttnPlan p{};
  constexpr int32_t tile = 32;
  const int32_t group = g.q_heads / g.kv_heads;
  p.head_tiles = (group + 15) / 16;
  p.max_len = length_bound(g);
  int64_t span = p.max_len;
  if (g.window > 0) span = std::min<int64_t>(span, (int64_t)g.window + tile);
  const int64_t all = (int64_t)g.kv_heads * p.head_tiles;
  p.items = g.rows * all;
  const int64_t slots = 256 * (g.head_dim <= 64 ? 4 : g.head_dim <= 128 ? 3 : 2);
  const int64_t steps = ceil_div(std::max<int64_t>(span, 1), kRangeWaves * tile);
  const int32_t group_waves = g.head_dim <= 128 ? 8 : 4;
  const int64_t few = (int64_t)group_waves * tile * 8;
  // As for 16-bit caches, whose reasons hold: few and short rows a workgroup each, many short
  // ones a wave each, the rest by ranges.  Rows of random lengths up to a bound, in us (a wave
  // each / a workgroup each / ranges):
  //   bf16, e4m3, 16 query and 4 key/value heads of 64: 16 rows up to 1024 31.5 / 10.7 / 17.5,
  //     up to 4096 108 / 23.4 / 18.6; 256 rows up to 256 13.2 / 13.7 / 18.2, up to 512 20.0 /
  //     17.1 / 23.2, up to 2048 59.4 / 34.3 / 38.8; 1024 rows up to 512 35.1 / 46.4 / 44.0, up to
  //     2048 130 / 110 / 121; 4096 rows up to 512 123 / 183 / 168
  //   bf16, int8, 32 and 8 of 128: 16 rows up to 1024 43.5 / 15.1 / 21.9, up to 4096 179 / 38.1 /
  //     28.6; 256 rows up to 256 24.3 / 42.0 / 34.4, up to 512 38.9 / 50.7 / 43.9, up to 1024 71.4
  //     / 72.6 / 63.0; 1024 rows up to 512 129 / 192 / 153
  //   bf16, int8, 8 and 4 of 256: 64 rows up to 512 36.0 / 18.2 / 24.4; 256 rows up to 512 39.6 /
  //     50.9 / 42.4
  //   f32, int8, 8 of 64: 64 rows up to 1024 46.3 / 21.9 / 31.0; 256 rows up to 512 34.0 / 42.8 /
  //     39.4, up to 1024 59.9 / 58.7 / 51.0
  // Wide heads and f32 leave registers for one workgroup of eight waves on a CU at a time, so
  // that many of them are slower than ranges (not with heads of 64 in 16 bits).
  const bool crowded = (g.head_dim > 64 || g.dtype == CTCPB_LM_F32) &&
                       p.items * group_waves >= 16 * slots;
  if (span <= few && p.items * 8 * tile >= slots * span) {
    p.waves = 1;
  } else if (span <= few && !crowded) {
    p.waves = group_waves;
  } else {
    p.ranges = (int32_t)std::max<int64_t>(1, std::min(slots / all, g.rows * steps));
    p.o_part = ((size_t)(g.rows + 1) * sizeof(int32_t) + 255) / 256 * 256;
    p.bytes = p.o_part +
              (size_t)p.ranges * all * 2 * part_floats(group, g.head_dim) * sizeof(float);
  }
  return p;
}

int check_attention8(const ctcpb_lm_attention8_args& g) {
  if (int rc = check_attention(g.base)) return rc;
  if (!code_ok(g.code)) return fail(CTCPB_ERR_INVALID, kBadCode);
  if (g.base.head_dim % 16) return fail(CTCPB_ERR_INVALID, "head_dim must be a multiple of 16");
  return CTCPB_OK;
}

template <typename T, typename C>
void launch_attention8(const Attn8Args& a, const AttnPlan& p, hipStream_t st) {
  if (a.D <= 64)
    launch_tiles_of<Tile8<T, C, 64>>(a, p, st);
  else if (a.D <= 128)
    launch_tiles_of<Tile8<T, C, 128>>(a, p, st);
  else
    launch_tiles_of<Tile8<T, C, 256>>(a, p, st);
}

template <typename T>
void launch_attention8(const Attn8Args& a, const AttnPlan& p, int32_t code, hipStream_t st) {
  if (code == CTCPB_LM_INT8)
    launch_attention8<T, Int8>(a, p, st);
  else
    launch_attention8<T, E4m3>(a, p, st);
}

// ---------------------------------------------------------------- linear --

constexpr int32_t kMostHidden = 131071;   // 128 * 128 * it is below 2^31

// Sizes and workspace offsets of a linear8 call.
struct LinearPlan {
  int32_t padded;             // hidden up to 16 bytes
  bool quantize, pad_x, pad_w;
  bool few;                   // one launch for few rows
  Cut cut;
  int32_t pitch;
  size_t o_x, o_scale, o_w, o_planes, bytes;
};

// Whether rows of codes begin where they can be read 16 bytes at a time (their addresses
// within a tile have 31 bits).
bool codes_aligned(const void* p, int64_t stride) {
  return aligned(p, 16) && stride % 16 == 0 && stride <= 1 << 23;
}

LinearPlan plan_linear8(const ctcpb_lm_linear8_args& g) {
  LinearPlan p{};
  const bool readable = g.flags & CTCPB_LM_READABLE;
  p.padded = (int32_t)up(g.hidden, 16);
  p.quantize = g.x_dtype != CTCPB_LM_CODES;
  // What lies behind a row's `hidden` codes, up to 16 bytes, is multiplied too: x has zeros
  // there, w may have anything.
  p.pad_x = !p.quantize && (g.hidden % 16 != 0 || !codes_aligned(g.x, g.stride_x));
  p.pad_w = (g.hidden % 16 != 0 && !readable) || !codes_aligned(g.w, g.stride_w);
  // On the GPU in us, with weights that its caches hold, one launch for few rows of codes / the
  // product's tiles: 5000 channels of 512 4.2 and 4.3 for a row, 4.8 and 4.3 for 16, 6.0 and 4.5 for
  // 32; 2048 of 2048 4.4 and 7.7, 4.7 and 7.2, 5.8 and 7.6; 8192 of 2048 5.7 and 8.4, 6.1 and 9.3,
  // 7.6 and 7.3; 50000 of 2048 25 and 18, 27 and 20 for 32.  x quantised there / before it, then one
  // launch / before it, then tiles, 5000 channels: 16 rows of 512 6.1, 7.9, 7.8; 32 8.4, 9.6, 8.1
  // (and a launch less for the host); 16 of 1024 7.3, 8.6, 9.5; 8 of 2048 7.9, 9.0, 11.4; 16 of
  // them before it 9.5, tiles 12.0.
  const int64_t values = (int64_t)g.rows * up(p.padded, 64);
  // quantised by the same launch
  const bool there = p.quantize && values <= kFewValues;
  p.few = g.rows <= (there || p.padded >= 1024 ? 32 : 16) && values <= kFewCodes && !p.pad_w &&
          g.features <= 64 * kCUs;
  if (p.few) {
    p.pad_x = false;
    p.quantize = p.quantize && !there;
  } else {
    p.cut = choose_cut(1, g.features, g.rows, p.padded, true);
  }
  p.pitch = (int32_t)up(g.features, 4);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  if (p.quantize || p.pad_x) p.o_x = take((size_t)g.rows * p.padded);
  if (p.quantize) p.o_scale = take((size_t)g.rows * sizeof(float));
  if (p.pad_w) p.o_w = take((size_t)g.features * p.padded);
  if (p.cut.splits > 1)
    p.o_planes = take((size_t)p.cut.splits * g.rows * p.pitch * sizeof(int32_t));
  p.bytes = at;
  return p;
}

int check_linear8(const ctcpb_lm_linear8_args& g) {
  if (!elem_size(g.dtype)) return fail(CTCPB_ERR_INVALID, kBadType);
  if (g.x_dtype != g.dtype && g.x_dtype != CTCPB_LM_CODES)
    return fail(CTCPB_ERR_INVALID, "x_dtype must be dtype or CTCPB_LM_CODES");
  if (g.flags & ~CTCPB_LM_READABLE) return fail(CTCPB_ERR_INVALID, "flags has unknown bits");
  if (g.rows < 0 || g.features < 1 || g.hidden < 1)
    return fail(CTCPB_ERR_INVALID, "need rows >= 0, features >= 1 and hidden >= 1");
  if (g.stride_x < 0 || g.stride_w < 0 || g.stride_out < g.features)
    return fail(CTCPB_ERR_INVALID, "need stride_x and stride_w >= 0, stride_out >= features");
  if (g.hidden > kMostHidden)
    return fail(CTCPB_ERR_UNSUPPORTED, "hidden above 131071, where sums leave 32 bits");
  if (g.features > 1 << 30 || g.rows > 1 << 30)
    return fail(CTCPB_ERR_UNSUPPORTED, "features or rows above 2^30");
  if ((int64_t)ceil_div(g.features, 64) * ceil_div(g.rows, 64) * 16 > INT_MAX)
    return fail(CTCPB_ERR_UNSUPPORTED, "too many tiles for one launch");
  return CTCPB_OK;
}

template <typename T, bool ANY>
void launch_quantize(const QuantArgs& a, hipStream_t st) {
  constexpr int N = 16 / (int)sizeof(T);
  // a wave to each row where there are enough to fill the card, and they fit its registers
  if (a.rows >= 1024 && a.per <= 64 * kQuantHeld)
    quantize_kernel<T, N, ANY, 1><<<(unsigned)((a.rows + 3) / 4), 256, 0, st>>>(a);
  else
    quantize_kernel<T, N, ANY, 4><<<(unsigned)a.rows, 256, 0, st>>>(a);
}

template <typename T>
void launch_quantize(const void* x, int64_t stride, int8_t* codes, int64_t codes_row, float* scales,
                     int32_t rows, int32_t hidden, int32_t padded, hipStream_t st) {
  constexpr int N = 16 / (int)sizeof(T);
  const QuantArgs a{static_cast<const char*>(x), stride * (int)sizeof(T), codes, codes_row, scales,
                    rows, hidden, padded, ceil_div(hidden, N)};
  const bool whole = hidden % N == 0 && aligned(x, 16) && a.x_row % 16 == 0 && aligned(codes, N) &&
                     codes_row % N == 0;
  if (whole)
    launch_quantize<T, false>(a, st);
  else
    launch_quantize<T, true>(a, st);
}

void launch_quantize(int32_t dtype, const void* x, int64_t stride, int8_t* codes, int64_t codes_row,
                     float* scales, int32_t rows, int32_t hidden, int32_t padded, hipStream_t st) {
  const auto f = dtype == CTCPB_LM_BF16  ? launch_quantize<__bf16>
                 : dtype == CTCPB_LM_F16 ? launch_quantize<_Float16>
                                         : launch_quantize<float>;
  constexpr int32_t most = 1 << 22;   // rows of a launch, which has 2^32 threads at most
  for (int64_t r = 0; r < rows; r += most)
    f(static_cast<const char*>(x) + r * stride * elem_size(dtype), stride, codes + r * codes_row,
      codes_row, scales + r, (int32_t)std::min<int64_t>(rows - r, most), hidden, padded, st);
}

Operand codes_of(const void* data, int64_t stride, int32_t rows, int32_t hidden, int32_t padded,
                 bool pad, char* copy, hipStream_t st) {
  if (!pad) return Operand{static_cast<const char*>(data), stride, rows, false};
  const int64_t all = (int64_t)rows * padded, blocks = std::min<int64_t>((all + 255) / 256, 8192);
  pad_kernel<uint8_t><<<(unsigned)blocks, 256, 0, st>>>(
      static_cast<const uint8_t*>(data), stride, reinterpret_cast<uint8_t*>(copy), rows, hidden,
      padded);
  return Operand{copy, padded, rows, false};
}

template <typename T, typename X, bool ANY, int NT>
void launch_few(const FewArgs& a, hipStream_t st) {
  const int tiles = ceil_div(a.features, 16);
  const size_t lds =
      (size_t)a.rows * (up(a.padded, 64) + 16) + 16 * NT * 1024 + a.rows * sizeof(float);
  static_assert(kFewCodes + 32 * 16 + 32 * 1024 + 32 * 4 <= kLds, "more LDS than there is");
  // Four waves to a tile, and four tiles at a time to a workgroup, where rows are too short for 16
  // and there are tiles enough
  if (tiles <= kCUs || a.padded >= 1024)
    launch_with_lds(linear8_few_kernel<T, X, ANY, NT, 16>, (unsigned)std::min(tiles, kCUs), 1024,
                    lds, a, st);
  else
    launch_with_lds(linear8_few_kernel<T, X, ANY, NT, 4>,
                    (unsigned)std::min(ceil_div(tiles, 4), kCUs), 1024, lds, a, st);
}

template <typename T, typename X, bool ANY>
void launch_few(const FewArgs& a, hipStream_t st) {
  if (a.rows <= 16)
    launch_few<T, X, ANY, 1>(a, st);
  else
    launch_few<T, X, ANY, 2>(a, st);
}

// x of type X, in pieces of 16 bytes, which are whole and aligned or not.
template <typename T, typename X>
void launch_few(FewArgs& a, const void* x, int64_t stride, hipStream_t st) {
  constexpr int N = 16 / (int)sizeof(X);
  a.x = static_cast<const char*>(x);
  a.x_row = stride * (int)sizeof(X);
  a.per = ceil_div(a.hidden, N);
  while (64 << a.ways_log < a.per && (2 << a.ways_log) * a.rows <= 16) ++a.ways_log;
  if (a.hidden % N == 0 && aligned(x, 16) && a.x_row % 16 == 0)
    launch_few<T, X, false>(a, st);
  else
    launch_few<T, X, true>(a, st);
}

template <typename T>
void run_few(const LinearPlan& p, const ctcpb_lm_linear8_args& g, char* ws, hipStream_t st) {
  FewArgs a{nullptr, 0, g.x_scale, g.w, g.stride_w, g.w_scale, g.bias, static_cast<char*>(g.out),
            g.stride_out, g.rows, g.hidden, g.features, p.padded, 0, 0};
  if (g.x_dtype == CTCPB_LM_CODES) return launch_few<T, int8_t>(a, g.x, g.stride_x, st);
  if (!p.quantize) return launch_few<T, T>(a, g.x, g.stride_x, st);   // (out has x's type)
  float* scales = reinterpret_cast<float*>(ws + p.o_scale);
  launch_quantize(g.x_dtype, g.x, g.stride_x, reinterpret_cast<int8_t*>(ws + p.o_x), p.padded,
                  scales, g.rows, g.hidden, p.padded, st);
  a.x_scale = scales;
  a.hidden = p.padded;   // zeros behind
  launch_few<T, int8_t>(a, ws + p.o_x, p.padded, st);
}

template <typename T>
void run_linear8(const LinearPlan& p, const ctcpb_lm_linear8_args& g, char* ws, hipStream_t st) {
  if (p.few) return run_few<T>(p, g, ws, st);
  const float* x_scale = g.x_scale;
  Operand x;
  if (p.quantize) {
    float* scales = reinterpret_cast<float*>(ws + p.o_scale);
    launch_quantize(g.x_dtype, g.x, g.stride_x, reinterpret_cast<int8_t*>(ws + p.o_x), p.padded,
                    scales, g.rows, g.hidden, p.padded, st);
    x_scale = scales;
    x = Operand{ws + p.o_x, p.padded, g.rows, false};
  } else {
    x = codes_of(g.x, g.stride_x, g.rows, g.hidden, p.padded, p.pad_x, ws + p.o_x, st);
  }
  const Operand w =
      codes_of(g.w, g.stride_w, g.features, g.hidden, p.padded, p.pad_w, ws + p.o_w, st);
  constexpr int per = 16 / (int)sizeof(T);
  int32_t* planes = p.cut.splits > 1 ? reinterpret_cast<int32_t*>(ws + p.o_planes) : nullptr;
  const bool wide = g.features % per == 0 && g.stride_out % per == 0 && aligned(g.out, 16);
  const auto run = [&](auto ep) {
    ep = decltype(ep){static_cast<T*>(g.out), g.stride_out, g.w_scale, g.bias, x_scale, planes,
                      p.pitch, g.features, g.rows};
    launch_cut<int8_t, true, true>(w, x, p.padded, p.cut, 0, ep, st);
  };
  if (wide)
    run(Linear8Epilogue<T, true>{});
  else
    run(Linear8Epilogue<T, false>{});
  if (planes) {
    const Linear8Epilogue<T, false> ep{static_cast<T*>(g.out), g.stride_out, g.w_scale, g.bias,
                                       x_scale, planes, p.pitch, g.features, g.rows};
    const int64_t blocks = ((int64_t)g.rows * (p.pitch / 4) + 255) / 256;
    linear8_join_kernel<T><<<(unsigned)std::min<int64_t>(blocks, 4096), 256, 0, st>>>(ep,
                                                                                      p.cut.splits);
  }
}

}  // namespace

extern "C" {

int ctcpb_lm_cache_store8(const ctcpb_lm_cache8_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_cache8(*args)) return rc;
    if (args->tokens == 0) return ok();
    // (as many as a plan has; a chunk's waves look up to 127 tokens past it, in 32 bits)
    if (args->tokens > 1 << 30)
      return fail(CTCPB_ERR_UNSUPPORTED, "too many tokens: above 2^30");
    bool wide;
    Cache8Args a = cache8_args(*args, wide);
    // A wave to each token while that makes no more than some waves to each place on the card, else
    // as many as hold a page's keys or values in registers, or one that holds both, to as many
    // tokens
    const int64_t one = (int64_t)a.tokens * a.heads * 2, pieces = (int64_t)args->page_size * a.per;
    const bool many = one > 1 << 16;
    const int waves = !many || pieces <= 64 * kStoreHeld ? 1 : pieces <= 128 * kStoreHeld ? 2 : 4;
    const bool both = many && pieces <= 32 * kStoreHeld;
    a.chunk = !many ? 1 : std::min(std::max(args->page_size, 16), 64);
    const int64_t units = (int64_t)ceil_div(a.tokens, a.chunk) * a.heads * (both ? 1 : 2);
    const int64_t blocks = waves == 1 ? (units + 3) / 4 : units;
    if (blocks >= kMostBlocks)
      return fail(CTCPB_ERR_UNSUPPORTED, "too many tokens for one launch");
    hipStream_t st = static_cast<hipStream_t>(stream);
    for_types(args->dtype, args->code, wide, [&](auto t, auto c, auto n) {
      typedef decltype(t) T;
      typedef decltype(c) C;
      constexpr int N = decltype(n)::value;
      if (both)
        store8_kernel<T, C, N, 1, 2><<<(unsigned)blocks, 256, 0, st>>>(a);
      else if (waves == 1)
        store8_kernel<T, C, N, 1, 1><<<(unsigned)blocks, 256, 0, st>>>(a);
      else if (waves == 2)
        store8_kernel<T, C, N, 2, 1><<<(unsigned)blocks, 128, 0, st>>>(a);
      else
        store8_kernel<T, C, N, 4, 1><<<(unsigned)blocks, 256, 0, st>>>(a);
    });
    return launched("store8_kernel");
  });
}

int ctcpb_lm_cache_load8(const ctcpb_lm_cache8_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_cache8(*args)) return rc;
    if (args->tokens == 0) return ok();
    bool wide;
    const Cache8Args a = cache8_args(*args, wide);
    const int64_t pieces = (int64_t)a.tokens * a.heads * a.per;
    const int64_t blocks = std::min<int64_t>((pieces + 255) / 256, 1 << 20);
    hipStream_t st = static_cast<hipStream_t>(stream);
    for_types(args->dtype, args->code, wide, [&](auto t, auto c, auto n) {
      load8_kernel<decltype(t), decltype(c), decltype(n)::value>
          <<<(unsigned)blocks, 256, 0, st>>>(a);
    });
    return launched("load8_kernel");
  });
}

int ctcpb_lm_attention8_workspace(const ctcpb_lm_attention8_args* args, size_t* out_bytes) {
  return guarded([&] {
    if (!args || !out_bytes) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_attention8(*args)) return rc;
    *out_bytes = plan_attention8(args->base).bytes;
    return ok();
  });
}

int ctcpb_lm_attention8(const ctcpb_lm_attention8_args* args, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_attention8(*args)) return rc;
    const ctcpb_lm_attention_args& g = args->base;
    const AttnPlan p = plan_attention8(g);
    Attn8Args a{};
    if (int rc = check_scales(args->k_scale)) return rc;
    if (int rc = check_scales(args->v_scale)) return rc;
    if (int rc = attention_args(g, p, 1, workspace, workspace_bytes,
                                "workspace smaller than ctcpb_lm_attention8_workspace", a))
      return rc;
    if (g.rows == 0) return ok();
    // (a wave to an item, four to a workgroup; four heads or more to a workgroup that joins)
    if ((int64_t)g.rows * g.q_heads >= 4 * kMostBlocks)
      return fail(CTCPB_ERR_UNSUPPORTED, "too many rows for one launch");
    a.ks = view(args->k_scale);
    a.vs = view(args->v_scale);
    if (std::max(a.kc.page, a.vc.page) > UINT32_MAX ||
        std::max(a.ks.page, a.vs.page) > UINT32_MAX / 4 ||
        std::max(a.kc.token, a.vc.token) > 1 << 23)
      return fail(CTCPB_ERR_UNSUPPORTED, "pages 4 GiB apart, or tokens of a page more than 8 MiB");
    a.k_page = (uint32_t)a.kc.page;
    a.v_page = (uint32_t)a.vc.page;
    a.k_token = (uint32_t)a.kc.token;
    a.v_token = (uint32_t)a.vc.token;
    a.ks_page = (uint32_t)(4 * a.ks.page);
    a.vs_page = (uint32_t)(4 * a.vs.page);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (g.dtype == CTCPB_LM_BF16)
      launch_attention8<__bf16>(a, p, args->code, st);
    else if (g.dtype == CTCPB_LM_F16)
      launch_attention8<_Float16>(a, p, args->code, st);
    else
      launch_attention8<float>(a, p, args->code, st);
    return launched("attn_kernel");
  });
}

int ctcpb_lm_quantize_rows(const ctcpb_lm_quantize_args* args, void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_quantize_args& g = *args;
    if (!elem_size(g.dtype)) return fail(CTCPB_ERR_INVALID, kBadType);
    if (g.rows < 0 || g.hidden < 1 || g.hidden > 1 << 30)
      return fail(CTCPB_ERR_INVALID, "need rows >= 0 and 1 <= hidden <= 2^30");
    if (g.stride_x < 0 || g.stride_codes < g.hidden)
      return fail(CTCPB_ERR_INVALID, "need stride_x >= 0 and stride_codes >= hidden");
    if (g.rows == 0) return ok();
    if (!g.x || !g.codes || !g.scales) return fail(CTCPB_ERR_INVALID, kNull);
    const int64_t padded = std::min<int64_t>(up(g.hidden, 16), g.stride_codes);
    launch_quantize(g.dtype, g.x, g.stride_x, g.codes, g.stride_codes, g.scales, g.rows, g.hidden,
                    (int32_t)padded, static_cast<hipStream_t>(stream));
    return launched("quantize_kernel");
  });
}

int ctcpb_lm_linear8_workspace(const ctcpb_lm_linear8_args* args, size_t* out_bytes) {
  return guarded([&] {
    if (!args || !out_bytes) return fail(CTCPB_ERR_INVALID, kNoArgs);
    if (int rc = check_linear8(*args)) return rc;
    *out_bytes = args->rows ? plan_linear8(*args).bytes : 0;
    return ok();
  });
}

int ctcpb_lm_linear8(const ctcpb_lm_linear8_args* args, void* workspace, size_t workspace_bytes,
                     void* stream) {
  return guarded([&] {
    if (!args) return fail(CTCPB_ERR_INVALID, kNoArgs);
    const ctcpb_lm_linear8_args& g = *args;
    if (int rc = check_linear8(g)) return rc;
    if (g.rows == 0) return ok();
    if (!g.x || !g.w || !g.w_scale || !g.out || (g.x_dtype == CTCPB_LM_CODES && !g.x_scale))
      return fail(CTCPB_ERR_INVALID, kNull);
    const LinearPlan p = plan_linear8(g);
    if (p.bytes && (!workspace || !aligned(workspace, 256)))
      return fail(CTCPB_ERR_INVALID, "workspace must be 256-byte aligned and not NULL");
    if (workspace_bytes < p.bytes)
      return fail(CTCPB_ERR_TOO_SMALL, "workspace smaller than ctcpb_lm_linear8_workspace");
    const auto f = g.dtype == CTCPB_LM_BF16  ? run_linear8<__bf16>
                   : g.dtype == CTCPB_LM_F16 ? run_linear8<_Float16>
                                             : run_linear8<float>;
    f(p, g, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
    return launched("linear8 kernels");
  });
}

}  // extern "C"
