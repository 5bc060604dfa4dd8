// What the entry points of libctcpb_lm.so share on the host: the error of the thread and
// the checks of arguments.
#pragma once
#include <climits>
#include <exception>
#include <string>

#include "common.h"
#include "ctcpb.h"
#include "ctcpb_lm.h"

namespace ctcpb_lm {

inline thread_local std::string g_err;

inline int ok() {
  g_err.clear();
  return CTCPB_OK;
}

inline int fail(int code, const char* msg) {
  g_err = msg;
  return code;
}

inline int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return ok();
  g_err = std::string(what) + " launch failed: " + hipGetErrorString(e);
  return CTCPB_ERR_DEVICE;
}

// No C++ exception leaves a C entry point (the only ones possible here are
// allocation failures of the error text).
template <typename F>
inline int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return CTCPB_ERR_DEVICE;
  }
}

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int32_t ceil_div(int64_t a, int64_t b) { return (int32_t)((a + b - 1) / b); }

inline int log2_of(int32_t v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

inline bool page_size_ok(int32_t ps) { return ps >= 4 && ps <= 256 && (ps & (ps - 1)) == 0; }

inline int elem_size(int32_t dtype) {
  return dtype == CTCPB_LM_BF16 || dtype == CTCPB_LM_F16 ? 2 : dtype == CTCPB_LM_F32 ? 4 : 0;
}

inline constexpr const char* kBadPage = "page_size must be a power of two in 4..256";
inline constexpr const char* kBadType = "dtype must be CTCPB_LM_BF16, CTCPB_LM_F16 or CTCPB_LM_F32";
inline constexpr const char* kNull = "a required pointer is NULL";
inline constexpr const char* kNoArgs = "args is NULL";

inline int check_table(int32_t rows, int64_t stride, int32_t width, int32_t page_size) {
  if (rows < 0 || width < 0) return fail(CTCPB_ERR_INVALID, "rows and table_width must be >= 0");
  if (!page_size_ok(page_size)) return fail(CTCPB_ERR_INVALID, kBadPage);
  if (stride < width) return fail(CTCPB_ERR_INVALID, "table_stride must be >= table_width");
  if ((int64_t)width * page_size > (1 << 30))
    return fail(CTCPB_ERR_INVALID, "table_width * page_size must be at most 2^30");
  return CTCPB_OK;
}

inline int check_pages(int32_t num_pages, int32_t page_size) {
  if (!page_size_ok(page_size)) return fail(CTCPB_ERR_INVALID, kBadPage);
  if (num_pages < 1 || (int64_t)num_pages * page_size > INT_MAX)
    return fail(CTCPB_ERR_INVALID, "num_pages must be >= 1 and num_pages * page_size below 2^31");
  return CTCPB_OK;
}

inline int check_cache(const ctcpb_lm_cache& c) {
  if (!c.data) return fail(CTCPB_ERR_INVALID, kNull);
  if (c.stride_page < 0 || c.stride_token < 0 || c.stride_head < 0)
    return fail(CTCPB_ERR_INVALID, "cache strides must be >= 0");
  return CTCPB_OK;
}

inline CacheView view(const ctcpb_lm_cache& c, int es) {
  return CacheView{static_cast<char*>(c.data), c.stride_page * es, c.stride_token * es,
                   c.stride_head * es};
}

inline bool wide_cache(const CacheView& v) {
  return aligned(v.data, 16) && v.page % 16 == 0 && v.token % 16 == 0 && v.head % 16 == 0;
}

}  // namespace ctcpb_lm
