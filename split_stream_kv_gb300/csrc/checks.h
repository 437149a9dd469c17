// checks.h -- checks of arguments that the C ABI of the paged cache shares.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "cache.h"
#include "lynx.h"

namespace lynx {

inline int fail(int code, const char* fmt, ...) {
  char msg[200];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return report_error(code, msg);
}

inline int check_ptr(const void* p, unsigned align, const char* what) {
  if (!p) return fail(LYNX_EINVAL, "%s: null pointer", what);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return fail(LYNX_EINVAL, "%s: not %u-byte aligned", what, align);
  return LYNX_OK;
}

// A buffer a call reads or writes, for the overlap check.
struct Span {
  const void* p;
  uint64_t bytes;
  const char* name;
};
inline int check_apart(const Span& w, const Span& r) {
  if (!w.p || !r.p || !w.bytes || !r.bytes) return LYNX_OK;
  const uint64_t a = reinterpret_cast<uintptr_t>(w.p), b = reinterpret_cast<uintptr_t>(r.p);
  if (a < b + r.bytes && b < a + w.bytes)
    return fail(LYNX_EINVAL, "%s overlaps %s", w.name, r.name);
  return LYNX_OK;
}

inline int check_layout(int batch, int64_t n_tokens, int H_q, int H_kv, int D, int page,
                 int64_t max_pages, int64_t num_blocks) {
  if (batch < 0 || n_tokens < 0) return fail(LYNX_ESHAPE, "need batch >= 0 and n_tokens >= 0");
  if (H_kv < 1 || H_q < 0) return fail(LYNX_ESHAPE, "need H_kv >= 1 and H_q >= 0");
  if (D != kCacheD) return fail(LYNX_EUNSUPPORTED, "D = %d: only D = 128 is built", D);
  if (page != 64 && page != 128 && page != 256 && page != 512)
    return fail(LYNX_EUNSUPPORTED, "page = %d: built for 64 ... 512 (powers of two)", page);
  if (max_pages < 1 || num_blocks < 1)
    return fail(LYNX_ESHAPE, "need max_pages >= 1 and num_blocks >= 1");
  if (num_blocks > (int64_t)INT32_MAX / page)
    return fail(LYNX_EUNSUPPORTED, "num_blocks * page must be < 2^31");
  if (max_pages > ((int64_t)INT32_MAX + 1 - 512) / page)
    return fail(LYNX_EUNSUPPORTED, "max_pages * page must be <= 2^31 - 512");
  if ((int64_t)batch * H_kv > INT32_MAX / 4)
    return fail(LYNX_EUNSUPPORTED, "batch * H_kv must be < 2^29");
  const int64_t heads = (int64_t)H_q + 2 * (int64_t)H_kv;
  if (n_tokens > INT32_MAX / heads)
    return fail(LYNX_EUNSUPPORTED, "n_tokens * heads must be < 2^31");
  return LYNX_OK;
}

inline int check_stride(int64_t stride, int heads, const char* what) {
  if (stride < (int64_t)heads * kCacheD || stride % 8)
    return fail(LYNX_ESHAPE, "%s = %lld: a multiple of 8 and at least %lld elements", what,
                (long long)stride, (long long)heads * kCacheD);
  if (stride > ((int64_t)1 << 31)) return fail(LYNX_EUNSUPPORTED, "%s: at most 2^31", what);
  return LYNX_OK;
}

inline uint64_t rows_bytes(int64_t n, int64_t stride, int heads) {
  return n < 1 ? 0 : ((uint64_t)(n - 1) * (uint64_t)stride + (uint64_t)heads * kCacheD) * 2;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(LYNX_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace lynx
