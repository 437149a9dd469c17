// tree_api.cu -- the extern "C" boundary of tree drafting and of the paged cache's
// books declared in include/lynx.h: argument checks and dispatch.
#include <algorithm>

#include "checks.h"
#include "common.cuh"
#include "tree.h"

namespace lynx {
namespace {

int check_tree(int batch, int T) {
  if (batch < 0) return fail(LYNX_ESHAPE, "need batch >= 0");
  if (T < 1) return fail(LYNX_ESHAPE, "T = %d must be >= 1", T);
  if (T > kTreeRoom) return fail(LYNX_EUNSUPPORTED, "T = %d: at most %d nodes", T, kTreeRoom);
  if (batch > INT32_MAX / kTreeRoom)
    return fail(LYNX_EUNSUPPORTED, "batch * %d must be < 2^31", kTreeRoom);
  return LYNX_OK;
}

int check_books(int batch, int page, int64_t max_pages, int64_t num_blocks) {
  return check_layout(batch, 0, 0, 1, kCacheD, page, max_pages, num_blocks);
}

// Every buffer that is written apart from the others and from what is read.
template <int W, int R>
int check_buffers(const Span (&written)[W], const Span (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    for (int j = i + 1; j < W; ++j)
      if (int rc = check_apart(written[i], written[j])) return rc;
    for (const Span& r : read)
      if (int rc = check_apart(written[i], r)) return rc;
  }
  return LYNX_OK;
}

// The same for many buffers, those that are written among them: sorted by address, each
// has to begin behind the written ones before it, and a written one behind all.
struct Used {
  Span s;
  bool written;
};
int check_many(Used* u, int n) {
  const auto at = [](const Used& x) { return reinterpret_cast<uintptr_t>(x.s.p); };
  std::sort(u, u + n, [&](const Used& x, const Used& y) { return at(x) < at(y); });
  const Used *far = nullptr, *far_written = nullptr;     // the ones that reach furthest
  const auto end = [&](const Used* x) { return x ? at(*x) + x->s.bytes : 0; };
  for (int i = 0; i < n; ++i) {
    if (!u[i].s.p || !u[i].s.bytes) continue;
    const Used* const before = u[i].written ? far : far_written;
    if (at(u[i]) < end(before))
      return fail(LYNX_EINVAL, "%s overlaps %s", u[i].s.name, before->s.name);
    if (end(&u[i]) > end(far)) far = &u[i];
    if (u[i].written && end(&u[i]) > end(far_written)) far_written = &u[i];
  }
  return LYNX_OK;
}

int done(cudaError_t e, const char* what) { return e == cudaSuccess ? LYNX_OK : cuda_fail(e, what); }

uint64_t table_bytes(int batch, int64_t max_pages) {
  return 4 * (uint64_t)batch * (uint64_t)max_pages;
}

}  // namespace
}  // namespace lynx

using namespace lynx;

extern "C" {

int lynx_token_logprobs(const void* logits, int dtype, int64_t row_stride, int64_t rows, int64_t V,
                        float scale, const int32_t* tokens, int n_given, int top, float* logprob,
                        float* entropy, float* top_logprob, int32_t* top_token, void* stream) {
  if (dtype != LYNX_BF16 && dtype != LYNX_FP32 && dtype != LYNX_FP16)
    return fail(LYNX_EINVAL, "dtype = %d: LYNX_BF16, LYNX_FP32 or LYNX_FP16", dtype);
  if (rows < 0 || V < 1) return fail(LYNX_ESHAPE, "need rows >= 0 and V >= 1");
  if (rows > 1 << 30 || V > 1 << 30)
    return fail(LYNX_EUNSUPPORTED, "rows and V must be <= 2^30");
  if (row_stride < V) return fail(LYNX_ESHAPE, "row_stride = %lld: at least V", (long long)row_stride);
  if (row_stride > ((int64_t)1 << 40)) return fail(LYNX_EUNSUPPORTED, "row_stride: at most 2^40");
  if (!(scale >= 1e-6f && scale <= 1e6f)) return fail(LYNX_EINVAL, "scale must lie in 1e-6 .. 1e6");
  if (n_given < 0 || top < 0) return fail(LYNX_ESHAPE, "need n_given >= 0 and top >= 0");
  if (n_given > 64) return fail(LYNX_EUNSUPPORTED, "n_given = %d: at most 64", n_given);
  if (top > 32) return fail(LYNX_EUNSUPPORTED, "top = %d: at most 32", top);
  if (top > V) return fail(LYNX_ESHAPE, "top = %d of %lld tokens", top, (long long)V);
  if (rows == 0) return LYNX_OK;
  const unsigned size = dtype == LYNX_FP32 ? 4 : 2;
  int rc = check_ptr(logits, size, "logits");
  if (rc) return rc;
  if (n_given && ((rc = check_ptr(tokens, 4, "tokens")) || (rc = check_ptr(logprob, 4, "logprob"))))
    return rc;
  if (entropy && (rc = check_ptr(entropy, 4, "entropy"))) return rc;
  if (top && ((rc = check_ptr(top_logprob, 4, "top_logprob")) ||
              (rc = check_ptr(top_token, 4, "top_token"))))
    return rc;
  if (!n_given && !entropy && !top) return LYNX_OK;
  const uint64_t n = (uint64_t)rows;
  const Span out[] = {{n_given ? logprob : nullptr, 4 * n * n_given, "logprob"},
                      {entropy, 4 * n, "entropy"},
                      {top ? top_logprob : nullptr, 4 * n * top, "top_logprob"},
                      {top ? top_token : nullptr, 4 * n * top, "top_token"}};
  const Span in[] = {{logits, ((n - 1) * (uint64_t)row_stride + (uint64_t)V) * size, "logits"},
                     {n_given ? tokens : nullptr, 4 * n * n_given, "tokens"}};
  if ((rc = check_buffers(out, in))) return rc;
  LogprobArgs a;
  a.logits = logits;
  a.dtype = dtype;
  a.stride = row_stride;
  a.rows = rows;
  a.V = V;
  a.scale = scale;
  a.tokens = tokens;
  a.given = n_given;
  a.top = top;
  a.logprob = n_given ? logprob : nullptr;
  a.entropy = entropy;
  a.top_logprob = top_logprob;
  a.top_token = top_token;
  return done(launch_token_logprobs(a, static_cast<cudaStream_t>(stream)), "lynx_token_logprobs");
}

int lynx_tree_plan(const int32_t* parents, const int32_t* kv_len, int batch, int T, uint64_t* mask,
                   int32_t* positions, void* stream) {
  int rc = check_tree(batch, T);
  if (rc) return rc;
  if (batch == 0) return LYNX_OK;
  if ((rc = check_ptr(parents, 4, "parents")) || (rc = check_ptr(kv_len, 4, "kv_len"))) return rc;
  if (mask && (rc = check_ptr(mask, 8, "mask"))) return rc;
  if (positions && (rc = check_ptr(positions, 4, "positions"))) return rc;
  if (!mask && !positions) return LYNX_OK;
  const uint64_t n = (uint64_t)batch * T;
  const Span out[] = {{mask, 8 * n, "mask"}, {positions, 4 * n, "positions"}};
  const Span in[] = {{parents, 4 * n, "parents"}, {kv_len, 4 * (uint64_t)batch, "kv_len"}};
  if ((rc = check_buffers(out, in))) return rc;
  return done(launch_tree_plan(parents, kv_len, batch, T, mask, positions,
                               static_cast<cudaStream_t>(stream)), "lynx_tree_plan");
}

int lynx_tree_verify(const int32_t* parents, const int32_t* tokens, const int32_t* answers,
                     int batch, int T, int32_t* path, int32_t* n_path, int32_t* next_token,
                     void* stream) {
  int rc = check_tree(batch, T);
  if (rc) return rc;
  if (batch == 0) return LYNX_OK;
  if ((rc = check_ptr(parents, 4, "parents")) || (rc = check_ptr(tokens, 4, "tokens")) ||
      (rc = check_ptr(answers, 4, "answers")) || (rc = check_ptr(path, 4, "path")) ||
      (rc = check_ptr(n_path, 4, "n_path")) || (rc = check_ptr(next_token, 4, "next_token")))
    return rc;
  const uint64_t one = 4 * (uint64_t)batch, n = one * T;
  const Span out[] = {{path, n, "path"}, {n_path, one, "n_path"}, {next_token, one, "next_token"}};
  const Span in[] = {{parents, n, "parents"}, {tokens, n, "tokens"}, {answers, n, "answers"}};
  if ((rc = check_buffers(out, in))) return rc;
  return done(launch_tree_verify(parents, tokens, answers, batch, T, path, n_path, next_token,
                                 static_cast<cudaStream_t>(stream)), "lynx_tree_verify");
}

int lynx_cache_fork(const int32_t* block_table, const int32_t* kv_len, int32_t* refs,
                    int64_t max_pages, int64_t num_blocks, int page, int batch,
                    const int32_t* source, int out_batch, int32_t* out_table, int32_t* out_len,
                    void* stream) {
  int rc = check_books(batch, page, max_pages, num_blocks);
  if (rc) return rc;
  if ((rc = check_books(out_batch, page, max_pages, num_blocks))) return rc;
  if (batch > INT32_MAX / 8 || out_batch > INT32_MAX / 8)
    return fail(LYNX_EUNSUPPORTED, "batch and out_batch must be < 2^28");
  if (batch == 0 && out_batch == 0) return LYNX_OK;
  if ((rc = check_ptr(refs, 4, "refs"))) return rc;
  if (batch && ((rc = check_ptr(block_table, 4, "block_table")) || (rc = check_ptr(kv_len, 4, "kv_len"))))
    return rc;
  if (out_batch && ((rc = check_ptr(source, 4, "source")) || (rc = check_ptr(out_table, 4, "out_table")) ||
                    (rc = check_ptr(out_len, 4, "out_len"))))
    return rc;
  const Span out[] = {{out_table, table_bytes(out_batch, max_pages), "out_table"},
                      {out_len, 4 * (uint64_t)out_batch, "out_len"},
                      {refs, 4 * (uint64_t)num_blocks, "refs"}};
  const Span in[] = {{block_table, table_bytes(batch, max_pages), "block_table"},
                     {kv_len, 4 * (uint64_t)batch, "kv_len"},
                     {source, 4 * (uint64_t)out_batch, "source"}};
  if ((rc = check_buffers(out, in))) return rc;
  const BookArgs a{const_cast<int32_t*>(block_table), const_cast<int32_t*>(kv_len), refs, max_pages,
                   num_blocks, batch, page};
  return done(launch_cache_fork(a, source, out_table, out_len, out_batch,
                                static_cast<cudaStream_t>(stream)), "lynx_cache_fork");
}

int lynx_cache_reserve(int32_t* block_table, int32_t* kv_len, int32_t* refs, int64_t max_pages,
                       int64_t num_blocks, int page, int batch, const int32_t* grow,
                       int32_t* granted, int32_t* copy_src, int32_t* copy_dst, void* stream) {
  int rc = check_books(batch, page, max_pages, num_blocks);
  if (rc) return rc;
  if (batch == 0) return LYNX_OK;
  if ((rc = check_ptr(block_table, 4, "block_table")) || (rc = check_ptr(kv_len, 4, "kv_len")) ||
      (rc = check_ptr(refs, 4, "refs")) || (rc = check_ptr(grow, 4, "grow")) ||
      (rc = check_ptr(granted, 4, "granted")) || (rc = check_ptr(copy_src, 4, "copy_src")) ||
      (rc = check_ptr(copy_dst, 4, "copy_dst")))
    return rc;
  const uint64_t one = 4 * (uint64_t)batch;
  const Span out[] = {{block_table, table_bytes(batch, max_pages), "block_table"},
                      {kv_len, one, "kv_len"},
                      {refs, 4 * (uint64_t)num_blocks, "refs"},
                      {granted, one, "granted"},
                      {copy_src, one, "copy_src"},
                      {copy_dst, one, "copy_dst"}};
  const Span in[] = {{grow, one, "grow"}};
  if ((rc = check_buffers(out, in))) return rc;
  const BookArgs a{block_table, kv_len, refs, max_pages, num_blocks, batch, page};
  return done(launch_cache_reserve(a, grow, granted, copy_src, copy_dst,
                                   static_cast<cudaStream_t>(stream)), "lynx_cache_reserve");
}

int lynx_cache_trim(int32_t* block_table, int32_t* kv_len, int32_t* refs, int64_t max_pages,
                    int64_t num_blocks, int page, int batch, const int32_t* keep, void* stream) {
  int rc = check_books(batch, page, max_pages, num_blocks);
  if (rc) return rc;
  if (batch == 0) return LYNX_OK;
  if ((rc = check_ptr(block_table, 4, "block_table")) || (rc = check_ptr(kv_len, 4, "kv_len")) ||
      (rc = check_ptr(refs, 4, "refs")) || (rc = check_ptr(keep, 4, "keep")))
    return rc;
  const Span out[] = {{block_table, table_bytes(batch, max_pages), "block_table"},
                      {kv_len, 4 * (uint64_t)batch, "kv_len"},
                      {refs, 4 * (uint64_t)num_blocks, "refs"}};
  const Span in[] = {{keep, 4 * (uint64_t)batch, "keep"}};
  if ((rc = check_buffers(out, in))) return rc;
  const BookArgs a{block_table, kv_len, refs, max_pages, num_blocks, batch, page};
  return done(launch_cache_trim(a, keep, static_cast<cudaStream_t>(stream)), "lynx_cache_trim");
}

int lynx_cache_compact(int32_t* block_table, int32_t* kv_len, int32_t* refs, int64_t max_pages,
                       int64_t num_blocks, int page, int batch, int32_t* copy_src,
                       int32_t* copy_dst, int32_t* count, void* stream) {
  int rc = check_books(batch, page, max_pages, num_blocks);
  if (rc) return rc;
  if ((rc = check_ptr(refs, 4, "refs")) || (rc = check_ptr(count, 4, "count"))) return rc;
  if (batch && ((rc = check_ptr(block_table, 4, "block_table")) || (rc = check_ptr(kv_len, 4, "kv_len"))))
    return rc;
  if (num_blocks > 1 && ((rc = check_ptr(copy_src, 4, "copy_src")) ||
                         (rc = check_ptr(copy_dst, 4, "copy_dst"))))
    return rc;
  const uint64_t moves = 4 * (uint64_t)(num_blocks / 2);
  const Span out[] = {{block_table, table_bytes(batch, max_pages), "block_table"},
                      {refs, 4 * (uint64_t)num_blocks, "refs"},
                      {copy_src, moves, "copy_src"},
                      {copy_dst, moves, "copy_dst"},
                      {count, 4, "count"}};
  const Span in[] = {{kv_len, 4 * (uint64_t)batch, "kv_len"}};
  if ((rc = check_buffers(out, in))) return rc;
  const BookArgs a{block_table, kv_len, refs, max_pages, num_blocks, batch, page};
  return done(launch_cache_compact(a, copy_src, copy_dst, count, static_cast<cudaStream_t>(stream)),
              "lynx_cache_compact");
}

int lynx_cache_copy_pages(void* const* pools, const int64_t* block_bytes, int n_pools,
                          int64_t num_blocks, const int32_t* copy_src, const int32_t* copy_dst,
                          int64_t n, const int32_t* count, void* stream) {
  if (n < 0 || n_pools < 0) return fail(LYNX_ESHAPE, "need n >= 0 and n_pools >= 0");
  if (n_pools > kMaxPools) return fail(LYNX_EUNSUPPORTED, "n_pools = %d: at most %d", n_pools, kMaxPools);
  if (num_blocks < 1) return fail(LYNX_ESHAPE, "need num_blocks >= 1");
  if (num_blocks > INT32_MAX || n > INT32_MAX)
    return fail(LYNX_EUNSUPPORTED, "num_blocks and n must be < 2^31");
  if (n == 0 || n_pools == 0) return LYNX_OK;
  if (!pools || !block_bytes) return fail(LYNX_EINVAL, "pools, block_bytes: null pointer");
  int rc;
  if ((rc = check_ptr(copy_src, 4, "copy_src")) || (rc = check_ptr(copy_dst, 4, "copy_dst")))
    return rc;
  if (count && (rc = check_ptr(count, 4, "count"))) return rc;
  Used used[kMaxPools + 3] = {{{copy_src, 4 * (uint64_t)n, "copy_src"}, false},
                              {{copy_dst, 4 * (uint64_t)n, "copy_dst"}, false},
                              {{count, 4, "count"}, false}};
  PoolList list;
  list.n = n_pools;
  for (int i = 0; i < n_pools; ++i) {
    if ((rc = check_ptr(pools[i], 16, "a pool"))) return rc;
    if (block_bytes[i] < 16 || block_bytes[i] % 16)
      return fail(LYNX_ESHAPE, "block_bytes[%d] = %lld: a multiple of 16", i, (long long)block_bytes[i]);
    if (block_bytes[i] > (int64_t)1 << 36)      // (256 of them in 32 KiB pieces: 2^29)
      return fail(LYNX_EUNSUPPORTED, "block_bytes[%d]: at most 2^36", i);
    used[3 + i] = {{pools[i], (uint64_t)num_blocks * (uint64_t)block_bytes[i], "a pool"}, true};
    list.base[i] = pools[i];
    list.bytes[i] = block_bytes[i];
  }
  if ((rc = check_many(used, 3 + n_pools))) return rc;
  return done(launch_cache_copy_pages(list, num_blocks, copy_src, copy_dst, n, count,
                                      static_cast<cudaStream_t>(stream)), "lynx_cache_copy_pages");
}

int lynx_cache_keep(const void* const* nodes, void* const* pools, int n_pools, const int32_t* path,
                    const int32_t* granted, const int32_t* kv_len, const int32_t* block_table,
                    int64_t max_pages, int64_t num_blocks, int batch, int T, int H_kv, int D,
                    int page, void* stream) {
  int rc = check_layout(batch, 0, 0, H_kv, D, page, max_pages, num_blocks);
  if (rc) return rc;
  if ((rc = check_tree(batch, T))) return rc;
  if (n_pools < 0) return fail(LYNX_ESHAPE, "need n_pools >= 0");
  if (n_pools > kMaxPools) return fail(LYNX_EUNSUPPORTED, "n_pools = %d: at most %d", n_pools, kMaxPools);
  if ((int64_t)n_pools * batch * H_kv > INT32_MAX)
    return fail(LYNX_EUNSUPPORTED, "n_pools * batch * H_kv must be < 2^31");
  if (batch == 0 || n_pools == 0) return LYNX_OK;
  if (!nodes || !pools) return fail(LYNX_EINVAL, "nodes, pools: null pointer");
  if ((rc = check_ptr(path, 4, "path")) || (rc = check_ptr(granted, 4, "granted")) ||
      (rc = check_ptr(kv_len, 4, "kv_len")) || (rc = check_ptr(block_table, 4, "block_table")))
    return rc;
  const uint64_t one = 4 * (uint64_t)batch;
  const uint64_t pool = (uint64_t)num_blocks * page * H_kv * D * 2;
  const uint64_t node = (uint64_t)batch * kTreeRoom * H_kv * D * 2;
  Used used[2 * kMaxPools + 4] = {
      {{path, one * T, "path"}, false},
      {{granted, one, "granted"}, false},
      {{kv_len, one, "kv_len"}, false},
      {{block_table, table_bytes(batch, max_pages), "block_table"}, false}};
  for (int i = 0; i < n_pools; ++i) {
    if ((rc = check_ptr(nodes[i], 16, "a node buffer")) || (rc = check_ptr(pools[i], 16, "a pool")))
      return rc;
    used[4 + 2 * i] = {{nodes[i], node, "a node buffer"}, false};
    used[5 + 2 * i] = {{pools[i], pool, "a pool"}, true};
  }
  if ((rc = check_many(used, 4 + 2 * n_pools))) return rc;
  KeepArgs a;
  a.c = CacheLayout{block_table, kv_len, nullptr, max_pages, num_blocks, 0, batch, T, H_kv, page};
  a.path = path;
  a.granted = granted;
  a.n_pools = n_pools;
  a.nodes = nodes;
  a.pools = pools;
  return done(launch_cache_keep(a, static_cast<cudaStream_t>(stream)), "lynx_cache_keep");
}

}  // extern "C"
