// tree.h -- drafting with trees of tokens and the paged cache's books: host-side
// interfaces between the C ABI and the kernels.
#pragma once

#include "cache.h"

namespace lynx {

constexpr int kMaxPools = 256;           // pools of one call

struct LogprobArgs {
  const void* logits;
  int dtype;
  int64_t stride, rows, V;
  float scale;
  const int32_t* tokens;
  int given, top;
  float *logprob, *entropy, *top_logprob;
  int32_t* top_token;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);

cudaError_t launch_tree_plan(const int32_t* parents, const int32_t* kv_len, int batch, int T,
                             uint64_t* mask, int32_t* positions, cudaStream_t stream);
cudaError_t launch_tree_verify(const int32_t* parents, const int32_t* tokens,
                               const int32_t* answers, int batch, int T, int32_t* path,
                               int32_t* n_path, int32_t* next_token, cudaStream_t stream);

// The books of a paged cache.
struct BookArgs {
  int32_t *table, *kv_len, *refs;
  int64_t max_pages, nblocks;
  int batch, page;
};
cudaError_t launch_cache_fork(const BookArgs& in, const int32_t* source, int32_t* out_table,
                              int32_t* out_len, int out_batch, cudaStream_t stream);
cudaError_t launch_cache_reserve(const BookArgs& a, const int32_t* grow, int32_t* granted,
                                 int32_t* src, int32_t* dst, cudaStream_t stream);
cudaError_t launch_cache_trim(const BookArgs& a, const int32_t* keep, cudaStream_t stream);
cudaError_t launch_cache_compact(const BookArgs& a, int32_t* src, int32_t* dst, int32_t* count,
                                 cudaStream_t stream);

struct PoolList {
  int n;
  void* base[kMaxPools];
  int64_t bytes[kMaxPools];              // of a block, a multiple of 16
};
cudaError_t launch_cache_copy_pages(const PoolList& pools, int64_t nblocks, const int32_t* src,
                                    const int32_t* dst, int64_t n, const int32_t* count,
                                    cudaStream_t stream);
struct KeepArgs {
  CacheLayout c;                         // T: nodes
  const int32_t *path, *granted;
  int n_pools;
  const void* const* nodes;              // HOST [n_pools]
  void* const* pools;
};
cudaError_t launch_cache_keep(const KeepArgs& a, cudaStream_t stream);

cudaError_t read_logprobs_flags(unsigned int* flag);
cudaError_t read_cache_pages_flags(unsigned int* flag);

}  // namespace lynx
