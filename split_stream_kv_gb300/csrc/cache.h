// cache.h -- the BF16 paged cache: what its writer (cache_append.cu) and its
// readers (cache_attn.cu) share.
//
// A pool is [num_blocks][page][H_kv][128] BF16; block_table[batch][max_pages]
// names the physical page of each (sequence, logical page).  kv_len[b] counts
// the cached tokens of sequence b including the ones the call brings, so token
// t of its n new tokens is at position kv_len[b] - n + t.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "internal.h"

namespace lynx {

constexpr int kCacheD = 128;             // channels per head
constexpr int kMaxAxes = 4;
constexpr int kTreeRoom = 64;            // nodes of a tree, at most: rows of the node buffers
constexpr int kRopeMaxFreq = kCacheD / 2;

struct CacheLayout {
  const int32_t* table;     // [batch][max_pages]
  const int32_t* kv_len;    // [batch]
  const int32_t* offsets;   // [batch + 1] packed-token offsets, or null: T tokens each
  int64_t max_pages, nblocks, n_tokens;
  int batch, T, Hkv, page;
};

struct RopeArgs {
  int rot_dim = 0;
  bool interleaved = false;
  int n_axes = 0;
  const int32_t* positions = nullptr;   // device [n_axes][n_tokens], or null
  uint64_t turns[kRopeMaxFreq];         // inv_freq / 2 pi, 2^64 to a turn
  uint8_t axis[kRopeMaxFreq];
};

struct CacheAppendArgs {
  CacheLayout c;
  const void *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;   // elements from one token to the next
  void *k_pool, *v_pool, *q_out;
  int Hq;                                 // 0: no queries
};
cudaError_t launch_cache_append(const CacheAppendArgs& a, const RopeArgs& rope,
                                cudaStream_t stream);

struct CacheAttnArgs {
  CacheLayout c;
  const void* q;
  int64_t q_stride;
  const void *k_pool, *v_pool;
  int Hq;
  float scale, softcap;
  int64_t window;
  const float* slopes;
  const int32_t* prefix;
  void* out;
  float* lse;
  void* workspace;
  // a tree of T drafted nodes a sequence, not in the cache: which node sees which, and the
  // nodes' own keys and values [batch][kTreeRoom][H_kv][128]; null: T new tokens in a row
  const uint64_t* mask = nullptr;
  const void *k_nodes = nullptr, *v_nodes = nullptr;
};
// How a call's work is shared out on `sms` SMs (the LYNX_CACHE_ values of lynx.h).
// T = 0: packed chunks; tree: T nodes of a tree.
int cache_attn_form(int batch, int T, int64_t n_tokens, int Hq, int Hkv, int64_t max_tokens,
                    int sms, bool tree = false);
// 0: the call needs none.
size_t cache_attn_workspace_bytes(int batch, int T, int64_t n_tokens, int Hq, int Hkv,
                                  int64_t max_tokens, bool tree = false);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream);

// Launches `fn` as a programmatic dependent of the kernel before it in the stream:
// the blocks may start while that one ends, so the kernel waits
// (griddepcontrol.wait) before it touches global memory, and reads with plain loads:
// ld.global.nc (__ldg) is only for what nobody writes while the kernel is resident.
// cluster: CTAs to a cluster, 0: none.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*fn)(Params...), dim3 grid, unsigned threads, size_t smem,
                             unsigned cluster, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_cache_append_flags(unsigned int* flag);
cudaError_t read_cache_attn_flags(unsigned int* flag);
cudaError_t read_cache_prefill_flags(unsigned int* flag);

}  // namespace lynx
