// tree.cu -- trees of drafted tokens: which nodes see which, and the walk down a
// tree along what the model answered.
//
// A sequence's T <= 64 nodes are numbered parents first; node 0 is the root (parent
// -1), node t > 0 a child of a node before it.  Any other parent means that there is
// no node in that place, nor below it.  One warp a sequence, two nodes a lane:
//  * plan: mask[t] = bit t and the bits of t's ancestors.  Node t starts with its own bit
//    and a pointer to its parent; in each of six rounds it takes over the bits of
//    the node it points at, and that node's pointer, so that 2^6 steps up are
//    covered.  What does not reach the root is no node.
//  * verify: from the root on, the child whose token is the answer at the node
//    reached, the lowest where several have it, until there is none.
// Both are a few dependent loads and some hundred cycles: launch latency bounds them (6.2 us
// for 32 trees of 64 nodes in a graph, where adding 1 to a number takes 4.2).
#include "common.cuh"
#include "tree.h"

namespace lynx {

namespace {

constexpr int kTreeWarps = 4;

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int lane) {
  return __shfl_sync(kFull, v, lane);
}
// What node i of the warp's tree holds (nodes 32 .. 63 in the lanes' second values).
__device__ __forceinline__ uint64_t of_node(const uint64_t (&v)[2], int i) {
  const uint64_t a = shfl64(v[0], i & 31), b = shfl64(v[1], i & 31);
  return i < 32 ? a : b;
}
__device__ __forceinline__ int of_node(const int (&v)[2], int i) {
  const int a = __shfl_sync(kFull, v[0], i & 31), b = __shfl_sync(kFull, v[1], i & 31);
  return i < 32 ? a : b;
}

// The parent of place t, or -1 where t is the root, or -2 where there is no node.
__device__ __forceinline__ int parent_of(const int32_t* parents, int64_t at, int t, int T) {
  if (t >= T) return -2;
  const int p = parents[at + t];
  if (t == 0) return p == -1 ? -1 : -2;
  return p >= 0 && p < t ? p : -2;
}

__global__ void __launch_bounds__(32 * kTreeWarps)
tree_plan_kernel(const int32_t* parents, const int32_t* kv_len, int batch, int T, uint64_t* mask,
                 int32_t* positions) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * kTreeWarps + (threadIdx.x >> 5);
  if (b >= batch) return;
  const int64_t at = b * T;
  const int kv = max(kv_len[b], 0);
  uint64_t bits[2];
  int up[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    up[e] = parent_of(parents, at, t, T);
    bits[e] = up[e] == -2 ? 0 : 1ull << t;
  }
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    uint64_t b2[2];
    int u2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = up[e] < 0 ? 0 : up[e];
      const uint64_t q = of_node(bits, i);
      const int u = of_node(up, i);
      b2[e] = up[e] < 0 ? bits[e] : bits[e] | q;
      u2[e] = up[e] < 0 ? up[e] : u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      bits[e] = b2[e];
      up[e] = u2[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    if (t >= T) continue;
    const bool is = up[e] == -1;             // its pointer has passed the root
    if (mask) mask[at + t] = is ? bits[e] : 0;
    if (positions) positions[at + t] = is ? kv + __popcll(bits[e]) - 1 : -1;
  }
}

__global__ void __launch_bounds__(32 * kTreeWarps)
tree_verify_kernel(const int32_t* parents, const int32_t* tokens, const int32_t* answers, int batch,
                   int T, int32_t* path, int32_t* n_path, int32_t* next_token) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * kTreeWarps + (threadIdx.x >> 5);
  if (b >= batch) return;
  const int64_t at = b * T;
  int up[2], token[2], answer[2], on[2] = {-1, -1};   // on: what the path holds in places t
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    up[e] = parent_of(parents, at, t, T);
    token[e] = t < T ? tokens[at + t] : 0;
    answer[e] = t < T ? answers[at + t] : 0;
  }
  int n = 0, next = -1;
  int here = __shfl_sync(kFull, up[0], 0) == -1 ? 0 : -1;
  while (here >= 0) {                        // (at most T turns: children come behind parents)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e == n) on[e] = here;
    ++n;
    next = of_node(answer, here);
    const unsigned lo = __ballot_sync(kFull, up[0] == here && token[0] == next);
    const unsigned hi = __ballot_sync(kFull, up[1] == here && token[1] == next);
    here = lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : -1;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < T) path[at + lane + 32 * e] = on[e];
  if (lane == 0) {
    n_path[b] = n;
    next_token[b] = next;
  }
}

}  // namespace

cudaError_t launch_tree_plan(const int32_t* parents, const int32_t* kv_len, int batch, int T,
                             uint64_t* mask, int32_t* positions, cudaStream_t stream) {
  return launch_dependent(tree_plan_kernel, dim3((unsigned)((batch + kTreeWarps - 1) / kTreeWarps)),
                          32 * kTreeWarps, 0, 0, stream, parents, kv_len, batch, T, mask, positions);
}

cudaError_t launch_tree_verify(const int32_t* parents, const int32_t* tokens,
                               const int32_t* answers, int batch, int T, int32_t* path,
                               int32_t* n_path, int32_t* next_token, cudaStream_t stream) {
  return launch_dependent(tree_verify_kernel,
                          dim3((unsigned)((batch + kTreeWarps - 1) / kTreeWarps)), 32 * kTreeWarps,
                          0, 0, stream, parents, tokens, answers, batch, T, path, n_path, next_token);
}

}  // namespace lynx
