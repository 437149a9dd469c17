// cache_attn.h -- parameters and device helpers shared by the kernels that
// read the BF16 paged cache.
#pragma once

#include <float.h>

#include "cache.h"
#include "common.cuh"

namespace lynx {

struct CacheParams {
  const uint16_t* q;
  int64_t q_stride;                          // elements from one token to the next
  const int32_t *table, *kv_len, *offsets;   // offsets null: T tokens a sequence
  int64_t max_pages, nblocks, n_tokens;
  int batch, T, Hq, Hkv, G, lgP;
  int RT;                                    // query rows per unit
  int window;                                // INT_MAX: none
  const int32_t* prefix;                     // or null
  const float* slopes;                       // or null
  // scores in base 2: s * qk, or cap_out * tanh(s * scale / softcap), the tanh
  // from 2^(s * cap_in)
  float qk, cap_in, cap_out;
  float cap_small, cap_poly[4];              // see cache_cap_factor
  uint16_t* out;
  float* lse;                                // or null
  float* part;                               // partials of the split, see cache_attn.cu
  const uint64_t* mask;                      // of a tree's nodes [batch][T], see Tensors
  int n_cta;
  int tail0, tail_parts;                     // cache_prefill.cu: units cut in parts, from tail0 on
};

// The tensors a kernel reads by TMA.  With TREE the T tokens of a sequence are nodes of
// a tree: their keys and values, rows 64 b .. of their own tensors, are one more tile behind
// the cache's, of which node t sees the columns that are set in its mask; its position
// is kv_len plus the number of its other bits (its depth) less one.
template <bool TREE>
struct Tensors {
  CUtensorMap k, v;
};
template <>
struct Tensors<true> {
  CUtensorMap k, v, k_nodes, v_nodes;
};

constexpr int kKeyTile = 64;    // cached tokens per tile: never across a page

// One sequence of a call.
struct Seq {
  int n;            // new tokens
  int64_t tok0;     // packed index of the first
  int pos0;         // its position (negative: fewer cached tokens than new ones)
  int kv;           // cached tokens
  int pf;           // tokens visible to every row
};

// EARLY: before the kernel's own wait, behind a kernel that has waited itself and only
// reads these.  They are in L2 then; what L1 holds is not ordered without a wait.
template <bool EARLY>
__device__ __forceinline__ int32_t load_len(const int32_t* p) {
  return EARLY ? __ldcg(p) : *p;
}
template <bool EARLY = false, bool TREE = false>
__device__ __forceinline__ Seq load_seq(const CacheParams& a, int b) {
  Seq s;
  if (a.offsets) {
    int64_t o0 = load_len<EARLY>(a.offsets + b), o1 = load_len<EARLY>(a.offsets + b + 1);
    o0 = o0 < 0 ? 0 : o0 > a.n_tokens ? a.n_tokens : o0;
    o1 = o1 < o0 ? o0 : o1 > a.n_tokens ? a.n_tokens : o1;
    s.tok0 = o0;
    s.n = (int)(o1 - o0);
  } else {
    s.tok0 = (int64_t)b * a.T;
    s.n = a.T;
  }
  const int64_t room = a.max_pages << a.lgP;
  int64_t kv = load_len<EARLY>(a.kv_len + b);
  kv = kv < 0 ? 0 : kv > room ? room : kv;
  s.kv = (int)kv;
  s.pos0 = TREE ? s.kv : s.kv - s.n;       // (of a tree: the root's)
  int pf = a.prefix ? load_len<EARLY>(a.prefix + b) : 0;
  s.pf = pf < 0 ? 0 : pf > s.kv ? s.kv : pf;
  return s;
}

template <int TILE>
__device__ __forceinline__ int node_tile(int kv) { return (kv + TILE - 1) / TILE; }

// Node t of a tree's mask, and its depth (-1: no node).
__device__ __forceinline__ uint64_t tree_mask(const CacheParams& a, int b, int t) {
  const uint64_t own = a.mask[(int64_t)b * a.T + t];
  return a.T < 64 ? own & ((1ull << a.T) - 1ull) : own;
}
__device__ __forceinline__ int tree_depth(const CacheParams& a, int b, int t) {
  return __popcll(tree_mask(a, b, t)) - 1;
}
// A lane's part of a tree's masks (nodes lane and lane + 32), and from the warp's parts
// the nodes that any node sees.  What is in the others' places may be anything.
struct MaskPart {
  uint64_t lo, hi;
};
__device__ __forceinline__ MaskPart mask_part(const CacheParams& a, int b, int lane) {
  MaskPart p;
  p.lo = lane < a.T ? tree_mask(a, b, lane) : 0;
  p.hi = lane + 32 < a.T ? tree_mask(a, b, lane + 32) : 0;
  return p;
}
__device__ __forceinline__ uint64_t any_sees(const MaskPart& p) {
  const uint64_t m = p.lo | p.hi;
  const uint32_t l = __reduce_or_sync(kFull, (uint32_t)m);
  return (uint64_t)__reduce_or_sync(kFull, (uint32_t)(m >> 32)) << 32 | l;
}
// The nodes that node t sees: its mask without those that lie outside of the window.
__device__ __forceinline__ uint64_t tree_sees(const CacheParams& a, int b, int t) {
  uint64_t m = tree_mask(a, b, t);
  if (a.window < 64) {                       // (a depth is below 64)
    const int depth = __popcll(m) - 1;
    for (uint64_t left = m; left; left &= left - 1) {
      const int c = __ffsll((long long)left) - 1;
      if (depth - tree_depth(a, b, c) >= a.window) m &= ~(1ull << c);
    }
  }
  return m;
}

// The key tiles that tokens t0 .. t1 of a sequence see: the tiles of the
// prefix, then those from the oldest window start to the newest position.
// Logical tile x is tile x for x < nA, else tile x - nA + B0.
struct TileRange {
  int nA, B0, nt;
  __device__ __forceinline__ int tile(int x) const { return x < nA ? x : x - nA + B0; }
};

// With TREE: what the root sees, and then the nodes' tile, which is node_tile().
template <int TILE, bool TREE = false>
__device__ __forceinline__ TileRange tiles_of(const CacheParams& a, const Seq& s, int t0, int t1) {
  TileRange r{0, 0, 0};
  const int pmax = s.pos0 + t1;
  if (s.n == 0 || (!TREE && pmax < 0)) return r;
  const int pmin = TREE ? s.pos0 : s.pos0 + t0 > 0 ? s.pos0 + t0 : 0;
  const int lo = pmin - a.window + 1 > 0 ? pmin - a.window + 1 : 0;
  const int B0 = lo / TILE;
  const int B1 = TREE ? node_tile<TILE>(s.kv) + 1 : pmax / TILE + 1;    // pmax < kv
  const int A1 = (s.pf + TILE - 1) / TILE;
  if (A1 == 0) {
    r.B0 = B0;
    r.nt = B1 - B0;
  } else if (A1 >= B0) {
    r.nt = A1 > B1 ? A1 : B1;
  } else {
    r.nA = A1;
    r.B0 = B0;
    r.nt = A1 + B1 - B0;
  }
  return r;
}

__device__ __forceinline__ float cache_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float cache_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The capped score of |s| <= cap_small, that is |x| <= 0.5 for the tanh's argument
// x: tanh(x) / x as a polynomial of degree 3 in x^2, fitted for the least relative
// error on that range (5.4e-07), with the scale and the cap folded into the
// coefficients: s * cache_cap_factor(s).
constexpr double kCapSmall = 0.5;
constexpr int kCapTerms = 4;
constexpr double kTanhPoly[kCapTerms] = {0.9999994557833092, -0.333263179620872,
                                         0.13190296708500462, -0.04440222620089697};
__device__ __forceinline__ f2 cache_cap_factor(const CacheParams& a, f2 s) {
  const f2 z = mul2(s, s);
  f2 r = make_float2(a.cap_poly[kCapTerms - 1], a.cap_poly[kCapTerms - 1]);
#pragma unroll
  for (int i = kCapTerms - 2; i >= 0; --i) r = fma2(z, r, make_float2(a.cap_poly[i], a.cap_poly[i]));
  return r;
}

// Raw product q.k to a base-2 score, before the distance bias.  Capped far from
// zero: tanh(x) = 1 - 2 / (1 + e^2x), two function-unit operations, within 2^-22
// of the cap.  (tanh.approx is off by up to 2^-11 of the score: at a score of 30,
// 2 % of a weight.)  Below half a cap, where 2^-22 of it would be much of the
// score, the polynomial keeps the relative error.
__device__ __forceinline__ float cache_cap_far(const CacheParams& a, float s) {
  const float e = cache_ex2(__fmul_rn(s, a.cap_in));
  return fmaf(-2.0f * a.cap_out, cache_rcp(__fadd_rn(1.0f, e)), a.cap_out);
}
template <bool CAP>
__device__ __forceinline__ float cache_score(const CacheParams& a, float s) {
  if constexpr (CAP) {
    const float z = __fmul_rn(s, s);
    float r = a.cap_poly[kCapTerms - 1];
#pragma unroll
    for (int i = kCapTerms - 2; i >= 0; --i) r = fmaf(z, r, a.cap_poly[i]);
    return fabsf(s) <= a.cap_small ? __fmul_rn(s, r) : cache_cap_far(a, s);
  } else {
    return __fmul_rn(s, a.qk);
  }
}

// Waits, whatever became of the CTA's other waits, until the copies of items 0 .. n - 1
// have landed, item i on barrier i % ring: the CTA's shared memory must not go before
// them.  An item is issued only when the one before it in its place has landed, so
// the last `ring` tell.  (Bounded as well.)
__device__ __forceinline__ void drain_copies(uint64_t* full, int ring, int n, unsigned int* flag) {
  for (int i = n > ring ? n - ring : 0; i < n; ++i)
    if (!mbar_wait(&full[i % ring], (uint32_t)(i / ring) & 1u)) atomicOr(flag, kFlagWaitTimeout);
}

// A head's slope in base 2.  Kept finite if it is: an infinite one would turn the
// distance of zero into a NaN.
__device__ __forceinline__ float cache_slope(float s) {
  const float v = __fmul_rn(s, 1.4426950408889634f);
  return fabsf(v) > FLT_MAX && fabsf(s) <= FLT_MAX ? copysignf(FLT_MAX, s) : v;
}

// A row's sum of weights l at its maximum m (base 2): what its output is divided by,
// and its log-sum.  A row that sees nothing has l = 0.  A query that is not a number has
// l = NaN (at any m: a maximum passes a NaN over), and NaN is its answer too.
__device__ __forceinline__ float cache_inv(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float cache_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// (m, l, o) of two parts of a row, base 2.  A part without weights is left out by its
// sum, not by its maximum, which is -inf for a NaN as well.
__device__ __forceinline__ void cache_merge(float& M, float& L, float4& O, float m, float l, float4 o) {
  if (l == 0.f) return;
  const float Mn = fmaxf(M, m);
  const float fo = cache_ex2(M - Mn), fn = cache_ex2(m - Mn);
  O.x = O.x * fo + fn * o.x;
  O.y = O.y * fo + fn * o.y;
  O.z = O.z * fo + fn * o.z;
  O.w = O.w * fo + fn * o.w;
  L = L * fo + fn * l;
  M = Mn;
}

// The many-row kernel (cache_prefill.cu).
int cache_prefill_form(int batch, int64_t n_tokens, int G, int Hkv, int64_t max_tokens, int sms,
                       bool tree);
size_t cache_prefill_workspace_bytes(int batch, int64_t n_tokens, int G, int Hkv,
                                     int64_t max_tokens, bool tree);
cudaError_t launch_cache_prefill(const CacheParams& p, bool cap, const Tensors<true>& maps,
                                 cudaStream_t stream);
// The maps a kernel without a tree takes.
template <bool TREE>
inline Tensors<TREE> tensors_of(const Tensors<true>& m) {
  if constexpr (TREE) return m;
  else return Tensors<false>{m.k, m.v};
}

}  // namespace lynx
