// logprobs.cu -- log probabilities of given tokens, the entropy and the likeliest
// tokens of rows of logits, in one pass over them.
//
//   z = scale x,  lse = ln sum e^z,  logprob(t) = z_t - lse,
//   H = lse - sum p z,  the k tokens of the largest x, the lowest first among equals
//
// One reading.  A thread holds a reference r near its largest logit, and with
// y = (x - r) scale log2 e the sums s = sum 2^y and t = sum 2^y y; r is raised only
// when a logit exceeds it by 2^8 in 2^y, so that most elements cost a subtraction, a
// product, a maximum, an exponential and two sums.  (The difference is taken before the
// product: rows whose logits are all the type's lowest value have a finite y.)  Parts
// join as in any softmax: s = sum f s_i, t = sum f (t_i + s_i d_i), d_i = (r_i - r) scale
// log2 e, f = 2^d_i.  Then lse = r scale + ln s and H = ln s - ln 2 t / s.
//
// The likeliest tokens.  Every element has a 64-bit key, its value's bits in an order
// of integers and the complement of its index, so that keys are distinct and the
// order of equals is part of them.  A block keeps a key that k others are known not
// to fall below, and collects in shared memory what does not fall below it: after
// the first elements that is seldom (rank k of n seen: k / n of what follows).
// Where many threads of a chunk of 4096 elements qualify, the bound is first raised to
// the k-th largest of the chunk's 64 group maxima, which k of its elements reach; what
// then remains lies in k groups of 64 elements.  So the buffer holds whatever comes
// (constant rows, sorted ones), and is ranked down to k when it holds more than 128.
// Keys decide, not arrival: the result does not depend on the order of the atomics.
//
// What bounds it: memory, with one exponential an element beside it (16 a cycle and SM).
// Few rows are split over clusters of up to eight CTAs, whose sums and candidates meet
// in the first one's shared memory.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "lynx.h"
#include "tree.h"

namespace lynx {

__device__ unsigned int g_logprobs_flags = 0;

cudaError_t read_logprobs_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_logprobs_flags, sizeof(unsigned int));
}

namespace lp {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 16;                       // elements a thread takes of a chunk
constexpr int kChunk = kPer * kThreads;
constexpr int kGroups = 64;                    // of four lanes: 64 elements of a chunk each
constexpr int kKeep = 128;                     // candidates that wait before they are ranked
constexpr int kFew = 64;                       // threads that may qualify without a new bound
constexpr int kMaxTop = 32;
static_assert(kMaxTop <= kGroups && kFew * kPer <= kMaxTop * (kChunk / kGroups), "the buffer");
constexpr int kBuffer = kKeep + kMaxTop * (kChunk / kGroups);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeast = -16384.f;             // 2^y is 0 long before

struct Params {
  const void* x;
  int64_t stride, rows, V;
  float scale, qs;                             // qs = scale log2 e
  float rise;                                  // logits by which 2^y grows by 2^8
  const int32_t* tokens;
  int given, top;
  float *logprob, *entropy, *top_logprob;
  int32_t* top_token;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Types: bits of -inf, values of a 16-byte vector.
template <class T> struct Type;
template <> struct Type<float> {
  static constexpr uint32_t none = 0xff800000u;
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};
template <> struct Type<__nv_bfloat16> {
  static constexpr uint32_t none = 0xff80ff80u;
  static __device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 p = bf2_to_f2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
};
template <> struct Type<__half> {
  static constexpr uint32_t none = 0xfc00fc00u;
  static __device__ __forceinline__ float value(__half x) { return __half2float(x); }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
};

// The key of a logit above -inf (both zeros are one value).
__device__ __forceinline__ uint64_t key_of(float x, int64_t index) {
  uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
  u ^= u >> 31 ? 0xffffffffu : 0x80000000u;
  return (uint64_t)u << 32 | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ int32_t index_of(uint64_t key) {
  return (int32_t)(0xffffffffu - (uint32_t)key);
}

// What a part of a row comes to.  r = -inf: nothing seen (s = t = 0, or NaN).
struct Sums {
  float r, s, t;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float qs) {
  Sums c;
  c.r = fmaxf(a.r, b.r);
  auto part = [&](const Sums& p) {
    const bool none = p.r == -INFINITY;
    const float d = none ? kLeast : max_nan(__fmul_rn(__fsub_rn(p.r, c.r), qs), kLeast);
    const float f = ex2(d);
    return make_float2(__fmul_rn(f, p.s), __fmul_rn(f, fmaf(p.s, d, p.t)));
  };
  const float2 x = part(a), y = part(b);
  c.s = __fadd_rn(x.x, y.x);
  c.t = __fadd_rn(x.y, y.y);
  return c;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint64_t ld_peer64(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_peer32(const void* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}

struct Shared {
  uint64_t buffer[kBuffer];
  uint64_t best[kMaxTop];                      // the largest keys in order, 0: none
  uint64_t group[kGroups];
  uint64_t bound;
  uint32_t votes[2][kWarps];
  uint32_t count;
  Sums part[kWarps];
  Sums total;
};

// The `top` largest of sh.buffer's n keys, in order, to sh.best (0 behind the last).
// All threads; the buffer may be written again after the caller's next barrier.
__device__ __forceinline__ void rank_buffer(Shared& sh, int n, int top) {
  if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t own = sh.buffer[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += sh.buffer[j] > own;
    if (above < top) sh.best[above] = own;
  }
  __syncthreads();
}

}  // namespace lp

template <class T>
__global__ void __launch_bounds__(lp::kThreads, 4)
token_logprobs_kernel(const __grid_constant__ lp::Params a) {
  using namespace lp;
  constexpr int VE = 16 / (int)sizeof(T), NV = kPer / VE;    // elements of a vector, vectors
  __shared__ Shared sh;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int csize = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t row = blockIdx.x / (unsigned)csize;
  const int top = a.top;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = 0;
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  // vectors of the row, the first one holding `off` elements before it
  const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int64_t nvec = (a.V + off + VE - 1) / VE;
  const int64_t share = (nvec + csize - 1) / csize;
  const int64_t v0 = share * rank < nvec ? share * rank : nvec;
  const int64_t v1 = v0 + share < nvec ? v0 + share : nvec;
  const int chunks = (int)((v1 - v0 + NV * kThreads - 1) / (NV * kThreads));

  auto load = [&](int c, uint4 (&raw)[NV]) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int64_t v = v0 + ((int64_t)c * NV + u) * kThreads + tid, e = v * VE - off;
      if (v < v1 && e >= 0 && e + VE <= a.V) {
        raw[u] = ld16(x + e);
      } else {                                 // the row's ends, and behind the share
        uint32_t q[4] = {Type<T>::none, Type<T>::none, Type<T>::none, Type<T>::none};
        if (v < v1) {
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (e + i >= 0 && e + i < a.V) {
              if constexpr (sizeof(T) == 4) {
                q[i] = *reinterpret_cast<const uint32_t*>(x + e + i);
              } else {
                const uint32_t h = *reinterpret_cast<const uint16_t*>(x + e + i);
                q[i >> 1] = i & 1 ? (q[i >> 1] & 0xffffu) | h << 16 : (q[i >> 1] & 0xffff0000u) | h;
              }
            }
        }
        raw[u] = make_uint4(q[0], q[1], q[2], q[3]);
      }
    }
  };

  Sums own = {-INFINITY, 0.f, 0.f};
  float minus_r = 0.f, trigger = -INFINITY;    // -r (0 without one), what raises it
  uint64_t bound = 0;
  float least = top > 0 ? -FLT_MAX : NAN;      // of a candidate
  bool full = false;                           // this thread's last candidate lies behind kKeep
  uint4 raw[2][NV];
  load(0, raw[0]);
#pragma unroll 1
  for (int c2 = 0; c2 < chunks; c2 += 2) {
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int c = c2 + odd;
      if (c >= chunks) break;
      if (c + 1 < chunks) load(c + 1, raw[odd ^ 1]);
      float f[kPer];
#pragma unroll
      for (int u = 0; u < NV; ++u) Type<T>::unpack(raw[odd][u], f + u * VE);
      float mx = f[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) mx = fmaxf(mx, f[i]);
      // ---- the sums
      if (mx > trigger) {
        const float d = own.r == -INFINITY
                            ? kLeast : max_nan(__fmul_rn(__fsub_rn(own.r, mx), a.qs), kLeast);
        const float g = ex2(d);
        own.t = __fmul_rn(g, fmaf(own.s, d, own.t));
        own.s = __fmul_rn(g, own.s);
        own.r = mx;
        minus_r = -mx;
        trigger = __fadd_rn(mx, a.rise);
      }
      f2 s = make_float2(own.s, 0.f), t = make_float2(own.t, 0.f);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const f2 y = mul2(add2(make_float2(f[i], f[i + 1]), make_float2(minus_r, minus_r)),
                          make_float2(a.qs, a.qs));
        const f2 z = make_float2(max_nan(y.x, kLeast), max_nan(y.y, kLeast));
        const f2 e = make_float2(ex2(z.x), ex2(z.y));
        s = add2(s, e);
        t = fma2(e, z, t);
      }
      own.s = __fadd_rn(s.x, s.y);
      own.t = __fadd_rn(t.x, t.y);
      // ---- candidates
      if (top == 0) continue;
      auto index = [&](int i) {
        return (v0 + ((int64_t)c * NV + i / VE) * kThreads + tid) * VE - off + i % VE;
      };
      const unsigned here = __ballot_sync(kFull, mx >= least);
      const unsigned over = __ballot_sync(kFull, full);
      if (lane == 0) sh.votes[c & 1][w] = (uint32_t)__popc(here) | (over ? 1u << 16 : 0u);
      __syncthreads();
      uint32_t sum = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += sh.votes[c & 1][i];
      if (sum == 0) continue;
      if (sum >> 16) {                         // many wait: the best stay
        rank_buffer(sh, (int)sh.count, top);
        if (tid < top) sh.buffer[tid] = sh.best[tid];
        bound = sh.best[top - 1] > bound ? sh.best[top - 1] : bound;
        if (tid == 0) sh.count = (uint32_t)top;
        full = false;
        least = bound ? value_of(bound) : least;
        __syncthreads();
      }
      if ((sum & 0xffffu) > (uint32_t)kFew) {
        // the k-th largest of the groups' maxima: k elements reach it
        uint64_t k = 0;
        if (mx > -INFINITY) {
          int at = 0;
#pragma unroll
          for (int i = kPer - 1; i >= 0; --i) at = f[i] == mx ? i : at;
          k = key_of(mx, index(at));
        }
#pragma unroll
        for (int o = 1; o < kThreads / kGroups; o <<= 1) {
          const uint64_t q = __shfl_xor_sync(kFull, k, o);
          k = q > k ? q : k;
        }
        if (lane % (kThreads / kGroups) == 0) sh.group[tid / (kThreads / kGroups)] = k;
        __syncthreads();
        if (tid < kGroups) {
          const uint64_t q = sh.group[tid];
          int above = 0;
#pragma unroll 8
          for (int j = 0; j < kGroups; ++j) above += sh.group[j] > q;
          if (q && above == top - 1) sh.bound = q;
        }
        __syncthreads();
        bound = sh.bound > bound ? sh.bound : bound;
        least = bound ? value_of(bound) : least;
      }
      if (mx >= least) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (f[i] >= least) {
            const uint64_t k = key_of(f[i], index(i));
            if (k >= bound) {
              const uint32_t at = atomicAdd(&sh.count, 1u);
              if (at < (uint32_t)kBuffer) sh.buffer[at] = k;
              full = full || at >= (uint32_t)kKeep;
            }
          }
      }
    }
  }
  // ---- the block's sums and its best
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sums p;
    p.r = __shfl_xor_sync(kFull, own.r, o);
    p.s = __shfl_xor_sync(kFull, own.s, o);
    p.t = __shfl_xor_sync(kFull, own.t, o);
    own = join(own, p, a.qs);
  }
  if (lane == 0) sh.part[w] = own;
  __syncthreads();
  if (top > 0) rank_buffer(sh, (int)sh.count, top);
  if (tid == 0) {
    Sums p = sh.part[0];
    for (int i = 1; i < kWarps; ++i) p = join(p, sh.part[i], a.qs);
    sh.total = p;
  }
  if (csize > 1) {
    cluster_sync();                            // every part is there
    if (rank == 0) {
      if (top > 0) {
        for (int i = tid; i < csize * top; i += kThreads)
          sh.buffer[i] = ld_peer64(&sh.best[i % top], (uint32_t)(i / top));
      }
      if (tid == 0) {
        Sums p = sh.total;
        for (int k = 1; k < csize; ++k) {
          Sums q;
          q.r = ld_peer32(&sh.total.r, (uint32_t)k);
          q.s = ld_peer32(&sh.total.s, (uint32_t)k);
          q.t = ld_peer32(&sh.total.t, (uint32_t)k);
          p = join(p, q, a.qs);
        }
        sh.part[0] = p;
      }
      __syncthreads();
      if (tid == 0) sh.total = sh.part[0];
      // (empty places hold 0 and rank behind every key; only keys are written)
      if (top > 0) {
        __syncthreads();
        if (tid < kMaxTop) sh.best[tid] = 0;
        __syncthreads();
        for (int i = tid; i < csize * top; i += kThreads) {
          const uint64_t k = sh.buffer[i];
          int above = 0;
          for (int j = 0; j < csize * top; ++j) above += sh.buffer[j] > k;
          if (k && above < top) sh.best[above] = k;
        }
      }
    }
    cluster_sync();                            // the parts have been read
    if (rank != 0) return;
  }
  __syncthreads();
  // ---- the row's answers
  const Sums all = sh.total;
  const bool none = all.r == -INFINITY && all.s == 0.f;        // every logit is -inf
  const float ln = none ? 0.f : logf(all.s);
  auto logprob = [&](float v) {
    return none || v == -INFINITY ? (all.s != all.s ? all.s : -INFINITY)
                                  : __fsub_rn(__fmul_rn(__fsub_rn(v, all.r), a.scale), ln);
  };
  if (a.entropy && tid == 0)
    a.entropy[row] = none ? 0.f : __fsub_rn(ln, __fmul_rn(__fdiv_rn(all.t, all.s), kLn2));
  if (tid < top) {
    const uint64_t k = sh.best[tid];
    if (a.top_logprob) a.top_logprob[row * top + tid] = k ? logprob(value_of(k)) : -INFINITY;
    if (a.top_token) a.top_token[row * top + tid] = k ? index_of(k) : -1;
  }
  if (a.logprob) {
    for (int i = tid; i < a.given; i += kThreads) {
      const int64_t token = a.tokens[row * a.given + i];
      float v = -INFINITY;
      const bool in = token >= 0 && token < a.V;
      if (in) v = logprob(Type<T>::value(x[token]));
      else if (token >= a.V) atomicOr(&g_logprobs_flags, kFlagBadToken);
      a.logprob[row * a.given + i] = v;
    }
  }
}

// CTAs to a row: as many as are resident at once (four to an SM), a chunk each at least.
static int cluster_for(int64_t rows, int64_t V, int sms) {
  int c = 1;
  while (c < 8 && 2 * c * rows <= 4 * sms && V >= (int64_t)2 * c * lp::kChunk) c *= 2;
  return c;
}

template <class T>
static cudaError_t run(const lp::Params& p, cudaStream_t stream) {
  const int c = cluster_for(p.rows, p.V, sm_count());
  return launch_dependent(token_logprobs_kernel<T>, dim3((unsigned)(p.rows * c)), lp::kThreads, 0,
                          (unsigned)c, stream, p);
}

cudaError_t launch_token_logprobs(const LogprobArgs& x, cudaStream_t stream) {
  lp::Params p;
  p.x = x.logits;
  p.stride = x.stride;
  p.rows = x.rows;
  p.V = x.V;
  p.scale = x.scale;
  p.qs = (float)((double)x.scale * 1.4426950408889634);
  p.rise = 8.f / p.qs;
  p.tokens = x.tokens;
  p.given = x.given;
  p.top = x.top;
  p.logprob = x.logprob;
  p.entropy = x.entropy;
  p.top_logprob = x.top_logprob;
  p.top_token = x.top_token;
  return x.dtype == LYNX_FP32 ? run<float>(p, stream)
         : x.dtype == LYNX_FP16 ? run<__half>(p, stream) : run<__nv_bfloat16>(p, stream);
}

}  // namespace lynx
