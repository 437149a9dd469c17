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
// order of equals is part of them.  A warp collects in shared memory the keys that do
// not fall below a bound that k others are known to reach.  The first bound of a row is
// the k-th largest of the maxima of 64 groups of its first chunk, near that chunk's k-th
// largest; the block ranks what its warps have collected, and keeps k, after three chunks
// and after every sixteenth (with more than eight alternatives after two and eight as
// well: the bound falls behind by k elements a chunk).  So few tokens are collected: of
// 128256 in random order some 40 for k = 5.  A warp whose 64 places do not suffice ranks
// its own: any order of the row is right, rising ones are slow (1024 rows of 128256: 0.87
// ms, 0.07 in random order).  Keys decide, not arrival.
//
// What bounds it: memory, and beside it the issue of some 11 instructions an element.
// 4096 rows of 128256 BF16 logits take 177 us without alternatives (5.95 TB/s), 205 us
// with five (5.12 TB/s), 281 with 32.  Blocks of 256 threads, four to an SM, take rows in
// turn; a ring of two chunks of 16 KB in shared memory is filled by bulk copies that run
// ahead, into the next row as well.  A chunk's place is given back as soon as it is in
// registers, and asked for anew after its sums: slow warps hold up no copies (221 us with
// the place held until the candidates were read from it).  A lane with candidates
// hands its vectors to its warp.  (A row's ends that are no whole 16-byte vector are
// read by one warp.)  Few rows are split over clusters of up to eight blocks, whose sums
// and candidates meet in the first one's shared memory.  Nothing is kept in local memory.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "cache_attn.h"
#include "lynx.h"
#include "tree.h"

namespace lynx {

__device__ unsigned int g_logprobs_flags = 0;

cudaError_t read_logprobs_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_logprobs_flags, sizeof(unsigned int));
}

namespace lp {

constexpr int kPlaces = 64;                    // candidates of a warp
constexpr int kGroups = 64;                    // of the threads, for a row's first bound
constexpr int kMaxTop = 32;
static_assert(kMaxTop <= kGroups && kMaxTop + 32 <= kPlaces, "the places suffice");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeast = -16384.f;             // 2^y is 0 long before
constexpr float kFloor = -1e30f;               // see Type::floor
// With |r| up to kNear, y of a value from kFloor on is finite at every scale: (1e30 + 1.25e29)
// 1e6 log2 e = 1.6e36; and kFloor is so far below r that its 2^y is 0 at every scale.
constexpr float kNear = 1.25e29f;

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
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Types: the values of a 16-byte vector, and the largest of two vectors.  floor: the
// vector with what lies below kFloor, -inf too, raised to it (a NaN stays), so that y is
// finite without a maximum for each where r is not beyond kNear; FP16, which does not reach
// that far, always takes the maximum.
template <class T> struct Type;
template <> struct Type<float> {
  static constexpr uint32_t none = 0xff800000u;            // -inf
  static constexpr bool kFloors = true;
  static __device__ __forceinline__ uint4 floor(const uint4& v) {
    auto up = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), kFloor)); };
    return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
  }
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float largest(const uint4& v, const uint4& w) {
    float f[8];
    unpack(v, f);
    unpack(w, f + 4);
    return max3(max3(f[0], f[1], f[2]), max3(f[3], f[4], f[5]), fmaxf(f[6], f[7]));
  }
};
__device__ __forceinline__ uint32_t half2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <> struct Type<__nv_bfloat16> {
  static constexpr uint32_t none = 0xff80ff80u;            // -inf
  static constexpr bool kFloors = true;
  static __device__ __forceinline__ uint4 floor(const uint4& v) {
    auto up = [](uint32_t w) {
      uint32_t r;
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(f2_to_bf2(kFloor, kFloor)));
      return r;
    };
    return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
  }
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
  static __device__ __forceinline__ float largest(const uint4& v, const uint4& w) {
    const uint32_t a = bf2_max(bf2_max(v.x, v.y), bf2_max(v.z, v.w));
    const uint32_t b = bf2_max(bf2_max(w.x, w.y), bf2_max(w.z, w.w));
    const f2 m = bf2_to_f2(bf2_max(a, b));
    return fmaxf(m.x, m.y);
  }
};
template <> struct Type<__half> {
  static constexpr uint32_t none = 0xfc00fc00u;            // -inf
  static constexpr bool kFloors = false;
  static __device__ __forceinline__ uint4 floor(const uint4& v) { return v; }
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
  static __device__ __forceinline__ float largest(const uint4& v, const uint4& w) {
    const uint32_t a = half2_max(half2_max(v.x, v.y), half2_max(v.z, v.w));
    const uint32_t b = half2_max(half2_max(w.x, w.y), half2_max(w.z, w.w));
    const uint32_t c = half2_max(a, b);
    const float2 m = __half22float2(*reinterpret_cast<const __half2*>(&c));
    return fmaxf(m.x, m.y);
  }
};

// The key of a logit above -inf (both zeros are one value).
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
  u ^= u >> 31 ? 0xffffffffu : 0x80000000u;
  return (uint64_t)u << 32 | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ float next_above(float x) {      // (x is no NaN and not +inf)
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float(x == 0.f ? 1u : u >> 31 ? u - 1u : u + 1u);
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

// All lanes' as one, to all of them: one rescaling each, to the largest r.
__device__ __forceinline__ Sums join_lanes(const Sums& p, float qs) {
  float r = p.r;                                 // (no NaN)
#pragma unroll
  for (int o = 16; o; o >>= 1) r = fmaxf(r, __shfl_xor_sync(kFull, r, o));
  Sums c = join(Sums{r, 0.f, 0.f}, p, qs);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    c.s = __fadd_rn(c.s, __shfl_xor_sync(kFull, c.s, o));
    c.t = __fadd_rn(c.t, __shfl_xor_sync(kFull, c.t, o));
  }
  return c;
}

// The next chunk to be copied: number c of `row`, which has n vectors left from `from` on.
struct Ahead {
  int64_t row;
  uint64_t from;
  int c, chunks, n, issued;
};

template <int THREADS>
struct __align__(128) Shared {
  static constexpr int kWarps = THREADS / 32;
  // 16-byte vectors a thread takes of a chunk, and chunks on their way: many rows gain
  // from longer turns, one row's share of a block is short
  static constexpr int kVecs = THREADS == 256 ? 4 : 2, kRing = THREADS == 256 ? 2 : 4;
  uint4 ring[kRing][kVecs * THREADS];
  uint4 turn[kWarps][kVecs];                   // a lane's vectors, for its warp
  uint64_t place[kWarps][kPlaces];             // the warps' candidates
  uint64_t list[kWarps * kPlaces + kMaxTop];   // all of them, to be ranked
  uint64_t best[kMaxTop];                      // the largest keys so far in order, 0: none
  float group[kGroups], bound;                 // maxima of a row's first vectors
  uint64_t full[kRing], empty[kRing];          // mbarriers
  int count[kWarps], carried;                  // the warps' candidates; keys in `best`
  Sums part[kWarps];
  Sums total;
  Ahead ahead;
  uint32_t gone;                               // a wait has been given up
};

// Bounded wait; once a wait of the block has run out, every wait returns at once (its
// threads run out their loops, so that the barriers stay matched) and the flag says so.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase, volatile uint32_t* gone) {
  if (mbar_try_wait(bar, phase)) return;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, phase)) {
    if (*gone) return;
    if (global_ns() - t0 > kWaitNs) {
      *gone = 1u;
      atomicOr(&g_logprobs_flags, kFlagWaitTimeout);
      return;
    }
  }
}

// Ranks the n keys of `list` and writes the `top` largest in order to `best`, 0 behind
// them.  By all THREADS threads; no key twice.
template <int THREADS>
__device__ __forceinline__ void rank_list(const uint64_t* list, int n, int top, uint64_t* best) {
  const int tid = (int)threadIdx.x;
  if (tid >= n && tid < top) best[tid] = 0;
  for (int i = tid; i < n; i += THREADS) {
    const uint64_t own = list[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += list[j] > own;
    if (above < top) best[above] = own;
  }
}

// A warp's own ranking: its n > top keys down to the `top` largest, in order.
__device__ __forceinline__ void rank_places(uint64_t* place, int n, int top, int lane) {
  __syncwarp();
  const uint64_t a = lane < n ? place[lane] : 0, b = lane + 32 < n ? place[lane + 32] : 0;
  int ra = 0, rb = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t k = place[j];
    ra += k > a;
    rb += k > b;
  }
  __syncwarp();
  if (a && ra < top) place[ra] = a;
  if (b && rb < top) place[rb] = b;
  __syncwarp();
}

// A row of logits: the `head` elements before its first whole 16-byte vector, the n
// vectors that are this CTA's, from element `first` on and in chunks, and what lies behind
// the last vector of all, from element `tail` on.
template <class T>
struct Row {
  const T* x;
  int head, first, tail, n, chunks;
};

// What a warp knows of the likeliest tokens.
struct Picks {
  uint64_t bound;          // a key that `top` of them reach, 0: none known
  int n;                   // the warp's candidates, in its places
  __device__ __forceinline__ void raise(uint64_t k) { bound = k > bound ? k : bound; }
  // What the largest of the elements from index `from` on has to reach for a candidate to
  // be among them: where all of them lie behind the bound's own index, an equal value
  // is not enough.
  __device__ __forceinline__ float least(int from) const {
    if (bound == 0) return -FLT_MAX;
    const float v = value_of(bound);
    return index_of(bound) < from ? next_above(v) : v;
  }
};

// Everything that the block has collected (sh.count of each warp's places) and kept before
// (sh.carried keys of sh.best), ranked: the `top` best stay.  By all threads.
template <int THREADS>
__device__ __noinline__ void rank_all(Shared<THREADS>* sh, int top) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  __syncthreads();
  const int c = sh->count[lane % kWarps], own = sh->count[w], carried = sh->carried;
  const unsigned in = lane < kWarps ? (unsigned)c : 0u;
  const int total = carried + (int)__reduce_add_sync(kFull, in);
  const int before = carried + (int)__reduce_add_sync(kFull, lane < w ? in : 0u);
  if (tid < carried) sh->list[tid] = sh->best[tid];
  for (int i = lane; i < own; i += 32) sh->list[before + i] = sh->place[w][i];
  __syncthreads();
  rank_list<THREADS>(sh->list, total, top, sh->best);
  if (tid == 0) sh->carried = total < top ? total : top;
  __syncthreads();
}

// This CTA's part of row `row`.
template <class T, int CHUNK>
__device__ __forceinline__ Row<T> row_at(const Params& a, int row, int lg, int rank) {
  constexpr int VE = 16 / (int)sizeof(T);
  Row<T> q;
  q.x = static_cast<const T*>(a.x) + row * a.stride;
  const int off = (int)((reinterpret_cast<uintptr_t>(q.x) & 15u) / sizeof(T)), V = (int)a.V;
  q.head = off ? (VE - off < V ? VE - off : V) : 0;
  const int nvec = (V - q.head) / VE, share = (nvec + (1 << lg) - 1) >> lg;
  q.tail = q.head + nvec * VE;
  const int v0 = share * rank < nvec ? share * rank : nvec;
  q.n = v0 + share < nvec ? share : nvec - v0;
  q.first = q.head + v0 * VE;
  q.chunks = (q.n + CHUNK - 1) / CHUNK;
  return q;
}

// The next chunk's copy, by one thread: its row and number are in shared memory, which
// spares all others the registers.
template <class T, int THREADS>
__device__ __forceinline__ void issue(const Params& a, Shared<THREADS>& sh, int rows_at_once,
                                      int lg, int rank) {
  constexpr int kRing = Shared<THREADS>::kRing, kChunk = Shared<THREADS>::kVecs * THREADS;
  volatile uint32_t* const gone = &sh.gone;
  Ahead q = sh.ahead;
  while (q.c >= q.chunks) {
    if (q.row + rows_at_once >= a.rows) return;      // (rows and rows_at_once are below 2^31)
    q.row += rows_at_once;
    const Row<T> r = row_at<T, kChunk>(a, (int)q.row, lg, rank);
    q.c = 0;
    q.chunks = r.chunks;
    q.n = r.n;
    q.from = reinterpret_cast<uint64_t>(r.x + checked_index(r.first, a.V + 1, &g_logprobs_flags));
  }
  const int st = q.issued % kRing;
  if (q.issued >= kRing) wait(&sh.empty[st], (uint32_t)(q.issued / kRing - 1) & 1u, gone);
  if (*gone) return;
  const uint32_t bytes = 16u * (uint32_t)(q.n < kChunk ? q.n : kChunk);
  mbar_expect_tx(&sh.full[st], bytes);
  bulk_load(sh.ring[st], reinterpret_cast<const void*>(q.from), bytes, &sh.full[st]);
  ++q.issued;
  ++q.c;
  q.n -= kChunk;
  q.from += 16 * kChunk;
  sh.ahead = q;
}

}  // namespace lp

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
token_logprobs_kernel(const __grid_constant__ lp::Params a) {
  using namespace lp;
  using Block = Shared<THREADS>;
  constexpr int VE = 16 / (int)sizeof(T), kWarps = THREADS / 32, kVecs = Block::kVecs,
                kRing = Block::kRing, kChunk = kVecs * THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  Block& sh = *reinterpret_cast<Block*>(smem);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int csize = (int)cluster_size(), rank = (int)cluster_rank();
  const int lg = 31 - __clz(csize);              // (a power of two)
  const int rows_at_once = (int)(gridDim.x >> lg);
  const int top = a.top;
  volatile uint32_t* const gone = &sh.gone;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    sh.gone = 0;
    sh.ahead = Ahead{(int64_t)(blockIdx.x >> lg) - rows_at_once, 0, 0, 0, 0, 0};
    fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0)
    for (int i = 0; i < kRing; ++i) issue<T, THREADS>(a, sh, rows_at_once, lg, rank);

  uint32_t st = 0, ph = 0;                       // the ring's next chunk
  for (int64_t row = blockIdx.x >> lg; row < a.rows; row += rows_at_once) {
    Sums own = {-INFINITY, 0.f, 0.f};
    float trigger = -INFINITY;                   // what raises r
    Picks picks = {0, 0};
    float least = top > 0 ? -FLT_MAX : NAN;
    if (tid == 0) sh.carried = 0;
    // (the given token's logit is asked for while the candidates are ranked)
    const bool asks = rank == 0 && tid < a.given;
    int32_t token = -1;
    if (asks) token = a.tokens[row * a.given + tid];
    int left, first;                             // vectors; the chunk's first element
    {
      const Row<T> now = row_at<T, kChunk>(a, (int)row, lg, rank);
      left = now.n;
      first = now.first;
      if (rank == 0 && w == 0) {
        // ---- the row's ends, an element to a lane
        const int e = lane < now.head ? lane : now.tail + lane - now.head;
        float f = -INFINITY;
        if (e < (int)a.V) f = Type<T>::value(now.x[e]);
        if (f != -INFINITY) {
          if (f == f) {
            own.r = f;
            trigger = __fadd_rn(f, a.rise);
          }
          const float z = max_nan(__fmul_rn(__fsub_rn(f, f), a.qs), kLeast);
          own.s = ex2(z);
          own.t = __fmul_rn(own.s, z);
        }
        if (top > 0) {
          const uint64_t k = f >= -FLT_MAX ? key_of(f, e) : 0;
          const unsigned m = __ballot_sync(kFull, k != 0);
          if (k) sh.place[0][__popc(m & ((1u << lane) - 1u))] = k;
          picks.n = __popc(m);
        }
      }
    }
#pragma unroll 1
    for (int c = 0; left > 0; ++c, left -= kChunk, first += kChunk * VE) {
      wait(&sh.full[st], ph, gone);
      const uint4* const chunk = sh.ring[st];
      uint4 raw[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) raw[u] = chunk[u * THREADS + tid];
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(&sh.empty[st])) : "memory");
      if (left < kChunk) {                       // behind the share there is nothing
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          if (u * THREADS + tid >= left)
            raw[u] = make_uint4(Type<T>::none, Type<T>::none, Type<T>::none, Type<T>::none);
      }
      float most = -INFINITY;
#pragma unroll
      for (int h = 0; h < kVecs; h += 2) most = fmaxf(most, Type<T>::largest(raw[h], raw[h + 1]));
      // ---- candidates
      bool more = top > 0 && c == 0;
      if (more) {
        // the k-th largest of the groups' maxima, which k elements reach (any index: of
        // equals all are candidates)
        float g = most;
#pragma unroll
        for (int i = 1; i < THREADS / kGroups; i <<= 1) g = fmaxf(g, __shfl_xor_sync(kFull, g, i));
        if (tid % (THREADS / kGroups) == 0) sh.group[tid / (THREADS / kGroups)] = g;
        if (tid == 0) sh.bound = -INFINITY;
        __syncthreads();
        if (tid < kGroups) {
          g = sh.group[tid];
          int above = 0, reach = 0;
#pragma unroll 8
          for (int j = 0; j < kGroups; ++j) {
            above += sh.group[j] > g;
            reach += sh.group[j] >= g;
          }
          if (above < top && reach >= top) sh.bound = g;    // (the same by all that do)
        }
        __syncthreads();
        if (sh.bound > -INFINITY) picks.raise(key_of(sh.bound, INT_MAX));
        least = picks.least(0);
      }
      unsigned here = __ballot_sync(kFull, most >= least);
      more = more || here;
      // the elements of one lane after the other, one to a lane
#pragma unroll 1
      for (; here; here &= here - 1) {
        const int from = __ffs(here) - 1;
        if (lane == from) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u) sh.turn[w][u] = raw[u];
        }
        __syncwarp();
        uint64_t k = 0;
        if (lane < kVecs * VE) {
          const float f = Type<T>::value(reinterpret_cast<const T*>(sh.turn[w])[lane]);
          const int at = lane / VE * THREADS + (tid & ~31) + from;
          if (f >= -FLT_MAX) k = key_of(f, first + at * VE + lane % VE);
        }
        unsigned m = __ballot_sync(kFull, k != 0 && k >= picks.bound);
        if (picks.n + __popc(m) > kPlaces) {       // the warp's own best make room
          rank_places(sh.place[w], picks.n, top, lane);
          picks.n = picks.n < top ? picks.n : top;
          if (picks.n == top) picks.raise(sh.place[w][top - 1]);
          m = __ballot_sync(kFull, k != 0 && k >= picks.bound);
        }
        if (m >> lane & 1u) sh.place[w][picks.n + __popc(m & ((1u << lane) - 1u))] = k;
        picks.n += __popc(m);
        __syncwarp();
      }
      // ---- the sums
      if (most > trigger) {
        const float d = own.r == -INFINITY
                            ? kLeast : max_nan(__fmul_rn(__fsub_rn(own.r, most), a.qs), kLeast);
        const float g = ex2(d);
        own.t = __fmul_rn(g, fmaf(own.s, d, own.t));
        own.s = __fmul_rn(g, own.s);
        own.r = most;
        trigger = __fadd_rn(most, a.rise);
      }
      const float minus_r = own.r == -INFINITY ? 0.f : -own.r;
      f2 s = make_float2(own.s, 0.f), t = make_float2(own.t, 0.f);
      // (rows of the type's lowest values have r near the floor or below it, and those with
      // its highest one so far above it that y would be -inf and 2^y y a NaN)
      if (Type<T>::kFloors && !__any_sync(kFull, fabsf(own.r) > kNear && own.r != -INFINITY)) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          float f[VE];
          Type<T>::unpack(Type<T>::floor(raw[u]), f);
#pragma unroll
          for (int i = 0; i < VE; i += 2) {
            const f2 y = mul2(add2(make_float2(f[i], f[i + 1]), make_float2(minus_r, minus_r)),
                              make_float2(a.qs, a.qs));
            const f2 e = make_float2(ex2(y.x), ex2(y.y));
            s = add2(s, e);
            t = fma2(e, y, t);
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          float f[VE];
          Type<T>::unpack(raw[u], f);
#pragma unroll
          for (int i = 0; i < VE; i += 2) {
            const f2 y = mul2(add2(make_float2(f[i], f[i + 1]), make_float2(minus_r, minus_r)),
                              make_float2(a.qs, a.qs));
            const f2 z = make_float2(max_nan(y.x, kLeast), max_nan(y.y, kLeast));
            const f2 e = make_float2(ex2(z.x), ex2(z.y));
            s = add2(s, e);
            t = fma2(e, z, t);
          }
        }
      }
      own.s = __fadd_rn(s.x, s.y);
      own.t = __fadd_rn(t.x, t.y);
      if (tid == 0) issue<T, THREADS>(a, sh, rows_at_once, lg, rank);
      __syncwarp();
      if (top > 0) {
        // (many alternatives: the bound pays earlier)
        if ((c == (top > 8 ? 1 : 2) || (top > 8 && c == 7) || (c & 15) == 15) && left > kChunk) {
          if (lane == 0) sh.count[w] = picks.n;
          __syncwarp();
          rank_all<THREADS>(&sh, top);
          picks.n = 0;
          if (sh.carried == top) picks.raise(sh.best[top - 1]);
          more = true;
        }
        if (more) least = picks.least(first + kChunk * VE);
      }
      if (++st == kRing) st = 0, ph ^= 1u;
    }
    // ---- the block's sums and its best
    float asked = -INFINITY;
    if (token >= 0 && token < a.V)
      asked = Type<T>::value(static_cast<const T*>(a.x)[row * a.stride + token]);
    else if (token >= 0)
      atomicOr(&g_logprobs_flags, kFlagBadToken);
    own = join_lanes(own, a.qs);
    if (lane == 0) {
      sh.part[w] = own;
      sh.count[w] = picks.n;
    }
    __syncwarp();
    if (top > 0) rank_all<THREADS>(&sh, top);
    else __syncthreads();
    Sums all = sh.part[lane % kWarps];
    if (lane >= kWarps) all = Sums{-INFINITY, 0.f, 0.f};
    all = join_lanes(all, a.qs);
    if (csize > 1) {
      if (tid == 0) sh.total = all;
      cluster_sync();                            // every part is there
      if (rank == 0) {
        all = Sums{-INFINITY, 0.f, 0.f};
        if (lane < csize) {
          all.r = ld_peer32(&sh.total.r, (uint32_t)lane);
          all.s = ld_peer32(&sh.total.s, (uint32_t)lane);
          all.t = ld_peer32(&sh.total.t, (uint32_t)lane);
        }
        __syncwarp();
        all = join_lanes(all, a.qs);
        if (top > 0) {                           // (0 where a part has fewer)
          uint64_t k = 0;
          if (tid < csize * top) k = ld_peer64(&sh.best[tid % top], (uint32_t)(tid / top));
          const unsigned m = __ballot_sync(kFull, k != 0);
          if (lane == 0) sh.count[w] = __popc(m);
          __syncthreads();
          const int c = sh.count[lane % kWarps];
          const unsigned in = lane < kWarps ? (unsigned)c : 0u;
          const int total = (int)__reduce_add_sync(kFull, in);
          const int before = (int)__reduce_add_sync(kFull, lane < w ? in : 0u);
          if (k) sh.list[before + __popc(m & ((1u << lane) - 1u))] = k;
          __syncthreads();
          rank_list<THREADS>(sh.list, total, top, sh.best);
        }
      }
      cluster_sync();                            // the parts have been read
    }
    // ---- the row's answers
    if (rank == 0) {
      const bool none = all.r == -INFINITY && all.s == 0.f;        // every logit is -inf
      const float ln = none ? 0.f : logf(all.s);
      auto logprob = [&](float v) {
        if (none || v == -INFINITY) return all.s != all.s ? all.s : -INFINITY;
        // (halves: the difference of two logits may be beyond float32, and z not)
        const float half = __fsub_rn(__fmul_rn(0.5f, v), __fmul_rn(0.5f, all.r));
        return __fsub_rn(__fmul_rn(2.f, __fmul_rn(half, a.scale)), ln);
      };
      if (a.entropy && tid == 0)
        a.entropy[row] = none ? 0.f : __fsub_rn(ln, __fmul_rn(__fdiv_rn(all.t, all.s), kLn2));
      if (tid < top) {
        const uint64_t k = sh.best[tid];
        a.top_logprob[row * top + tid] = k ? logprob(value_of(k)) : -INFINITY;
        a.top_token[row * top + tid] = k ? index_of(k) : -1;
      }
      if (asks)
        a.logprob[row * a.given + tid] = token >= 0 && token < a.V ? logprob(asked) : -INFINITY;
    }
    __syncwarp();
    __syncthreads();                             // before the next row's parts
  }
  // (where a wait was given up, copies may still be on their way)
  if (tid == 0 && *gone) drain_copies(sh.full, kRing, sh.ahead.issued, &g_logprobs_flags);
}

template <class T, int THREADS>
static cudaError_t run(const lp::Params& p, unsigned grid, unsigned cluster, cudaStream_t stream) {
  auto fn = token_logprobs_kernel<T, THREADS>;
  constexpr size_t kBytes = sizeof(lp::Shared<THREADS>);
  static thread_local int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  return launch_dependent(fn, dim3(grid), THREADS, kBytes, cluster, stream, p);
}

// Blocks of 256 threads, four to an SM, where there are rows for most of the SMs, or few
// enough chunks to a block that long turns gain nothing; else blocks of 1024 threads.
// Both in clusters of up to eight to a row, as many as the GPU holds at once (in
// clusters of four the larger ones do not fill every SM: 38 rows would take two rounds).
// Five alternatives, 256 and 1024 threads, us: 300 rows of 128256 BF16 logits 22.6 (a block a
// row 23.6) and 29.2, 152 rows 16.4 and 15.9, 76 rows 14.4 and 13.3, 38 rows 10.8 and 13.3,
// 8 rows 8.7 and 9.2, 1 row of FP32 11.0 and 10.0, 100 rows of 8000 5.7 and 7.2.
template <class T>
static cudaError_t run_rows(const lp::Params& p, cudaStream_t stream) {
  constexpr int64_t kSmall = 256 * lp::Shared<256>::kVecs * (16 / (int)sizeof(T));
  constexpr int64_t kLarge = 1024 * lp::Shared<1024>::kVecs * (16 / (int)sizeof(T));
  const int64_t sms = sm_count();
  int64_t c = 1;
  while (c < 8 && 2 * c * p.rows <= (p.rows > sms ? 4 : 2) * sms && p.V >= 2 * c * kSmall) c *= 2;
  if (p.rows > sms || p.V <= 2 * c * kSmall) {
    const int64_t most = 4 * sms, n = p.rows * c, grid = c > 1 || n < most ? n : most;
    return run<T, 256>(p, (unsigned)grid, (unsigned)c, stream);
  }
  c = 1;
  while (c < 8 && 2 * c * p.rows <= (c == 1 ? sms : sms * 3 / 4) && p.V >= 2 * c * kLarge) c *= 2;
  return run<T, 1024>(p, (unsigned)(p.rows * c), (unsigned)c, stream);
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
  return x.dtype == LYNX_FP32 ? run_rows<float>(p, stream)
         : x.dtype == LYNX_FP16 ? run_rows<__half>(p, stream) : run_rows<__nv_bfloat16>(p, stream);
}

}  // namespace lynx
