// cache_pages.cu -- the paged cache's books (which pages a sequence has, how many
// places name a page) and the pages themselves: sequences that share pages, new pages,
// pages given back, pages moved to the front, and tokens kept of a tree.
//
// A row of the table names the ceil(kv_len / page) pages that its tokens need, in
// order, and -1 behind them.  refs[p] counts the places that name page p; a page
// with none is free.  So a row is forked by copying its entries and raising the
// counts, and pages are given back by lowering them.  Only sums are made with
// atomics, and free pages are taken in the order of their numbers by sequences in theirs:
// results do not depend on timing.
//
// What bounds them.  The books: latency.  One pass over the counts finds the free pages:
// each warp counts those of a contiguous part, the parts' sums meet in shared memory (of
// a cluster of up to eight CTAs where there are many pages), and in a second pass each
// warp numbers its own without waiting for others.  Copies: memory.  In a graph of one
// kernel, where adding 1 to a number takes 4.2 us: fork and trim 6.2 (48 sequences), reserve 8.3,
// compact 9.3 (248 moves of 48 sequences), keep 8.3 (32 sequences, 32 pools, 64 nodes).
#include "cache_attn.h"
#include "tree.h"

namespace lynx {

// Set when a table entry that was read lay outside the pools, or a sequence named
// one that is not there; read through read_cache_pages_flags(), never reset.
__device__ unsigned int g_cache_pages_flags = 0;

cudaError_t read_cache_pages_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_cache_pages_flags, sizeof(unsigned int));
}

namespace pg {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct Books {
  int32_t *table, *kv_len, *refs;
  int64_t max_pages, nblocks;
  int batch, lgP;
  __device__ __forceinline__ int64_t pages(int64_t tokens) const {
    return (tokens + (1 << lgP) - 1) >> lgP;
  }
  __device__ __forceinline__ int64_t length(int b) const {
    const int64_t n = kv_len[b], room = max_pages << lgP;
    return n < 0 ? 0 : n > room ? room : n;
  }
  __device__ __forceinline__ bool is_page(int32_t p) const { return p >= 0 && p < nblocks; }
};

__device__ __forceinline__ void start() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void bad_entry() { atomicOr(&g_cache_pages_flags, kFlagBadBlock); }

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
// (release and acquire at the cluster's scope: global memory too)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int32_t ld_peer(const void* p, uint32_t rank) {
  uint32_t at;
  int32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// ------------------------------------------------------------------ fork, trim

// Block y < out_batch makes output row y, the others give back input row y - out_batch.
__global__ void __launch_bounds__(128)
cache_fork_kernel(const __grid_constant__ Books a, const int32_t* source, int32_t* out_table,
                  int32_t* out_len, int out_batch) {
  start();
  const int y = blockIdx.x;
  if (y < out_batch) {
    const int from = source[y];
    const bool there = from >= 0 && from < a.batch;
    if (from >= a.batch && threadIdx.x == 0) bad_entry();
    const int64_t n = there ? a.length(from) : 0, have = a.pages(n);
    for (int64_t m = threadIdx.x; m < a.max_pages; m += blockDim.x) {
      int32_t p = -1;
      if (m < have) {
        p = a.table[(int64_t)from * a.max_pages + m];
        if (a.is_page(p)) atomicAdd(a.refs + p, 1);
        else bad_entry(), p = -1;
      }
      out_table[(int64_t)y * a.max_pages + m] = p;
    }
    if (threadIdx.x == 0) out_len[y] = (int32_t)n;
  } else {
    const int b = y - out_batch;
    const int64_t have = a.pages(a.length(b));
    for (int64_t m = threadIdx.x; m < have; m += blockDim.x) {
      const int32_t p = a.table[(int64_t)b * a.max_pages + m];
      if (a.is_page(p)) atomicAdd(a.refs + p, -1);
      else bad_entry();
    }
  }
}

__global__ void __launch_bounds__(128)
cache_trim_kernel(const __grid_constant__ Books a, const int32_t* keep) {
  start();
  const int b = blockIdx.x;
  const int64_t n = a.length(b), k = keep[b] < 0 ? 0 : keep[b];
  const int64_t left = k < n ? k : n, have = a.pages(n);
  __syncthreads();                           // the length has been read
  for (int64_t m = a.pages(left) + threadIdx.x; m < have; m += blockDim.x) {
    int32_t* e = a.table + (int64_t)b * a.max_pages + m;
    if (a.is_page(*e)) atomicAdd(a.refs + *e, -1);
    else bad_entry();
    *e = -1;
  }
  if (threadIdx.x == 0) a.kv_len[b] = (int32_t)left;
}

// ------------------------------------------------------------------ new pages

struct Part {
  int64_t lo, hi;          // the warp's pages
};
// The contiguous part of the pages that is warp w's of CTA `rank` of `csize`.
__device__ __forceinline__ Part part_of(const Books& a, int csize, int rank, int w) {
  const int lg = 31 - __clz(csize * kWarps);   // (powers of two)
  const int64_t each = (((a.nblocks + (1ll << lg) - 1) >> lg) + 31) & ~31ll;
  const int64_t lo = each * ((int64_t)rank * kWarps + w);
  Part p;
  p.lo = lo < a.nblocks ? lo : a.nblocks;
  p.hi = p.lo + each < a.nblocks ? p.lo + each : a.nblocks;
  return p;
}
// How many of pages lo .. hi - 1 are free (FREE) or in use, to all lanes.
template <bool FREE>
__device__ __forceinline__ int count(const Books& a, int64_t lo, int64_t hi, int lane) {
  int n = 0;
  int64_t p = lo + lane;
  for (; p + 7 * 32 < hi; p += 8 * 32) {     // eight loads in flight
    int32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = a.refs[p + 32 * i];
#pragma unroll
    for (int i = 0; i < 8; ++i) n += (r[i] <= 0) == FREE;
  }
  for (; p < hi; p += 32) n += (a.refs[p] <= 0) == FREE;
  return (int)__reduce_add_sync(kFull, (unsigned)n);
}
// Sums of the warps' counts in mine[kWarps] of each CTA: those before warp w of CTA
// `rank`, and all.  Behind a cluster barrier; by whole warps.
__device__ __forceinline__ int64_t before(const int32_t* mine, int csize, int rank, int w, int lane,
                                          int64_t& all) {
  int64_t b = 0;
  all = 0;
  for (int c = 0; c < csize; ++c) {
    const int v = ld_peer(mine + lane, (uint32_t)c);
    const unsigned sum = __reduce_add_sync(kFull, (unsigned)v);
    all += sum;
    if (c < rank) b += sum;
    if (c == rank) b += __reduce_add_sync(kFull, lane < w ? (unsigned)v : 0u);
  }
  return b;
}

// One cluster.  granted, src and dst are the call's outputs; until the last phase
// they hold, for each sequence, the pages it needs (-1: its row has no room), its shared
// last page (-1: none), and the sum of the needs before it.
__global__ void __launch_bounds__(kThreads, 1)
cache_reserve_kernel(const __grid_constant__ Books a, const int32_t* grow, int32_t* granted,
                     int32_t* src, int32_t* dst) {
  __shared__ int32_t free_of[kWarps];
  __shared__ int64_t sums[kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int csize = (int)cluster_size(), rank = (int)cluster_rank();
  start();
  const Part part = part_of(a, csize, rank, w);
  const int n_free = count<true>(a, part.lo, part.hi, lane);
  if (lane == 0) free_of[w] = n_free;
  // ---- what each sequence needs, and the needs before it
  if (rank == 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int b = b0 + tid;
      int64_t need = 0;
      int32_t old = -1;
      bool fits = true;
      if (b < a.batch) {
        const int64_t kv = a.length(b), n = grow[b] < 0 ? 0 : grow[b];
        const int64_t have = a.pages(kv);
        fits = kv + n <= a.max_pages << a.lgP;
        if (fits && n > 0) {
          need = a.pages(kv + n) - have;
          if (kv & ((1 << a.lgP) - 1)) {
            const int32_t p = a.table[(int64_t)b * a.max_pages + have - 1];
            if (!a.is_page(p)) bad_entry();
            else if (a.refs[p] > 1) old = p, ++need;
          }
        }
      }
      int64_t v = need;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t m = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += m;
      }
      if (lane == 31) sums[w] = v;
      __syncthreads();
      int64_t first = base;
      for (int i = 0; i < kWarps; ++i) {
        if (i < w) first += sums[i];
        base += sums[i];
      }
      __syncthreads();
      if (b < a.batch) {
        const int64_t at = first + v - need;
        granted[b] = fits ? (int32_t)need : -1;
        src[b] = old;
        dst[b] = at < INT_MAX ? (int32_t)at : INT_MAX;   // (more than there are pages)
      }
    }
  }
  cluster_sync();
  // ---- free page number r goes to the sequence whose needs hold place r
  int64_t total;
  int64_t r = before(free_of, csize, rank, w, lane, total);
  auto found = [&](int b) {                  // whether sequence b's needs are met
    return granted[b] >= 0 && (granted[b] == 0 || (int64_t)dst[b] + granted[b] <= total);
  };
  const int64_t wanted = a.batch ? (int64_t)dst[a.batch - 1] + max(granted[a.batch - 1], 0) : 0;
  for (int64_t p0 = part.lo; p0 < part.hi && r < wanted; p0 += 32) {
    const int64_t p = p0 + lane;
    const bool is = p < part.hi && a.refs[p] <= 0;
    const unsigned m = __ballot_sync(kFull, is);
    const int64_t x = r + __popc(m & ((1u << lane) - 1u));
    r += __popc(m);
    if (!is || x >= wanted) continue;
    int lo = 0, hi = a.batch;                // the last sequence with dst <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (dst[mid] <= x) lo = mid;
      else hi = mid;
    }
    const int64_t k = x - dst[lo];
    if (k >= granted[lo] || !found(lo)) continue;
    const int64_t at = a.pages(a.length(lo)) - (src[lo] >= 0) + k;
    a.table[(int64_t)lo * a.max_pages + at] = (int32_t)p;
    a.refs[p] = 1;
  }
  cluster_sync();
  // ---- the outputs
  for (int b = rank * kThreads + tid; b < a.batch; b += csize * kThreads) {
    const bool ok = found(b);
    const int32_t n = ok && grow[b] > 0 ? grow[b] : 0, old = src[b];
    const int64_t kv = a.length(b);
    int32_t own = -1;
    if (ok && old >= 0) {
      atomicAdd(a.refs + old, -1);
      own = a.table[(int64_t)b * a.max_pages + a.pages(kv) - 1];
    }
    granted[b] = n;
    src[b] = ok ? old : -1;
    dst[b] = own;
    a.kv_len[b] = (int32_t)(kv + n);
  }
  cluster_sync();                            // peers may still read this CTA's counts
}

// The same by one CTA, a thread a sequence: what the phases hand on stays in registers and
// shared memory, so that three loads follow one another instead of ten (32 sequences, 200
// pages: 12.4 us in a graph as above, 8.3 like this).  Pages are below 2^25, and sums are cut
// off behind them, so that they fit in 32 bits.
__global__ void __launch_bounds__(kThreads, 1)
cache_reserve_small_kernel(const __grid_constant__ Books a, const int32_t* grow, int32_t* granted,
                           int32_t* src, int32_t* dst) {
  __shared__ int32_t free_of[kWarps], need_of[kWarps];
  __shared__ int32_t first[kThreads], needs[kThreads], own[kThreads];
  __shared__ int64_t place[kThreads];        // of a sequence's first new page in the table
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  start();
  const int b = tid;
  const bool is = b < a.batch;
  const int64_t kv = is ? a.length(b) : 0, n = is && grow[b] > 0 ? grow[b] : 0;
  const int64_t have = a.pages(kv), at = b * a.max_pages + have;
  const bool fits = kv + n <= a.max_pages << a.lgP;
  const bool open = fits && n > 0 && (kv & ((1 << a.lgP) - 1));     // a last page with room
  const int32_t last = open ? a.table[at - 1] : -1;
  const Part part = part_of(a, 1, 0, w);
  const int n_free = count<true>(a, part.lo, part.hi, lane);
  int32_t old = -1;
  if (open) {
    if (!a.is_page(last)) bad_entry();
    else if (a.refs[last] > 1) old = last;
  }
  const int most = (int)a.nblocks + 1;
  int need = 0;
  if (fits && n > 0) need = (int)(a.pages(kv + n) - have) + (old >= 0);
  int v = need < most ? need : most;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int m = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v = v + m < most ? v + m : most;
  }
  if (lane == 0) free_of[w] = n_free;
  if (lane == 31) need_of[w] = v;
  __syncthreads();
  const unsigned f = (unsigned)free_of[lane], d = (unsigned)need_of[lane];
  const int total = (int)__reduce_add_sync(kFull, f);
  int r = (int)__reduce_add_sync(kFull, lane < w ? f : 0u);
  const unsigned wanted = __reduce_add_sync(kFull, d);
  const unsigned begin = __reduce_add_sync(kFull, lane < w ? d : 0u);
  // (need pages from `from` on; cut off, they lie behind all there are)
  const int from = (int)(begin < (unsigned)most ? begin : (unsigned)most) + (v < most ? v - need : most);
  const bool ok = fits && (need == 0 || from + need <= total);
  first[b] = from;
  needs[b] = ok ? need : 0;
  place[b] = at - (old >= 0);
  __syncthreads();
  for (int64_t p0 = part.lo; p0 < part.hi && (unsigned)r < wanted; p0 += 32) {
    const int64_t p = p0 + lane;
    const bool free = p < part.hi && a.refs[p] <= 0;
    const unsigned m = __ballot_sync(kFull, free);
    const int x = r + __popc(m & ((1u << lane) - 1u));
    r += __popc(m);
    if (!free) continue;
    int lo = 0, hi = a.batch;                // the last sequence with first <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= x) lo = mid;
      else hi = mid;
    }
    // (below the first sequence's where that alone needs more than there is)
    const int k = x - first[lo];
    if (k < 0 || k >= needs[lo]) continue;
    a.table[checked_index(place[lo] + k, a.max_pages * a.batch, &g_cache_pages_flags)] = (int32_t)p;
    a.refs[p] = 1;
    if (k == 0) own[lo] = (int32_t)p;
  }
  __syncthreads();
  if (!is) return;
  const int32_t got = ok ? (int32_t)n : 0;
  const bool copy = ok && old >= 0;
  if (copy) atomicAdd(a.refs + old, -1);
  granted[b] = got;
  src[b] = copy ? old : -1;
  dst[b] = copy ? own[b] : -1;
  a.kv_len[b] = (int32_t)(kv + got);
}

// ------------------------------------------------------------------ compaction

// Where page p is after n moves, src in ascending order.
__device__ __forceinline__ int32_t moved_to(int32_t p, const int32_t* src, const int32_t* dst, int n) {
  if (n == 0 || p < src[0]) return p;
  int lo = 0, hi = n;                        // the last place with src <= p
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (src[mid] <= p) lo = mid;
    else hi = mid;
  }
  return src[lo] == p ? dst[lo] : p;
}

// The table's entries first, first + step, ... after n moves.  One that is no page stays as
// it is; where its row's length needs a page it is reported, whether there are moves or not.
// I: an integer that holds twice the entries.
template <class I>
__device__ __forceinline__ void retable(const Books& a, const int32_t* src, const int32_t* dst, int n,
                                        I first, I step, I entries) {
  if (first >= entries) return;
  const I width = (I)a.max_pages, rows = step / width, rest = step - rows * width;
  I b = first / width, m = first - b * width;     // of entry i
  for (I i = first; i < entries; i += step) {
    const int32_t p = a.table[i];
    if (!a.is_page(p)) {
      if (m < a.pages(a.length((int)b))) bad_entry();
    } else {
      const int32_t q = moved_to(p, src, dst, n);
      if (q != p) a.table[i] = q;
    }
    b += rows;
    m += rest;
    if (m >= width) m -= width, ++b;
  }
}

// One cluster.  With U pages in use, the i-th of them from U on moves to the i-th free
// one below U.  entries: how many of the table's it brings in line itself.
__global__ void __launch_bounds__(kThreads, 1)
cache_compact_kernel(const __grid_constant__ Books a, int32_t* src, int32_t* dst, int32_t* moved,
                     int64_t entries) {
  __shared__ int32_t used_of[kWarps];
  __shared__ int32_t below[kWarps];          // of those, pages below U
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int csize = (int)cluster_size(), rank = (int)cluster_rank();
  start();
  const Part part = part_of(a, csize, rank, w);
  const int n_used = count<false>(a, part.lo, part.hi, lane);
  if (lane == 0) used_of[w] = n_used;
  cluster_sync();
  int64_t U;
  const int64_t first = before(used_of, csize, rank, w, lane, U);
  int under = 0;
  if (U >= part.hi) under = n_used;
  else if (U > part.lo) under = count<false>(a, part.lo, U, lane);
  if (lane == 0) below[w] = under;
  cluster_sync();
  int64_t W;                                 // pages in use below U
  (void)before(below, csize, rank, w, lane, W);
  const int64_t n = U - W;
  int64_t r = first;                         // pages in use before p0
  if (n > 0) {
    for (int64_t p0 = part.lo; p0 < part.hi; p0 += 32) {
      const int64_t p = p0 + lane;
      const bool in = p < part.hi, used = in && a.refs[p] > 0;
      const unsigned m = __ballot_sync(kFull, used);
      const int64_t x = r + __popc(m & ((1u << lane) - 1u));
      r += __popc(m);
      if (in && !used && p < U) dst[p - x] = (int32_t)p;
      if (used && p >= U) src[x - W] = (int32_t)p;
    }
  }
  for (int64_t i = n + rank * kThreads + tid; i < a.nblocks / 2; i += csize * kThreads)
    src[i] = dst[i] = -1;
  cluster_sync();
  for (int64_t i = rank * kThreads + tid; i < n; i += csize * kThreads) {
    a.refs[dst[i]] = a.refs[src[i]];
    a.refs[src[i]] = 0;
  }
  retable<int>(a, src, dst, (int)n, rank * kThreads + tid, csize * kThreads, (int)entries);
  if (rank == 0 && tid == 0) *moved = (int32_t)n;
  cluster_sync();                            // peers may still read this CTA's counts
}

// The table's entries, where they are many.
__global__ void __launch_bounds__(256)
cache_retable_kernel(const __grid_constant__ Books a, const int32_t* src, const int32_t* dst,
                     const int32_t* moved) {
  start();
  retable<int64_t>(a, src, dst, *moved, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
          (int64_t)gridDim.x * blockDim.x, a.max_pages * a.batch);
}

// ------------------------------------------------------------------ copies

// Eight 16-byte loads in flight a thread: 248 pages of 128 KB in eight pools (520 MB) take
// 166 us, 6.27 TB/s, 170 with four (a plain copy of 520 MB 170, 6.42 TB/s); more or
// larger blocks and loads past L1 change nothing.
constexpr int kCopyThreads = 256, kCopyDepth = 8;
constexpr int kPiece = kCopyThreads * kCopyDepth * 16;    // bytes a CTA copies at once

struct CopyParams {
  uint64_t base[kMaxPools];
  int64_t bytes[kMaxPools];
  int32_t first[kMaxPools + 1];              // pieces of the pools before, of one block
  int n_pools;
  int64_t nblocks, n;
  const int32_t *src, *dst, *count;
};

__global__ void __launch_bounds__(kCopyThreads)
cache_copy_kernel(const __grid_constant__ CopyParams a) {
  start();
  int64_t n = a.n;
  if (a.count) {
    const int64_t c = *a.count;
    n = c < 0 ? 0 : c < n ? c : n;
  }
  const int per = a.first[a.n_pools];
  for (int64_t x = blockIdx.x; x < n * per; x += gridDim.x) {
    const int64_t i = x / per;
    const int piece = (int)(x - i * per);
    const int64_t from = a.src[i], to = a.dst[i];
    if (from < 0 || to < 0) continue;        // no copy in this place
    if (from >= a.nblocks || to >= a.nblocks) {
      if (threadIdx.x == 0) bad_entry();
      continue;
    }
    int lo = 0, hi = a.n_pools;              // the last pool with first <= piece
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first[mid] <= piece) lo = mid;
      else hi = mid;
    }
    const int64_t size = a.bytes[lo], at = (int64_t)(piece - a.first[lo]) * kPiece;
    const uint8_t* s = reinterpret_cast<const uint8_t*>(a.base[lo]) + from * size;
    uint8_t* d = reinterpret_cast<uint8_t*>(a.base[lo]) + to * size;
    uint4 v[kCopyDepth];
#pragma unroll
    for (int k = 0; k < kCopyDepth; ++k) {
      const int64_t o = at + (k * kCopyThreads + threadIdx.x) * 16;
      if (o < size) v[k] = *reinterpret_cast<const uint4*>(s + o);
    }
#pragma unroll
    for (int k = 0; k < kCopyDepth; ++k) {
      const int64_t o = at + (k * kCopyThreads + threadIdx.x) * 16;
      if (o < size) *reinterpret_cast<uint4*>(d + o) = v[k];
    }
  }
}

// ------------------------------------------------------------------ nodes kept

struct KeepParams {
  const uint16_t* nodes[kMaxPools];
  uint16_t* pools[kMaxPools];
  const int32_t *path, *granted, *kv_len, *table;
  int64_t max_pages, nblocks, jobs;
  int batch, T, lgP, row, segs;              // row: values of a token; segs: of 256 values
};

constexpr int kKeepWarps = 8, kKeepDepth = 4;

// A warp takes one sequence, pool and 512 bytes of its rows, four nodes at once: rows are
// 256 bytes a KV head, and where they go is known after two loads that follow one another.
__global__ void __launch_bounds__(32 * kKeepWarps)
cache_keep_kernel(const __grid_constant__ KeepParams a) {
  start();
  const int lane = threadIdx.x & 31;
  const int64_t job = (int64_t)blockIdx.x * kKeepWarps + (threadIdx.x >> 5);
  if (job >= a.jobs) return;
  const int seg = (int)(job % a.segs);
  const int64_t rest = job / a.segs;
  const int b = (int)(rest % a.batch), pool = (int)(rest / a.batch);
  const int granted = a.granted[b], n = granted < a.T ? granted : a.T;
  const int64_t pos0 = (int64_t)a.kv_len[b] - granted;
  const int c = seg * 256 + 8 * lane;        // the lane's values of a row
  for (int i0 = 0; i0 < n; i0 += kKeepDepth) {
    uint4 v[kKeepDepth];
    int64_t slot[kKeepDepth];
#pragma unroll
    for (int k = 0; k < kKeepDepth; ++k) {
      const int i = i0 + k;
      slot[k] = -1;
      if (i >= n) continue;
      const int64_t pos = pos0 + i, page = pos >> a.lgP;
      const int node = a.path[(int64_t)b * a.T + i];
      if (node < 0 || pos < 0) continue;       // a place that no node takes
      int64_t blk = -1;
      if (page < a.max_pages) blk = a.table[(int64_t)b * a.max_pages + page];
      if (blk < 0 || blk >= a.nblocks || node >= kTreeRoom) {
        if (lane == 0) bad_entry();
        continue;
      }
      slot[k] = (blk << a.lgP) + (pos & ((1 << a.lgP) - 1));
      if (c < a.row)
        v[k] = *reinterpret_cast<const uint4*>(a.nodes[pool] +
                                               ((int64_t)b * kTreeRoom + node) * a.row + c);
    }
#pragma unroll
    for (int k = 0; k < kKeepDepth; ++k)
      if (slot[k] >= 0 && c < a.row) {
        const int64_t at = checked_index(slot[k], a.nblocks << a.lgP, &g_cache_pages_flags);
        *reinterpret_cast<uint4*>(a.pools[pool] + at * a.row + c) = v[k];
      }
  }
}

}  // namespace pg

// ------------------------------------------------------------------ host

static pg::Books books_of(const BookArgs& a) {
  return pg::Books{a.table, a.kv_len, a.refs, a.max_pages, a.nblocks, a.batch,
                   __builtin_ctz((unsigned)a.page)};
}
// CTAs of the cluster that reads the counts: one for up to 16K pages, then eight.
static unsigned cluster_of(int64_t nblocks) {
  return nblocks <= 16384 ? 1 : pg::kMaxCluster;
}

cudaError_t launch_cache_fork(const BookArgs& in, const int32_t* source, int32_t* out_table,
                              int32_t* out_len, int out_batch, cudaStream_t stream) {
  return launch_dependent(pg::cache_fork_kernel, dim3((unsigned)(in.batch + out_batch)), 128, 0, 0,
                          stream, books_of(in), source, out_table, out_len, out_batch);
}

cudaError_t launch_cache_trim(const BookArgs& a, const int32_t* keep, cudaStream_t stream) {
  return launch_dependent(pg::cache_trim_kernel, dim3((unsigned)a.batch), 128, 0, 0, stream,
                          books_of(a), keep);
}

cudaError_t launch_cache_reserve(const BookArgs& a, const int32_t* grow, int32_t* granted,
                                 int32_t* src, int32_t* dst, cudaStream_t stream) {
  const unsigned c = cluster_of(a.nblocks);
  if (c == 1 && a.batch <= pg::kThreads)
    return launch_dependent(pg::cache_reserve_small_kernel, dim3(1), pg::kThreads, 0, 0, stream,
                            books_of(a), grow, granted, src, dst);
  return launch_dependent(pg::cache_reserve_kernel, dim3(c), pg::kThreads, 0, c, stream, books_of(a),
                          grow, granted, src, dst);
}

// Up to four table entries a thread are brought in line by the cluster that finds the moves;
// more by a kernel of their own over the whole GPU (another launch: 3 us on the device, 5
// to 10 us on the host).
cudaError_t launch_cache_compact(const BookArgs& a, int32_t* src, int32_t* dst, int32_t* count,
                                 cudaStream_t stream) {
  const unsigned c = cluster_of(a.nblocks);
  const int64_t entries = a.max_pages * a.batch;
  const bool few = entries <= 4 * (int64_t)c * pg::kThreads;
  cudaError_t e = launch_dependent(pg::cache_compact_kernel, dim3(c), pg::kThreads, 0, c, stream,
                                   books_of(a), src, dst, count, few ? entries : (int64_t)0);
  if (e != cudaSuccess || few) return e;
  const int64_t blocks = (entries + 255) / 256, most = 8 * sm_count();
  return launch_dependent(pg::cache_retable_kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                          256, 0, 0, stream, books_of(a), static_cast<const int32_t*>(src),
                          static_cast<const int32_t*>(dst), static_cast<const int32_t*>(count));
}

cudaError_t launch_cache_copy_pages(const PoolList& pools, int64_t nblocks, const int32_t* src,
                                    const int32_t* dst, int64_t n, const int32_t* count,
                                    cudaStream_t stream) {
  pg::CopyParams p;
  p.first[0] = 0;
  for (int i = 0; i < pools.n; ++i) {
    p.base[i] = reinterpret_cast<uint64_t>(pools.base[i]);
    p.bytes[i] = pools.bytes[i];
    p.first[i + 1] = p.first[i] + (int32_t)((pools.bytes[i] + pg::kPiece - 1) / pg::kPiece);
  }
  p.n_pools = pools.n;
  p.nblocks = nblocks;
  p.n = n;
  p.src = src;
  p.dst = dst;
  p.count = count;
  const int64_t pieces = n * p.first[pools.n], most = 8 * (int64_t)sm_count();
  return launch_dependent(pg::cache_copy_kernel, dim3((unsigned)(pieces < most ? pieces : most)),
                          pg::kCopyThreads, 0, 0, stream, p);
}

cudaError_t launch_cache_keep(const KeepArgs& x, cudaStream_t stream) {
  pg::KeepParams p;
  for (int i = 0; i < x.n_pools; ++i) {
    p.nodes[i] = static_cast<const uint16_t*>(x.nodes[i]);
    p.pools[i] = static_cast<uint16_t*>(x.pools[i]);
  }
  p.path = x.path;
  p.granted = x.granted;
  p.kv_len = x.c.kv_len;
  p.table = x.c.table;
  p.max_pages = x.c.max_pages;
  p.nblocks = x.c.nblocks;
  p.batch = x.c.batch;
  p.T = x.c.T;
  p.lgP = __builtin_ctz((unsigned)x.c.page);
  p.row = x.c.Hkv * kCacheD;
  p.segs = (p.row + 255) / 256;
  p.jobs = (int64_t)x.n_pools * x.c.batch * p.segs;
  return launch_dependent(pg::cache_keep_kernel,
                          dim3((unsigned)((p.jobs + pg::kKeepWarps - 1) / pg::kKeepWarps)),
                          32 * pg::kKeepWarps, 0, 0, stream, p);
}

}  // namespace lynx
