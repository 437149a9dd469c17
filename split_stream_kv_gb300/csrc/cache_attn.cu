// cache_attn.cu -- attention over the BF16 paged cache, split over its length
// and joined: a few new tokens per sequence against all that is cached.
//
//   s_ij = scale q_i.k_j, capped, minus slope |p_i - j|, over the visible j;
//   lse_i = ln sum_j e^s_ij,  out_i = sum_j e^(s_ij - lse_i) v_j
//
// Work.  A unit is one (sequence, KV head, group of RT = 16 WR query rows; row
// r is token r / G, query head h G + r % G, so that the G query heads of a KV
// head share one reading of it).  A unit's cache is cut into tiles of 64
// tokens; all tiles of all units form one line, cut into equal shares, one per
// CTA.  The lengths are read on the device, so a captured graph follows them.
// A share's first and last unit may continue in other CTAs: their (m, l, o)
// go to the workspace, and the join (launched as a programmatic dependent)
// merges them.  A unit inside one share is written at once.
//
// Where contexts are short, a unit is one cluster of up to eight CTAs instead:
// its parts meet in shared memory, without a workspace or a second kernel.
//
// A CTA: one warp feeds a ring of tiles by TMA (each tile as two boxes of 64
// channels, 128-byte swizzle); four warps, WR across rows and 4 / WR
// across the tile's tokens, keep a running maximum, sum and output in
// registers: S = Q K^T and O += P V on m16n8k16 MMAs, P going from the
// accumulators of the first to the operand of the second without leaving
// registers.  The token warps of a unit merge once, at its end.
//
// A tree of drafted nodes (TREE): the nodes' own keys and values are one more tile of a
// unit, behind the cache's; of it a row sees the bits of its node's mask, of the cache all
// but what its window leaves out.  Positions, and with them windows and biases, go by
// the node's depth.  16 sequences up to 12001 tokens, 6 nodes, 40 / 8 heads: 56 us.
//
// What bounds it: reading the cache.  512 bytes of K and V per token and KV
// head meet 4 * 128 flop per row, at most 32 flop a byte: the register MMAs
// suffice, and spare the tensor-memory round trip of tcgen05.  (More rows are
// cache_prefill.cu's, but for short contexts.)  1 x 131071 tokens, 64 query heads
// over 8: 89 to 92 us, 5.8 to 6.0 TB/s, of which 11 us are the start, ends that lie 8 us
// apart (some SMs are served more slowly than others when all read) and the join; 8 x
// 32767 tokens, 32 rows: 172 to 178 us, 6.0 to 6.3 TB/s.
//
// Rounding: P is rounded to BF16 for the second product (its terms are
// weights in [0, 1], each off by at most 2^-8 of itself, at random, as the
// BF16 output is); l sums the unrounded weights; everything else is float32.
#include <math.h>

#include "cache_attn.h"
#include "lynx.h"

namespace lynx {

__device__ unsigned int g_cache_attn_flags = 0;

cudaError_t read_cache_attn_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_cache_attn_flags, sizeof(unsigned int));
}

namespace ca {

constexpr int kWarps = 4;                       // consumers
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;
constexpr uint32_t kBox = kKeyTile * 128;       // 64 tokens x 64 channels
constexpr uint32_t kStageBytes = 4 * kBox;      // K: two boxes, V: two boxes
constexpr uint32_t kScratch = kStages * kStageBytes;   // merge of the token warps: 2 x 8 KiB
constexpr uint32_t kMl = kScratch + 2 * 16 * 128 * 4;  // [4 warps][16 rows][m, l]
constexpr uint32_t kBars = kMl + kWarps * 16 * 2 * 4;
constexpr uint32_t kMisc = kBars + 8 * 2 * kStages;    // abort word, the scan's words
constexpr uint32_t kSmem = kMisc + 8 + 8 * (2 * (kWarps + 1) + 6);
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void sync_consumers() {
  asm volatile("barrier.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
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
// What CTA `rank` of the cluster has where this one has `p`, in shared memory.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_peer2(const void* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
               : "=f"(v.x), "=f"(v.y) : "r"(peer(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(const void* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer(p, rank)) : "memory");
  return v;
}

// Bounded wait; once a wait of the CTA has run out, every wait returns at once
// (the roles then run out their iterations, so that the barriers stay
// matched) and the call's flag word says so.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase, volatile uint32_t* gone) {
  if (mbar_try_wait(bar, phase)) return;
  if (*gone) return;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, phase)) {
    if (*gone) return;
    if (global_ns() - t0 > kWaitNs) {
      *gone = 1u;
      atomicOr(&g_cache_attn_flags, kFlagWaitTimeout);
      return;
    }
  }
}

// Rows per unit and the CTA's share, walked in step by all roles.
template <bool TREE>
struct Walk {
  Seq s;
  TileRange tr;       // of the whole sequence
  int b, u, units;    // sequence, unit of it (h * row groups + group), units of it
  int x;              // logical tile
  __device__ __forceinline__ int groups(const CacheParams& a) const {
    return (s.n * a.G + a.RT - 1) / a.RT;
  }
  template <bool EARLY = false>
  __device__ __forceinline__ void load(const CacheParams& a) {
    s = load_seq<EARLY, TREE>(a, b);
    tr = tiles_of<kKeyTile, TREE>(a, s, 0, s.n - 1);
    units = a.Hkv * groups(a);
  }
  // n tiles on; behind the last one b == batch
  __device__ __forceinline__ void advance(const CacheParams& a, int n) {
    x += n;
    while (x >= tr.nt) {
      x -= tr.nt;
      if (++u < units) continue;
      u = 0;
      do {
        if (++b >= a.batch) {
          x = 0;
          return;
        }
        load(a);
      } while (tr.nt == 0 || units == 0);
    }
  }
};

// The line: every unit takes its tiles and kUnitCost places more, what its
// queries and its merge cost beside them, so that a share of many short units
// is no longer work than one of a few long ones (a batch of 8 with sequences
// of 0 and 1 tokens beside 32K: 18 us above the time to read its cache without
// this, 15 with 1, 12 with 3, 12 with 4; full batches do not change).
constexpr int kUnitCost = 3;

// Where place `x` of the line lies: sequence b, the places before it, the tiles
// before it.
struct Place {
  int b;
  int64_t at, tiles;
  // tiles before place x, nt and the units being those of sequence b
  __device__ __forceinline__ int64_t tiles_before(int64_t x, int nt) const {
    const int64_t u = (x - at) / (nt + kUnitCost), r = (x - at) - u * (nt + kUnitCost);
    return tiles + u * nt + (r < nt ? r : nt);
  }
};
struct Line {
  int64_t N, tiles;        // places, tiles
  Place p[2];
};

// A block's view of the line.  want(i, N): the i-th place sought (a place behind
// the end is not found), or, with seq >= 0, the place of sequence seq.
// WARPS warps, all threads; scan: 2 WARPS + 6 words of shared memory.  EARLY: see load_len.
template <int WARPS, bool EARLY, bool TREE, class Want>
__device__ __forceinline__ Line line_of(const CacheParams& a, int64_t* scan, Want want, int seq) {
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  int64_t* found = scan + 2 * WARPS;
  Line r;
  r.N = 0;
  if (a.batch <= 32) {
    // few sequences, one per lane: every warp finds out by itself, without a barrier
    // (one sequence of 131071 tokens 91.4 -> 90.5 us, 8 of 32768 tokens 91.0 -> 90.5 us)
    int64_t own = 0, v = 0, t = 0;
    if (lane < a.batch) {
      Walk<TREE> k;
      k.b = lane;
      k.template load<EARLY>(a);
      t = (int64_t)k.tr.nt * k.units;
      v = own = k.tr.nt ? t + (int64_t)kUnitCost * k.units : 0;
    }
    const int64_t own_t = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t m = __shfl_up_sync(kFull, v, o), n = __shfl_up_sync(kFull, t, o);
      if (lane >= o) {
        v += m;
        t += n;
      }
    }
    r.N = __shfl_sync(kFull, v, 31);
    r.tiles = __shfl_sync(kFull, t, 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t x = seq < 0 ? want(i, r.N) : 0;
      const unsigned here = __ballot_sync(kFull, seq >= 0 ? lane == seq : v - own <= x && x < v);
      const int l = here ? __ffs(here) - 1 : 0;
      r.p[i] = Place{l, __shfl_sync(kFull, v - own, l), __shfl_sync(kFull, t - own_t, l)};
    }
    return r;
  }
  // up to 32 WARPS sequences are read once
  const bool once = a.batch <= 32 * WARPS;
  for (int pass = once ? 1 : 0; pass < 2; ++pass) {
    int64_t places = 0, tiles = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32 * WARPS) {
      const int b = b0 + tid;
      int64_t own = 0, v = 0, t = 0;
      if (b < a.batch) {
        Walk<TREE> k;
        k.b = b;
        k.template load<EARLY>(a);
        t = (int64_t)k.tr.nt * k.units;
        v = own = k.tr.nt ? t + (int64_t)kUnitCost * k.units : 0;
      }
      const int64_t own_t = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t m = __shfl_up_sync(kFull, v, o), n = __shfl_up_sync(kFull, t, o);
        if (lane >= o) {
          v += m;
          t += n;
        }
      }
      __syncthreads();
      if (lane == 31) {
        scan[2 * w] = v;
        scan[2 * w + 1] = t;
      }
      __syncthreads();
      int64_t bv = places, bt = tiles;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        if (i < w) {
          bv += scan[2 * i];
          bt += scan[2 * i + 1];
        }
        places += scan[2 * i];
        tiles += scan[2 * i + 1];
      }
      if (once) r.N = places;
      if (pass == 1) {
        const int64_t lo = bv + v - own;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t x = seq < 0 ? want(i, r.N) : 0;
          if (seq >= 0 ? b == seq : b < a.batch && lo <= x && x < lo + own) {
            found[3 * i] = b;
            found[3 * i + 1] = lo;
            found[3 * i + 2] = bt + t - own_t;
          }
        }
      }
    }
    r.N = places;
    r.tiles = tiles;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) r.p[i] = Place{(int)found[3 * i], found[3 * i + 1], found[3 * i + 2]};
  return r;
}

}  // namespace ca

// The CTA of a place of the line: share c of N places is [N c / n, N (c + 1) / n).
__device__ __forceinline__ int cta_of(int64_t x, int64_t N, int n) {
  return (int)(((x + 1) * n - 1) / N);
}

template <int WR, bool CAP, bool BIAS, bool CL, bool TREE>
__global__ void __launch_bounds__(ca::kThreads, 2)
cache_attn_kernel(const __grid_constant__ CacheParams a,
                  const __grid_constant__ Tensors<TREE> maps) {
  using namespace ca;
  constexpr int WT = kWarps / WR;            // warps across a tile's tokens
  constexpr int NT = kKeyTile / WT;          // tokens a warp takes of a tile
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBars);
  uint64_t* empty = full + kStages;
  volatile uint32_t* gone = reinterpret_cast<volatile uint32_t*>(smem + kMisc);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + kMisc + 8);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    *gone = 0u;
    fence_barrier_init();
  }
  if (w == kWarps && lane < 2)
    asm volatile("prefetch.tensormap [%0];" :: "l"(lane ? &maps.v : &maps.k) : "memory");
  if constexpr (TREE) {
    if (w == kWarps && lane < 2)
      asm volatile("prefetch.tensormap [%0];" :: "l"(lane ? &maps.v_nodes : &maps.k_nodes) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what came before may have written anything
  Walk<TREE> wk;
  int total = 0;                             // tiles of this CTA
  if constexpr (CL) {
    // ---- the cluster's unit, cut evenly over its CTAs
    const int csize = (int)cluster_size(), rank = (int)cluster_rank();
    const int per = a.Hkv * ((a.T * a.G + a.RT - 1) / a.RT), unit = cta / csize;
    wk.b = unit / per;
    wk.load(a);
    wk.u = unit - wk.b * per;
    wk.x = (int)((int64_t)wk.tr.nt * rank / csize);
    total = (int)((int64_t)wk.tr.nt * (rank + 1) / csize) - wk.x;
    __syncthreads();
  } else {
    __syncthreads();                           // the barriers are there
    // ---- this CTA's share of the line, never an empty one (the join reads every
    // CTA between a unit's ends), and the tiles in it
    const Line line = line_of<kWarps + 1, false, TREE>(
        a, scan,
        [&](int i, int64_t N) {
          const int64_t n = N < a.n_cta ? (N > 0 ? N : 1) : a.n_cta;
          return N * (cta + i) / n;
        },
        -1);
    const int64_t N = line.N;
    const int n_cta = N < a.n_cta ? (int)N : a.n_cta;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (cta >= n_cta) return;
    const int64_t begin = N * cta / n_cta, end = N * (cta + 1) / n_cta;

    int64_t last_tile = line.tiles;
    if (end < N) {
      wk.b = line.p[1].b;
      wk.load(a);
      last_tile = line.p[1].tiles_before(end, wk.tr.nt);
    }
    wk.b = line.p[0].b;
    wk.load(a);
    total = (int)(last_tile - line.p[0].tiles_before(begin, wk.tr.nt));
    if (total == 0) return;                    // nothing but the cost of a unit before
    wk.u = (int)((begin - line.p[0].at) / (wk.tr.nt + kUnitCost));
    wk.x = (int)((begin - line.p[0].at) - (int64_t)wk.u * (wk.tr.nt + kUnitCost));
    if (wk.x >= wk.tr.nt) {                    // behind a unit's tiles: the next unit
      wk.x = wk.tr.nt - 1;
      wk.advance(a, 1);
    }
  }

  if (w == kWarps) {
    // ================= the feeding warp.  Lane l looks up the page of tile
    // i + l, so that a table entry is read 32 tiles ahead of its copy.
    int row_l = 0, x_l = 0, issued = 0;
    for (int i = 0; i < total; ++i) {
      if ((i & 31) == 0) {
        Walk<TREE> f = wk;
        f.advance(a, lane);
        if (i + lane < total) {
          row_l = f.tr.tile(f.x) * kKeyTile;
          x_l = (f.u / f.groups(a)) * kCacheD;
          if (TREE && row_l >= f.s.kv) {
            row_l = ~(f.b * kTreeRoom);      // rows of the nodes' tensors
          } else {
            int64_t blk = a.table[(int64_t)f.b * a.max_pages + (row_l >> a.lgP)];
            if (blk < 0 || blk >= a.nblocks) {
              atomicOr(&g_cache_attn_flags, kFlagBadBlock);
              blk = 0;
            }
            row_l = (int)checked_index((blk << a.lgP) + (row_l & ((1 << a.lgP) - 1)),
                                       a.nblocks << a.lgP, &g_cache_attn_flags);
          }
        }
        __syncwarp();
        if (i + 32 < total) wk.advance(a, 32);
      }
      int row = __shfl_sync(kFull, row_l, i & 31);
      const int x = __shfl_sync(kFull, x_l, i & 31);
      const CUtensorMap *km = &maps.k, *vm = &maps.v;
      if constexpr (TREE) {
        if (row < 0) {
          row = ~row;
          km = &maps.k_nodes;
          vm = &maps.v_nodes;
        }
      }
      const int st = i % kStages;
      if (i >= kStages) wait(&empty[st], (uint32_t)(i / kStages - 1) & 1u, gone);
      if (lane == 0 && !*gone) {
        uint8_t* at = smem + st * kStageBytes;
        mbar_expect_tx(&full[st], kStageBytes);
        tma_load_2d(at, km, x, row, &full[st]);
        tma_load_2d(at + kBox, km, x + 64, row, &full[st]);
        tma_load_2d(at + 2 * kBox, vm, x, row, &full[st]);
        tma_load_2d(at + 3 * kBox, vm, x + 64, row, &full[st]);
        ++issued;
      }
      __syncwarp();
    }
    if (lane == 0) drain_copies(full, kStages, issued, &g_cache_attn_flags);
    __syncwarp();
    if constexpr (CL) {
      cluster_sync();                        // the parts are there
      cluster_sync();                        // and have been read
    }
    return;
  }

  // ================= the four computing warps
  const int wr = w / WT, wt = w % WT;         // its rows, its tokens of a tile
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  uint32_t qf[8][4];
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (CL && total == 0) {
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  }
  int p[2], pf[2];                            // position and prefix of the thread's two rows
  float slope[2];
  int tu0 = 0, tu1 = 0;                       // the unit's tokens
  int h = 0, r0 = 0, rows = 0;
  bool fresh = true, live[2] = {true, true};  // (of a tree: there is a node)

  for (int i = 0; i < total; ++i) {
    if (fresh) {
      // ---- a unit begins: its queries, rows past the end as zeros
      fresh = false;
      const int ng = wk.groups(a);
      h = wk.u / ng;
      r0 = (wk.u % ng) * a.RT;
      rows = wk.s.n * a.G - r0;
      if (rows > a.RT) rows = a.RT;
      tu0 = r0 / a.G;
      tu1 = (r0 + rows - 1) / a.G;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * wr + g + 8 * e;
        const bool in = r < rows;
        const int t = in ? (r0 + r) / a.G : 0, gq = in ? (r0 + r) - t * a.G : 0;
        const int hq = h * a.G + gq;
        if constexpr (TREE) {
          // (rows of no node ask for no masks: their sums are dropped at the unit's end)
          const int depth = in ? tree_depth(a, wk.b, t) : -1;
          live[e] = depth >= 0;
          p[e] = wk.s.pos0 + (depth > 0 ? depth : 0);
        } else {
          p[e] = in ? wk.s.pos0 + t : -1;
        }
        pf[e] = p[e] >= 0 ? wk.s.pf : 0;
        slope[e] = BIAS && in ? cache_slope(a.slopes[hq]) : 0.f;
        const uint16_t* qr = a.q + (wk.s.tok0 + t) * a.q_stride + hq * kCacheD + c2;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          qf[k][e] = in ? *reinterpret_cast<const uint32_t*>(qr + 16 * k) : 0u;
          qf[k][e + 2] = in ? *reinterpret_cast<const uint32_t*>(qr + 16 * k + 8) : 0u;
        }
        m[e] = -INFINITY;
        l[e] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    }
    const int st = i % kStages;
    const int j0 = wk.tr.tile(wk.x) * kKeyTile;         // first token of the tile
    // masks: none if every row sees the whole tile; no work if none sees any
    const bool nodes = TREE && j0 >= wk.s.kv;
    const int q0 = wk.s.pos0 + (TREE ? 0 : tu0), q1 = wk.s.pos0 + (TREE ? wk.s.n - 1 : tu1);
    const bool inside = j0 + kKeyTile <= wk.s.pf && q0 >= 0;
    const bool all = TREE ? j0 + kKeyTile <= wk.s.kv && (inside || q1 - j0 < a.window)
                          : inside || (j0 + kKeyTile - 1 <= q0 && q1 - j0 < a.window);
    const bool none = !nodes && j0 >= wk.s.pf &&
                      (j0 > q1 || (q0 > 0 ? q0 : 0) - (j0 + kKeyTile - 1) >= a.window);
    MaskPart masks{0, 0};
    if (TREE && nodes) masks = mask_part(a, wk.b, lane);
    wait(&full[st], (uint32_t)(i / kStages) & 1u, gone);
    // the warp's tokens of a nodes' tile: those behind the last node are left out, by 16
    const int held = TREE && nodes ? wk.s.n - wt * NT : NT;
    if (!none && held > 0) {
      const uint32_t kb = smem_u32(smem + st * kStageBytes), vb = kb + 2 * kBox;
      const int tw = wt * NT;                           // first token of the warp's part
      if (j0 + kKeyTile > wk.s.kv) {
        // values behind the last token, or of a node that none sees, may hold anything, a
        // NaN too, and their weight of zero would not clear it
        const int from = nodes ? 0 : wk.s.kv - j0 > tw ? wk.s.kv - j0 - tw : 0;
        const int to = TREE && nodes && held < NT ? (held + 15) & ~15 : NT;
        const uint64_t seen = TREE && nodes ? any_sees(masks) : 0;
        for (int t = tw + from; t < tw + to; ++t) {
          if (seen >> t & 1) continue;
          *reinterpret_cast<uint2*>(smem + st * kStageBytes + (2 + (lane >> 4)) * kBox + t * 128 +
                                    (lane & 15) * 8) = make_uint2(0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
      }
      float s[NT / 8][4];
#pragma unroll
      for (int n = 0; n < NT / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      {
        // K as the second operand: rows are tokens, 16 bytes are 8 channels
        const int tr = ((lane >> 4) & 1) * 8 + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int n = 0; n < NT / 16; ++n) {
            const int t = tw + 16 * n + tr, cc = 2 * (k & 3) + ch;
            uint32_t f[4];
            ldsm4(kb + (k >> 2) * kBox + t * 128 + ((cc ^ (t & 7)) << 4), f);
            mma(s[2 * n], qf[k], f[0], f[1]);
            mma(s[2 * n + 1], qf[k], f[2], f[3]);
          }
      }
      // ---- scores, masks, the running maximum
      uint64_t sees[2] = {0, 0};                        // of the nodes, by the two rows
      if constexpr (TREE) {
        if (nodes)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * wr + g + 8 * e;
            if (live[e]) sees[e] = tree_sees(a, wk.b, (r0 + r) / a.G);
          }
      }
      float mx[2] = {m[0], m[1]};
      if constexpr (TREE) {
        // (one loop a rule, and the capped scores' function-unit operations only where a
        // score of the warp is past half a cap.  16 x 6 nodes over 12001, a cap: 92.7 us
        // with all of it in one loop, 72 to 74 us like this)
        bool far = false;
        if constexpr (CAP) {
          float size = 0.f;
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) size = fmaxf(size, fabsf(s[n][e]));
          far = __any_sync(kFull, !(size <= a.cap_small));
        }
        if (CAP && !far) {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const f2 x = make_float2(s[n][e], s[n][e + 1]), v = mul2(x, cache_cap_factor(a, x));
              s[n][e] = v.x;
              s[n][e + 1] = v.y;
            }
        } else {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = cache_score<CAP>(a, s[n][e]);
        }
        if (BIAS) {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = tw + 8 * n + c2 + (e & 1);
              const int away = !nodes ? p[e >> 1] - (j0 + c)
                               : p[e >> 1] - wk.s.pos0 - (c < wk.s.n ? tree_depth(a, wk.b, c) : 0);
              s[n][e] = fmaf(-slope[e >> 1], fabsf((float)away), s[n][e]);
            }
        }
        if (nodes) {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(sees[e >> 1] >> (tw + 8 * n + c2 + (e & 1)) & 1u)) s[n][e] = -INFINITY;
        } else if (!all) {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = e >> 1, j = j0 + tw + 8 * n + c2 + (e & 1);
              if (!(j < wk.s.kv && (p[r] - j < a.window || j < pf[r]))) s[n][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int n = 0; n < NT / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      } else {
#pragma unroll
      for (int n = 0; n < NT / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1, j = j0 + tw + 8 * n + c2 + (e & 1);
          float v = cache_score<CAP>(a, s[n][e]);
          if constexpr (BIAS) v = fmaf(-slope[r], fabsf((float)(p[r] - j)), v);
          if (!all) {
            const bool vis = (j <= p[r] && p[r] - j < a.window) || j < pf[r];
            v = vis ? v : -INFINITY;
          }
          s[n][e] = v;
          mx[r] = fmaxf(mx[r], v);
        }
      }
      float mr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 2));
        mr[r] = mx[r] == -INFINITY ? 0.f : mx[r];       // a row that sees nothing yet
      }
      if (__any_sync(kFull, mx[0] != m[0] || mx[1] != m[1])) {
        const float f0 = cache_ex2(m[0] - mr[0]), f1 = cache_ex2(m[1] - mr[1]);
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
        m[0] = mx[0];
        m[1] = mx[1];
      }
      // ---- weights and the second product
      const int tv = ((lane >> 3) & 1) * 8 + (lane & 7), cv = lane >> 4;
#pragma unroll
      for (int n = 0; n < NT / 16; ++n) {
        if (TREE && 16 * n >= held) break;
        uint32_t pa[4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float* e = s[2 * n + hh];
          const float e0 = cache_ex2(e[0] - mr[0]), e1 = cache_ex2(e[1] - mr[0]);
          const float e2 = cache_ex2(e[2] - mr[1]), e3 = cache_ex2(e[3] - mr[1]);
          l[0] += e0 + e1;
          l[1] += e2 + e3;
          pa[2 * hh] = f2_to_bf2(e0, e1);
          pa[2 * hh + 1] = f2_to_bf2(e2, e3);
        }
        const int t = tw + 16 * n + tv;
#pragma unroll
        for (int d = 0; d < 8; ++d) {                   // 16 channels
          const int cc = 2 * (d & 3) + cv;
          uint32_t f[4];
          ldsm4t(vb + (d >> 2) * kBox + t * 128 + ((cc ^ (t & 7)) << 4), f);
          mma(o[2 * d], pa, f[0], f[1]);
          mma(o[2 * d + 1], pa, f[2], f[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) arrive(&empty[st]);

    const bool last = i == total - 1 || wk.x + 1 == wk.tr.nt;
    if (last) {
      // ---- the unit ends here: row sums over the quad, then the token warps
      float* ml = reinterpret_cast<float*>(smem + kMl);
      if constexpr (TREE) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!live[e]) {
            m[e] = -INFINITY;
            l[e] = 0.f;
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n][2 * e] = o[n][2 * e + 1] = 0.f;
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(kFull, l[r], 1);
        l[r] += __shfl_xor_sync(kFull, l[r], 2);
      }
      auto put = [&](int slot) {
        float4* sc = reinterpret_cast<float4*>(smem + kScratch + slot * 8192);
#pragma unroll
        for (int n = 0; n < 16; ++n) sc[n * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
        if ((lane & 3) == 0) {
          ml[slot * 32 + 2 * g] = m[0];
          ml[slot * 32 + 2 * g + 1] = l[0];
          ml[slot * 32 + 16 + 2 * g] = m[1];
          ml[slot * 32 + 16 + 2 * g + 1] = l[1];
        }
      };
      auto get = [&](int slot) {
        const float4* sc = reinterpret_cast<const float4*>(smem + kScratch + slot * 8192);
        float fo[2], fn[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mo = ml[slot * 32 + 16 * r + 2 * g], lo = ml[slot * 32 + 16 * r + 2 * g + 1];
          const float mn = fmaxf(m[r], mo), mz = mn == -INFINITY ? 0.f : mn;
          fo[r] = cache_ex2(m[r] - mz);
          fn[r] = cache_ex2(mo - mz);
          l[r] = l[r] * fo[r] + lo * fn[r];
          m[r] = mn;
        }
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float4 v = sc[n * 32 + lane];
          o[n][0] = o[n][0] * fo[0] + v.x * fn[0];
          o[n][1] = o[n][1] * fo[0] + v.y * fn[0];
          o[n][2] = o[n][2] * fo[1] + v.z * fn[1];
          o[n][3] = o[n][3] * fo[1] + v.w * fn[1];
        }
      };
      if constexpr (WT == 4) {
        if (w >= 2) put(w - 2);
        sync_consumers();
        if (w < 2) get(w);
        sync_consumers();
        if (w == 1) put(0);
        sync_consumers();
        if (w == 0) get(0);
        sync_consumers();                               // before the next unit's put
      } else if constexpr (WT == 2) {
        if (wt == 1) put(wr);
        sync_consumers();
        if (wt == 0) get(wr);
        sync_consumers();
      }
      if (!CL && wt == 0) {
        const bool started = i - wk.x >= 0;             // the unit's first tile is in this share
        const bool whole = started && wk.x + 1 == wk.tr.nt;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * wr + g + 8 * e;
            if (r < rows) {
              const int t = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - t * a.G;
              const float inv = cache_inv(l[e]);
              const int64_t at = checked_index((wk.s.tok0 + t) * a.Hq + hq, a.n_tokens * a.Hq,
                                               &g_cache_attn_flags);
#pragma unroll
              for (int n = 0; n < 16; ++n)
                *reinterpret_cast<uint32_t*>(a.out + at * kCacheD + 8 * n + c2) =
                    f2_to_bf2(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
              if (a.lse && (lane & 3) == 0) a.lse[at] = cache_lse(m[e], l[e]);
            }
          }
        } else {
          float* ps = a.part + (int64_t)(2 * cta + (started ? 1 : 0)) * (a.RT * (kCacheD + 2));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * wr + g + 8 * e;
            if ((lane & 3) == 0) {
              ps[2 * r] = m[e];
              ps[2 * r + 1] = l[e];
            }
#pragma unroll
            for (int n = 0; n < 16; ++n)
              *reinterpret_cast<float2*>(ps + 2 * a.RT + r * kCacheD + 8 * n + c2) =
                  make_float2(o[n][2 * e], o[n][2 * e + 1]);
          }
        }
      }
      fresh = true;
    }
    if (i + 1 < total) wk.advance(a, 1);
  }
  if constexpr (CL) {
    // ---- the CTAs' parts meet in shared memory (the ring's, which is done with);
    // each CTA merges every csize-th row
    const int csize = (int)cluster_size(), rank = (int)cluster_rank();
    constexpr int kPitch = kCacheD + 4;
    float* so = reinterpret_cast<float*>(smem);
    float2* sml = reinterpret_cast<float2*>(so + 16 * WR * kPitch);
    sync_consumers();                        // every warp is done with the last tile
    if (wt == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * wr + g + 8 * e;
        if ((lane & 3) == 0) sml[r] = make_float2(m[e], l[e]);
#pragma unroll
        for (int n = 0; n < 16; ++n)
          *reinterpret_cast<float2*>(so + r * kPitch + 8 * n + c2) =
              make_float2(o[n][2 * e], o[n][2 * e + 1]);
      }
    }
    cluster_sync();
    const int ng = wk.groups(a);
    const int u = (cta / csize) % (a.Hkv * ng), hh = u / ng, first = (u % ng) * a.RT;
    const int b = (cta / csize) / (a.Hkv * ng);
    const int left = a.T * a.G - first, n = left < a.RT ? left : a.RT;
    for (int r = rank + csize * w; r < n; r += csize * kWarps) {
      float M = -INFINITY, L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < csize; ++k) {
        const float2 q = ld_peer2(sml + r, (uint32_t)k);
        const float4 v = ld_peer4(so + r * kPitch + 4 * lane, (uint32_t)k);
        cache_merge(M, L, O, q.x, q.y, v);
      }
      const float inv = cache_inv(L);
      const int t = (first + r) / a.G;
      const int64_t at = checked_index(((int64_t)b * a.T + t) * a.Hq + hh * a.G + first + r - t * a.G,
                                       a.n_tokens * a.Hq, &g_cache_attn_flags);
      *reinterpret_cast<uint2*>(a.out + at * kCacheD + 4 * lane) =
          make_uint2(f2_to_bf2(O.x * inv, O.y * inv), f2_to_bf2(O.z * inv, O.w * inv));
      if (a.lse && lane == 0) a.lse[at] = cache_lse(M, L);
    }
    cluster_sync();
  }
}

// The join.  Four warps, W of them to an output row, each merging every W-th
// partial with four channels a lane.  Rows of a unit that one CTA wrote are
// left alone; rows that see nothing get zeros.  All that does not need the
// partials is worked out before the wait for the grid that writes them.
constexpr int kJoinWarps = 4;
constexpr int kJoinBatch = 8;

template <int W, bool TREE>
__global__ void __launch_bounds__(32 * kJoinWarps)
cache_join_kernel(const __grid_constant__ CacheParams a) {
  constexpr int kRows = kJoinWarps / W;        // rows of the block, of one sequence
  __shared__ int64_t scan[2 * kJoinWarps + 6];
  __shared__ float4 so[W > 1 ? kJoinWarps : 1][32];
  __shared__ float2 sm[kJoinWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int all = a.T * a.Hq, per = (all + kRows - 1) / kRows;
  const int b = (int)(blockIdx.x / (unsigned)per);
  const int idx = (int)(blockIdx.x % (unsigned)per) * kRows + w / W;
  const ca::Line line = ca::line_of<kJoinWarps, true, TREE>(
      a, scan, [](int, int64_t) { return (int64_t)0; }, b);
  ca::Walk<TREE> wk;
  wk.b = b;
  wk.template load<true>(a);
  const int t = idx / a.Hq, hq = idx - t * a.Hq, h = hq / a.G, row = t * a.G + hq - h * a.G;
  const int r = row % a.RT;
  int k0 = 0, k1 = -1;
  if (wk.tr.nt > 0) {
    const int64_t x0 = line.p[0].at +
                       (int64_t)(h * wk.groups(a) + row / a.RT) * (wk.tr.nt + ca::kUnitCost);
    const int n_cta = line.N < a.n_cta ? (int)line.N : a.n_cta;
    k0 = cta_of(x0, line.N, n_cta);
    k1 = cta_of(x0 + wk.tr.nt - 1, line.N, n_cta);
  }
  // (every thread waits, also where there is nothing to join: this grid must not end
  // before the one it depends on)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // rows that one CTA wrote are left (for the whole block, where warps share a row)
  if (idx >= all || (k1 >= 0 && k0 == k1)) return;
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int kb = k0 + w % W; kb <= k1; kb += W * kJoinBatch) {
    float2 ml[kJoinBatch];
    float4 ov[kJoinBatch];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      const int k = kb + W * i;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k <= k1) {
        const int slot = k == k0 ? 1 : 0;      // the unit begins in k0's share
        const float* ps = a.part + checked_index(2 * (int64_t)k + slot, 2 * (int64_t)a.n_cta,
                                                 &g_cache_attn_flags) * (a.RT * (kCacheD + 2));
        ml[i] = *reinterpret_cast<const float2*>(ps + 2 * r);
        ov[i] = *reinterpret_cast<const float4*>(ps + 2 * a.RT + r * kCacheD + 4 * lane);
      }
    }
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) cache_merge(M, L, O, ml[i].x, ml[i].y, ov[i]);
  }
  if constexpr (W > 1) {
    so[w][lane] = O;
    if (lane == 0) sm[w] = make_float2(M, L);
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int i = 1; i < W; ++i) cache_merge(M, L, O, sm[i].x, sm[i].y, so[i][lane]);
  }
  const float inv = cache_inv(L);
  const int64_t z = (int64_t)b * all + idx;
  *reinterpret_cast<uint2*>(a.out + z * kCacheD + 4 * lane) =
      make_uint2(f2_to_bf2(O.x * inv, O.y * inv), f2_to_bf2(O.z * inv, O.w * inv));
  if (a.lse && lane == 0) a.lse[z] = cache_lse(M, L);
}

// ------------------------------------------------------------------ host

// Tensor map of BF16 rows[rows][inner] for boxes of box_rows x 64 with the 128-byte
// swizzle.  (cuTensorMapEncodeTiled through the runtime: no -lcuda.)
static cudaError_t tensor_map_rows(CUtensorMap* map, const void* base, int64_t inner, int64_t rows,
                                   int box_rows) {
  using Fn = decltype(&cuTensorMapEncodeTiled);
  static const Fn encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                           cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Fn>(p)
                                                                    : nullptr;
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows per unit: the smallest of 16, 32, 64 that holds a sequence's rows.
static int rows_per_unit(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

constexpr int kMaxCtas = 512;   // two per SM, of up to 256 SMs: what the workspace is sized for

// Rows for which the register MMAs are slower than memory: the many-row kernel
// takes them, in shares.  8 sequences of 32767 tokens, 8 KV heads: 32 rows 171 us
// here, 172 there (floor 158); 64 rows 245 here, 177 there; 128 rows 475 here (in
// two units), 179 there.  2 x 16000, 128 rows: 78 and 39 us.
static bool many_rows(int R) { return R > 32; }

// Whether units are clusters: contexts of at most kClusterTiles tiles (the table
// has room for no more) and all units resident at once.  1 x 1000 tokens, 8 KV
// heads: 7.5 us as clusters, 8.5 us split and joined, and 4 us less on the host;
// 4 x 1000 8.7 and 11.3 us, 1 x 2000 9.2 us either way; 32 ragged up to 4000 60.8
// and 53.0 us, since a cluster's share does not follow the lengths.  Many rows: only
// where every unit gets eight CTAs.  1 x 2000, 64 rows: 13.9 us as clusters, 23.5 us on
// the many-row kernel; 8 x 2000 28.4 and 25.1, 32 x 2000 81.7 and 50.2 us.
constexpr int kClusterTiles = 32, kClusterUnits = 304;
static bool in_clusters(int64_t units, int R, int64_t max_tokens) {
  return max_tokens <= (int64_t)kClusterTiles * kKeyTile &&
         units <= (many_rows(R) ? kClusterUnits / 8 : kClusterUnits);
}
static int64_t units_of(int batch, int T, int G, int Hkv) {
  const int RT = rows_per_unit(T * G);
  return (int64_t)batch * Hkv * ((T * G + RT - 1) / RT);
}

size_t cache_attn_workspace_bytes(int batch, int T, int64_t n_tokens, int Hq, int Hkv,
                                  int64_t max_tokens, bool tree) {
  const int G = Hq / Hkv;
  if (T && in_clusters(units_of(batch, T, G, Hkv), T * G, max_tokens)) return 0;
  if (!T || many_rows(T * G))
    return cache_prefill_workspace_bytes(batch, n_tokens, G, Hkv, max_tokens, tree);
  return (size_t)2 * kMaxCtas * rows_per_unit(T * G) * (kCacheD + 2) * sizeof(float);
}

int cache_attn_form(int batch, int T, int64_t n_tokens, int Hq, int Hkv, int64_t max_tokens,
                    int sms, bool tree) {
  const int G = Hq / Hkv;
  if (T && in_clusters(units_of(batch, T, G, Hkv), T * G, max_tokens)) return LYNX_CACHE_CLUSTERS;
  if (T && !many_rows(T * G)) return LYNX_CACHE_SPLIT;
  return cache_prefill_form(batch, n_tokens, G, Hkv, max_tokens, sms, tree);
}

template <int W, bool TREE>
static cudaError_t run_join(const CacheParams& p, cudaStream_t stream) {
  constexpr int kRows = kJoinWarps / W;
  return launch_dependent(cache_join_kernel<W, TREE>,
                          dim3((unsigned)((int64_t)p.batch * ((p.T * p.Hq + kRows - 1) / kRows))),
                          32 * kJoinWarps, 0, 0, stream, p);
}

// csize: CTAs to a unit, 0 for shares of the line and a join
template <int WR, bool CAP, bool BIAS, bool CL, bool TREE>
static cudaError_t run(const CacheParams& p, int csize, const Tensors<true>& m,
                       cudaStream_t stream) {
  const Tensors<TREE> maps = tensors_of<TREE>(m);
  auto fn = cache_attn_kernel<WR, CAP, BIAS, CL, TREE>;
  static thread_local int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ca::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  const int64_t units = units_of(p.batch, p.T, p.G, p.Hkv);
  if constexpr (CL)
    return launch_dependent(fn, dim3((unsigned)(units * csize)), ca::kThreads, ca::kSmem,
                            (unsigned)csize, stream, p, maps);
  e = launch_dependent(fn, dim3((unsigned)p.n_cta), ca::kThreads, ca::kSmem, 0, stream, p, maps);
  if (e != cudaSuccess) return e;
  // as many warps to a row as its units are likely to be split over CTAs
  return p.n_cta >= 8 * units ? run_join<4, TREE>(p, stream) : run_join<1, TREE>(p, stream);
}

template <int WR, bool CL, bool TREE>
static cudaError_t run_score(const CacheParams& p, bool cap, int csize, const Tensors<true>& m,
                             cudaStream_t stream) {
  if (cap) return p.slopes ? run<WR, true, true, CL, TREE>(p, csize, m, stream)
                           : run<WR, true, false, CL, TREE>(p, csize, m, stream);
  return p.slopes ? run<WR, false, true, CL, TREE>(p, csize, m, stream)
                  : run<WR, false, false, CL, TREE>(p, csize, m, stream);
}

template <int WR, bool TREE>
static cudaError_t run_rows(const CacheParams& p, bool cap, int csize, const Tensors<true>& m,
                            cudaStream_t stream) {
  return csize ? run_score<WR, true, TREE>(p, cap, csize, m, stream)
               : run_score<WR, false, TREE>(p, cap, csize, m, stream);
}

template <bool TREE>
static cudaError_t run_call(const CacheParams& p, bool cap, int csize, const Tensors<true>& m,
                            cudaStream_t stream) {
  return p.RT == 16 ? run_rows<1, TREE>(p, cap, csize, m, stream)
         : p.RT == 32 ? run_rows<2, TREE>(p, cap, csize, m, stream)
                      : run_score<4, true, TREE>(p, cap, csize, m, stream);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& x, cudaStream_t stream) {
  constexpr double kLog2e = 1.4426950408889634;
  CacheParams p;
  p.q = static_cast<const uint16_t*>(x.q);
  p.q_stride = x.q_stride;
  p.table = x.c.table;
  p.kv_len = x.c.kv_len;
  p.offsets = x.c.offsets;
  p.max_pages = x.c.max_pages;
  p.nblocks = x.c.nblocks;
  p.n_tokens = x.c.n_tokens;
  p.batch = x.c.batch;
  p.T = x.c.T;
  p.Hq = x.Hq;
  p.Hkv = x.c.Hkv;
  p.G = x.Hq / x.c.Hkv;
  p.lgP = __builtin_ctz((unsigned)x.c.page);
  p.window = x.window > 0 && x.window < INT_MAX ? (int)x.window : INT_MAX;
  p.prefix = x.prefix;
  p.slopes = x.slopes;
  p.mask = x.mask;
  // (kept finite: an infinite factor would turn a score of zero into a NaN, and half of
  // the range leaves room for cap_out to be doubled)
  auto factor = [](double f) { return (float)(f < FLT_MAX / 2 ? f : FLT_MAX / 2); };
  p.qk = factor(x.scale * kLog2e);
  p.cap_in = x.softcap > 0 ? factor(2.0 * kLog2e * x.scale / x.softcap) : 0.f;
  p.cap_out = factor(x.softcap * kLog2e);
  p.cap_small = 0.f;
  for (int i = 0; i < kCapTerms; ++i) p.cap_poly[i] = 0.f;
  if (x.softcap > 0) {
    const double to_x = (double)x.scale / x.softcap;     // q.k to the tanh's argument
    double f = (double)x.softcap * kLog2e * to_x;
    bool fits = true;                                    // of caps of any sensible size
    for (int i = 0; i < kCapTerms; ++i, f *= to_x * to_x) {
      p.cap_poly[i] = (float)(kTanhPoly[i] * f);
      fits = fits && fabs(kTanhPoly[i] * f) < 1e30;
    }
    p.cap_small = !fits ? -1.f : kCapSmall / to_x < 1e15 ? (float)(kCapSmall / to_x) : 1e15f;
  }
  p.out = static_cast<uint16_t*>(x.out);
  p.lse = x.lse;
  p.part = static_cast<float*>(x.workspace);
  p.RT = rows_per_unit(p.T * p.G);
  const int sms = sm_count();
  p.n_cta = 2 * (sms < kMaxCtas / 2 ? sms : kMaxCtas / 2);
  Tensors<true> maps;
  cudaError_t e;
  const int64_t rows = x.c.nblocks * x.c.page, width = (int64_t)p.Hkv * kCacheD;
  if ((e = tensor_map_rows(&maps.k, x.k_pool, width, rows, kKeyTile)) != cudaSuccess) return e;
  if ((e = tensor_map_rows(&maps.v, x.v_pool, width, rows, kKeyTile)) != cudaSuccess) return e;
  if (x.mask) {
    const int64_t n = (int64_t)p.batch * kTreeRoom;
    static_assert(kTreeRoom == kKeyTile, "a sequence's nodes are one tile");
    if ((e = tensor_map_rows(&maps.k_nodes, x.k_nodes, width, n, kKeyTile)) != cudaSuccess) return e;
    if ((e = tensor_map_rows(&maps.v_nodes, x.v_nodes, width, n, kKeyTile)) != cudaSuccess) return e;
  }
  const bool cap = x.softcap > 0;
  const int64_t max_tokens = p.max_pages << p.lgP;
  const int form =
      cache_attn_form(p.batch, p.T, p.n_tokens, p.Hq, p.Hkv, max_tokens, sms, p.mask != nullptr);
  if (form != LYNX_CACHE_CLUSTERS && form != LYNX_CACHE_SPLIT)
    return launch_cache_prefill(p, cap, maps, stream);
  // CTAs to a unit: as many as fill the GPU, at most one to a tile and eight
  int csize = 0;
  if (form == LYNX_CACHE_CLUSTERS) {
    const int64_t units = units_of(p.batch, p.T, p.G, p.Hkv);
    csize = 1;
    while (csize < 8 && 2 * csize * units <= 2 * sms && 2 * csize * kKeyTile <= max_tokens)
      csize *= 2;
  }
  return p.mask ? run_call<true>(p, cap, csize, maps, stream)
                : run_call<false>(p, cap, csize, maps, stream);
}

}  // namespace lynx
