// cache_prefill.cu -- attention of packed chunks over the BF16 paged cache on
// the tensor-memory path: the many-row side of cache_attn.cu.
//
//   s_ij = scale q_i.k_j, capped, minus slope |p_i - j|, over the visible j;
//   lse_i = ln sum_j e^s_ij,  out_i = sum_j e^(s_ij - lse_i) v_j
//
// What bounds it: 4 * 128 flop per (query head, visible key) on the tensor
// cores, and beside them one exponential per pair.  A turn (256 rows by 128 keys)
// takes 2430 cycles, 2048 of them tensor work: a row half's softmax is a little
// longer than the other half's two products.  2 x 8192 tokens, 32 heads over 8,
// causal: 0.62 ms, 1.77 PFLOP/s, in bursts; 0.69 to 0.71 ms under the power cap.
//
// Work.  A unit is one (sequence, KV head, 256 query rows); row r is token
// r / G, query head h G + r % G.  The cache comes in tiles of 128 tokens; one CTA
// per SM walks units.  Either whole ones, the longest row blocks of a sequence
// first, taken as the CTAs become free.  Or, where there are few and they are
// long, equal shares of the line of all tiles: a share may then begin and end
// inside a unit, whose parts (m, l, o) go to the workspace and are merged by a
// join, so that a few rows over a long cache use the whole GPU.  Or whole units,
// the last of them in equal parts, where they are all long and would leave CTAs
// idle in a last round.  Units of trees, which are as many as the call says, go
// otherwise: see tree_form() and lend().
//
// A tree of drafted nodes (TREE, see cache_attn.cu): the last tile of a unit holds the
// nodes' keys in its first half, and nothing in the second.  8 x 32768 tokens, 64 nodes, 64
// heads over 4: 0.35 ms in a graph, 0.37 to 0.38 call by call (1.57 and 1.44 to 1.49 PFLOP/s),
// 128 units on as many SMs.
//
// Warps:
//  * 0-7 and 8-15, the softmax of 128 rows each, two threads a row: a row's
//    scores from tensor memory to registers (64 a thread), its maximum (the
//    two threads' through shared memory), weights 2^(s - m) as BF16 back to
//    tensor memory over the scores, where they are the first operand of the
//    second product.  m is raised (and the output rescaled) only when a score
//    exceeds it by 2^8: the weights then stay below 2^8, which BF16 and the
//    float32 sum hold as exactly as [0, 1].
//  * 16 feeds a ring of five 32 KiB buffers (K, V, K, V, ...) by TMA, each tile
//    as 64-token boxes, since a page may be 64 tokens.
//  * 18 works out the CTA's units and announces them to the others.
//  * 17 issues the tcgen05 MMAs: S = Q K^T and O += P V, each 128 x 128 x 128,
//    for the two row halves in turn, so that one half's softmax runs under the
//    other half's products.
// Tensor memory: S (then P) of both halves, O of both halves: 512 columns.
//
// Rounding: as cache_attn.cu: P to BF16, the rest float32.
#include <math.h>

#include "cache_attn.h"
#include "lynx.h"

namespace lynx {

__device__ unsigned int g_cache_prefill_flags = 0;

cudaError_t read_cache_prefill_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_cache_prefill_flags, sizeof(unsigned int));
}

namespace cp {

constexpr int kTile = 128;                  // cached tokens per tile
constexpr int kHalf = 128;                  // rows of a softmax warpgroup
constexpr int kUnit = 2 * kHalf;            // rows per unit
constexpr int kSoftWarps = 16;
constexpr int kThreads = 32 * (kSoftWarps + 4);   // setmaxnreg acts on four warps at once
constexpr int kCols = kTile / 2;            // scores of a row per thread
constexpr int kRing = 5;
constexpr int kSlots = 1;                   // units announced ahead of the one under way
constexpr uint32_t kBox = 64 * 128;         // 64 rows x 64 channels
constexpr uint32_t kBuf = 4 * kBox;         // 128 rows x 128 channels: [channel half][row]
constexpr uint32_t kQ = 0;
constexpr uint32_t kKv = 2 * kBuf;
constexpr uint32_t kBars = kKv + kRing * kBuf;
// mbarriers: ring full / empty, then per half Q, S, P (of 64 tokens each), O,
// then units announced / taken, a claim's answer, a unit's last tile on its way,
// all products (where waits were given up), a tree's values
constexpr int kBFull = 0, kBEmpty = kRing, kBQ = 2 * kRing, kBS = kBQ + 2, kBP = kBS + 2,
              kBO = kBP + 4, kBUnit = kBO + 2, kBUsed = kBUnit + kSlots,
              kBClaim = kBUsed + kSlots, kBFed = kBClaim + 1, kBDone = kBFed + 1,
              kBNodes = kBDone + 1, kBCount = kBNodes + 1;
// tensor-memory address, abort word, tiles of the longest unit
constexpr uint32_t kMisc = kBars + 8 * kBCount;
constexpr uint32_t kMax = kMisc + 16;                // [half][column half][row] floats
constexpr uint32_t kUnits = (kMax + 2 * 2 * kHalf * 4 + 15) / 16 * 16;
constexpr uint32_t kClaim = kUnits + kSlots * 64;    // 16 bytes
constexpr uint32_t kSmem = kClaim + 16;
static_assert(kSmem <= 227 * 1024, "one CTA per SM");
// how units are shared out
constexpr int kWhole = 0, kShares = 1, kTail = 2;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 for the second half

// kind::f16, float32 accumulator, BF16 operands, M = N = 128; b_mn: B is
// N-major
constexpr uint32_t idesc(int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((128u >> 3) << 17) |
         ((128u >> 4) << 24);
}
// Shared-memory descriptor with the 128-byte swizzle: lbo the bytes between
// 64-element blocks of an MN-major operand, sbo between groups of 8 rows.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3fffu) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc(0)), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc(1)), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
      :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void ld32(uint32_t taddr, float* r) {
  uint32_t v[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
         "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
         "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ld8(uint32_t taddr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                 "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void st8(uint32_t taddr, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]),
                  "f"(r[6]), "f"(r[7])
               : "memory");
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Asks to take over a block of the grid that has not been launched; the answer, 16
// bytes of shared memory, completes the barrier.
__device__ __forceinline__ void claim(uint64_t* bar, void* answer) {
  mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" :: "r"(smem_u32(answer)), "r"(smem_u32(bar)) : "memory");
}
// Whether there was one (no more claims are made after a no), and which.
__device__ __forceinline__ bool claimed(const void* answer, uint32_t& x) {
  uint32_t yes, id;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n"
      " mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
      : "=r"(yes), "=r"(id) : "r"(smem_u32(answer)) : "memory");
  fence_proxy_async();                     // read before the next answer is written
  __syncwarp();
  if (yes) x = id;
  return yes != 0;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// The low n bits, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t below(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Bounded wait, as in cache_attn.cu; false if it was given up.  A unit may have to
// end first: the limit grows by 100 us for each tile of the longest one announced
// (gone[1]).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t phase, volatile uint32_t* gone,
                                         uint64_t limit_ns, unsigned int* flag) {
  if (mbar_try_wait(bar, phase)) return true;
  if (*gone) return false;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, phase)) {
    if (*gone) return false;
    if (global_ns() - t0 > limit_ns + (uint64_t)gone[1] * 100000u) {
      *gone = 1u;
      atomicOr(flag, kFlagWaitTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase, volatile uint32_t* gone) {
  return wait_for(bar, phase, gone, kWaitNs, &g_cache_prefill_flags);
}
// Waits for every product issued so far, by the warp that issued them and whatever
// became of its other waits: tensor memory must not go before them.  (That warp runs a
// unit of `tiles` tiles to its end without waiting, so the limit grows with them.)
__device__ __forceinline__ bool drain_products(uint64_t* done, bool one, uint32_t tiles,
                                               unsigned int* flag) {
  if (one) commit(done);
  __syncwarp();
  const uint64_t t0 = global_ns();
  bool ok = mbar_try_wait(done, 0);
  while (!ok && global_ns() - t0 <= kWaitNs + (uint64_t)tiles * 100000u)
    ok = mbar_try_wait(done, 0);
  if (!ok) atomicOr(flag, kFlagWaitTimeout);
  return ok;
}

__device__ __forceinline__ int row_blocks(const CacheParams& a, const Seq& s) {
  return (int)(((int64_t)s.n * a.G + kUnit - 1) / kUnit);
}

// One unit of the walk, as announced in shared memory.
struct __align__(16) Unit {     // the first 64 bytes are announced
  int nt;                   // tiles; -1: no more units
  int rows;                 // 1 .. 256
  int b, h, row0;           // sequence, KV head, first row in the sequence
  int tok0, pos0, kv, pf;   // see Seq
  int nA, B0;               // see TileRange
  int lo, hi;               // the keys its rows see lie in [lo, hi) or the prefix
  int x0;                   // the first of its tiles in this share
  int last;                 // index here of the unit's last tile (>= nt: not here)
  int slot;                 // -1: all of it is here; else the place of this part in the
                            // workspace: twice the share, plus one if the unit begins there
  int part;                 // (not announced) -1, 0, 1 accordingly
  int unused[3];
  __device__ __forceinline__ bool active(int half) const { return rows > half * kHalf; }
  __device__ __forceinline__ int tile(int i) const {
    return x0 + i < nA ? x0 + i : x0 + i - nA + B0;
  }
  // whether the 64 tokens from j on are read (of the nodes' tile the first 64)
  template <bool TREE>
  __device__ __forceinline__ bool needs(int j) const {
    if (TREE && j >= node_tile<kTile>(kv) * kTile) return j % kTile == 0;
    return (j < hi && j + 64 > lo) || j < pf;
  }
};
static_assert(sizeof(Unit) == 80, "kUnits");

__device__ __forceinline__ Unit unit_at(const uint8_t* smem, int slot) {
  Unit u;
  const int4* src = reinterpret_cast<const int4*>(smem + kUnits + slot * 64);
  int4* dst = reinterpret_cast<int4*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[i] = src[i];
  return u;
}

// The line of units: row blocks in the order of the sequences, within one the
// longest first, each with its KV heads; a unit takes its tiles and kUnitCost
// places more.  Walked by one warp, 32 sequences at a time (lane l holds
// sequence b0 + l).
constexpr int kUnitCost = 3;
// A part of a unit that another CTA lends a hand with costs it this many tiles more, and is
// worth a join (10 us) from this many on and from a sixth of the longest unit on.
constexpr int kLendCost = 4, kLendLeast = 16;
template <bool TREE>
struct Walk {
  int b0, own, incl, tot;         // row blocks: the lane's, up to and with it, of all 32
  Seq s;
  __device__ __forceinline__ void load(const CacheParams& a, int lane) {
    s.n = 0;
    if (b0 + lane < a.batch) s = load_seq<false, TREE>(a, b0 + lane);
    own = row_blocks(a, s);
    incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int m = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += m;
    }
    tot = __shfl_sync(kFull, incl, 31);
  }
  // Row block j of these sequences (j < tot), j the lane's own or the same for all
  __device__ __forceinline__ Unit block(const CacheParams& a, int j) const {
    int l = 0;                    // the first lane with incl > j
#pragma unroll
    for (int o = 16; o; o >>= 1)
      if (__shfl_sync(kFull, incl, l + o - 1) <= j) l += o;
    Unit u;
    Seq q;
    const int end = __shfl_sync(kFull, incl, l);
    q.n = __shfl_sync(kFull, s.n, l);
    q.pos0 = __shfl_sync(kFull, s.pos0, l);
    q.kv = __shfl_sync(kFull, s.kv, l);
    q.pf = __shfl_sync(kFull, s.pf, l);
    u.tok0 = __shfl_sync(kFull, (int)s.tok0, l);
    u.b = b0 + l;
    u.row0 = (end - 1 - j) * kUnit;
    const int64_t n = (int64_t)q.n * a.G - u.row0;
    u.rows = n < kUnit ? (int)n : kUnit;
    const int t0 = u.row0 / a.G, t1 = (u.row0 + u.rows - 1) / a.G;
    const TileRange tr = tiles_of<kTile, TREE>(a, q, t0, t1);
    u.nt = tr.nt;
    u.nA = tr.nA;
    u.B0 = tr.B0;
    u.pos0 = q.pos0;
    u.kv = q.kv;
    u.pf = q.pf;
    const int pmin = TREE ? q.pos0 : q.pos0 + t0 > 0 ? q.pos0 + t0 : 0;
    u.lo = pmin - a.window + 1 > 0 ? pmin - a.window + 1 : 0;
    u.hi = TREE ? q.kv : q.pos0 + t1 + 1;
    return u;
  }
  // Places of the next 32 row blocks from j on, summed up to each lane.
  __device__ __forceinline__ int64_t places(const CacheParams& a, int j, int lane) const {
    const Unit u = block(a, j + lane < tot ? j + lane : tot - 1);
    int64_t v = j + lane < tot ? (int64_t)(u.nt + kUnitCost) * a.Hkv : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t m = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += m;
    }
    return v;
  }
};

// A unit that began in an earlier share, for the join: which CTAs hold its parts.
struct __align__(16) Seam {
  int k0, k1;               // k1 = -1: this share begins with a unit
  int rows, row0, tok0, h;
  int unused[2];
};

// Partial `i` in the workspace, behind the seams: m [256 rows], l [256], then o
// [128 channels][256 rows], since a warp writes 32 rows at once.
constexpr int kMaxCtas = 160;
constexpr int kPartFloats = kUnit * (kCacheD + 2);
__device__ __forceinline__ float* part_of(const CacheParams& a, int i) {
  return a.part + kMaxCtas * sizeof(Seam) / sizeof(float) + (int64_t)i * kPartFloats;
}

// Channels 64 ch .. 64 ch + 63 of the warp's 32 rows of a unit's half into the
// operand's layout: two blocks of 64 channels, rows of 128 bytes, 16-byte
// pieces swizzled by the row.  r: the lane's row.  Each lane finds its own
// row; eight lanes then copy a row's 128 bytes.
__device__ __forceinline__ void load_q(const CacheParams& a, const Unit& u, uint32_t dst, int half,
                                       int r, int ch, int lane) {
  const int row = u.row0 + half * kHalf + r;
  const bool in = half * kHalf + r < u.rows;
  const int t = in ? row / a.G : 0, g = in ? row - t * a.G : 0;
  const uint64_t own = in ? reinterpret_cast<uint64_t>(
      a.q + (int64_t)(u.tok0 + t) * a.q_stride + (u.h * a.G + g) * kCacheD + 64 * ch) : 0;
  const int c = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int from = 4 * i + (lane >> 3), rr = (r & ~31) + from;
    const uint64_t src = __shfl_sync(kFull, own, from);
    const uint32_t at = dst + ch * 2 * kBox + rr * 128 + ((c ^ (rr & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(at), "l"(src ? src + 16 * c : reinterpret_cast<uint64_t>(a.q)),
                    "r"(src ? 16u : 0u) : "memory");
  }
}

// 32 bytes of output: a whole sector in one store where the output is aligned
// to it (callers owe 16 bytes).
__device__ __forceinline__ void st_sector(uint16_t* p, const uint32_t (&v)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                    "r"(v[6]), "r"(v[7]) : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace cp

template <bool CAP, bool BIAS, int MODE, bool TREE>
__global__ void __launch_bounds__(cp::kThreads, 1)
cache_prefill_kernel(const __grid_constant__ CacheParams a,
                     const __grid_constant__ Tensors<TREE> maps) {
  using namespace cp;
  constexpr bool SPLIT = MODE != kWhole;       // parts go to the workspace
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, w = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kBars);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + kMisc);
  volatile uint32_t* gone = misc + 1;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar[kBFull + i], 1);
      mbar_init(&bar[kBEmpty + i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar[kBQ + t], 2 * kHalf);
      mbar_init(&bar[kBS + t], 1);
      mbar_init(&bar[kBP + 2 * t], 2 * kHalf);
      mbar_init(&bar[kBP + 2 * t + 1], 2 * kHalf);
      mbar_init(&bar[kBO + t], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar[kBUnit + i], 1);
      mbar_init(&bar[kBUsed + i], kSoftWarps + 2);
    }
    mbar_init(&bar[kBClaim], 1);
    mbar_init(&bar[kBFed], 1);
    mbar_init(&bar[kBDone], 1);
    mbar_init(&bar[kBNodes], 1);
    gone[0] = gone[1] = 0u;
    fence_barrier_init();
  }
  if (w == kSoftWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(smem_u32(smem + kMisc)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what came before may have written anything
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = __shfl_sync(kFull, misc[0], 0);
  // Unit k, once announced (nt = -1 behind the last one, and once a wait has been
  // given up); taken: the warp needs its slot no more.
  auto peek = [&](int k) {
    const bool told = wait(&bar[kBUnit + k % kSlots], (uint32_t)(k / kSlots) & 1u, gone);
    Unit u = unit_at(smem, k % kSlots);
    if (!__all_sync(kFull, told)) u.nt = -1;
    return u;
  };
  auto take = [&](int k) {
    const Unit u = peek(k);
    __syncwarp();
    if (lane == 0) arrive(&bar[kBUsed + k % kSlots]);
    return u;
  };
  if (w >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (w == kSoftWarps) {
      // ================= the feeding warp: item n of the ring is K (n even) or
      // V of tile n / 2
      int item = 0, issued = 0, trees = 0;
      for (int k = 0;; ++k) {
        const Unit u = take(k);
        if (u.nt < 0) break;
        int row_l = -1;
        for (int i = 0; i < u.nt; ++i) {
          if ((i & 15) == 0) {
            // lane l: the first pool row of 64-token piece l of the next 16 tiles
            const int x = i + (lane >> 1);
            row_l = -1;
            if (x < u.nt) {
              const int j = u.tile(x) * kTile + 64 * (lane & 1);
              if (TREE && j >= u.kv && u.needs<TREE>(j)) {
                row_l = -2;                // the nodes
              } else if (j < u.kv && u.needs<TREE>(j)) {
                int64_t blk = a.table[(int64_t)u.b * a.max_pages + (j >> a.lgP)];
                if (blk < 0 || blk >= a.nblocks) {
                  atomicOr(&g_cache_prefill_flags, kFlagBadBlock);
                  blk = 0;
                }
                row_l = (int)checked_index((blk << a.lgP) + (j & ((1 << a.lgP) - 1)),
                                           a.nblocks << a.lgP, &g_cache_prefill_flags);
              }
            }
          }
          const int r0 = __shfl_sync(kFull, row_l, 2 * (i & 15));
          const int r1 = __shfl_sync(kFull, row_l, 2 * (i & 15) + 1);
          const uint32_t bytes = ((TREE ? r0 != -1 : r0 >= 0) ? 2 * kBox : 0) + (r1 >= 0 ? 2 * kBox : 0);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++item) {
            const int st = item % kRing;
            if (item >= kRing)
              wait(&bar[kBEmpty + st], (uint32_t)(item / kRing - 1) & 1u, gone);
            if constexpr (TREE) {
              if (kv && r0 == -2) {
                // Values of places that no node sees may be anything, a NaN too: they are
                // cleared before the issuing warp is told.  (With that warp doing it
                // each tile of a unit took 75 cycles longer.)
                const MaskPart masks = mask_part(a, u.b, lane);
                uint8_t* at = smem + kKv + st * kBuf;
                const bool go = __shfl_sync(kFull, *gone, 0) == 0u;
                if (!go) continue;
                if (lane == 0) {
                  mbar_expect_tx(&bar[kBNodes], 2 * kBox);
                  tma_load_2d(at, &maps.v_nodes, u.h * kCacheD, u.b * kTreeRoom, &bar[kBNodes]);
                  tma_load_2d(at + 2 * kBox, &maps.v_nodes, u.h * kCacheD + 64, u.b * kTreeRoom,
                              &bar[kBNodes]);
                }
                __syncwarp();
                const uint64_t seen = any_sees(masks);
                at += (lane >> 4) * 2 * kBox + (lane & 15) * 8;
                for (int r = kTreeRoom; r < kTile; ++r)
                  *reinterpret_cast<uint2*>(at + r * 128) = make_uint2(0u, 0u);
                wait(&bar[kBNodes], (uint32_t)trees++ & 1u, gone);
                for (uint64_t left = ~seen; left; left &= left - 1)
                  *reinterpret_cast<uint2*>(at + (__ffsll((long long)left) - 1) * 128) =
                      make_uint2(0u, 0u);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                  arrive(&bar[kBFull + st]);
                  ++issued;
                }
                continue;
              }
            }
            if (lane == 0 && !*gone) {
              const CUtensorMap* map = kv ? &maps.v : &maps.k;
              if constexpr (TREE) {
                if (r0 == -2) map = &maps.k_nodes;
              }
              const int from = TREE && r0 == -2 ? u.b * kTreeRoom : r0;
              uint8_t* at = smem + kKv + st * kBuf;
              uint64_t* fb = &bar[kBFull + st];
              mbar_expect_tx(fb, bytes);
              ++issued;
              if (from >= 0) {
                tma_load_2d(at, map, u.h * kCacheD, from, fb);
                tma_load_2d(at + 2 * kBox, map, u.h * kCacheD + 64, from, fb);
              }
              if (r1 >= 0) {
                tma_load_2d(at + kBox, map, u.h * kCacheD, r1, fb);
                tma_load_2d(at + 3 * kBox, map, u.h * kCacheD + 64, r1, fb);
              }
            }
            __syncwarp();
          }
        }
        if (MODE != kShares && lane == 0) arrive(&bar[kBFed]);
      }
      if (lane == 0) {
        drain_copies(&bar[kBFull], kRing, issued, &g_cache_prefill_flags);
        if (TREE) drain_copies(&bar[kBNodes], 1, trees, &g_cache_prefill_flags);
      }
      __syncwarp();
    } else if (w == kSoftWarps + 1) {
      // ================= the issuing warp.  One elected lane issues; everything
      // that the descriptors and branches depend on is uniform over the warp
      // and known to the compiler to be (counters, and broadcasts of what was
      // loaded): with operands it took for per-lane values an MMA needed
      // 110 cycles to issue, nearly twice its 64 cycles of work.
      const bool one = elect_one();
      const uint64_t qd = sdesc(smem_u32(smem + kQ), 16, 1024);
      const uint64_t kd = sdesc(smem_u32(smem + kKv), 16, 1024);
      const uint64_t vd = sdesc(smem_u32(smem + kKv), 2 * kBox, 1024);
      uint32_t st = 0, ph = 0;             // the ring's next item
      int items = 0;                       // tiles so far
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      for (int k = 0;; ++k) {
        const Unit u = take(k);
        const int nt = __shfl_sync(kFull, u.nt, 0);
        if (nt < 0) break;
        if (nt == 0) continue;
        const int halves = __shfl_sync(kFull, u.rows, 0) > kHalf ? 2 : 1;
        // tiles of which a part is not read, or lies behind the last token: the
        // last one, and any where a window or a prefix ends
        const bool ragged = a.window != INT_MAX || a.prefix != nullptr;
        // The ring's item for tile i, waited for.  Values that were not read may be
        // anything, a NaN too, and a weight of zero would not clear it: they are
        // cleared here.
        auto ready_v = [&](int i, uint32_t buf, uint32_t phase) {
          wait(&bar[kBFull + buf], phase, gone);
          if (TREE ? i != u.last && (ragged || i == u.last - 1) : ragged || i == u.last) {
            const int j0 = u.tile(i) * kTile;
            const bool miss0 = !u.needs<TREE>(j0), miss1 = !u.needs<TREE>(j0 + 64);
            if (j0 + kTile > u.kv || miss0 || miss1) {
              for (int r = 0; r < kTile; ++r) {
                if (j0 + r >= u.kv || (r < 64 ? miss0 : miss1))
                  *reinterpret_cast<uint2*>(smem + kKv + buf * kBuf + (lane >> 4) * 2 * kBox +
                                            r * 128 + (lane & 15) * 8) = make_uint2(0u, 0u);
              }
              fence_proxy_async();
            }
            __syncwarp();
          }
        };
        // Each turn: the second product of tile i - 1, the first of tile i.  The
        // ring is waited for where the tensor cores have work queued: K behind the
        // first half's second product, V behind its first.
        uint32_t vst = 0;                  // V of the tile before
        for (int i = 0; i <= nt; ++i) {
          uint32_t kst = st, kph = ph;
          if (i < nt && ++st == kRing) st = 0, ph ^= 1u;
          uint32_t nvst = st;              // V of this tile
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t < halves) {
              if (i > 0) {                 // O_t += P_t V
                const uint64_t d = vd + (uint64_t)(vst * (kBuf >> 4));
#pragma unroll
                for (int q = 0; q < 2; ++q) {   // 64 tokens as soon as their weights are there
                  wait(&bar[kBP + 2 * t + q], np[t], gone);
                  fence_after();
                  if (one) {
#pragma unroll
                    for (int c = 4 * q; c < 4 * q + 4; ++c)
                      mma_ts(tm + kColO + 128 * t, tm + kColS + 128 * t + 8 * c,
                             d + (2048 >> 4) * c, (c > 0 || i > 1) ? 1u : 0u);
                    if (q) commit(&bar[kBO + t]);
                  }
                }
                np[t] ^= 1u;
                if (one && t + 1 == halves) commit(&bar[kBEmpty + vst]);
              }
              if (i < nt) {                // S_t = Q_t K^T
                if (t == 0) wait(&bar[kBFull + kst], kph, gone);
                if (i == 0) {
                  wait(&bar[kBQ + t], nq[t], gone);
                  nq[t] ^= 1u;
                }
                fence_after();
                if (one) {
                  const uint64_t dq = qd + (uint64_t)(t * (kBuf >> 4));
                  const uint64_t dk = kd + (uint64_t)(kst * (kBuf >> 4));
#pragma unroll
                  for (int c = 0; c < kCacheD / 16; ++c) {
                    const uint32_t off = ((c >> 2) * 2 * kBox + (c & 3) * 32) >> 4;
                    mma_ss(tm + kColS + 128 * t, dq + off, dk + off, c > 0 ? 1u : 0u);
                  }
                  commit(&bar[kBS + t]);
                  if (t + 1 == halves) commit(&bar[kBEmpty + kst]);
                }
              }
            }
            if (t == 0 && i < nt) {
              ready_v(i, st, ph);
              if (++st == kRing) st = 0, ph ^= 1u;
            }
          }
          vst = nvst;
        }
        items += nt;
      }
      // every release has landed before the barriers go
      for (int n = 2 * items > kRing ? 2 * items - kRing : 0; n < 2 * items; ++n)
        wait(&bar[kBEmpty + n % kRing], (uint32_t)(n / kRing) & 1u, gone);
      // (where a wait was given up, that loop waited for nothing)
      if (__any_sync(kFull, *gone != 0u))
        drain_products(&bar[kBDone], one, gone[1], &g_cache_prefill_flags);
    } else if (w == kSoftWarps + 2) {
      // ================= the announcing warp
      Walk<TREE> wk;
      wk.b0 = 0;
      wk.load(a, lane);
      int k = 0;
      auto announce = [&](const Unit& u) {
        if (k >= kSlots &&
            !__all_sync(kFull, wait(&bar[kBUsed + k % kSlots], (uint32_t)(k / kSlots - 1) & 1u, gone)))
          return false;                    // given up: nothing is overwritten
        if (lane == 0 && u.nt > (int)gone[1]) gone[1] = (uint32_t)u.nt;
        if (lane < 4)
          reinterpret_cast<int4*>(smem + kUnits + (k % kSlots) * 64)[lane] =
              lane == 0 ? make_int4(u.nt, u.rows, u.b, u.h)
              : lane == 1 ? make_int4(u.row0, u.tok0, u.pos0, u.kv)
              : lane == 2 ? make_int4(u.pf, u.nA, u.B0, u.lo)
                          : make_int4(u.hi, u.x0, u.last, u.part < 0 ? -1 : u.slot);
        __syncwarp();
        if (lane == 0) arrive(&bar[kBUnit + k % kSlots]);
        ++k;
        return true;
      };
      bool going = true;                   // false: a wait was given up
      if constexpr (MODE != kShares) {
        // Whole units, one to a block of the grid: this block's, then those of blocks
        // that it takes over before they are launched, so that a CTA is never
        // without work while there is some.  The units under way and the last
        // ones to be taken are then short ones, which even out the end.
        uint32_t x = blockIdx.x, phase = 0;
        int base = 0;                      // row blocks before these sequences
        for (;;) {
          // kTail: blocks from tail0 on are parts of units, tail_parts each; part y of
          // all is share y of the join, which meets its unit at the second part
          uint32_t unit = x;
          int part = 0, y = -1;
          if (MODE == kTail && x >= (uint32_t)a.tail0) {
            y = (int)(x - (uint32_t)a.tail0);
            unit = (uint32_t)a.tail0 + (uint32_t)(y / a.tail_parts);
            part = y % a.tail_parts;
          }
          const int blk = (int)(unit / (uint32_t)a.Hkv);
          if (blk < base) {                // (should blocks ever come out of order)
            base = 0;
            wk.b0 = 0;
            wk.load(a, lane);
          }
          while (blk >= base + wk.tot && wk.b0 + 32 < a.batch) {
            base += wk.tot;
            wk.b0 += 32;
            wk.load(a, lane);
          }
          const bool real = blk < base + wk.tot;   // the grid may have more blocks than units
          Seam seam = {0, -1, 0, 0, 0, 0, {0, 0}};
          if (real) {
            Unit u = wk.block(a, blk - base);
            u.h = (int)(unit - (uint32_t)blk * (uint32_t)a.Hkv);
            u.x0 = 0;
            u.last = u.nt - 1;
            u.part = -1;
            if (MODE == kTail && y >= 0) {
              if (part == 1)
                seam = Seam{y - 1, y - 2 + a.tail_parts, u.rows, u.row0, u.tok0, u.h, {0, 0}};
              const int nt = u.nt;
              u.x0 = (int)((int64_t)nt * part / a.tail_parts);
              u.nt = (int)((int64_t)nt * (part + 1) / a.tail_parts) - u.x0;
              u.last = nt - 1 - u.x0;
              u.part = part == 0 ? 1 : 0;
              u.slot = 2 * y + u.part;
            }
            going = announce(u);
          }
          if (MODE == kTail && y >= 0 && lane == 0) reinterpret_cast<Seam*>(a.part)[y] = seam;
          if (real) {
            // the next one is claimed when this one's last tile is on its way: taken
            // earlier, it might wait here while other CTAs have nothing to do (2048
            // tokens, 1.7 units a CTA: 40 us when claimed as a unit begins, 32 us like this)
            if (!going || !__all_sync(kFull, wait(&bar[kBFed], (uint32_t)(k - 1) & 1u, gone)))
              break;
          }
          if (lane == 0) claim(&bar[kBClaim], smem + kClaim);
          if (!__all_sync(kFull, wait(&bar[kBClaim], phase, gone))) {
            (void)mbar_wait(&bar[kBClaim], phase);   // the answer is still to be written
            going = false;
            break;
          }
          phase ^= 1u;
          if (!claimed(smem + kClaim, x)) break;
        }
      } else if (TREE && a.tail0 > 0) {
        // Units and lenders: CTA c has unit c, of which the tiles from `cut` on go to CTAs
        // without a unit or with a short one, a unit's to one of them.  (Sequences are
        // lanes, all here; their units are `per` each and as long as one another.)
        const int units = a.tail0, per = units / a.batch, idle = (int)gridDim.x - units;
        const int nt = lane < a.batch ? tiles_of<kTile, TREE>(a, wk.s, 0, wk.s.n - 1).nt : 0;
        const int longest = __reduce_max_sync(kFull, nt);
        // the shortest cut, of one for each lane, that leaves room for what is cut off: a part
        // takes its tiles and kLendCost more
        int cut = longest - longest * lane / 64;
        {
          const int part = longest - cut + kLendCost;
          const float each = 1.f / (float)part;
          auto holds = [&](int left) {       // left / part, without a division
            if (left < part) return 0;
            const int q = (int)((float)left * each);     // off by one at most
            return q * part > left ? q - 1 : (q + 1) * part <= left ? q + 1 : q;
          };
          int cuts = 0, room = 0;
          for (int b = 0; b < a.batch; ++b) {
            const int n = __shfl_sync(kFull, nt, b);
            if (n > cut) ++cuts;
            else room += holds(cut - n - kLendCost);
          }
          const bool fits = longest - cut >= max(kLendLeast, longest / 6) &&
                            idle * holds(cut) + per * room >= per * cuts;
          const unsigned m = __ballot_sync(kFull, fits);
          cut = m ? __shfl_sync(kFull, cut, 31 - __clz(m)) : longest;
        }
        const int part = longest - cut + kLendCost;
        // how many parts the CTAs of the lane's sequence take, and those without a unit
        const int takes = lane < a.batch && nt <= cut && nt + kLendCost < cut
                              ? (cut - nt - kLendCost) / part : 0;
        const int idle_takes = cut / part;
        const unsigned cuts = __ballot_sync(kFull, nt > cut);
        const int cta = blockIdx.x, mine = cta / per;    // (mine: a sequence, or none)
        // tiles x0 .. x0 + n - 1 of a unit
        auto give = [&](int unit, int x0, int n, int first) {
          Unit v = wk.block(a, unit / a.Hkv);
          v.h = unit % a.Hkv;
          v.x0 = x0;
          v.last = v.nt - 1 - x0;
          v.part = n == v.nt ? -1 : first;
          v.nt = n;
          v.slot = 2 * (unit + 1 - first) + first;
          going = announce(v);
          return v;
        };
        int can = idle_takes;
        if (cta < units) {
          const int n = __shfl_sync(kFull, nt, mine);
          can = __shfl_sync(kFull, takes, mine);
          const Unit v = give(cta, 0, n < cut ? n : cut, 1);
          Seam seam = {0, -1, 0, 0, 0, 0, {0, 0}};
          if (n > cut) seam = Seam{cta, cta + 1, v.rows, v.row0, v.tok0, v.h, {0, 0}};
          if (lane == 0) reinterpret_cast<Seam*>(a.part)[cta + 1] = seam;
        }
        // round by round, a part each: row blocks over the same keys are then under way
        // at the same time
        int at = 0;                          // parts of the rounds before
        for (int round = 0; going && round < can && longest > cut; ++round) {
          const unsigned take = __ballot_sync(kFull, takes > round);
          const int of_units = per * __popc(take);
          const int place = cta >= units ? of_units + cta - units
                                         : per * __popc(take & ((1u << mine) - 1u)) + cta - per * mine;
          int i = at + place;
          at += of_units + (idle_takes > round ? idle : 0);
          if (i >= per * __popc(cuts)) break;
          unsigned left = cuts;              // the sequence of part i
          for (; i >= per; i -= per) left &= left - 1;
          const int b = __ffs(left) - 1;
          give(per * b + i, cut, __shfl_sync(kFull, nt, b) - cut, 0);
        }
      } else {
        int64_t N = 0;
        for (;;) {
          for (int j = 0; j < wk.tot; j += 32) N += __shfl_sync(kFull, wk.places(a, j, lane), 31);
          if (wk.b0 + 32 >= a.batch) break;
          wk.b0 += 32;
          wk.load(a, lane);
        }
        // shares of eight places at least: a smaller one costs more than it saves
        const int most = (int)((N + 7) / 8 < gridDim.x ? (N + 7) / 8 : gridDim.x);
        const int cta = blockIdx.x;
        const int64_t begin = cta < most ? N * cta / most : N;
        const int64_t end = cta < most ? N * (cta + 1) / most : N;
        Seam seam = {0, -1, 0, 0, 0, 0, {0, 0}};
        if (begin < end) {
          // the row block that holds the share's first place
          int64_t left = end - begin;
          int64_t at = 0;                  // places before these sequences' block j
          int j = 0;
          if (wk.b0) {
            wk.b0 = 0;
            wk.load(a, lane);
          }
          for (;;) {
            if (j >= wk.tot) {
              wk.b0 += 32;
              if (wk.b0 >= a.batch) break; // (lengths that changed under the call)
              wk.load(a, lane);
              j = 0;
              continue;
            }
            const int64_t v = wk.places(a, j, lane);
            const unsigned past = __ballot_sync(kFull, at + v > begin);
            if (past) {
              const int l = __ffs(past) - 1;
              const int64_t before = __shfl_sync(kFull, v, l > 0 ? l - 1 : 0);
              if (l > 0) at += before;
              j += l;
              break;
            }
            at += __shfl_sync(kFull, v, 31);
            j += 32;
          }
          if (wk.b0 >= a.batch) {
            wk.tot = 0;
            left = 0;
          }
          Unit u = wk.block(a, j);
          u.h = (int)((begin - at) / (u.nt + kUnitCost));
          int x = (int)((begin - at) - (int64_t)u.h * (u.nt + kUnitCost));
          if (left > 0 && x > 0 && x < u.nt) {
            const int64_t first = begin - x;
            seam = Seam{(int)(((first + 1) * most - 1) / N), (int)(((first + u.nt) * most - 1) / N),
                        u.rows, u.row0, u.tok0, u.h, {0, 0}};
          }
          while (going && left > 0) {
            if (x < u.nt || x == 0) {
              Unit v = u;
              v.nt = u.nt - x < left ? u.nt - x : (int)left;
              v.x0 = x;
              v.last = u.nt - 1 - x;
              v.part = v.nt == u.nt ? -1 : x == 0 ? 1 : 0;
              v.slot = 2 * cta + v.part;
              going = announce(v);
            }
            left -= u.nt + kUnitCost - x;
            if (left <= 0) break;
            x = 0;
            if (++u.h < a.Hkv) continue;
            while (++j >= wk.tot && wk.b0 + 32 < a.batch) {
              wk.b0 += 32;
              wk.load(a, lane);
              j = -1;
            }
            if (j >= wk.tot) break;        // (as above)
            u = wk.block(a, j);
            u.h = 0;
          }
        }
        if (lane == 0) reinterpret_cast<Seam*>(a.part)[cta] = seam;
      }
      if (going) {
        Unit u = {};
        u.nt = -1;
        announce(u);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ================= softmax: thread = row `r` of half t, 32 columns (tokens)
    // of each 64: 32 ch .. and 64 + 32 ch ..
    const int t = w >> 3, ch = (w >> 2) & 1, r = 32 * (w & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (w & 3)) << 16;
    const uint32_t ts = tm + kColS + 128 * t + lanes, to = tm + kColO + 128 * t + 64 * ch + lanes;
    const uint32_t qdst = smem_u32(smem + kQ + t * kBuf);
    // this thread's word of the exchange, and that of the row's other thread
    volatile float* mine = reinterpret_cast<float*>(smem + kMax) + (t * 2 + ch) * kHalf + r;
    volatile float* other = reinterpret_cast<float*>(smem + kMax) + (t * 2 + 1 - ch) * kHalf + r;
    const int pair = 1 + 4 * t + (w & 3);   // named barrier of the two warps of 32 rows
    // whether any of the pair's 64 threads says yes
    auto vote_pair = [&](bool yes) {
      uint32_t any;
      asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
                   " barrier.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                   : "=r"(any) : "r"((uint32_t)yes), "r"(pair) : "memory");
      return any != 0;
    };
    auto sync_pair = [&]() { asm volatile("barrier.sync %0, 64;" :: "r"(pair) : "memory"); };
    uint32_t ns = 0;                        // tiles of this half so far
    bool loaded = false;                    // the next unit's queries are on their way
    for (int k = 0;; ++k) {
      const Unit u = take(k);
      const int nt = u.nt;
      if (vote_pair(nt < 0)) break;         // both warps, whatever each was told
      const bool in = t * kHalf + r < u.rows;
      const int row = u.row0 + t * kHalf + r;
      const int tok = in ? row / a.G : 0, g = in ? row - tok * a.G : 0;
      const int hq = in ? u.h * a.G + g : 0;
      float m = -INFINITY, l = 0.f;
      bool live = true;                     // (of a tree: there is a node)
      if (nt > 0 && u.active(t)) {
        if (!loaded) {
          load_q(a, u, qdst, t, r, ch, lane);
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async();
          arrive(&bar[kBQ + t]);
        }
        loaded = false;
        // rows of no token see everything, so that they ask for no masks
        // (nor do places of a tree without a node: their sums are dropped at the end)
        auto place = [&]() {
          if constexpr (TREE) {
            const int depth = tree_depth(a, u.b, tok);
            live = depth >= 0;
            return live ? u.pos0 + depth : INT_MAX;
          } else {
            return u.pos0 + tok;
          }
        };
        const int p = in ? place() : INT_MAX;
        const int pf = in && p >= 0 && live ? u.pf : 0;
        const float slope = BIAS && in ? cache_slope(a.slopes[hq]) : 0.f;
        for (int i = 0; i < nt; ++i, ++ns) {
          const int j0 = u.tile(i) * kTile;
          // columns [c_lo, c_end) and those below c_pf are visible
          const bool nodes = TREE && j0 >= u.kv;
          const int c_end = p == INT_MAX ? kTile : p < 0 ? 0 : TREE ? u.kv - j0 : p - j0 + 1;
          const int c_lo = p == INT_MAX || p < a.window ? 0 : p - a.window + 1 - j0;
          const int c_pf = pf - j0;
          auto visible = [&](int q) {       // of the 32 columns from 64 q + 32 ch on
            const int c0 = 64 * q + 32 * ch;
            return (below(c_end - c0) & ~below(c_lo - c0)) | below(c_pf - c0);
          };
          const bool all = (c_lo <= 0 && c_end >= kTile) || c_pf >= kTile;
          const bool masked = !__all_sync(kFull, TREE ? all && !nodes : all);
          // What a tree's node sees of the nodes is a word.  Capped scores are masked twice
          // and take the words of a tile's masks as they are (16 x 26 nodes over 12001: 102 us,
          // and 105 with words made for each masking); the others make them where they
          // are needed (8 x 64 nodes over 32768: 370 us, and 381 with words made before).
          uint32_t sees = 0, words[2] = {0u, 0u};
          if (TREE && nodes && in && live) sees = (uint32_t)(tree_sees(a, u.b, tok) >> (32 * ch));
          auto word = [&](int q) {
            return TREE && nodes ? (q == 0 ? sees : 0u) : visible(q);
          };
          if (TREE && CAP && masked) {
            words[0] = word(0);
            words[1] = word(1);
          }
          // scores that are not seen become `v`: 32 columns as the bits of a word
          auto hide = [&](float (&s)[kCols], float v) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t vis = TREE && CAP ? words[q] : word(q);
#pragma unroll
              for (int c = 0; c < 32; ++c) s[32 * q + c] = vis & (1u << c) ? s[32 * q + c] : v;
            }
          };
          wait(&bar[kBS + t], ns & 1u, gone);
          fence_after();
          if (i == nt - 1) {                // this half's last S has read the queries
            const Unit nx = peek(k + 1);
            loaded = nx.nt > 0 && nx.active(t);
            if (loaded) load_q(a, nx, qdst, t, r, ch, lane);
          }
          float s[kCols];
          ld32(ts + 32 * ch, s);
          ld32(ts + 64 + 32 * ch, s + 32);
          wait_ld();
          // Capped scores.  Three function-unit operations a score would outweigh the
          // products; where the warp's scores are all within half a cap, as most are,
          // a polynomial takes the place of two, and its last product is fused with the
          // maximum's subtraction below.  The cap keeps the order of the scores, so
          // their maximum can be taken before it.
          bool small = false;
          float size = 0.f;                 // of the thread's largest score
          if constexpr (CAP) {
            if (masked) hide(s, 0.f);       // what is not seen may be anything
            float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kCols; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) am[e] = max3(am[e], fabsf(s[c + e]), fabsf(s[c + 4 + e]));
            size = max3(am[0], am[1], fmaxf(am[2], am[3]));
            small = __all_sync(kFull, size <= a.cap_small);
            if (!small) {
#pragma unroll
              for (int c = 0; c < kCols; ++c) s[c] = cache_cap_far(a, s[c]);
            } else if (BIAS || masked) {
#pragma unroll
              for (int c = 0; c < kCols; c += 2) {
                const f2 x = make_float2(s[c], s[c + 1]), v = mul2(x, cache_cap_factor(a, x));
                s[c] = v.x;
                s[c + 1] = v.y;
              }
            }
          } else if constexpr (BIAS) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) s[c] = __fmul_rn(s[c], a.qk);
          }
          if constexpr (BIAS) {
            if (TREE && nodes) {
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const int n = 32 * ch + c;
                const int away = p - u.pos0 - (n < a.T ? tree_depth(a, u.b, n) : 0);
                s[c] = fmaf(-slope, fabsf((float)away), s[c]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < kCols; ++c)
                s[c] = fmaf(-slope, fabsf((float)(p - (j0 + 32 * ch + c + (c & 32)))), s[c]);
            }
          }
          if (masked) hide(s, -INFINITY);
          auto row_max = [&]() {
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mx[e] = max3(max3(s[e], s[8 + e], s[16 + e]), max3(s[24 + e], s[32 + e], s[40 + e]),
                           fmaxf(s[48 + e], s[56 + e]));
            return max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
          };
          // (capped: the largest size of a score bounds the maximum, and mostly that is
          // enough to know that it does not rise)
          const bool fused = CAP && !BIAS && small && !masked;
          float mt;
          if (fused)
            mt = __fmul_rn(size, cache_cap_factor(a, make_float2(size, size)).x);
          else
            mt = CAP || BIAS ? row_max() : __fmul_rn(row_max(), a.qk);
          // (the vote also says that both warps of the rows have read their scores,
          // which the weights overwrite; a NaN does not raise)
          if (vote_pair(i == 0 || mt > m + 8.f)) {
            if (fused) {
              mt = row_max();
              mt = __fmul_rn(mt, cache_cap_factor(a, make_float2(mt, mt)).x);
            }
            *mine = mt;
            sync_pair();
            mt = fmaxf(mt, *other);
            const float mn = fmaxf(m, mt);
            const float f = mn == -INFINITY ? 1.f : cache_ex2(m - mn);
            m = mn;
            l *= f;
            if (i > 0) {
              wait(&bar[kBO + t], (ns - 1) & 1u, gone);
              fence_after();
#pragma unroll 1
              for (int c = 0; c < kCols; c += 8) {   // (few registers beside the scores)
                float o[8];
                ld8(to + c, o);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= f;
                st8(to + c, o);
              }
            }
          }
          const float mz = m == -INFINITY ? 0.f : m;
          f2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto weights = [&](auto score) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pw[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const f2 x = score(make_float2(s[32 * q + 2 * c], s[32 * q + 2 * c + 1]));
                const f2 e = make_float2(cache_ex2(x.x), cache_ex2(x.y));
                sum[c & 1] = add2(sum[c & 1], e);
                pw[c] = f2_to_bf2(e.x, e.y);
              }
              st16(ts + 32 * q + 16 * ch, pw);
              wait_st();
              fence_before();
              arrive(&bar[kBP + 2 * t + q]);
            }
          };
          const f2 less = make_float2(-mz, -mz);
          if constexpr (!CAP && !BIAS) {
            weights([&](f2 x) { return fma2(x, make_float2(a.qk, a.qk), less); });
          } else if (fused) {
            weights([&](f2 x) { return fma2(x, cache_cap_factor(a, x), less); });
          } else {
            weights([&](f2 x) { return add2(x, less); });
          }
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
        }
        if (loaded) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async();
          arrive(&bar[kBQ + t]);
        }
        sync_pair();                        // the last maxima have been read
        *mine = l;
        sync_pair();
        l += *other;
        sync_pair();                        // both have, before the next maxima
        wait(&bar[kBO + t], (ns - 1) & 1u, gone);
        fence_after();
      }
      if (TREE && !live) l = 0.f;
      if (u.active(t)) {
        const int64_t at = in ? checked_index((int64_t)(u.tok0 + tok) * a.Hq + hq, a.n_tokens * a.Hq,
                                              &g_cache_prefill_flags) : 0;
        const float inv = cache_inv(l);     // (0 in a unit without tiles)
        const bool aligned = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        uint16_t* dst = a.out + at * kCacheD + kCols * ch;
        if (in && a.lse && ch == 0 && u.slot < 0)
          a.lse[at] = cache_lse(m, l);
        if (SPLIT && u.slot >= 0) {         // (the same for the whole unit)
          if (!TREE || t * kHalf + 32 * (w & 3) < u.rows) {    // (no rows: not read by the join)
            float* ps = part_of(a, u.slot) + t * kHalf + r;
            if (ch == 0) {
              ps[0] = m;
              ps[kUnit] = l;
            }
            ps += (2 + kCols * ch) * kUnit;
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
              float o[32];
              ld32(to + c, o);
              wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ps[(c + e) * kUnit] = o[e];
            }
          }
        } else if (nt > 0) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            float o[32];
            ld32(to + c, o);
            wait_ld();
            if (in)
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                uint32_t v[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                  v[d] = TREE && !live ? 0u
                                       : f2_to_bf2(o[e + 2 * d] * inv, o[e + 2 * d + 1] * inv);
                st_sector(dst + c + e, v, aligned);
              }
          }
        } else if (in) {
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            const uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            st_sector(dst + c, v, aligned);
          }
        }
        fence_before();
      }
    }
  }
  if (SPLIT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ---- every product has been waited for: tensor memory goes
  fence_before();
  __syncthreads();
  fence_after();
  if (w == kSoftWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tm));
}

// The join: block (c, y, z) merges rows 32 y .. and channels 32 z .. of the unit
// that is open where share c begins, if it began in share c - 1.  Lane = row,
// a warp takes four channels; the output goes through shared memory to be written
// by rows.
constexpr int kSeamWarps = 8;
constexpr int kSeamRows = 32, kSeamCols = 32;
__global__ void __launch_bounds__(32 * kSeamWarps)
cache_seam_kernel(const __grid_constant__ CacheParams a) {
  using namespace cp;
  constexpr int kCh = kSeamCols / kSeamWarps, kBatch = 6;
  __shared__ uint32_t tile[kSeamRows][kSeamCols / 2 + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Seam s = reinterpret_cast<const Seam*>(a.part)[c];
  const int r0 = blockIdx.y * kSeamRows, r = r0 + lane, c0 = blockIdx.z * kSeamCols;
  if (s.k1 < 0 || s.k0 != c - 1 || r0 >= s.rows) return;
  float M = -INFINITY, L = 0.f, O[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) O[i] = 0.f;
  for (int k = s.k0; k <= s.k1; k += kBatch) {
    float m[kBatch], l[kBatch], o[kBatch][kCh];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      l[b] = 0.f;
      if (k + b <= s.k1) {
        const float* ps = part_of(a, (int)checked_index(2 * (k + b) + (k + b == s.k0 ? 1 : 0),
                                                        2 * kMaxCtas, &g_cache_prefill_flags)) + r;
        m[b] = ps[0];
        l[b] = ps[kUnit];
#pragma unroll
        for (int i = 0; i < kCh; ++i) o[b][i] = ps[(2 + c0 + kCh * w + i) * kUnit];
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (r >= s.rows || l[b] == 0.f) continue;   // (rows of no token hold anything)
      const float Mn = fmaxf(M, m[b]), fo = cache_ex2(M - Mn), fn = cache_ex2(m[b] - Mn);
#pragma unroll
      for (int i = 0; i < kCh; ++i) O[i] = O[i] * fo + o[b][i] * fn;
      L = L * fo + l[b] * fn;
      M = Mn;
    }
  }
  const float inv = cache_inv(L);
#pragma unroll
  for (int i = 0; i < kCh; i += 2)
    tile[lane][(kCh * w + i) / 2] = f2_to_bf2(O[i] * inv, O[i + 1] * inv);
  auto place = [&](int rr) {                            // output row of unit row rr
    const int row = s.row0 + rr, t = row / a.G;
    return checked_index((int64_t)(s.tok0 + t) * a.Hq + s.h * a.G + row - t * a.G,
                         a.n_tokens * a.Hq, &g_cache_prefill_flags);
  };
  if (c0 == 0 && w == 0 && r < s.rows && a.lse)
    a.lse[place(r)] = cache_lse(M, L);
  __syncthreads();
  const int rr = threadIdx.x >> 3, q = threadIdx.x & 7;  // 8 lanes a row of 64 bytes
  if (r0 + rr < s.rows)
    *reinterpret_cast<uint2*>(a.out + place(r0 + rr) * kCacheD + c0 + 4 * q) =
        make_uint2(tile[rr][2 * q], tile[rr][2 * q + 1]);
}

// ------------------------------------------------------------ wait self-test

// How a CTA of these kernels ends when a wait runs out.  Warp 1 waits, with limit_ns,
// for what nothing completes; it must give up, raise the abort word and record it.  Then
// warp 0 starts copies (five on a ring of three) and products, and drains both although
// the abort word is up: the copies' bytes and the products must be there.
// *status = 5 if all held, else 6.  The flag word is the CTA's own.
__device__ uint4 g_selftest_src[256];          // zeros
constexpr uint32_t kTestRing = 2 * cp::kBuf, kTestCopy = sizeof g_selftest_src;
constexpr uint32_t kTestSmem = kTestRing + 3 * kTestCopy;
__global__ void __launch_bounds__(64, 1)
cache_wait_selftest_kernel(uint64_t limit_ns, unsigned int* status) {
  using namespace cp;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[5];    // three of copies, products, never
  __shared__ uint32_t tmem, gone[2], good;
  __shared__ unsigned int flags;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  // operands of ones (BF16 0x3f80), a ring of ones bits
  for (uint32_t i = tid; i < kTestSmem / 4; i += 64)
    reinterpret_cast<uint32_t*>(smem)[i] = i < kTestRing / 4 ? 0x3f803f80u : 0xffffffffu;
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(&bars[i], 1);
    gone[0] = gone[1] = good = flags = 0u;
    fence_barrier_init();
  }
  if (w == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(smem_u32(&tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_proxy_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = tmem;
  if (w == 1) {
    const bool ok = wait_for(&bars[4], 0, gone, limit_ns, &flags);
    if (lane == 0 && !ok && gone[0] && (flags & kFlagWaitTimeout)) atomicAdd(&good, 1u);
  }
  __syncthreads();
  if (w == 0) {
    const bool one = elect_one();
    if (lane == 0) {
      for (int i = 0; i < 5; ++i) {
        if (i >= 3) (void)mbar_wait(&bars[i % 3], 0);
        mbar_expect_tx(&bars[i % 3], kTestCopy);
        bulk_load(smem + kTestRing + (i % 3) * kTestCopy, g_selftest_src, kTestCopy, &bars[i % 3]);
      }
      flags = 0u;
      drain_copies(bars, 3, 5, &flags);
      uint32_t bits = flags;
      for (uint32_t i = 0; i < 3 * kTestCopy / 4; ++i)
        bits |= reinterpret_cast<const volatile uint32_t*>(smem + kTestRing)[i];
      if (bits == 0u) atomicAdd(&good, 1u);
    }
    __syncwarp();
    if (one) {
      const uint64_t a = sdesc(smem_u32(smem), 16, 1024), b = sdesc(smem_u32(smem + kBuf), 16, 1024);
      for (int c = 0; c < 64; ++c) mma_ss(tm, a, b, c > 0 ? 1u : 0u);   // 16 channels of ones
    }
    const bool done = drain_products(&bars[3], one, 0, &flags);
    fence_after();
    float s[32];
    ld32(tm, s);
    wait_ld();
    bool right = done;
    for (int i = 0; i < 32; ++i) right = right && s[i] == 64.f * 16.f;
    right = __all_sync(kFull, right);
    if (lane == 0 && right) atomicAdd(&good, 1u);
    fence_before();
  }
  __syncthreads();
  fence_after();
  if (w == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tm));
  if (tid == 0) *status = good == 3u ? 5u : 6u;
}

cudaError_t launch_cache_wait_selftest(uint64_t limit_ns, unsigned int* status,
                                       cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(
      cache_wait_selftest_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTestSmem);
  if (e != cudaSuccess) return e;
  cache_wait_selftest_kernel<<<1, 64, kTestSmem, stream>>>(limit_ns, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ host

// shares: how many the join looks through
template <bool CAP, bool BIAS, int MODE, bool TREE>
static cudaError_t run(const CacheParams& p, int grid, int shares, const Tensors<true>& m,
                       cudaStream_t stream) {
  const Tensors<TREE> maps = tensors_of<TREE>(m);
  auto fn = cache_prefill_kernel<CAP, BIAS, MODE, TREE>;
  static thread_local int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cp::kSmem);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  e = launch_dependent(fn, dim3((unsigned)grid), cp::kThreads, cp::kSmem, 0, stream, p, maps);
  if (e != cudaSuccess || MODE == cp::kWhole || shares < 2) return e;
  return launch_dependent(cache_seam_kernel,
                          dim3((unsigned)(shares - 1), cp::kUnit / kSeamRows, kCacheD / kSeamCols),
                          32 * kSeamWarps, 0, 0, stream, p);
}

template <int MODE, bool TREE>
static cudaError_t run_score(const CacheParams& p, int grid, int shares, bool cap,
                             const Tensors<true>& m, cudaStream_t stream) {
  if (cap) return p.slopes ? run<true, true, MODE, TREE>(p, grid, shares, m, stream)
                           : run<true, false, MODE, TREE>(p, grid, shares, m, stream);
  return p.slopes ? run<false, true, MODE, TREE>(p, grid, shares, m, stream)
                  : run<false, false, MODE, TREE>(p, grid, shares, m, stream);
}
template <int MODE>
static cudaError_t run_mode(const CacheParams& p, int grid, int shares, bool cap,
                            const Tensors<true>& m, cudaStream_t stream) {
  return p.mask ? run_score<MODE, true>(p, grid, shares, cap, m, stream)
                : run_score<MODE, false>(p, grid, shares, cap, m, stream);
}

// Units of a call, at most.
static int64_t units_of(int batch, int64_t n_tokens, int G, int Hkv) {
  return (n_tokens * G / cp::kUnit + batch) * Hkv;
}
// Units are cut where contexts may be long (the table has room for more than
// 2048 tokens) and whole ones would leave half of the CTAs idle or more: 100
// tokens over 32K (16 units) take 330 us whole and 61 us cut, 16 over 128K 1216
// and 96.  300 tokens over 1200 take 21 us whole and 29 us cut, over 2000 29 us
// either way.  More units share keys better whole, row blocks of a head running
// over them side by side: 1000 tokens over 32K (128 units) take 338 us whole and
// 365 us cut, a causal prompt of 4096 (512 units) 93 and 128 us.
static bool cut(int64_t units, int64_t max_tokens, int sms) {
  return max_tokens > 16 * cp::kTile && 2 * units <= sms;
}

// The last round's units are cut where all may be equally long (the table has
// room for four times the mean chunk or more), so that the round would be as long as
// the others with CTAs idle, and where there are few rounds: 2 x 1023 tokens over
// 16K, 512 units, 3.4 rounds, take 0.91 ms whole and 0.84 ms with the last 56
// in two parts each.
static bool long_contexts(int batch, int64_t n_tokens, int64_t units, int64_t max_tokens, int sms) {
  return max_tokens > 16 * cp::kTile && max_tokens >= 4 * n_tokens / batch && units < 8 * sms;
}

// With one row block to a sequence (a few new tokens each) no keys are shared, so
// nothing is lost by cutting more units, and equal shares follow the lengths: 8 x 8
// tokens over 32767, 8 KV heads (64 units), take 295 us whole and 177 us cut.
static bool cut_few(int batch, int64_t n_tokens, int G, int64_t units, int64_t max_tokens,
                    int sms) {
  return n_tokens * G <= (int64_t)cp::kUnit * batch && max_tokens > 16 * cp::kTile &&
         units < 8 * sms;
}

// Units of a tree's call: as many rows to every sequence.
static int64_t tree_units(int batch, int64_t n_tokens, int G, int Hkv) {
  const int64_t rows = n_tokens / batch * G;
  return (rows + cp::kUnit - 1) / cp::kUnit * batch * Hkv;
}
// The rows of a tree's sequence are few blocks over the same keys, so that little is lost
// by cutting them: shares where whole units would leave more than three SMs in ten idle (64
// units over 16384 tokens 179 us whole and 107 cut, 96 units 181 and 156, 112 units 183
// and 187; over 4096 tokens, where each share's parts weigh more, 64 units 56 and 48, 96
// units 58 and 62).  More units than SMs: the last round's in parts.
static int tree_form(int64_t units, int64_t max_tokens, int sms) {
  if (max_tokens <= 16 * cp::kTile) return LYNX_CACHE_WHOLE;
  if (2 * units <= sms || (10 * units < 7 * sms && max_tokens > 32 * cp::kTile))
    return LYNX_CACHE_SHARES;
  const int64_t last = units % sms;
  return units > sms && units < 8 * sms && last > 0 && 2 * last <= sms ? LYNX_CACHE_PARTS
                                                                       : LYNX_CACHE_WHOLE;
}
// A tree's units that have an SM each: CTAs without a unit, or with a short one, take parts of
// the long ones, by the sequences' lengths.  Equal and ragged ones, whole and like this: 112
// units over 8192 tokens 105 and 113, 103 and 80 us; 128 units over 12000 150 and 160, 142
// and 105; 136 units over 8192 115 and 121, 103 and 97.  Several row blocks over the same
// keys gain by equal lengths as well, up to where most SMs are busy: 112 units over 16384
// tokens 181 and 168, 128 units 185 and 197.
static bool lend(const CacheParams& p, int64_t units, int sms) {
  const int64_t room = p.max_pages << p.lgP, most = room < p.window ? room : p.window;
  const bool blocks = (int64_t)p.T * p.G > cp::kUnit;
  return p.batch <= 32 && 10 * units >= 7 * sms && 20 * units <= (blocks ? 16 : 17) * sms &&
         units < cp::kMaxCtas && most >= 64 * cp::kTile;
}

size_t cache_prefill_workspace_bytes(int batch, int64_t n_tokens, int G, int Hkv,
                                     int64_t max_tokens, bool tree) {
  // (a tree's calls: whatever the number of SMs)
  if (tree && max_tokens > 16 * cp::kTile &&
      tree_units(batch, n_tokens, G, Hkv) < 8 * cp::kMaxCtas)
    return cp::kMaxCtas * (sizeof(cp::Seam) + 2 * cp::kPartFloats * sizeof(float));
  if (tree) return 0;
  const int64_t units = units_of(batch, n_tokens, G, Hkv);
  if (!cut(units, max_tokens, cp::kMaxCtas) && !cut_few(batch, n_tokens, G, units, max_tokens, cp::kMaxCtas) &&
      !long_contexts(batch, n_tokens, units, max_tokens, cp::kMaxCtas))
    return 0;
  return cp::kMaxCtas * (sizeof(cp::Seam) + 2 * cp::kPartFloats * sizeof(float));
}

int cache_prefill_form(int batch, int64_t n_tokens, int G, int Hkv, int64_t max_tokens, int sms,
                       bool tree) {
  if (sms > cp::kMaxCtas) sms = cp::kMaxCtas;
  if (tree) return tree_form(tree_units(batch, n_tokens, G, Hkv), max_tokens, sms);
  const int64_t units = units_of(batch, n_tokens, G, Hkv);
  if (cut(units, max_tokens, sms) || cut_few(batch, n_tokens, G, units, max_tokens, sms))
    return LYNX_CACHE_SHARES;
  const int last = (int)(units % sms);
  return long_contexts(batch, n_tokens, units, max_tokens, sms) && last > 0 && 2 * last <= sms
             ? LYNX_CACHE_PARTS : LYNX_CACHE_WHOLE;
}

cudaError_t launch_cache_prefill(const CacheParams& x, bool cap, const Tensors<true>& m,
                                 cudaStream_t stream) {
  CacheParams p = x;
  const int sms = sm_count() < cp::kMaxCtas ? sm_count() : cp::kMaxCtas;
  const bool tree = p.mask != nullptr;
  const int64_t units = tree ? tree_units(p.batch, p.n_tokens, p.G, p.Hkv)
                             : units_of(p.batch, p.n_tokens, p.G, p.Hkv);
  const int form =
      cache_prefill_form(p.batch, p.n_tokens, p.G, p.Hkv, p.max_pages << p.lgP, sms, tree);
  if (tree && lend(p, units, sms)) {
    p.tail0 = (int)units;
    return run_mode<cp::kShares>(p, sms, (int)units + 1, cap, m, stream);
  }
  p.tail0 = 0;
  if (form == LYNX_CACHE_SHARES)
    return run_mode<cp::kShares>(p, sms, sms, cap, m, stream);
  if (form == LYNX_CACHE_PARTS) {
    const int last = (int)(units % sms);
    p.tail_parts = sms / last < 8 ? sms / last : 8;
    p.tail0 = (int)(units - last);
    return run_mode<cp::kTail>(p, p.tail0 + last * p.tail_parts, last * p.tail_parts, cap, m,
                               stream);
  }
  return run_mode<cp::kWhole>(p, (int)units, 0, cap, m, stream);   // (below 2^31, as n_tokens * H_q)
}

}  // namespace lynx
