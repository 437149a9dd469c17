// cache_append.cu -- new tokens into the BF16 paged cache: keys (and queries)
// rotated by their positions, keys and values written to their pages.
//
// Rotation.  Pair i of a head, (x1, x2), turns by a_i = pos * f_i:
//   x1' = x1 cos a_i - x2 sin a_i,  x2' = x2 cos a_i + x1 sin a_i,
// pos the position on axis[i].  Only the angle's fraction of a turn matters,
// and a float32 product pos * f_i would lose it for far positions (2^17 * 1.0
// has a last place of 2^-7).  So the frequency is held as a 64-bit fraction
// of a turn, F_i = f_i / 2 pi * 2^64 rounded to the nearest: pos * F_i mod 2^64, with two
// integer multiplications, is the fraction of a turn to within 2^-34 at any 32-bit
// position.  Its top 32 bits become the angle in [-pi, pi], where sin.approx and
// cos.approx are within 2^-21 of the value: 2^-12 of a BF16 half step of a
// unit vector's length, so the library's slower sincosf would change nothing
// that survives the one rounding to BF16.
//
// What bounds it: memory, each value read and written once (15525 tokens of 64 + 8
// heads: 92.6 us, 6.87 TB/s; the copy rate, and the last writes of a pass are still in L2
// when it ends).  A warp takes one token and 4 * U of its heads (queries, keys and
// values in one list): 8 lanes a head, 16 channels a lane as two 16-byte vectors that
// hold 8 whole pairs in either pairing, so a lane computes its 8 angles once and keeps
// them for its U heads; all loads of the U heads are in flight at once.
#include <math.h>

#include "cache.h"
#include "common.cuh"

namespace lynx {

// Set when a block-table entry was outside [0, num_blocks) or a token lay
// beyond the table; read through read_cache_append_flags(), never reset.
__device__ unsigned int g_cache_append_flags = 0;

cudaError_t read_cache_append_flags(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_cache_append_flags, sizeof(unsigned int));
}

struct AppendParams {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_pool, *v_pool;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *table, *kv_len, *offsets, *positions;
  int64_t max_pages, nblocks, n_tokens;
  int batch, Hq, Hkv, lgP, nseg, rot_dim, interleaved;
};

// Heads a warp takes: four at once, U times.  5042 tokens of 56 heads: 27.7 us with
// U = 3, 28.1 with 4, 30.5 with 6, 33.0 with 8; 15525 tokens of 80 heads 92.3, 92.6,
// 101.5, 96.2.
constexpr int kAppendWarps = 8, U = 4;

// Sequence of packed token t: the last b with offsets[b] <= t, found by a
// warp 32 boundaries at a time.  Returns -1 for a token before the first or
// behind the last sequence.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int batch, int64_t t,
                                           int lane) {
  int lo = 0, n = batch + 1;             // offsets[lo .. lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && offsets[lo + i] <= t;
    const int c = __popc(__ballot_sync(kFull, le));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
  }
  const bool le = lane < n && offsets[lo + lane] <= t;
  const int c = __popc(__ballot_sync(kFull, le));
  if (c == 0) return -1;
  const int b = lo + c - 1;
  return b < batch ? b : -1;
}

__global__ void __launch_bounds__(32 * kAppendWarps)
cache_append_kernel(const __grid_constant__ AppendParams a, const __grid_constant__ RopeArgs rope) {
  // (a lane reads its own eight: from the parameters that would be eight addresses a
  // load, one after the other; 5042 tokens on three axes 29.7 us, 27.9 us like this)
  __shared__ uint64_t turns[kRopeMaxFreq];
  __shared__ uint32_t axis[kRopeMaxFreq];
  if (threadIdx.x < kRopeMaxFreq) {
    turns[threadIdx.x] = rope.turns[threadIdx.x];
    axis[threadIdx.x] = rope.axis[threadIdx.x];
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, item = lane & 7, sub = lane >> 3;
  const int64_t job = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int64_t t = job / a.nseg;
  if (t >= a.n_tokens) return;
  const int b = sequence_of(a.offsets, a.batch, t, lane);
  if (b < 0) return;                     // a padding row: left as it is
  const int head0 = (int)(job % a.nseg) * (4 * U) + sub;
  const int HT = a.Hq + 2 * a.Hkv;
  const bool turned = 16 * item < a.rot_dim;
  // the lane's two vectors of 8 channels
  const int half = a.rot_dim >> 1;
  const int c0 = turned && !a.interleaved ? 8 * item : 16 * item;
  const int c1 = turned && !a.interleaved ? half + 8 * item : 16 * item + 8;

  uint4 x[U], y[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + 4 * u;
    if (h < HT) {
      const uint16_t* p = h < a.Hq ? a.q + t * a.q_stride + h * kCacheD
                          : h < a.Hq + a.Hkv ? a.k + t * a.k_stride + (h - a.Hq) * kCacheD
                                             : a.v + t * a.v_stride + (h - a.Hq - a.Hkv) * kCacheD;
      x[u] = *reinterpret_cast<const uint4*>(p + c0);
      y[u] = *reinterpret_cast<const uint4*>(p + c1);
    }
  }
  // where the token goes
  const int64_t first = a.offsets[b], after = a.offsets[b + 1];
  const int64_t pos = (int64_t)a.kv_len[b] - (after - first) + (t - first);
  int64_t slot = -1;                     // token row of the pools
  if (pos >= 0) {
    const int64_t pg = pos >> a.lgP;
    int64_t blk = -1;
    if (pg < a.max_pages) blk = a.table[(int64_t)b * a.max_pages + pg];
    if (blk >= 0 && blk < a.nblocks)
      slot = (blk << a.lgP) + (pos & ((1 << a.lgP) - 1));
    else if (lane == 0)
      atomicOr(&g_cache_append_flags, kFlagBadBlock);
  }
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = 8 * item + i;
      const int64_t p = a.positions ? (int64_t)a.positions[axis[f] * a.n_tokens + t] : pos;
      const uint64_t ph = (uint64_t)p * turns[f];
      const float ang = (float)(int32_t)(uint32_t)(ph >> 32) * 1.4629180792671596e-09f;  // 2 pi / 2^32
      cs[i] = __cosf(ang);
      sn[i] = __sinf(ang);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + 4 * u;
    if (h >= HT) continue;
    uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, yw[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
    if (turned && h < a.Hq + a.Hkv) {
      if (a.interleaved) {               // (2i, 2i + 1): pairs 0..3 in x, 4..7 in y
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 p = bf2_to_f2(xw[i]), r = bf2_to_f2(yw[i]);
          xw[i] = f2_to_bf2(fmaf(p.x, cs[i], -__fmul_rn(p.y, sn[i])),
                            fmaf(p.y, cs[i], __fmul_rn(p.x, sn[i])));
          yw[i] = f2_to_bf2(fmaf(r.x, cs[4 + i], -__fmul_rn(r.y, sn[4 + i])),
                            fmaf(r.y, cs[4 + i], __fmul_rn(r.x, sn[4 + i])));
        }
      } else {                           // (i, i + half): x holds the firsts, y the seconds
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 p = bf2_to_f2(xw[i]), r = bf2_to_f2(yw[i]);
          const int j = 2 * i;
          xw[i] = f2_to_bf2(fmaf(p.x, cs[j], -__fmul_rn(r.x, sn[j])),
                            fmaf(p.y, cs[j + 1], -__fmul_rn(r.y, sn[j + 1])));
          yw[i] = f2_to_bf2(fmaf(r.x, cs[j], __fmul_rn(p.x, sn[j])),
                            fmaf(r.y, cs[j + 1], __fmul_rn(p.y, sn[j + 1])));
        }
      }
    }
    uint16_t* o;
    if (h < a.Hq) {
      o = a.q_out + (t * a.Hq + h) * kCacheD;
    } else {
      if (slot < 0) continue;
      const bool key = h < a.Hq + a.Hkv;
      const int64_t at = checked_index(slot * a.Hkv + h - a.Hq - (key ? 0 : a.Hkv),
                                       (a.nblocks << a.lgP) * a.Hkv, &g_cache_append_flags);
      o = (key ? a.k_pool : a.v_pool) + at * kCacheD;
    }
    *reinterpret_cast<uint4*>(o + c0) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
    *reinterpret_cast<uint4*>(o + c1) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
  }
}

cudaError_t launch_cache_append(const CacheAppendArgs& x, const RopeArgs& rope,
                                cudaStream_t stream) {
  AppendParams p;
  p.q = static_cast<const uint16_t*>(x.q);
  p.k = static_cast<const uint16_t*>(x.k);
  p.v = static_cast<const uint16_t*>(x.v);
  p.q_out = static_cast<uint16_t*>(x.q_out);
  p.k_pool = static_cast<uint16_t*>(x.k_pool);
  p.v_pool = static_cast<uint16_t*>(x.v_pool);
  p.q_stride = x.q_stride;
  p.k_stride = x.k_stride;
  p.v_stride = x.v_stride;
  p.table = x.c.table;
  p.kv_len = x.c.kv_len;
  p.offsets = x.c.offsets;
  p.positions = rope.positions;
  p.max_pages = x.c.max_pages;
  p.nblocks = x.c.nblocks;
  p.n_tokens = x.c.n_tokens;
  p.batch = x.c.batch;
  p.Hq = x.Hq;
  p.Hkv = x.c.Hkv;
  p.lgP = __builtin_ctz((unsigned)x.c.page);
  p.rot_dim = rope.rot_dim;
  p.interleaved = rope.interleaved;
  const int HT = p.Hq + 2 * p.Hkv;
  p.nseg = (HT + 4 * U - 1) / (4 * U);
  const int64_t blocks = (p.n_tokens * p.nseg + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_dependent(cache_append_kernel, dim3((unsigned)blocks), 32 * kAppendWarps, 0, 0,
                          stream, p, rope);
}

}  // namespace lynx
