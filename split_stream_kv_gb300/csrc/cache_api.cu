// cache_api.cu -- the extern "C" boundary of the BF16 paged cache declared in
// include/lynx.h: argument checks and dispatch.
#include <math.h>
#include <string.h>

#include "checks.h"
#include "common.cuh"

namespace lynx {
namespace {

// 1 / (2 pi), the bits behind the binary point, first ones first: as many as the largest
// double's fraction of a turn needs.
constexpr int kInvWords = 19;
constexpr uint64_t kInv2Pi[kInvWords] = {
    0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull,
    0x7f9458eaf7aef158ull, 0x6dc91b8e909374b8ull, 0x01924bba82746487ull,
    0x3f877ac72c4a69cfull, 0xba208d7d4baed121ull, 0x3a671c09ad17df90ull,
    0x4e64758e60d4ce7dull, 0x272117e2ef7e4a0eull, 0xc7fe25fff7816603ull,
    0xfbcbc462d6829b47ull, 0xdb4d9fb3c9f2c26dull, 0xd3d18fd9a797fa8bull,
    0x5d49eeb1faf97c5eull, 0xcf41ce7de294a4baull, 0x9afed7ec47e35742ull,
    0x1580cc11bf1edaeaull,
};
// The 64 bits from bit `at` on (bits before the first and behind the last are zero).
inline uint64_t inv_2pi_bits(int at) {
  const int i = at >> 6, d = at & 63;          // word i starts d bits before `at`
  const uint64_t x = i >= 0 && i < kInvWords ? kInv2Pi[i] : 0;
  const uint64_t y = i >= -1 && i < kInvWords - 1 ? kInv2Pi[i + 1] : 0;
  return d ? x << d | y >> (64 - d) : x;
}

// inv_freq / 2 pi as a fraction of a turn, 2^64 to a turn, rounded to the nearest; its
// whole turns, which no integer position sees, are left out.  (As Payne and Hanek reduce
// an argument: inv_freq = m 2^e with an integer m, and the bits of 1 / (2 pi) from e on are
// all that m has to be multiplied by.  A double quotient would be off by up to 2^-54 of the
// turns, at position 2^31 and a frequency of 1e6 that is a few per cent of one.)
uint64_t turns_of(double inv_freq) {
  uint64_t bits;
  memcpy(&bits, &inv_freq, sizeof bits);
  const int biased = (int)(bits >> 52) & 0x7ff;
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (biased ? 1ull << 52 : 0);
  const int e = (biased ? biased : 1) - 1075;
  // m times the 192 bits from e on, modulo a turn
  unsigned __int128 lo = (unsigned __int128)m * inv_2pi_bits(e + 128);
  lo = (lo >> 64) + (unsigned __int128)m * inv_2pi_bits(e + 64);
  const uint64_t below = (uint64_t)lo;
  const uint64_t f = (uint64_t)(lo >> 64) + m * inv_2pi_bits(e) + (below >> 63);
  return inv_freq < 0 ? 0 - f : f;
}

}  // namespace
}  // namespace lynx

using namespace lynx;

extern "C" {

int lynx_cache_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      const void* q, int64_t q_stride, void* q_out, const int32_t* q_offsets,
                      const int32_t* kv_len, const int32_t* block_table, int64_t max_pages,
                      int64_t num_blocks, int batch, int64_t n_tokens, int H_q, int H_kv, int D,
                      int page, const lynx_rope* rope, void* k_pool, void* v_pool, void* stream) {
  if (!q) H_q = 0;
  int rc = check_layout(batch, n_tokens, H_q, H_kv, D, page, max_pages, num_blocks);
  if (rc) return rc;
  if (q && H_q < 1) return fail(LYNX_ESHAPE, "H_q = %d with queries", H_q);
  if ((rc = check_stride(k_stride, H_kv, "k_stride"))) return rc;
  if ((rc = check_stride(v_stride, H_kv, "v_stride"))) return rc;
  if (q && (rc = check_stride(q_stride, H_q, "q_stride"))) return rc;
  RopeArgs ra;
  memset(ra.turns, 0, sizeof ra.turns);
  memset(ra.axis, 0, sizeof ra.axis);
  if (rope) {
    if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 16)
      return fail(LYNX_EUNSUPPORTED, "rot_dim = %d: a multiple of 16 up to D", (int)rope->rot_dim);
    if (rope->interleaved != 0 && rope->interleaved != 1)
      return fail(LYNX_EINVAL, "interleaved must be 0 or 1");
    if (rope->n_axes < 1 || rope->n_axes > kMaxAxes)
      return fail(LYNX_EUNSUPPORTED, "n_axes = %d: 1 to %d", (int)rope->n_axes, kMaxAxes);
    if (rope->rot_dim > 0) {
      if (!rope->inv_freq) return fail(LYNX_EINVAL, "inv_freq: null pointer");
      if (rope->n_axes > 1 && (!rope->positions || !rope->axis))
        return fail(LYNX_EINVAL, "several axes need positions and axis");
      for (int i = 0; i < rope->rot_dim / 2; ++i) {
        if (!isfinite(rope->inv_freq[i])) return fail(LYNX_EINVAL, "inv_freq[%d] is not finite", i);
        ra.turns[i] = turns_of(rope->inv_freq[i]);
        ra.axis[i] = rope->axis ? rope->axis[i] : 0;
        if (ra.axis[i] >= rope->n_axes)
          return fail(LYNX_EINVAL, "axis[%d] = %d with %d axes", i, ra.axis[i], (int)rope->n_axes);
      }
      ra.rot_dim = rope->rot_dim;
      ra.interleaved = rope->interleaved != 0;
      ra.n_axes = rope->n_axes;
      ra.positions = rope->positions;
    }
  }
  if (batch == 0 || n_tokens == 0) return LYNX_OK;
  if ((rc = check_ptr(k, 16, "k")) || (rc = check_ptr(v, 16, "v")) ||
      (rc = check_ptr(k_pool, 16, "k_pool")) || (rc = check_ptr(v_pool, 16, "v_pool")) ||
      (rc = check_ptr(q_offsets, 4, "q_offsets")) || (rc = check_ptr(kv_len, 4, "kv_len")) ||
      (rc = check_ptr(block_table, 4, "block_table")))
    return rc;
  if (q && ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(q_out, 16, "q_out")))) return rc;
  if (ra.positions && (rc = check_ptr(ra.positions, 4, "positions"))) return rc;
  const uint64_t pool = (uint64_t)num_blocks * page * H_kv * D * 2;
  const Span ins[] = {{k, rows_bytes(n_tokens, k_stride, H_kv), "k"},
                      {v, rows_bytes(n_tokens, v_stride, H_kv), "v"},
                      {q, rows_bytes(n_tokens, q_stride, H_q), "q"},
                      {q_offsets, 4 * ((uint64_t)batch + 1), "q_offsets"},
                      {kv_len, 4 * (uint64_t)batch, "kv_len"},
                      {block_table, 4 * (uint64_t)batch * (uint64_t)max_pages, "block_table"},
                      {ra.positions, 4 * (uint64_t)ra.n_axes * (uint64_t)n_tokens, "positions"}};
  const Span kp{k_pool, pool, "k_pool"}, vp{v_pool, pool, "v_pool"};
  const Span qo{q ? q_out : nullptr, rows_bytes(n_tokens, (int64_t)H_q * D, H_q), "q_out"};
  if ((rc = check_apart(kp, vp)) || (rc = check_apart(qo, kp)) || (rc = check_apart(qo, vp)))
    return rc;
  // dense queries may be rotated in place: only they, not what else starts at their address
  const Span* const in_place = q_out == q && q_stride == (int64_t)H_q * D ? &ins[2] : nullptr;
  for (const Span& s : ins) {
    if ((rc = check_apart(kp, s)) || (rc = check_apart(vp, s))) return rc;
    if (&s != in_place && (rc = check_apart(qo, s))) return rc;
  }
  CacheAppendArgs a;
  a.c = CacheLayout{block_table, kv_len, q_offsets, max_pages, num_blocks, n_tokens,
                    batch, 0, H_kv, page};
  a.k = k;
  a.v = v;
  a.q = q;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.q_out = q_out;
  a.Hq = H_q;
  cudaError_t e = launch_cache_append(a, ra, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LYNX_OK : cuda_fail(e, "lynx_cache_append");
}

static int check_heads(int batch, int H_q, int H_kv) {
  if (H_q < 1 || H_kv < 1 || H_q % H_kv)
    return fail(LYNX_ESHAPE, "H_q = %d is not a multiple of H_kv = %d", H_q, H_kv);
  // A CTA of the many-row kernel passes over sequences without tokens to find its next
  // unit: 2^22 of them take 72 ms, so 2^26 take 1.2 s, and its other warps wait for 2 s.
  if ((int64_t)batch * H_kv > (1 << 26))
    return fail(LYNX_EUNSUPPORTED, "batch * H_kv must be <= 2^26");
  return LYNX_OK;
}

static int check_T(int T) {
  if (T < 1) return fail(LYNX_ESHAPE, "T = %d must be >= 1", T);
  if (T > 64) return fail(LYNX_EUNSUPPORTED, "T = %d: at most 64 query tokens", T);
  return LYNX_OK;
}

static int rows_workspace(int batch, int T, int H_q, int H_kv, int D, int page, int64_t max_pages,
                          bool tree, size_t* bytes) {
  if (!bytes) return fail(LYNX_EINVAL, "null pointer");
  int rc = check_T(T);
  if (rc) return rc;
  if ((rc = check_layout(batch, (int64_t)batch * T, H_q, H_kv, D, page, max_pages, 1))) return rc;
  if ((rc = check_heads(batch, H_q, H_kv))) return rc;
  *bytes = batch ? cache_attn_workspace_bytes(batch, T, (int64_t)batch * T, H_q, H_kv,
                                              max_pages * page, tree) : 0;
  return LYNX_OK;
}

int lynx_cache_attn_decode_workspace_bytes(int batch, int T, int H_q, int H_kv, int D, int page,
                                           int64_t max_pages, size_t* bytes) {
  return rows_workspace(batch, T, H_q, H_kv, D, page, max_pages, false, bytes);
}

int lynx_cache_attn_prefill_workspace_bytes(int64_t n_tokens, int batch, int H_q, int H_kv, int D,
                                            int page, int64_t max_pages, size_t* bytes) {
  if (!bytes) return fail(LYNX_EINVAL, "null pointer");
  int rc = check_layout(batch, n_tokens, H_q, H_kv, D, page, max_pages, 1);
  if (rc) return rc;
  if ((rc = check_heads(batch, H_q, H_kv))) return rc;
  *bytes = batch && n_tokens
               ? cache_attn_workspace_bytes(batch, 0, n_tokens, H_q, H_kv, max_pages * page) : 0;
  return LYNX_OK;
}

int lynx_cache_attn_form(int64_t n_tokens, int batch, int T, int H_q, int H_kv, int D, int page,
                         int64_t max_pages, int sms, int* form) {
  if (!form) return fail(LYNX_EINVAL, "null pointer");
  if (sms < 1) return fail(LYNX_EINVAL, "sms = %d: at least 1", sms);
  int rc = T ? check_T(T) : LYNX_OK;
  if (rc) return rc;
  if (T && n_tokens != (int64_t)batch * T)
    return fail(LYNX_ESHAPE, "n_tokens must be batch * T where T is not 0");
  if ((rc = check_layout(batch, n_tokens, H_q, H_kv, D, page, max_pages, 1))) return rc;
  if ((rc = check_heads(batch, H_q, H_kv))) return rc;
  *form = batch && n_tokens
              ? cache_attn_form(batch, T, n_tokens, H_q, H_kv, max_pages * page, sms) : 0;
  return LYNX_OK;
}

static int attn(const void* q, int64_t q_stride, const int32_t* q_offsets, int64_t n_tokens,
                int batch, int T, int H_q, const void* k_pool, const void* v_pool,
                const int32_t* block_table, int64_t max_pages, int64_t num_blocks,
                const int32_t* kv_len, int H_kv, int D, int page, const lynx_score* score,
                void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream,
                const char* what, const uint64_t* mask = nullptr, const void* k_nodes = nullptr,
                const void* v_nodes = nullptr) {
  int rc = check_layout(batch, n_tokens, H_q, H_kv, D, page, max_pages, num_blocks);
  if (rc) return rc;
  if ((rc = check_heads(batch, H_q, H_kv))) return rc;
  if ((rc = check_stride(q_stride, H_q, "q_stride"))) return rc;
  lynx_score sc = {(float)(1.0 / sqrt((double)kCacheD)), 0.f, 0, nullptr, nullptr};
  if (score) sc = *score;
  if (!(sc.scale > 0.f) || !isfinite(sc.scale))
    return fail(LYNX_EINVAL, "scale must be finite and > 0");
  if (!(sc.softcap >= 0.f) || !isfinite(sc.softcap))
    return fail(LYNX_EINVAL, "softcap must be finite and >= 0");
  if (sc.window < 0) return fail(LYNX_EINVAL, "window must be >= 0");
  if (batch == 0 || n_tokens == 0) return LYNX_OK;
  if ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(k_pool, 16, "k_pool")) ||
      (rc = check_ptr(v_pool, 16, "v_pool")) || (rc = check_ptr(block_table, 4, "block_table")) ||
      (rc = check_ptr(kv_len, 4, "kv_len")) || (rc = check_ptr(out, 16, "out")))
    return rc;
  if (!T && (rc = check_ptr(q_offsets, 4, "q_offsets"))) return rc;
  if (lse && (rc = check_ptr(lse, 4, "lse"))) return rc;
  if (sc.slopes && (rc = check_ptr(sc.slopes, 4, "slopes"))) return rc;
  if (sc.prefix && (rc = check_ptr(sc.prefix, 4, "prefix"))) return rc;
  const size_t need = cache_attn_workspace_bytes(batch, T, n_tokens, H_q, H_kv, max_pages * page,
                                                 mask != nullptr);
  if (need && (rc = check_ptr(workspace, 16, "workspace"))) return rc;
  if (workspace_bytes < need)
    return fail(LYNX_EWORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  const uint64_t pool = (uint64_t)num_blocks * page * H_kv * D * 2;
  const Span ins[] = {{q, rows_bytes(n_tokens, q_stride, H_q), "q"},
                      {k_pool, pool, "k_pool"},
                      {v_pool, pool, "v_pool"},
                      {T ? nullptr : q_offsets, 4 * ((uint64_t)batch + 1), "q_offsets"},
                      {kv_len, 4 * (uint64_t)batch, "kv_len"},
                      {block_table, 4 * (uint64_t)batch * (uint64_t)max_pages, "block_table"},
                      {sc.slopes, 4 * (uint64_t)H_q, "slopes"},
                      {sc.prefix, 4 * (uint64_t)batch, "prefix"},
                      {mask, 8 * (uint64_t)n_tokens, "mask"},
                      {k_nodes, (uint64_t)batch * kTreeRoom * H_kv * D * 2, "k_nodes"},
                      {v_nodes, (uint64_t)batch * kTreeRoom * H_kv * D * 2, "v_nodes"}};
  const Span o{out, (uint64_t)n_tokens * H_q * D * 2, "out"};
  const Span ls{lse, (uint64_t)n_tokens * H_q * 4, "lse"};
  const Span ws{need ? workspace : nullptr, need, "workspace"};
  if ((rc = check_apart(o, ls)) || (rc = check_apart(o, ws)) || (rc = check_apart(ls, ws)))
    return rc;
  for (const Span& s : ins)
    if ((rc = check_apart(o, s)) || (rc = check_apart(ls, s)) || (rc = check_apart(ws, s)))
      return rc;
  CacheAttnArgs a;
  a.c = CacheLayout{block_table, kv_len, T ? nullptr : q_offsets, max_pages, num_blocks, n_tokens,
                    batch, T, H_kv, page};
  a.q = q;
  a.q_stride = q_stride;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.Hq = H_q;
  a.scale = sc.scale;
  a.softcap = sc.softcap;
  a.window = sc.window;
  a.slopes = sc.slopes;
  a.prefix = sc.prefix;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.mask = mask;
  a.k_nodes = k_nodes;
  a.v_nodes = v_nodes;
  cudaError_t e = launch_cache_attn(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LYNX_OK : cuda_fail(e, what);
}

int lynx_cache_attn_decode(const void* q, int64_t q_stride, int batch, int T, int H_q,
                           const void* k_pool, const void* v_pool, const int32_t* block_table,
                           int64_t max_pages, int64_t num_blocks, const int32_t* kv_len, int H_kv,
                           int D, int page, const lynx_score* score, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_T(T);
  if (rc) return rc;
  return attn(q, q_stride, nullptr, (int64_t)batch * T, batch, T, H_q, k_pool, v_pool,
              block_table, max_pages, num_blocks, kv_len, H_kv, D, page, score, out, lse,
              workspace, workspace_bytes, stream, "lynx_cache_attn_decode");
}

int lynx_cache_attn_tree_workspace_bytes(int batch, int T, int H_q, int H_kv, int D, int page,
                                         int64_t max_pages, size_t* bytes) {
  return rows_workspace(batch, T, H_q, H_kv, D, page, max_pages, true, bytes);
}

int lynx_cache_attn_tree(const void* q, int64_t q_stride, int batch, int T, int H_q,
                         const void* k_nodes, const void* v_nodes, const uint64_t* mask,
                         const void* k_pool, const void* v_pool, const int32_t* block_table,
                         int64_t max_pages, int64_t num_blocks, const int32_t* kv_len, int H_kv,
                         int D, int page, const lynx_score* score, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_T(T);
  if (rc) return rc;
  if (batch > INT32_MAX / kTreeRoom)
    return fail(LYNX_EUNSUPPORTED, "batch * %d must be < 2^31", kTreeRoom);
  if (batch > 0 && ((rc = check_ptr(mask, 8, "mask")) || (rc = check_ptr(k_nodes, 16, "k_nodes")) ||
                    (rc = check_ptr(v_nodes, 16, "v_nodes"))))
    return rc;
  return attn(q, q_stride, nullptr, (int64_t)batch * T, batch, T, H_q, k_pool, v_pool,
              block_table, max_pages, num_blocks, kv_len, H_kv, D, page, score, out, lse,
              workspace, workspace_bytes, stream, "lynx_cache_attn_tree", mask, k_nodes, v_nodes);
}

int lynx_cache_attn_prefill(const void* q, int64_t q_stride, const int32_t* q_offsets,
                            int64_t n_tokens, int batch, int H_q, const void* k_pool,
                            const void* v_pool, const int32_t* block_table, int64_t max_pages,
                            int64_t num_blocks, const int32_t* kv_len, int H_kv, int D, int page,
                            const lynx_score* score, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return attn(q, q_stride, q_offsets, n_tokens, batch, 0, H_q, k_pool, v_pool, block_table,
              max_pages, num_blocks, kv_len, H_kv, D, page, score, out, lse, workspace,
              workspace_bytes, stream, "lynx_cache_attn_prefill");
}

}  // extern "C"
