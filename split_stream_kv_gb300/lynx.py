"""ctypes binding of liblynx.so (include/lynx.h), one Python function per C
entry point with the same name.  Only argument marshalling happens here:
tensors become device pointers and sizes, the current CUDA stream is passed
along, and output tensors are allocated with torch when the caller gives none.
There is no CPU path: non-CUDA tensors are rejected.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# LYNX_LIBRARY=checked selects the checked build (liblynx_checked.so: kernels
# that verify their index arithmetic and report a failed check through
# lynx_device_errors); the default is the regular build.
LIB_PATH = os.path.join(_HERE, "liblynx_checked.so" if os.environ.get("LYNX_LIBRARY") == "checked"
                        else "liblynx.so")

LYNX_OK, LYNX_EINVAL, LYNX_ESHAPE, LYNX_EUNSUPPORTED, LYNX_ECUDA, LYNX_EWORKSPACE = (
    0, -1, -2, -3, -4, -5)
LYNX_ANCHOR, LYNX_FULL = 0, 1
LYNX_OUT_BF16, LYNX_OUT_FP32 = 0, 1
LYNX_BF16, LYNX_FP32, LYNX_FP16 = 0, 1, 2
(LYNX_CACHE_CLUSTERS, LYNX_CACHE_SPLIT, LYNX_CACHE_WHOLE, LYNX_CACHE_SHARES,
 LYNX_CACHE_PARTS) = range(1, 6)

_lib = None


class LynxError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str):
        super().__init__(f"{what}: {detail} ({code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load liblynx.so (build it first with split_stream_kv_gb300._build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "split_stream_kv_gb300._build.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I, F, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                        ctypes.c_size_t)
    PSZ = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "lynx_encoded_sizes": ([I64, I64, I, I, I, I, PSZ, PSZ, PSZ], I),
        "lynx_encode": ([P, I64, I64, I, I, I, I, F, P, P, P, P], I),
        "lynx_decode_anchor": ([P, P, I64, I64, I, I, I, I, F, P, I, P], I),
        "lynx_decode_full": ([P, P, P, I64, I64, I, I, I, I, F, P, I, P], I),
        "lynx_attn_workspace_bytes": ([I, I, I, I64, I, I, I, PSZ], I),
        "lynx_attn_decode": ([P, I, I, I, P, P, P, P, P, P, I64, I, I, I, I, F, I, P, P, SZ, P],
                             I),
        "lynx_attn_decode_tail": ([P, I, I, I, P, P, P, P, P, P, I64, I, I, I, I, F, I, P, P, P, P,
                                   SZ, P], I),
        "lynx_attn_decode_paged": ([P, I, I, I, P, P, P, P, P, P, P, I64, I64, I, I, I, I, F, I,
                                    P, P, P, P, SZ, P], I),
        "lynx_encode_paged": ([P, I64, I64, I, I, I, I, F, P, I64, P, P, P, P], I),
        "lynx_decode_paged": ([P, P, P, P, I64, I64, I64, I, I, I, I, F, I, P, I, P], I),
        "lynx_device_errors": ([ctypes.POINTER(ctypes.c_uint)], I),
        "lynx_spec_verify": ([P, P, P, P, P, I, I, I64, P, P, P], I),
        "lynx_attn_decode_noalloc": ([P, I, I, I, P, P, P, P, P, P, I64, I, I, I, I, F, I, P, P],
                                     I),
        "lynx_split_plan": ([I64, I64, I, I, I, I, I64, I, I, P, I64,
                             ctypes.POINTER(ctypes.c_int64)], I),
        "lynx_split_receive": ([P, P, P, P, P, P, I64, I64, I, I, I, I, F, I64, P, I, P, P, P,
                                P, P], I),
        "lynx_split_send": ([P, I64, I64, I, I, I, I, F, P, P, P, P, P, P, I64, P, P, P, P], I),
        "lynx_header_init": ([P, I64, I64, I, I, I, I, F, I], I),
        "lynx_header_check": ([P], I),
        "lynx_int_encode": ([P, I64, I, I, P, P, P], I),
        "lynx_int_decode": ([P, P, I64, I, I, P, I, P], I),
        "lynx_split_bits": ([P, P, I64, I, I, P, P, P], I),
        "lynx_join_bits": ([P, P, I64, I, I, P, P, P], I),
        "lynx_decode_anchor_bits": ([P, P, I64, I64, I, I, I, I, F, I, P, I, P], I),
        "lynx_a1_encode": ([P, I64, I64, I, I, I, F, P, P, P, P], I),
        "lynx_a1_decode": ([P, P, P, I64, I64, I, I, I, F, P, I, P], I),
        "lynx_cache_append": ([P, I64, P, I64, P, I64, P, P, P, P, I64, I64, I, I64, I, I, I, I,
                               P, P, P, P], I),
        "lynx_cache_attn_decode_workspace_bytes": ([I, I, I, I, I, I, I64, PSZ], I),
        "lynx_cache_attn_prefill_workspace_bytes": ([I64, I, I, I, I, I, I64, PSZ], I),
        "lynx_cache_attn_form": ([I64, I, I, I, I, I, I, I64, I, ctypes.POINTER(I)], I),
        "lynx_cache_attn_decode": ([P, I64, I, I, I, P, P, P, I64, I64, P, I, I, I, P, P, P, P,
                                    SZ, P], I),
        "lynx_cache_attn_prefill": ([P, I64, P, I64, I, I, P, P, P, I64, I64, P, I, I, I, P, P, P,
                                     P, SZ, P], I),
        "lynx_cache_attn_tree_workspace_bytes": ([I, I, I, I, I, I, I64, PSZ], I),
        "lynx_cache_attn_tree": ([P, I64, I, I, I, P, P, P, P, P, P, I64, I64, P, I, I, I, P, P, P,
                                  P, SZ, P], I),
        "lynx_token_logprobs": ([P, I, I64, I64, I64, F, P, I, I, P, P, P, P, P], I),
        "lynx_tree_plan": ([P, P, I, I, P, P, P], I),
        "lynx_tree_verify": ([P, P, P, I, I, P, P, P, P], I),
        "lynx_cache_fork": ([P, P, P, I64, I64, I, I, P, I, P, P, P], I),
        "lynx_cache_reserve": ([P, P, P, I64, I64, I, I, P, P, P, P, P], I),
        "lynx_cache_trim": ([P, P, P, I64, I64, I, I, P, P], I),
        "lynx_cache_compact": ([P, P, P, I64, I64, I, I, P, P, P, P], I),
        "lynx_cache_copy_pages": ([P, P, I, I64, P, P, I64, P, P], I),
        "lynx_cache_keep": ([P, P, I, P, P, P, P, I64, I64, I, I, I, I, I, P], I),
        "lynx_wait_selftest": ([ctypes.c_uint64, I, P, P], I),
        "lynx_compander_thresholds": ([F, P], I),
        "lynx_expand_table": ([F, P], I),
        "lynx_compander_selfcheck": ([F, P, P], I),
        "lynx_wait_timeouts": ([ctypes.POINTER(ctypes.c_uint)], I),
        "lynx_status_string": ([I], ctypes.c_char_p),
        "lynx_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != LYNX_OK:
        detail = lib().lynx_last_error().decode(errors="replace")
        raise LynxError(rc, what, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("lynx: tensors must be contiguous CUDA tensors")


def _expect(t, shape, dtype, device, what):
    """The C ABI sees pointers only: a caller's tensor of the wrong size or
    type would be read or written out of bounds on the device, so every
    tensor is checked against the sizes the call implies before it is
    passed."""
    if t is None:
        raise ValueError(f"{what} is required")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected {dtype} of shape {tuple(shape)}, got {t.dtype} "
                         f"of shape {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")


# ----------------------------------------------------------------- codec

def lynx_encoded_sizes(B: int, L: int, H_kv: int, D: int, page: int, C: int):
    a, r, m = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().lynx_encoded_sizes(B, L, H_kv, D, page, C, ctypes.byref(a), ctypes.byref(r),
                                    ctypes.byref(m)), "lynx_encoded_sizes")
    return a.value, r.value, m.value


def stream_shapes(B: int, L: int, H_kv: int, D: int, page: int, C: int):
    """Tensor shapes of (anchor, residual, meta) for a kv[B][L][H_kv][D]."""
    NB = L // page
    codes = (B, NB, H_kv, page, D // 2)
    return codes, codes, (B, NB, H_kv, 2 + 2 * (page // C), D)


def lynx_encode(kv: torch.Tensor, page: int, C: int, alpha: float, anchor=None, residual=None,
                meta=None):
    """Encode kv[B][L][H_kv][D] (bf16, CUDA).  Returns (anchor, residual, meta)."""
    _need_cuda(kv, anchor, residual, meta)
    if kv.dtype != torch.bfloat16 or kv.dim() != 4:
        raise ValueError("lynx_encode: kv must be a 4-D bfloat16 tensor")
    B, L, H, D = kv.shape
    ca, cr, cm = stream_shapes(B, L, H, D, page, C)
    dev = kv.device
    if anchor is None:
        anchor = torch.empty(ca, dtype=torch.uint8, device=dev)
    if residual is None:
        residual = torch.empty(cr, dtype=torch.uint8, device=dev)
    if meta is None:
        meta = torch.empty(cm, dtype=torch.float32, device=dev)
    _expect(anchor, ca, torch.uint8, dev, "lynx_encode: anchor")
    _expect(residual, cr, torch.uint8, dev, "lynx_encode: residual")
    _expect(meta, cm, torch.float32, dev, "lynx_encode: meta")
    _check(lib().lynx_encode(_ptr(kv), B, L, H, D, page, C, alpha, _ptr(anchor), _ptr(residual),
                             _ptr(meta), _stream(dev)), "lynx_encode")
    return anchor, residual, meta


def _decode_out(anchor, L, out_dtype, out):
    B, NB, H, page, half = anchor.shape
    if out is None:
        out = torch.empty((B, L, H, half * 2), dtype=out_dtype, device=anchor.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("lynx decode: output must be bfloat16 or float32")
    _expect(out, (B, L, H, half * 2), out.dtype, anchor.device, "lynx decode: out")
    code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    return out, code, B, H, page, half * 2


def _check_decode_streams(what, anchor, residual, meta, L, page, C):
    if anchor.dim() != 5 or anchor.dtype != torch.uint8:
        raise ValueError(f"{what}: anchor must be uint8 [B][L/page][H_kv][page][D/2]")
    B, _, H, _, half = anchor.shape
    ca, cr, cm = stream_shapes(B, L, H, half * 2, page, C)
    _expect(anchor, ca, torch.uint8, anchor.device, f"{what}: anchor")
    if residual is not None:
        _expect(residual, cr, torch.uint8, anchor.device, f"{what}: residual")
    _expect(meta, cm, torch.float32, anchor.device, f"{what}: meta")


def lynx_decode_anchor(anchor, meta, L: int, page: int, C: int, alpha: float,
                       out_dtype=torch.bfloat16, out=None):
    """Anchor-only reconstruction -> out[B][L][H_kv][D]."""
    _need_cuda(anchor, meta, out)
    _check_decode_streams("lynx_decode_anchor", anchor, None, meta, L, page, C)
    out, code, B, H, P, D = _decode_out(anchor, L, out_dtype, out)
    _check(lib().lynx_decode_anchor(_ptr(anchor), _ptr(meta), B, L, H, D, page, C, alpha,
                                    _ptr(out), code, _stream(anchor.device)),
           "lynx_decode_anchor")
    return out


def lynx_decode_full(anchor, residual, meta, L: int, page: int, C: int, alpha: float,
                     out_dtype=torch.bfloat16, out=None):
    """Anchor + Residual reconstruction -> out[B][L][H_kv][D]."""
    _need_cuda(anchor, residual, meta, out)
    _check_decode_streams("lynx_decode_full", anchor, residual, meta, L, page, C)
    if residual is None:
        raise ValueError("lynx_decode_full: residual is required")
    out, code, B, H, P, D = _decode_out(anchor, L, out_dtype, out)
    _check(lib().lynx_decode_full(_ptr(anchor), _ptr(residual), _ptr(meta), B, L, H, D, page, C,
                                  alpha, _ptr(out), code, _stream(anchor.device)),
           "lynx_decode_full")
    return out


# ----------------------------------------------------------------- paged

def paged_pool_shapes(num_blocks: int, H_kv: int, D: int, page: int, C: int):
    """Tensor shapes of the (anchor, residual, meta) pools of num_blocks pages."""
    codes = (num_blocks, H_kv, page, D // 2)
    return codes, codes, (num_blocks, H_kv, 2 + 2 * (page // C), D)


def _check_table(block_table, B, NB):
    if block_table.dtype != torch.int32 or tuple(block_table.shape) != (B, NB):
        raise ValueError(f"block_table must be int32 [{B}][{NB}]")


def lynx_encode_paged(kv: torch.Tensor, page: int, C: int, alpha: float, block_table,
                      num_blocks: int, anchor_pool=None, residual_pool=None, meta_pool=None):
    """lynx_encode into pools of num_blocks pages through block_table [B][L/page]
    (int32).  Returns (anchor_pool, residual_pool, meta_pool)."""
    _need_cuda(kv, block_table, anchor_pool, residual_pool, meta_pool)
    if kv.dtype != torch.bfloat16 or kv.dim() != 4:
        raise ValueError("lynx_encode_paged: kv must be a 4-D bfloat16 tensor")
    B, L, H, D = kv.shape
    _check_table(block_table, B, L // page)
    ca, cr, cm = paged_pool_shapes(num_blocks, H, D, page, C)
    dev = kv.device
    if anchor_pool is None:
        anchor_pool = torch.empty(ca, dtype=torch.uint8, device=dev)
    if residual_pool is None:
        residual_pool = torch.empty(cr, dtype=torch.uint8, device=dev)
    if meta_pool is None:
        meta_pool = torch.empty(cm, dtype=torch.float32, device=dev)
    _expect(anchor_pool, ca, torch.uint8, dev, "lynx_encode_paged: anchor pool")
    _expect(residual_pool, cr, torch.uint8, dev, "lynx_encode_paged: residual pool")
    _expect(meta_pool, cm, torch.float32, dev, "lynx_encode_paged: meta pool")
    _check(lib().lynx_encode_paged(_ptr(kv), B, L, H, D, page, C, alpha, _ptr(block_table),
                                   num_blocks, _ptr(anchor_pool), _ptr(residual_pool),
                                   _ptr(meta_pool), _stream(dev)), "lynx_encode_paged")
    return anchor_pool, residual_pool, meta_pool


def lynx_decode_paged(anchor_pool, residual_pool, meta_pool, block_table, L: int, page: int,
                      C: int, alpha: float, mode: int, out_dtype=torch.bfloat16, out=None):
    """Decode paged streams (mode LYNX_ANCHOR or LYNX_FULL) -> out[B][L][H_kv][D]."""
    _need_cuda(anchor_pool, residual_pool, meta_pool, block_table, out)
    num_blocks, H, P, half = anchor_pool.shape
    B = block_table.shape[0]
    _check_table(block_table, B, L // page)
    if out is None:
        out = torch.empty((B, L, H, half * 2), dtype=out_dtype, device=anchor_pool.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("lynx decode: output must be bfloat16 or float32")
    dev = anchor_pool.device
    shapes = paged_pool_shapes(num_blocks, H, half * 2, page, C)
    _expect(anchor_pool, shapes[0], torch.uint8, dev, "lynx_decode_paged: anchor pool")
    if mode == LYNX_FULL:
        _expect(residual_pool, shapes[1], torch.uint8, dev, "lynx_decode_paged: residual pool")
    _expect(meta_pool, shapes[2], torch.float32, dev, "lynx_decode_paged: meta pool")
    _expect(out, (B, L, H, half * 2), out.dtype, dev, "lynx_decode_paged: out")
    code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    _check(lib().lynx_decode_paged(_ptr(anchor_pool), _ptr(residual_pool), _ptr(meta_pool),
                                   _ptr(block_table), num_blocks, B, L, H, half * 2, page, C,
                                   alpha, mode, _ptr(out), code, _stream(anchor_pool.device)),
           "lynx_decode_paged")
    return out


def lynx_spec_verify(p, q, draft_tokens, u, r, n_accepted=None, next_token=None):
    """Eq. 10-11 for a batch: p [batch][T+1][V] f32, q [batch][T][V] f32,
    draft_tokens [batch][T] int32, u [batch][T] f32, r [batch] int32 holding
    uint32 bits.  Returns (n_accepted, next_token), int32 [batch]."""
    _need_cuda(p, q, draft_tokens, u, r, n_accepted, next_token)
    batch, T1, V = p.shape
    T = T1 - 1
    if p.dtype != torch.float32 or q.dtype != torch.float32 or u.dtype != torch.float32:
        raise ValueError("lynx_spec_verify: p, q and u must be float32")
    if draft_tokens.dtype != torch.int32 or r.dtype != torch.int32:
        raise ValueError("lynx_spec_verify: draft_tokens and r must be int32 tensors")
    if tuple(q.shape) != (batch, T, V) or tuple(draft_tokens.shape) != (batch, T) or \
            tuple(u.shape) != (batch, T) or tuple(r.shape) != (batch,):
        raise ValueError("lynx_spec_verify: shapes")
    if n_accepted is None:
        n_accepted = torch.empty(batch, dtype=torch.int32, device=p.device)
    if next_token is None:
        next_token = torch.empty(batch, dtype=torch.int32, device=p.device)
    _check(lib().lynx_spec_verify(_ptr(p), _ptr(q), _ptr(draft_tokens), _ptr(u), _ptr(r), batch,
                                  T, V, _ptr(n_accepted), _ptr(next_token), _stream(p.device)),
           "lynx_spec_verify")
    return n_accepted, next_token


def lynx_wait_selftest(limit_ns: int, arrive, device) -> int:
    """Run the bounded-wait check; returns 1 (barrier completed) or 2 (the
    wait gave up after limit_ns); with arrive == 2 the verification pass's
    wait and abort word: 3 (both waits ended as they must) or 4; with 3 the paged
    cache's: 5 (what was in flight arrived after a wait was given up) or 6."""
    st = torch.zeros(1, dtype=torch.int32, device=device)
    _check(lib().lynx_wait_selftest(limit_ns, int(arrive), _ptr(st), _stream(st.device)),
           "lynx_wait_selftest")
    return int(st.item())


def lynx_device_errors() -> int:
    bits = ctypes.c_uint()
    _check(lib().lynx_device_errors(ctypes.byref(bits)), "lynx_device_errors")
    return bits.value


# ------------------------------------------------------- split-stream transfer

LYNX_OP_ENCODE, LYNX_OP_COPY_ANCHOR, LYNX_OP_COPY_META, LYNX_OP_COPY_RESIDUAL = 0, 1, 2, 3
LYNX_OP_DECODE_ANCHOR, LYNX_OP_UPGRADE, LYNX_OP_NONE = 4, 5, -1
LYNX_Q_COPY, LYNX_Q_HI, LYNX_Q_LO = 0, 1, 2


class SplitOp(ctypes.Structure):
    """lynx_split_op of include/lynx.h."""
    _fields_ = [("kind", ctypes.c_int32), ("queue", ctypes.c_int32), ("group", ctypes.c_int64),
                ("page0", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("offset", ctypes.c_int64), ("bytes", ctypes.c_int64),
                ("wait_kind", ctypes.c_int32 * 2), ("wait_group", ctypes.c_int64 * 2)]


class LynxHeader(ctypes.Structure):
    """lynx_header of include/lynx.h (128 bytes)."""
    _fields_ = [("magic", ctypes.c_char * 8), ("version", ctypes.c_uint32),
                ("header_bytes", ctypes.c_uint32), ("B", ctypes.c_int64), ("L", ctypes.c_int64),
                ("H_kv", ctypes.c_int32), ("D", ctypes.c_int32), ("page", ctypes.c_int32),
                ("C", ctypes.c_int32), ("alpha", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("anchor_offset", ctypes.c_uint64), ("anchor_bytes", ctypes.c_uint64),
                ("meta_offset", ctypes.c_uint64), ("meta_bytes", ctypes.c_uint64),
                ("residual_offset", ctypes.c_uint64), ("residual_bytes", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64), ("reserved", ctypes.c_uint32 * 3),
                ("header_crc", ctypes.c_uint32)]


def lynx_split_plan(B: int, L: int, H_kv: int, D: int, page: int, C: int, pages_per_group: int,
                    send: bool = False, with_decode: bool = True):
    """The transfer schedule as a list of dicts, in issue order."""
    n = ctypes.c_int64()
    rc = lib().lynx_split_plan(B, L, H_kv, D, page, C, pages_per_group, int(send),
                               int(with_decode), None, 0, ctypes.byref(n))
    if rc not in (LYNX_OK, LYNX_EWORKSPACE):
        _check(rc, "lynx_split_plan")
    buf = (SplitOp * max(1, n.value))()
    _check(lib().lynx_split_plan(B, L, H_kv, D, page, C, pages_per_group, int(send),
                                 int(with_decode), buf, n.value, ctypes.byref(n)),
           "lynx_split_plan")
    return [{"kind": o.kind, "queue": o.queue, "group": o.group, "page0": o.page0,
             "n_pages": o.n_pages, "offset": o.offset, "bytes": o.bytes,
             "waits": [(o.wait_kind[i], o.wait_group[i]) for i in range(2)
                       if o.wait_kind[i] != LYNX_OP_NONE]} for o in buf[:n.value]]


def _need_host(*ts):
    for t in ts:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("lynx: host buffers must be contiguous CPU tensors (pinned)")


def _raw_stream(s):
    return ctypes.c_void_p(s.cuda_stream) if s is not None else None


def _raw_event(ev, stream):
    """Handle of a torch.cuda.Event, created (by a first record) if still lazy."""
    if ev is None:
        return None
    if not ev.cuda_event:
        ev.record(stream if stream is not None else torch.cuda.current_stream())
    return ctypes.c_void_p(ev.cuda_event)


def lynx_split_receive(host, dev, L: int, page: int, C: int, alpha: float, pages_per_group: int,
                       out=None, copy_stream=None, hi_stream=None, lo_stream=None,
                       anchor_ready=None, full_ready=None):
    """Receiver side: host = (anchor, residual, meta) CPU tensors, dev = the
    same three CUDA tensors (stream_shapes); out (optional) is decoded from
    the Anchor as it lands and upgraded in place to the full decode."""
    ha, hr, hm = host
    da, dr, dm = dev
    _need_host(ha, hr, hm)
    _need_cuda(da, dr, dm, out)
    B, NB, H, P, half = da.shape
    code = LYNX_OUT_BF16
    if out is not None:
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("lynx_split_receive: out must be bfloat16 or float32")
        code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    _check(lib().lynx_split_receive(_ptr(ha), _ptr(hm), _ptr(hr), _ptr(da), _ptr(dm), _ptr(dr),
                                    B, L, H, half * 2, page, C, alpha, pages_per_group, _ptr(out),
                                    code, _raw_stream(copy_stream), _raw_stream(hi_stream),
                                    _raw_stream(lo_stream), _raw_event(anchor_ready, hi_stream),
                                    _raw_event(full_ready, lo_stream)),
           "lynx_split_receive")


def lynx_split_send(kv, page: int, C: int, alpha: float, dev, host, pages_per_group: int,
                    hi_stream=None, copy_stream=None, anchor_sent=None, all_sent=None):
    """Sender side: encode kv into dev = (anchor, residual, meta) group by
    group and copy each group to host = (anchor, residual, meta) CPU tensors,
    every Residual after the last Anchor."""
    da, dr, dm = dev
    ha, hr, hm = host
    _need_cuda(kv, da, dr, dm)
    _need_host(ha, hr, hm)
    B, L, H, D = kv.shape
    _check(lib().lynx_split_send(_ptr(kv), B, L, H, D, page, C, alpha, _ptr(da), _ptr(dm),
                                 _ptr(dr), _ptr(ha), _ptr(hm), _ptr(hr), pages_per_group,
                                 _raw_stream(hi_stream), _raw_stream(copy_stream),
                                 _raw_event(anchor_sent, copy_stream),
                                 _raw_event(all_sent, copy_stream)),
           "lynx_split_send")


def lynx_header_init(B: int, L: int, H_kv: int, D: int, page: int, C: int, alpha: float,
                     with_residual: bool = True) -> bytes:
    """The 128-byte header of a serialized request."""
    h = LynxHeader()
    _check(lib().lynx_header_init(ctypes.byref(h), B, L, H_kv, D, page, C, alpha,
                                  int(with_residual)), "lynx_header_init")
    return bytes(h)


def lynx_header_check(buf: bytes) -> LynxHeader:
    """Validate a header; returns it parsed, or raises LynxError."""
    if len(buf) < ctypes.sizeof(LynxHeader):
        raise ValueError("lynx_header_check: fewer than 128 bytes")
    h = LynxHeader.from_buffer_copy(bytes(buf[:ctypes.sizeof(LynxHeader)]))
    _check(lib().lynx_header_check(ctypes.byref(h)), "lynx_header_check")
    return h


# ------------------------------------------------------- comparison points

def lynx_int_encode(kv, bits: int, codes=None, meta=None):
    """Linear INT-`bits` baseline (Eq. 4) of kv[..][128] BF16: one scale and
    zero point per row of 128 channels.  Returns (codes, meta)."""
    _need_cuda(kv, codes, meta)
    if kv.dtype != torch.bfloat16 or kv.shape[-1] != 128:
        raise ValueError("lynx_int_encode: kv must be bfloat16 with 128 channels")
    rows = kv.numel() // 128
    if codes is None:
        codes = torch.empty(kv.shape[:-1] + (128 * bits // 8,), dtype=torch.uint8,
                            device=kv.device)
    if meta is None:
        meta = torch.empty(kv.shape[:-1] + (2,), dtype=torch.float32, device=kv.device)
    _check(lib().lynx_int_encode(_ptr(kv), rows, 128, bits, _ptr(codes), _ptr(meta),
                                 _stream(kv.device)), "lynx_int_encode")
    return codes, meta


def lynx_int_decode(codes, meta, bits: int, out_dtype=torch.bfloat16, out=None):
    _need_cuda(codes, meta, out)
    rows = meta.numel() // 2
    if out is None:
        out = torch.empty(meta.shape[:-1] + (128,), dtype=out_dtype, device=codes.device)
    code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    _check(lib().lynx_int_decode(_ptr(codes), _ptr(meta), rows, 128, bits, _ptr(out), code,
                                 _stream(codes.device)), "lynx_int_decode")
    return out


def lynx_split_bits(anchor, residual, k: int, anchor_k=None, residual_k=None):
    """Re-split 4+4 streams [B][NB][H][P][64] into a k + (8-k) split:
    returns (anchor_k [B][NB][H][P][16k], residual_k [..][16(8-k)])."""
    _need_cuda(anchor, residual, anchor_k, residual_k)
    shp = anchor.shape[:-1]
    rows = anchor.numel() // 64
    if anchor_k is None:
        anchor_k = torch.empty(shp + (16 * k,), dtype=torch.uint8, device=anchor.device)
    if residual_k is None:
        residual_k = torch.empty(shp + (16 * (8 - k),), dtype=torch.uint8, device=anchor.device)
    _check(lib().lynx_split_bits(_ptr(anchor), _ptr(residual), rows, 128, k, _ptr(anchor_k),
                                 _ptr(residual_k), _stream(anchor.device)), "lynx_split_bits")
    return anchor_k, residual_k


def lynx_join_bits(anchor_k, residual_k, k: int, anchor=None, residual=None):
    _need_cuda(anchor_k, residual_k, anchor, residual)
    shp = anchor_k.shape[:-1]
    rows = anchor_k.numel() // (16 * k)
    if anchor is None:
        anchor = torch.empty(shp + (64,), dtype=torch.uint8, device=anchor_k.device)
    if residual is None:
        residual = torch.empty(shp + (64,), dtype=torch.uint8, device=anchor_k.device)
    _check(lib().lynx_join_bits(_ptr(anchor_k), _ptr(residual_k), rows, 128, k, _ptr(anchor),
                                _ptr(residual), _stream(anchor_k.device)), "lynx_join_bits")
    return anchor, residual


def lynx_decode_anchor_bits(anchor_k, meta, L: int, page: int, C: int, alpha: float, k: int,
                            out_dtype=torch.bfloat16, out=None):
    """Anchor-only decode of a k-bit Anchor stream [B][NB][H][P][16k]."""
    _need_cuda(anchor_k, meta, out)
    B, NB, H = anchor_k.shape[:3]
    if out is None:
        out = torch.empty((B, L, H, 128), dtype=out_dtype, device=anchor_k.device)
    code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    _check(lib().lynx_decode_anchor_bits(_ptr(anchor_k), _ptr(meta), B, L, H, 128, page, C, alpha,
                                         k, _ptr(out), code, _stream(anchor_k.device)),
           "lynx_decode_anchor_bits")
    return out


def lynx_a1_encode(kv, page: int, alpha: float = 100.0):
    """The Appendix A.1 variant of kv[B][L][H][128] BF16: returns (anchor,
    residual, meta[B][L/page][H][1 + page/16][128])."""
    _need_cuda(kv)
    if kv.dtype != torch.bfloat16 or kv.dim() != 4:
        raise ValueError("lynx_a1_encode: kv must be a 4-D bfloat16 tensor")
    B, L, H, D = kv.shape
    codes = (B, L // page, H, page, D // 2)
    anchor = torch.empty(codes, dtype=torch.uint8, device=kv.device)
    residual = torch.empty(codes, dtype=torch.uint8, device=kv.device)
    meta = torch.empty((B, L // page, H, 1 + page // 16, D), dtype=torch.float32,
                       device=kv.device)
    _check(lib().lynx_a1_encode(_ptr(kv), B, L, H, D, page, alpha, _ptr(anchor), _ptr(residual),
                                _ptr(meta), _stream(kv.device)), "lynx_a1_encode")
    return anchor, residual, meta


def lynx_a1_decode(anchor, residual, meta, L: int, page: int, alpha: float = 100.0,
                   out_dtype=torch.bfloat16, out=None):
    """Decode of the A.1 variant; residual None gives the Anchor-only decode."""
    _need_cuda(anchor, residual, meta, out)
    B, NB, H, P, half = anchor.shape
    if out is None:
        out = torch.empty((B, L, H, half * 2), dtype=out_dtype, device=anchor.device)
    code = LYNX_OUT_BF16 if out.dtype == torch.bfloat16 else LYNX_OUT_FP32
    _check(lib().lynx_a1_decode(_ptr(anchor), _ptr(residual), _ptr(meta), B, L, H, half * 2, page,
                                alpha, _ptr(out), code, _stream(anchor.device)),
           "lynx_a1_decode")
    return out


# ----------------------------------------------------------------- attention

def lynx_attn_workspace_bytes(batch: int, T: int, H_q: int, L: int, H_kv: int, D: int,
                              page: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().lynx_attn_workspace_bytes(batch, T, H_q, L, H_kv, D, page, ctypes.byref(n)),
           "lynx_attn_workspace_bytes")
    return n.value


def _check_attn_io(what, q, ks, vs, L, page, C, mode, out, workspace, need, pools=False):
    """Shapes, types and devices of everything an attention call reads or
    writes: q [batch][T][H_q][D] bf16; K and V streams of one layout (dense
    [batch][L/page][H_kv][...], or pools [num_blocks][H_kv][...]); residuals
    present in full mode; out [batch][T][H_q][D] float32; a workspace of at
    least `need` bytes."""
    batch, T, H_q, D = q.shape
    dev = q.device
    for name, (a, r, m) in (("k", ks), ("v", vs)):
        if a.dtype != torch.uint8 or a.dim() != (4 if pools else 5):
            raise ValueError(f"{what}: {name} anchor must be uint8 "
                             + ("[num_blocks][H_kv][page][D/2]" if pools
                                else "[batch][L/page][H_kv][page][D/2]"))
        if pools:
            nb, H_kv = a.shape[0], a.shape[1]
            codes = (nb, H_kv, page, D // 2)
            mshape = (nb, H_kv, 2 + 2 * (page // C), D)
        else:
            H_kv = a.shape[2]
            codes, _, mshape = stream_shapes(batch, L, H_kv, D, page, C)
        _expect(a, codes, torch.uint8, dev, f"{what}: {name} anchor")
        if mode == LYNX_FULL:
            _expect(r, codes, torch.uint8, dev, f"{what}: {name} residual")
        _expect(m, mshape, torch.float32, dev, f"{what}: {name} meta")
    if tuple(ks[0].shape) != tuple(vs[0].shape):
        raise ValueError(f"{what}: K and V streams differ in shape")
    _expect(out, (batch, T, H_q, D), torch.float32, dev, f"{what}: out")
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError(f"{what}: workspace on {workspace.device}, expected {dev}")
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"{what}: workspace holds "
                             f"{workspace.numel() * workspace.element_size()} bytes, "
                             f"the call needs {need}")


def lynx_attn_decode(q, k_streams, v_streams, L: int, page: int, C: int, alpha: float,
                     mode: int, out=None, workspace=None, k_tail=None, v_tail=None):
    """q[batch][T][H_q][D] bf16; k_streams / v_streams = (anchor, residual or
    None, meta) from lynx_encode of K and V.  With k_tail / v_tail
    ([batch][T][H_kv][D] bf16, the draft tokens' own keys and values) query
    token t also attends to draft tokens 0..t (lynx_attn_decode_tail).
    Returns out[batch][T][H_q][D] f32."""
    ka, kr, km = k_streams
    va, vr, vm = v_streams
    _need_cuda(q, ka, kr, km, va, vr, vm, out, workspace, k_tail, v_tail)
    if (k_tail is None) != (v_tail is None):
        raise ValueError("lynx_attn_decode: give both k_tail and v_tail, or neither")
    if q.dtype != torch.bfloat16 or q.dim() != 4:
        raise ValueError("lynx_attn_decode: q must be a 4-D bfloat16 tensor")
    batch, T, H_q, D = q.shape
    if ka.dim() != 5:
        raise ValueError("lynx_attn_decode: streams must be [batch][L/page][H_kv][...]")
    H_kv = ka.shape[2]
    if out is None:
        out = torch.empty((batch, T, H_q, D), dtype=torch.float32, device=q.device)
    need = lynx_attn_workspace_bytes(batch, T, H_q, L, H_kv, D, page)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check_attn_io("lynx_attn_decode", q, k_streams, v_streams, L, page, C, mode, out,
                   workspace, need)
    if k_tail is not None:
        for t in (k_tail, v_tail):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != (batch, T, H_kv, D) or \
                    not t.is_contiguous():
                raise ValueError("lynx_attn_decode: tails must be contiguous bfloat16 "
                                 "[batch][T][H_kv][D]")
        _check(lib().lynx_attn_decode_tail(_ptr(q), batch, T, H_q, _ptr(ka), _ptr(kr),
                                           _ptr(km), _ptr(va), _ptr(vr), _ptr(vm), L, H_kv, D,
                                           page, C, alpha, mode, _ptr(k_tail), _ptr(v_tail),
                                           _ptr(out), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(q.device)), "lynx_attn_decode_tail")
        return out
    _check(lib().lynx_attn_decode(_ptr(q), batch, T, H_q, _ptr(ka), _ptr(kr), _ptr(km),
                                  _ptr(va), _ptr(vr), _ptr(vm), L, H_kv, D, page, C, alpha,
                                  mode, _ptr(out), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream(q.device)), "lynx_attn_decode")
    return out


def lynx_attn_decode_tail(q, k_streams, v_streams, L: int, page: int, C: int, alpha: float,
                          mode: int, k_tail, v_tail, out=None, workspace=None):
    """lynx_attn_decode_tail: query token t attends to the L cached tokens and
    to the draft tokens 0..t given by k_tail / v_tail ([batch][T][H_kv][D] bf16)."""
    if k_tail is None or v_tail is None:
        raise ValueError("lynx_attn_decode_tail: k_tail and v_tail are required")
    return lynx_attn_decode(q, k_streams, v_streams, L, page, C, alpha, mode, out=out,
                            workspace=workspace, k_tail=k_tail, v_tail=v_tail)


def lynx_attn_decode_paged(q, k_pools, v_pools, block_table, L: int, page: int, C: int,
                           alpha: float, mode: int, out=None, workspace=None, k_tail=None,
                           v_tail=None):
    """lynx_attn_decode(_tail) over paged K and V pools (anchor, residual or None,
    meta) read through block_table [batch][L/page] (int32)."""
    ka, kr, km = k_pools
    va, vr, vm = v_pools
    _need_cuda(q, ka, kr, km, va, vr, vm, block_table, out, workspace, k_tail, v_tail)
    if (k_tail is None) != (v_tail is None):
        raise ValueError("lynx_attn_decode_paged: give both k_tail and v_tail, or neither")
    if q.dtype != torch.bfloat16 or q.dim() != 4:
        raise ValueError("lynx_attn_decode_paged: q must be a 4-D bfloat16 tensor")
    batch, T, H_q, D = q.shape
    if ka.dim() != 4:
        raise ValueError("lynx_attn_decode_paged: pools must be [num_blocks][H_kv][...]")
    num_blocks, H_kv = ka.shape[0], ka.shape[1]
    _check_table(block_table, batch, L // page)
    if out is None:
        out = torch.empty((batch, T, H_q, D), dtype=torch.float32, device=q.device)
    need = lynx_attn_workspace_bytes(batch, T, H_q, L, H_kv, D, page)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check_attn_io("lynx_attn_decode_paged", q, k_pools, v_pools, L, page, C, mode, out,
                   workspace, need, pools=True)
    if k_tail is not None:
        for t in (k_tail, v_tail):
            _expect(t, (batch, T, H_kv, D), torch.bfloat16, q.device,
                    "lynx_attn_decode_paged: tail")
    _check(lib().lynx_attn_decode_paged(_ptr(q), batch, T, H_q, _ptr(ka), _ptr(kr), _ptr(km),
                                        _ptr(va), _ptr(vr), _ptr(vm), _ptr(block_table),
                                        num_blocks, L, H_kv, D, page, C, alpha, mode,
                                        _ptr(k_tail), _ptr(v_tail), _ptr(out), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(q.device)),
           "lynx_attn_decode_paged")
    return out


def lynx_attn_decode_noalloc(q, k_streams, v_streams, L: int, page: int, C: int,
                             alpha: float, mode: int, out=None):
    """lynx_attn_decode with the library's built-in scratch instead of a
    workspace (for callers that cannot allocate device memory).  `out` must
    be given by such callers; if it is None it is allocated here for
    convenience."""
    ka, kr, km = k_streams
    va, vr, vm = v_streams
    _need_cuda(q, ka, kr, km, va, vr, vm, out)
    if q.dtype != torch.bfloat16 or q.dim() != 4:
        raise ValueError("lynx_attn_decode_noalloc: q must be a 4-D bfloat16 tensor")
    batch, T, H_q, D = q.shape
    if ka.dim() != 5:
        raise ValueError("lynx_attn_decode_noalloc: streams must be [batch][L/page][H_kv][...]")
    H_kv = ka.shape[2]
    if out is None:
        out = torch.empty((batch, T, H_q, D), dtype=torch.float32, device=q.device)
    _check_attn_io("lynx_attn_decode_noalloc", q, k_streams, v_streams, L, page, C, mode, out,
                   None, 0)
    _check(lib().lynx_attn_decode_noalloc(_ptr(q), batch, T, H_q, _ptr(ka), _ptr(kr), _ptr(km),
                                          _ptr(va), _ptr(vr), _ptr(vm), L, H_kv, D, page, C,
                                          alpha, mode, _ptr(out), _stream(q.device)),
           "lynx_attn_decode_noalloc")
    return out


# ----------------------------------------------------------- BF16 paged cache

class LynxRope(ctypes.Structure):
    """lynx_rope of include/lynx.h."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("axis", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


class LynxScore(ctypes.Structure):
    """lynx_score of include/lynx.h."""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int64), ("slopes", ctypes.c_void_p),
                ("prefix", ctypes.c_void_p)]


class Rope:
    """A model's rotation, made once: inv_freq, radians a position of each pair
    of channels (rope_frequencies gives the usual ones); axis, the axis of
    each pair where positions have several (None: one); interleaved, pairs
    (2i, 2i + 1) instead of (i, i + rot_dim / 2)."""

    def __init__(self, inv_freq, axis=None, interleaved: bool = False):
        f = [float(x) for x in inv_freq]
        if axis is not None:
            axis = [int(x) for x in axis]
            if len(axis) != len(f):
                raise ValueError(f"Rope: {len(axis)} axes for {len(f)} frequencies")
            if any(x < 0 or x > 255 for x in axis):
                raise ValueError("Rope: axes are small non-negative numbers")
        self.rot_dim = 2 * len(f)
        self.interleaved = bool(interleaved)
        self.n_axes = 1 if not axis else max(axis) + 1
        self._f = (ctypes.c_double * max(1, len(f)))(*f)
        self._a = None if axis is None else (ctypes.c_uint8 * max(1, len(axis)))(*axis)
        self._f_at = ctypes.addressof(self._f)
        self._a_at = None if self._a is None else ctypes.addressof(self._a)

    def _c(self, positions) -> LynxRope:
        return LynxRope(self.rot_dim, self.interleaved, self.n_axes, 0, self._f_at, self._a_at,
                        None if positions is None else positions.data_ptr())


def rope_frequencies(theta: float, rot_dim: int):
    """theta^(-2i / rot_dim) for i < rot_dim / 2."""
    return [theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]


# The calls of a decode step are short: the checks below cost about as long as
# the kernels, so they read each property once and pass pointers as integers.

def _token_rows(t, heads, what, device):
    """Packed token rows [n][heads][128] BF16; the rows may lie apart (views of
    a fused projection).  Returns (n, heads, stride in elements)."""
    shape = t.shape
    if t.dtype != torch.bfloat16 or len(shape) != 3 or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what}: expected bfloat16 [n_tokens][{heads or 'heads'}][D], got "
                         f"{t.dtype} of shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    n, h, d = shape
    apart, head, one = t.stride()
    if d != 1 and one != 1 or h > 1 and head != d:
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    if n <= 1:
        return n, h, h * d
    if apart < h * d or apart % 8:
        raise ValueError(f"{what}: tokens {apart} elements apart; a multiple of 8 and at "
                         f"least {h * d} is needed")
    return n, h, apart


def _dense(t, shape, dtype, device, what):
    """A contiguous tensor of just this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} of shape {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _check_cache(what, k_pool, v_pool, block_table, kv_len):
    """Pools [num_blocks][page][H_kv][D] BF16, block_table [batch][max_pages] and
    kv_len [batch] int32, contiguous and on one device.  Returns the device,
    the pools' shape and the table's."""
    dev, shape, table = k_pool.device, k_pool.shape, block_table.shape
    if dev.type != "cuda":
        raise ValueError(f"{what}: tensors must be CUDA tensors")
    if len(shape) != 4 or len(table) != 2:
        raise ValueError(f"{what}: pools must be [num_blocks][page][H_kv][D], block_table "
                         "[batch][max_pages]")
    if (k_pool.dtype != torch.bfloat16 or v_pool.dtype != torch.bfloat16 or v_pool.shape != shape or
            v_pool.device != dev or not k_pool.is_contiguous() or not v_pool.is_contiguous()):
        raise ValueError(f"{what}: K and V pools must be contiguous bfloat16 of one shape and device")
    if (block_table.dtype != torch.int32 or block_table.device != dev or
            not block_table.is_contiguous()):
        raise ValueError(f"{what}: block_table must be contiguous int32 on {dev}")
    if (kv_len.dtype != torch.int32 or kv_len.shape != table[:1] or kv_len.device != dev or
            not kv_len.is_contiguous()):
        raise ValueError(f"{what}: kv_len must be contiguous int32 [{table[0]}] on {dev}")
    return dev, shape, table


class _on:
    """Makes `index` the current device for a launch, where it is not."""

    def __init__(self, index):
        self.to, self.was = index, None

    def __enter__(self):
        self.was = torch.cuda.current_device()
        torch.cuda.set_device(self.to)

    def __exit__(self, *exc):
        torch.cuda.set_device(self.was)
        return False


def _launch(fn, what, dev, *args):
    """fn(*args, the current stream of `dev`), launched with `dev` current."""
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with _on(index):
            rc = fn(*args, stream)
    if rc:
        _check(rc, what)


def lynx_cache_append(k, v, q_offsets, kv_len, block_table, k_pool, v_pool, q=None, q_out=None,
                      rope=None, positions=None):
    """New tokens into the BF16 paged cache: k (rotated) and v [n_tokens][H_kv][D]
    to their slots of the pools [num_blocks][page][H_kv][D], q [n_tokens][H_q][D]
    rotated into q_out (which may be q itself).  q_offsets [batch + 1] names each
    sequence's packed tokens, kv_len [batch] its length in the cache with them;
    rope is a Rope (None: no rotation), positions int32 [n_axes][n_tokens] (None:
    the position in the cache).  Returns q_out, None without q."""
    what = "lynx_cache_append"
    dev, (num_blocks, page, H_kv, D), (batch, max_pages) = _check_cache(what, k_pool, v_pool,
                                                                        block_table, kv_len)
    n, _, k_stride = _token_rows(k, H_kv, "lynx_cache_append: k", dev)
    _, _, v_stride = _token_rows(v, H_kv, "lynx_cache_append: v", dev)
    if v.shape != k.shape or k.shape[2] != D:
        raise ValueError(f"{what}: k and v must both be [n_tokens][{H_kv}][{D}]")
    at = _dense(q_offsets, (batch + 1,), torch.int32, dev, "lynx_cache_append: q_offsets")
    H_q = q_stride = 0
    qp = qo = None
    if q is not None:
        m, H_q, q_stride = _token_rows(q, None, "lynx_cache_append: q", dev)
        if m != n or q.shape[2] != D:
            raise ValueError(f"{what}: q must be [{n}][H_q][{D}]")
        if q_out is None:
            q_out = torch.empty((n, H_q, D), dtype=torch.bfloat16, device=dev)
        qp = q.data_ptr()
        qo = _dense(q_out, (n, H_q, D), torch.bfloat16, dev, "lynx_cache_append: q_out")
    elif q_out is not None:
        raise ValueError(f"{what}: q_out without q")
    c_rope = None
    if rope is not None:
        if positions is not None:
            if positions.dim() == 1 and rope.n_axes == 1:
                positions = positions[None]
            _dense(positions, (rope.n_axes, n), torch.int32, dev, "lynx_cache_append: positions")
        c_rope = ctypes.byref(rope._c(positions))
    elif positions is not None:
        raise ValueError(f"{what}: positions without rope")
    _launch(lib().lynx_cache_append, what, dev, k.data_ptr(), k_stride, v.data_ptr(), v_stride, qp,
            q_stride, qo, at, kv_len.data_ptr(), block_table.data_ptr(), max_pages, num_blocks,
            batch, n, H_q, H_kv, D, page, c_rope, k_pool.data_ptr(), v_pool.data_ptr())
    return q_out


def lynx_cache_attn_decode_workspace_bytes(batch: int, T: int, H_q: int, H_kv: int, D: int,
                                           page: int, max_pages: int) -> int:
    """Bytes of workspace lynx_cache_attn_decode needs; 0: none."""
    n = ctypes.c_size_t()
    _check(lib().lynx_cache_attn_decode_workspace_bytes(batch, T, H_q, H_kv, D, page, max_pages,
                                                        ctypes.byref(n)),
           "lynx_cache_attn_decode_workspace_bytes")
    return n.value


def lynx_cache_attn_prefill_workspace_bytes(n_tokens: int, batch: int, H_q: int, H_kv: int,
                                            D: int, page: int, max_pages: int) -> int:
    """Bytes of workspace lynx_cache_attn_prefill needs; 0: none."""
    n = ctypes.c_size_t()
    _check(lib().lynx_cache_attn_prefill_workspace_bytes(n_tokens, batch, H_q, H_kv, D, page,
                                                         max_pages, ctypes.byref(n)),
           "lynx_cache_attn_prefill_workspace_bytes")
    return n.value


def lynx_cache_attn_form(n_tokens: int, batch: int, T: int, H_q: int, H_kv: int, D: int, page: int,
                         max_pages: int, sms: int) -> int:
    """How a call's work is shared out on a GPU of `sms` SMs, one of LYNX_CACHE_*, or
    0 for a call without tokens; T = 0: lynx_cache_attn_prefill."""
    form = ctypes.c_int()
    _check(lib().lynx_cache_attn_form(n_tokens, batch, T, H_q, H_kv, D, page, max_pages, sms,
                                      ctypes.byref(form)), "lynx_cache_attn_form")
    return form.value


_decode_bytes = functools.lru_cache(maxsize=256)(lynx_cache_attn_decode_workspace_bytes)
_prefill_bytes = functools.lru_cache(maxsize=256)(lynx_cache_attn_prefill_workspace_bytes)


def _cache_attn(what, q, shape, batch, T, n, H_q, D, stride, offsets, k_pool, v_pool,
                block_table, kv_len, scale, softcap, window, slopes, prefix, out, lse, workspace,
                tree=None):
    """The attention calls: q of shape `shape`, its n token rows `stride` elements apart;
    tree: the nodes' keys, values and mask."""
    dev, (num_blocks, page, H_kv, pool_D), (seqs, max_pages) = _check_cache(
        what, k_pool, v_pool, block_table, kv_len)
    if q.dtype != torch.bfloat16 or q.device != dev:
        raise ValueError(f"{what}: q must be bfloat16 on {dev}, got {q.dtype} on {q.device}")
    if pool_D != D:
        raise ValueError(f"{what}: q has {D} channels, the pools {pool_D}")
    if batch != seqs:
        raise ValueError(f"{what}: q holds {batch} sequences, block_table {seqs}")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        op = out.data_ptr()
    else:
        op = _dense(out, shape, torch.bfloat16, dev, what)
    lp = None if lse is None else _dense(lse, shape[:-1], torch.float32, dev, what)
    score = LynxScore(D ** -0.5 if scale is None else scale, softcap, window,
                      None if slopes is None else _dense(slopes, (H_q,), torch.float32, dev, what),
                      None if prefix is None else _dense(prefix, (batch,), torch.int32, dev, what))
    wp, size = None, 0
    if workspace is None:
        size = (_tree_bytes(batch, T, H_q, H_kv, D, page, max_pages) if tree is not None else
                _decode_bytes(batch, T, H_q, H_kv, D, page, max_pages) if T else
                _prefill_bytes(n, batch, H_q, H_kv, D, page, max_pages))
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
            wp = workspace.data_ptr()
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"{what}: workspace must be contiguous on {dev}")
        wp = workspace.data_ptr()
    if tree is not None:
        k_nodes, v_nodes, mask = tree
        nodes = (batch, TREE_ROOM, H_kv, D)
        _launch(lib().lynx_cache_attn_tree, what, dev, q.data_ptr(), stride, batch, T, H_q,
                _dense(k_nodes, nodes, torch.bfloat16, dev, what),
                _dense(v_nodes, nodes, torch.bfloat16, dev, what),
                _dense(mask, (batch, T), torch.int64, dev, what), k_pool.data_ptr(),
                v_pool.data_ptr(), block_table.data_ptr(), max_pages, num_blocks,
                kv_len.data_ptr(), H_kv, D, page, ctypes.byref(score), op, lp, wp, size)
    elif T:
        _launch(lib().lynx_cache_attn_decode, what, dev, q.data_ptr(), stride, batch, T, H_q,
                k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(), max_pages,
                num_blocks, kv_len.data_ptr(), H_kv, D, page, ctypes.byref(score), op, lp, wp,
                size)
    else:
        at = _dense(offsets, (batch + 1,), torch.int32, dev, what)
        _launch(lib().lynx_cache_attn_prefill, what, dev, q.data_ptr(), stride, at, n, batch, H_q,
                k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(), max_pages,
                num_blocks, kv_len.data_ptr(), H_kv, D, page, ctypes.byref(score), op, lp, wp,
                size)
    return out


def lynx_cache_attn_decode(q, k_pool, v_pool, block_table, kv_len, scale=None,
                           softcap: float = 0.0, window: int = 0, slopes=None, prefix=None,
                           out=None, lse=None, workspace=None):
    """Attention of the T newest tokens of each sequence, q [batch][T][H_q][D] BF16,
    over the BF16 paged cache that holds them (lynx_cache_append).  softcap,
    window, slopes [H_q] and prefix [batch] as lynx_score in include/lynx.h; lse
    [batch][T][H_q] float32 is written if given.  Returns out, BF16 as q."""
    what = "lynx_cache_attn_decode"
    batch, T, H_q, D, step = _sequence_rows(q, what)
    return _cache_attn(what, q, q.shape, batch, T, batch * T, H_q, D, step, None, k_pool, v_pool,
                       block_table, kv_len, scale, softcap, window, slopes, prefix, out, lse,
                       workspace)


def _sequence_rows(q, what):
    """q [batch][T][H_q][D], its tokens evenly spaced: its shape and their stride."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"{what}: q must be [batch][T][H_q][D]")
    batch, T, H_q, D = shape
    if T < 1:
        raise ValueError(f"{what}: q holds no token")
    apart, step, head, one = q.stride()
    if T == 1:                      # (the stride of a dimension of one means nothing)
        step = apart if batch > 1 else H_q * D
    elif batch > 1 and apart != T * step:
        raise ValueError(f"{what}: the tokens of q must be evenly spaced")
    if D != 1 and one != 1 or H_q > 1 and head != D or step < H_q * D or step % 8:
        raise ValueError(f"{what}: the heads of a token must be contiguous, the tokens a multiple "
                         f"of 8 elements apart and at least {H_q * D}")
    return batch, T, H_q, D, step


def lynx_cache_attn_prefill(q, q_offsets, k_pool, v_pool, block_table, kv_len, scale=None,
                            softcap: float = 0.0, window: int = 0, slopes=None, prefix=None,
                            out=None, lse=None, workspace=None):
    """Attention of packed chunks, q [n_tokens][H_q][D] BF16 with q_offsets
    [batch + 1], over the BF16 paged cache they were appended to; the rest as
    lynx_cache_attn_decode.  Rows of no sequence are left as they were."""
    what = "lynx_cache_attn_prefill"
    n, H_q, stride = _token_rows(q, None, what, q.device)
    shape = q.shape
    return _cache_attn(what, q, shape, block_table.shape[0], 0, n, H_q, shape[2], stride,
                       q_offsets, k_pool, v_pool, block_table, kv_len, scale, softcap, window,
                       slopes, prefix, out, lse, workspace)


# ----------------------------------------------------- drafting with trees

TREE_ROOM = 64                  # nodes of a tree, at most: rows of a sequence's node buffer
_LOGIT_TYPES = {torch.bfloat16: LYNX_BF16, torch.float32: LYNX_FP32, torch.float16: LYNX_FP16}


# Calls this short are the host's time: checks are made in few calls of their own, and
# addresses go in arrays that need no conversion.
_I32, _F32, _empty = torch.int32, torch.float32, torch.empty


def _given(t, shape, dtype, device, what):
    """The caller's own output tensor, checked."""
    _dense(t, shape, dtype, device, what)
    return t


def _cuda(t, what):
    if t.device.type != "cuda":
        raise ValueError(f"{what}: tensors must be CUDA tensors")
    return t.device


def lynx_token_logprobs(logits, tokens=None, top: int = 0, scale: float = 1.0, logprob=None,
                        entropy=None, top_logprob=None, top_token=None):
    """Log probabilities of rows of logits [rows][V] (bfloat16, float16 or float32;
    the rows may lie apart) times `scale`: of the given tokens, int32 [rows] or
    [rows][n], the entropy [rows] and the `top` likeliest tokens [rows][top], the
    lowest first among equals.  Returns (logprob, entropy, top_logprob, top_token); logprob
    has the shape of tokens (None without them).  Nothing is recorded for a gradient."""
    what = "lynx_token_logprobs"
    dev = _cuda(logits, what)
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise ValueError(f"{what}: logits must be bfloat16, float16 or float32 [rows][V], got "
                         f"{logits.dtype} of shape {tuple(logits.shape)}")
    rows, V = logits.shape
    apart, one = logits.stride()
    if V > 1 and one != 1:
        raise ValueError(f"{what}: the logits of a row must be contiguous")
    if rows <= 1:
        apart = V
    elif apart < V:
        raise ValueError(f"{what}: rows {apart} elements apart; at least {V} is needed")
    given, tp, lp = 0, None, None
    if tokens is not None:
        if tokens.dim() not in (1, 2) or tokens.shape[0] != rows:
            raise ValueError(f"{what}: tokens must be int32 [{rows}] or [{rows}][n]")
        given = 1 if tokens.dim() == 1 else tokens.shape[1]
        tp = _dense(tokens, tokens.shape, _I32, dev, what)
        logprob = (_empty(tokens.shape, dtype=_F32, device=dev) if logprob is None else
                   _given(logprob, tokens.shape, _F32, dev, what))
        lp = logprob.data_ptr()
    elif logprob is not None:
        raise ValueError(f"{what}: logprob without tokens")
    entropy = (_empty((rows,), dtype=_F32, device=dev) if entropy is None else
               _given(entropy, (rows,), _F32, dev, what))
    top_logprob = (_empty((rows, top), dtype=_F32, device=dev) if top_logprob is None else
                   _given(top_logprob, (rows, top), _F32, dev, what))
    top_token = (_empty((rows, top), dtype=_I32, device=dev) if top_token is None else
                 _given(top_token, (rows, top), _I32, dev, what))
    _launch(lib().lynx_token_logprobs, what, dev, logits.data_ptr(), kind, apart, rows, V, scale, tp,
            given, top, lp, entropy.data_ptr(), top_logprob.data_ptr(), top_token.data_ptr())
    return logprob, entropy, top_logprob, top_token


def lynx_tree_plan(parents, kv_len, mask=None, positions=None):
    """Which node of each tree sees which: parents int32 [batch][T] (-1 for node 0, a
    smaller node for the others, anything else: no node), kv_len int32 [batch], the
    cached tokens.  Returns (mask, positions): int64 [batch][T], bit a of word t for each
    node a that t sees, itself included; int32 [batch * T], as lynx_cache_append takes
    them, -1 without a node."""
    what = "lynx_tree_plan"
    dev = _cuda(parents, what)
    if parents.dim() != 2:
        raise ValueError(f"{what}: parents must be int32 [batch][T]")
    batch, T = shape = parents.shape
    pp = _dense(parents, shape, _I32, dev, what)
    kp = _dense(kv_len, (batch,), _I32, dev, what)
    mask = (_empty(shape, dtype=torch.int64, device=dev) if mask is None else
            _given(mask, shape, torch.int64, dev, what))
    positions = (_empty((batch * T,), dtype=_I32, device=dev) if positions is None else
                 _given(positions, (batch * T,), _I32, dev, what))
    _launch(lib().lynx_tree_plan, what, dev, pp, kp, batch, T, mask.data_ptr(),
            positions.data_ptr())
    return mask, positions


def lynx_cache_attn_tree_workspace_bytes(batch: int, T: int, H_q: int, H_kv: int, D: int,
                                         page: int, max_pages: int) -> int:
    """Bytes of workspace lynx_cache_attn_tree needs; 0: none."""
    n = ctypes.c_size_t()
    _check(lib().lynx_cache_attn_tree_workspace_bytes(batch, T, H_q, H_kv, D, page, max_pages,
                                                      ctypes.byref(n)),
           "lynx_cache_attn_tree_workspace_bytes")
    return n.value


_tree_bytes = functools.lru_cache(maxsize=256)(lynx_cache_attn_tree_workspace_bytes)


def lynx_cache_attn_tree(q, k_nodes, v_nodes, mask, k_pool, v_pool, block_table, kv_len, scale=None,
                         softcap: float = 0.0, window: int = 0, slopes=None, prefix=None, out=None,
                         lse=None, workspace=None):
    """Attention of a tree's nodes, q [batch][T][H_q][D] BF16, over the BF16 paged cache
    (kv_len tokens, the nodes not among them) and one another: k_nodes and v_nodes
    [batch][64][H_kv][D], mask [batch][T] of lynx_tree_plan; the rest as
    lynx_cache_attn_decode."""
    what = "lynx_cache_attn_tree"
    batch, T, H_q, D, step = _sequence_rows(q, what)
    return _cache_attn(what, q, q.shape, batch, T, batch * T, H_q, D, step, None, k_pool, v_pool,
                       block_table, kv_len, scale, softcap, window, slopes, prefix, out, lse,
                       workspace, (k_nodes, v_nodes, mask))


def lynx_tree_verify(parents, tokens, answers, path=None, n_path=None, next_token=None):
    """The walk down each tree along the answers: all int32 [batch][T], tokens the
    nodes', answers what the model says follows each.  Returns (path [batch][T], the nodes
    met and -1 behind them, n_path [batch], how many, next_token [batch], the answer at
    the last of them)."""
    what = "lynx_tree_verify"
    dev = _cuda(parents, what)
    if parents.dim() != 2:
        raise ValueError(f"{what}: parents must be int32 [batch][T]")
    batch, T = shape = parents.shape
    ins = [_dense(t, shape, _I32, dev, what) for t in (parents, tokens, answers)]
    path = (_empty(shape, dtype=_I32, device=dev) if path is None else
            _given(path, shape, _I32, dev, what))
    n_path = (_empty((batch,), dtype=_I32, device=dev) if n_path is None else
              _given(n_path, (batch,), _I32, dev, what))
    next_token = (_empty((batch,), dtype=_I32, device=dev) if next_token is None else
                  _given(next_token, (batch,), _I32, dev, what))
    _launch(lib().lynx_tree_verify, what, dev, *ins, batch, T, path.data_ptr(), n_path.data_ptr(),
            next_token.data_ptr())
    return path, n_path, next_token


# ------------------------------------------------------ the paged cache's books

def _check_books(what, block_table, kv_len, refs):
    """block_table [batch][max_pages], kv_len [batch] and refs [num_blocks], int32,
    contiguous and on one device.  Returns it, their addresses and sizes."""
    dev = _cuda(block_table, what)
    if block_table.dim() != 2 or refs.dim() != 1:
        raise ValueError(f"{what}: block_table must be [batch][max_pages], refs [num_blocks]")
    batch, max_pages = shape = block_table.shape
    count = refs.shape
    return (dev, (_dense(block_table, shape, _I32, dev, what), _dense(kv_len, (batch,), _I32, dev, what),
                  _dense(refs, count, _I32, dev, what)), batch, max_pages, count[0])


def lynx_cache_fork(block_table, kv_len, refs, source, page: int, out_table=None, out_len=None):
    """Sequences that go on from others: output sequence i has the row and length of
    sequence source[i] (int32; negative: an empty one) and shares its pages; refs, changed
    in place, counts them and no longer counts the input's.  Returns (out_table, out_len)."""
    what = "lynx_cache_fork"
    dev, books, batch, max_pages, num_blocks = _check_books(what, block_table, kv_len, refs)
    if source.dim() != 1:
        raise ValueError(f"{what}: source must be int32 [out_batch]")
    n = source.shape[0]
    sp = _dense(source, (n,), _I32, dev, what)
    out_table = (_empty((n, max_pages), dtype=_I32, device=dev) if out_table is None else
                 _given(out_table, (n, max_pages), _I32, dev, what))
    out_len = (_empty((n,), dtype=_I32, device=dev) if out_len is None else
               _given(out_len, (n,), _I32, dev, what))
    _launch(lib().lynx_cache_fork, what, dev, *books, max_pages, num_blocks, page, batch, sp, n,
            out_table.data_ptr(), out_len.data_ptr())
    return out_table, out_len


def lynx_cache_reserve(block_table, kv_len, refs, grow, page: int, granted=None, copy_src=None,
                       copy_dst=None):
    """Room for grow[b] (int32) more tokens of each sequence; block_table, kv_len and refs
    are changed in place.  Returns (granted, copy_src, copy_dst), int32 [batch]: grow, or
    0 where the pages ran out, and the shared last pages to copy to pages of the
    sequence's own (lynx_cache_copy_pages; -1: none)."""
    what = "lynx_cache_reserve"
    dev, books, batch, max_pages, num_blocks = _check_books(what, block_table, kv_len, refs)
    gp = _dense(grow, (batch,), _I32, dev, what)
    granted = (_empty((batch,), dtype=_I32, device=dev) if granted is None else
               _given(granted, (batch,), _I32, dev, what))
    copy_src = (_empty((batch,), dtype=_I32, device=dev) if copy_src is None else
                _given(copy_src, (batch,), _I32, dev, what))
    copy_dst = (_empty((batch,), dtype=_I32, device=dev) if copy_dst is None else
                _given(copy_dst, (batch,), _I32, dev, what))
    _launch(lib().lynx_cache_reserve, what, dev, *books, max_pages, num_blocks, page, batch, gp,
            granted.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr())
    return granted, copy_src, copy_dst


def lynx_cache_trim(block_table, kv_len, refs, keep, page: int):
    """Cuts each sequence back to keep[b] tokens (int32; 0 frees it) and gives back the
    pages behind them; block_table, kv_len and refs are changed in place."""
    what = "lynx_cache_trim"
    dev, books, batch, max_pages, num_blocks = _check_books(what, block_table, kv_len, refs)
    kp = _dense(keep, (batch,), _I32, dev, what)
    _launch(lib().lynx_cache_trim, what, dev, *books, max_pages, num_blocks, page, batch, kp)


def lynx_cache_compact(block_table, kv_len, refs, page: int, copy_src=None, copy_dst=None,
                       count=None):
    """The pages in use to the front of the pools; block_table and refs are changed in
    place.  Returns (copy_src, copy_dst, count), int32 [num_blocks // 2] and [1]: the
    moves that lynx_cache_copy_pages has to make, and that a caller has to follow who
    holds a page without a sequence."""
    what = "lynx_cache_compact"
    dev, books, batch, max_pages, num_blocks = _check_books(what, block_table, kv_len, refs)
    copy_src = (_empty((num_blocks // 2,), dtype=_I32, device=dev) if copy_src is None else
                _given(copy_src, (num_blocks // 2,), _I32, dev, what))
    copy_dst = (_empty((num_blocks // 2,), dtype=_I32, device=dev) if copy_dst is None else
                _given(copy_dst, (num_blocks // 2,), _I32, dev, what))
    count = (_empty((1,), dtype=_I32, device=dev) if count is None else
             _given(count, (1,), _I32, dev, what))
    _launch(lib().lynx_cache_compact, what, dev, *books, max_pages, num_blocks, page, batch,
            copy_src.data_ptr(), copy_dst.data_ptr(), count.data_ptr())
    return copy_src, copy_dst, count


def lynx_cache_copy_pages(pools, copy_src, copy_dst, count=None):
    """Block copy_src[i] to block copy_dst[i] (int32) in each of the pools, tensors
    [num_blocks][...] of any type, for all i (with count, int32 [1]: for i < count);
    negative entries copy nothing."""
    what = "lynx_cache_copy_pages"
    n = len(pools)
    if not n:
        return
    dev = _cuda(copy_src, what)
    if copy_src.dim() != 1:
        raise ValueError(f"{what}: copy_src must be int32 [n]")
    sp = _dense(copy_src, copy_src.shape, _I32, dev, what)
    dp = _dense(copy_dst, copy_src.shape, _I32, dev, what)
    cp = None if count is None else _dense(count, (1,), _I32, dev, what)
    at, size = array.array("Q"), array.array("q")
    num_blocks = pools[0].shape[0] if pools[0].dim() else 0
    shape = kind = block = None
    for t in pools:
        if t.shape != shape or t.dtype != kind:
            shape, kind = t.shape, t.dtype
            block = t.numel() * t.element_size() // max(1, num_blocks)
            if not t.dim() or shape[0] != num_blocks:
                block = None
        if block is None or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: pools must be contiguous [{num_blocks}][...] on {dev}")
        at.append(t.data_ptr())
        size.append(block)
    _launch(lib().lynx_cache_copy_pages, what, dev, at.buffer_info()[0], size.buffer_info()[0], n,
            num_blocks, sp, dp, copy_src.shape[0], cp)


def lynx_cache_keep(nodes, pools, path, granted, kv_len, block_table):
    """The kept nodes' keys and values to the pages: nodes, a list of node buffers
    [batch][64][H_kv][D], and pools, as many pools [num_blocks][page][H_kv][D] (keys and
    values of all layers), BF16.  Row path[b][i] goes to position kv_len[b] - granted[b]
    + i, for i < granted[b]: path [batch][T] of lynx_tree_verify, granted and kv_len
    of lynx_cache_reserve.  Places of -1 in the path, and those behind it, are left as
    they are."""
    what = "lynx_cache_keep"
    n = len(pools)
    if n != len(nodes):
        raise ValueError(f"{what}: {len(nodes)} node buffers for {n} pools")
    if not n:
        return
    dev = _cuda(block_table, what)
    if block_table.dim() != 2 or path.dim() != 2 or pools[0].dim() != 4:
        raise ValueError(f"{what}: block_table must be [batch][max_pages], path [batch][T], pools "
                         "[num_blocks][page][H_kv][D]")
    batch, max_pages = block_table.shape
    shape = pools[0].shape
    num_blocks, page, H_kv, D = shape
    T = path.shape[1]
    bp = _dense(block_table, block_table.shape, _I32, dev, what)
    lp = _dense(kv_len, (batch,), _I32, dev, what)
    pp = _dense(path, (batch, T), _I32, dev, what)
    gp = _dense(granted, (batch,), _I32, dev, what)
    kind, one = torch.bfloat16, (batch, TREE_ROOM, H_kv, D)
    ins = array.array("Q", [_dense(t, one, kind, dev, what) for t in nodes])
    outs = array.array("Q", [_dense(t, shape, kind, dev, what) for t in pools])
    _launch(lib().lynx_cache_keep, what, dev, ins.buffer_info()[0], outs.buffer_info()[0], n, pp, gp,
            lp, bp, max_pages, num_blocks, batch, T, H_kv, D, page)


def lynx_compander_thresholds(alpha: float):
    buf = (ctypes.c_float * 127)()
    _check(lib().lynx_compander_thresholds(alpha, ctypes.cast(buf, ctypes.c_void_p)),
           "lynx_compander_thresholds")
    return list(buf)


def lynx_expand_table(alpha: float):
    buf = (ctypes.c_float * 128)()
    _check(lib().lynx_expand_table(alpha, ctypes.cast(buf, ctypes.c_void_p)),
           "lynx_expand_table")
    return list(buf)


def lynx_compander_selfcheck(alpha: float, device="cuda"):
    """[values checked, wrong unflagged, flagged, max |error| in 2^-32 of Y]."""
    counts = torch.zeros(4, dtype=torch.int64, device=device)
    _check(lib().lynx_compander_selfcheck(alpha, _ptr(counts), _stream(counts.device)),
           "lynx_compander_selfcheck")
    return [int(v) for v in counts.cpu().tolist()]


def lynx_wait_timeouts() -> int:
    flag = ctypes.c_uint()
    _check(lib().lynx_wait_timeouts(ctypes.byref(flag)), "lynx_wait_timeouts")
    return flag.value


def lynx_status_string(code: int) -> str:
    return lib().lynx_status_string(code).decode()


def lynx_last_error() -> str:
    return lib().lynx_last_error().decode(errors="replace")
