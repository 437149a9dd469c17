"""Refusals of the BF16 paged cache's calls, and their host-only parts: no GPU."""
import ctypes

import pytest

OK = ctypes.c_void_p(0x100000)          # aligned, never dereferenced: each call fails first
FAR = [ctypes.c_void_p((i + 1) << 40) for i in range(12)]   # apart from one another
BAD = ctypes.c_void_p(0x100008)


def _append(lib, lynx, **over):
    a = dict(k=FAR[0], k_stride=1024, v=FAR[1], v_stride=1024, q=FAR[2], q_stride=4096,
             q_out=FAR[3], off=FAR[4], kv=FAR[5], table=FAR[6], max_pages=4, blocks=9, batch=2,
             n=3, H_q=32, H_kv=8, D=128, page=64, rope=None, k_pool=FAR[7], v_pool=FAR[8])
    a.update(over)
    return lib.lynx_cache_append(a["k"], a["k_stride"], a["v"], a["v_stride"], a["q"],
                                 a["q_stride"], a["q_out"], a["off"], a["kv"], a["table"],
                                 a["max_pages"], a["blocks"], a["batch"], a["n"], a["H_q"],
                                 a["H_kv"], a["D"], a["page"],
                                 None if a["rope"] is None else ctypes.byref(a["rope"]),
                                 a["k_pool"], a["v_pool"], None)


@pytest.mark.parametrize("over,code", [
    (dict(D=64), -3), (dict(page=32), -3), (dict(page=1024), -3), (dict(page=96), -3),
    (dict(H_kv=0), -2), (dict(H_q=0), -2), (dict(batch=-1), -2), (dict(n=-1), -2),
    (dict(max_pages=0), -2), (dict(blocks=0), -2),
    (dict(blocks=1 << 25), -3),               # num_blocks * page = 2^31
    (dict(max_pages=1 << 25), -3), (dict(n=1 << 31), -3), (dict(batch=1 << 27), -3),
    (dict(k_stride=1016), -2), (dict(k_stride=1028), -2), (dict(v_stride=0), -2),
    (dict(q_stride=4088), -2),
    (dict(k=None), -1), (dict(v=BAD), -1), (dict(q_out=None), -1), (dict(q_out=BAD), -1),
    (dict(off=None), -1), (dict(kv=ctypes.c_void_p(0x100002)), -1), (dict(table=None), -1),
    (dict(k_pool=None), -1), (dict(v_pool=BAD), -1),
    (dict(v_pool=FAR[7]), -1),                # one pool for both
    (dict(q_out=FAR[0]), -1),                 # queries over the keys
    (dict(k=FAR[7]), -1),                     # keys inside the pool
    (dict(q_out=FAR[2], q_stride=6144), -1),  # in place, but not dense
    (dict(q_out=ctypes.c_void_p((3 << 40) + 16)), -1),
])
def test_append_rejects(lynx_lib, over, code):
    assert _append(lynx_lib.lib(), lynx_lib, **over) == code, lynx_lib.lynx_last_error()


def test_append_takes_nothing_without_looking(lynx_lib):
    lib = lynx_lib.lib()
    assert _append(lib, lynx_lib, n=0, k=None, off=None) == 0
    assert _append(lib, lynx_lib, batch=0, k=None, off=None) == 0


@pytest.mark.parametrize("rot,axes,axis,inter,freq,pos,code", [
    (24, 1, None, 0, 1.0, None, -3),          # not a multiple of 16
    (144, 1, None, 0, 1.0, None, -3), (-16, 1, None, 0, 1.0, None, -3),
    (64, 0, None, 0, 1.0, None, -3), (64, 5, [0] * 32, 0, 1.0, OK, -3),
    (64, 2, [0, 1] * 16, 0, 1.0, None, -1),   # two axes, no positions
    (64, 2, None, 0, 1.0, OK, -1),
    (64, 2, [0, 2] * 16, 0, 1.0, OK, -1),     # an axis that is not there
    (64, 1, None, 2, 1.0, None, -1),
    (64, 1, None, 0, float("nan"), None, -1), (64, 1, None, 0, float("inf"), None, -1),
    (64, 1, None, 0, 1.0, ctypes.c_void_p(0x100002), -1),
])
def test_append_rejects_rotations(lynx_lib, rot, axes, axis, inter, freq, pos, code):
    f = (ctypes.c_double * 72)(*([1.0] * 72))
    f[7] = freq
    ax = None if axis is None else (ctypes.c_uint8 * len(axis))(*axis)
    r = lynx_lib.LynxRope(rot, inter, axes, 0, ctypes.addressof(f),
                          None if ax is None else ctypes.addressof(ax),
                          None if pos is None else pos.value)
    assert _append(lynx_lib.lib(), lynx_lib, rope=r) == code, lynx_lib.lynx_last_error()


def _attn(lib, prefill=False, score=None, **over):
    a = dict(q=FAR[0], q_stride=4096, off=FAR[1], n=6, batch=2, T=3, H_q=32, k_pool=FAR[2],
             v_pool=FAR[3], table=FAR[4], max_pages=4, blocks=9, kv=FAR[5], H_kv=8, D=128,
             page=64, out=FAR[6], lse=FAR[7], ws=FAR[8], ws_bytes=1 << 40)
    a.update(over)
    tail = (a["k_pool"], a["v_pool"], a["table"], a["max_pages"], a["blocks"], a["kv"], a["H_kv"],
            a["D"], a["page"], None if score is None else ctypes.byref(score), a["out"], a["lse"],
            a["ws"], a["ws_bytes"], None)
    if prefill:
        return lib.lynx_cache_attn_prefill(a["q"], a["q_stride"], a["off"], a["n"], a["batch"],
                                           a["H_q"], *tail)
    return lib.lynx_cache_attn_decode(a["q"], a["q_stride"], a["batch"], a["T"], a["H_q"], *tail)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(D=256), -3), (dict(page=16), -3), (dict(H_q=30), -2), (dict(H_q=0), -2),
    (dict(H_kv=0), -2), (dict(q_stride=2048), -2), (dict(q_stride=4100), -2),
    (dict(batch=-1), -2), (dict(blocks=1 << 25), -3), (dict(max_pages=0), -2),
    (dict(q=None), -1), (dict(q=BAD), -1), (dict(k_pool=None), -1), (dict(table=None), -1),
    (dict(kv=None), -1), (dict(out=None), -1), (dict(lse=ctypes.c_void_p(0x100002)), -1),
    (dict(out=FAR[0]), -1), (dict(out=FAR[2]), -1), (dict(lse=FAR[6]), -1),
    # a workspace is needed where contexts may be long
    (dict(ws=None, max_pages=99), -1), (dict(ws_bytes=0, max_pages=99), -5),
    (dict(ws=FAR[3], max_pages=99), -1), (dict(ws=FAR[6], max_pages=99), -1),
])
def test_attention_rejects(lynx_lib, prefill, over, code):
    assert _attn(lynx_lib.lib(), prefill, **over) == code, lynx_lib.lynx_last_error()


def test_attention_rejects_its_own(lynx_lib):
    lib = lynx_lib.lib()
    assert _attn(lib, T=0) == -2
    assert _attn(lib, T=65) == -3
    assert _attn(lib, True, off=None) == -1
    assert _attn(lib, True, n=-1) == -2
    assert _attn(lib, True, n=0, q=None) == 0
    assert _attn(lib, batch=0, q=None) == 0
    need = lynx_lib.lynx_cache_attn_decode_workspace_bytes(2, 3, 32, 8, 128, 64, 99)
    assert need > 0
    assert _attn(lib, max_pages=99, ws_bytes=need - 1) == -5
    need = lynx_lib.lynx_cache_attn_prefill_workspace_bytes(6, 2, 32, 8, 128, 64, 99)
    assert need > 0
    assert _attn(lib, True, max_pages=99, ws_bytes=need - 1) == -5
    # short contexts and whole prompts need none
    assert lynx_lib.lynx_cache_attn_decode_workspace_bytes(2, 3, 32, 8, 128, 64, 16) == 0
    assert lynx_lib.lynx_cache_attn_prefill_workspace_bytes(6, 2, 32, 8, 128, 64, 16) == 0
    assert lynx_lib.lynx_cache_attn_prefill_workspace_bytes(9000, 2, 32, 8, 128, 64, 99) == 0


@pytest.mark.parametrize("kw", [
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
    dict(window=-1), dict(slopes=0x100002), dict(prefix=0x100001)])
def test_attention_rejects_scores(lynx_lib, kw):
    a = dict(scale=0.1, softcap=0.0, window=0, slopes=None, prefix=None)
    a.update(kw)
    score = lynx_lib.LynxScore(a["scale"], a["softcap"], a["window"], a["slopes"], a["prefix"])
    for prefill in (False, True):
        assert _attn(lynx_lib.lib(), prefill, score) == -1, lynx_lib.lynx_last_error()


def test_workspace_bytes_rejects(lynx_lib):
    for bad in (dict(batch=-1), dict(H_q=7), dict(H_kv=0), dict(D=64), dict(page=32),
                dict(max_pages=0), dict(T=0), dict(T=65)):
        a = dict(batch=1, T=1, H_q=8, H_kv=2, D=128, page=64, max_pages=9)
        a.update(bad)
        with pytest.raises(lynx_lib.LynxError):
            lynx_lib.lynx_cache_attn_decode_workspace_bytes(**a)
        if "T" in bad:
            continue
        del a["T"]
        with pytest.raises(lynx_lib.LynxError):
            lynx_lib.lynx_cache_attn_prefill_workspace_bytes(n_tokens=5, **a)
    with pytest.raises(lynx_lib.LynxError):
        lynx_lib.lynx_cache_attn_prefill_workspace_bytes(-1, 1, 8, 2, 128, 64, 9)


def test_binding_rejects_what_the_pointers_would_hide(lynx_lib):
    """Shapes, types, strides and devices, before anything is launched (CPU
    tensors are refused first, so the helpers are called themselves)."""
    import torch
    lynx = lynx_lib
    dev = torch.device("cpu")
    bf = torch.bfloat16
    rows = torch.zeros((4, 8, 128), dtype=bf)
    assert lynx._token_rows(rows, 8, "t", dev) == (4, 8, 1024)
    fused = torch.zeros((4, 48, 128), dtype=bf)
    assert lynx._token_rows(fused[:, 32:40], 8, "t", dev) == (4, 8, 6144)
    assert lynx._token_rows(fused[:1, 32:40], 8, "t", dev) == (1, 8, 1024)
    for bad in (rows.float(), rows[0], rows[:, :7], rows.expand(4, 8, 128).transpose(0, 1),
                rows[:1].expand(4, 8, 128), torch.zeros((4, 8, 256), dtype=bf)[..., ::2],
                torch.zeros(4 * 1026, dtype=bf).as_strided((4, 8, 128), (1026, 128, 1))):
        with pytest.raises(ValueError):
            lynx._token_rows(bad, 8, "t", dev)
    with pytest.raises(ValueError):
        lynx._token_rows(rows, 8, "t", torch.device("meta"))
    for bad in (rows.float(), rows[:3], rows.transpose(0, 1), fused[:, :8]):
        with pytest.raises(ValueError):
            lynx._dense(bad, (4, 8, 128), bf, dev, "t")
    with pytest.raises(ValueError):
        lynx._dense(rows, (4, 8, 128), bf, torch.device("meta"), "t")
    pool = torch.zeros((3, 64, 8, 128), dtype=bf)
    with pytest.raises(ValueError):         # not CUDA tensors
        lynx._check_cache("t", pool, pool.clone(), torch.zeros((1, 2), dtype=torch.int32),
                          torch.zeros(1, dtype=torch.int32))
    q = torch.zeros((3, 2, 8, 128), dtype=bf)
    for bad in (q[0], q[:, :0], q.expand(3, 2, 8, 128).transpose(0, 1), q.transpose(2, 3),
                torch.zeros((3, 4, 8, 128), dtype=bf)[:, :2],          # tokens unevenly spaced
                q[:1].expand(3, 2, 8, 128), q[:, :1].expand(3, 2, 8, 128)):
        with pytest.raises(ValueError, match="q must be|no token|evenly|contiguous"):
            lynx.lynx_cache_attn_decode(bad, pool, pool, torch.zeros((3, 2), dtype=torch.int32),
                                        torch.zeros(3, dtype=torch.int32))
    for args in (([1.0], [0, 1]), ([1.0], [300]), ([1.0], [-1])):
        with pytest.raises(ValueError):
            lynx.Rope(*args)
    assert lynx.Rope(lynx.rope_frequencies(1e4, 64), [0, 1] * 16).n_axes == 2
    assert lynx.rope_frequencies(1e4, 4) == [1.0, 0.01]
