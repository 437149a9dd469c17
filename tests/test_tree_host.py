"""Refusals of tree drafting and of the paged cache's books: no GPU."""
import ctypes

import pytest

FAR = [ctypes.c_void_p((i + 1) << 40) for i in range(16)]   # apart, never dereferenced
BAD = ctypes.c_void_p(0x100002)


def _call(fn, names, base, over):
    a = dict(base)
    a.update(over)
    return fn(*(a[n] for n in names), None)


LOGPROBS = dict(x=FAR[0], dtype=1, stride=100, rows=3, V=100, scale=1.0, tokens=FAR[1], given=2,
                top=4, lp=FAR[2], h=FAR[3], tl=FAR[4], tt=FAR[5])


@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(rows=-1), -2), (dict(V=0), -2),
    (dict(rows=1 << 31), -3), (dict(V=1 << 31, stride=1 << 31), -3), (dict(stride=99), -2),
    (dict(stride=(1 << 40) + 1), -3),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(scale=1e-7), -1), (dict(scale=2e6), -1),
    (dict(given=-1), -2), (dict(given=65), -3), (dict(top=-1), -2), (dict(top=33), -3),
    (dict(top=9, V=8), -2), (dict(x=None), -1), (dict(x=BAD), -1), (dict(tokens=None), -1),
    (dict(lp=None), -1), (dict(tl=None), -1), (dict(tt=None), -1), (dict(tt=BAD), -1),
    (dict(h=BAD), -1), (dict(lp=FAR[1]), -1), (dict(h=FAR[0]), -1), (dict(tl=FAR[5]), -1),
    (dict(tt=ctypes.c_void_p((1 << 40) + 1196)), -1),
])
def test_logprobs_rejects(lynx_lib, over, code):
    assert _call(lynx_lib.lib().lynx_token_logprobs, LOGPROBS, LOGPROBS, over) == code, \
        lynx_lib.lynx_last_error()


def test_logprobs_takes_nothing_without_looking(lynx_lib):
    fn = lynx_lib.lib().lynx_token_logprobs
    assert _call(fn, LOGPROBS, LOGPROBS, dict(rows=0, x=None, lp=None)) == 0
    assert _call(fn, LOGPROBS, LOGPROBS, dict(given=0, top=0, h=None)) == 0


PLAN = dict(parents=FAR[0], kv=FAR[1], batch=2, T=8, mask=FAR[2], pos=FAR[3])
VERIFY = dict(parents=FAR[0], tokens=FAR[1], answers=FAR[2], batch=2, T=8, path=FAR[3], n=FAR[4],
              next=FAR[5])


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), -2), (dict(T=0), -2), (dict(T=65), -3), (dict(batch=1 << 26), -3),
    (dict(parents=None), -1), (dict(parents=BAD), -1)])
def test_trees_reject(lynx_lib, over, code):
    lib = lynx_lib.lib()
    assert _call(lib.lynx_tree_plan, PLAN, PLAN, over) == code
    assert _call(lib.lynx_tree_verify, VERIFY, VERIFY, over) == code


def test_trees_reject_their_own(lynx_lib):
    lib = lynx_lib.lib()
    for over in (dict(kv=None), dict(mask=ctypes.c_void_p(0x100004)), dict(pos=BAD),
                 dict(mask=FAR[0]), dict(pos=FAR[1]), dict(pos=FAR[2])):
        assert _call(lib.lynx_tree_plan, PLAN, PLAN, over) == -1
    for over in (dict(tokens=None), dict(answers=BAD), dict(path=None), dict(n=None),
                 dict(next=None), dict(path=FAR[0]), dict(n=FAR[5]), dict(next=FAR[2])):
        assert _call(lib.lynx_tree_verify, VERIFY, VERIFY, over) == -1
    assert _call(lib.lynx_tree_plan, PLAN, PLAN, dict(batch=0, parents=None)) == 0
    assert _call(lib.lynx_tree_plan, PLAN, PLAN, dict(mask=None, pos=None)) == 0
    assert _call(lib.lynx_tree_verify, VERIFY, VERIFY, dict(batch=0, path=None)) == 0


BOOKS = dict(table=FAR[0], kv=FAR[1], refs=FAR[2], max_pages=4, blocks=9, page=64, batch=2)
FORK = dict(BOOKS, source=FAR[3], out_batch=3, out_table=FAR[4], out_len=FAR[5])
RESERVE = dict(BOOKS, grow=FAR[3], granted=FAR[4], src=FAR[5], dst=FAR[6])
TRIM = dict(BOOKS, keep=FAR[3])
COMPACT = dict(BOOKS, src=FAR[4], dst=FAR[5], count=FAR[6])
CALLS = {"fork": FORK, "reserve": RESERVE, "trim": TRIM, "compact": COMPACT}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(page=32), -3), (dict(page=96), -3), (dict(page=1024), -3), (dict(max_pages=0), -2),
    (dict(blocks=0), -2), (dict(blocks=1 << 25), -3), (dict(max_pages=1 << 25), -3),
    (dict(batch=-1), -2), (dict(batch=1 << 29), -3), (dict(table=None), -1), (dict(kv=BAD), -1),
    (dict(refs=None), -1), (dict(refs=BAD), -1), (dict(refs=FAR[0]), -1), (dict(kv=FAR[2]), -1)])
def test_books_reject(lynx_lib, name, over, code):
    fn = getattr(lynx_lib.lib(), "lynx_cache_" + name)
    assert _call(fn, CALLS[name], CALLS[name], over) == code, lynx_lib.lynx_last_error()


def test_books_reject_their_own(lynx_lib):
    lib = lynx_lib.lib()
    for over in (dict(source=None), dict(out_table=None), dict(out_len=BAD), dict(out_table=FAR[0]),
                 dict(out_len=FAR[1]), dict(source=FAR[4])):
        assert _call(lib.lynx_cache_fork, FORK, FORK, over) == -1
    assert _call(lib.lynx_cache_fork, FORK, FORK, dict(out_batch=-1)) == -2
    for k in ("grow", "granted", "src", "dst"):
        for v in (None, BAD, FAR[1]):
            assert _call(lib.lynx_cache_reserve, RESERVE, RESERVE, {k: v}) == -1
    for v in (None, BAD, FAR[0], FAR[2]):
        assert _call(lib.lynx_cache_trim, TRIM, TRIM, dict(keep=v)) == -1
    for k in ("src", "dst", "count"):
        for v in (None, BAD, FAR[2]):
            assert _call(lib.lynx_cache_compact, COMPACT, COMPACT, {k: v}) == -1
    assert _call(lib.lynx_cache_fork, FORK, FORK, dict(batch=0, out_batch=0, refs=None)) == 0
    assert _call(lib.lynx_cache_reserve, RESERVE, RESERVE, dict(batch=0, grow=None)) == 0
    assert _call(lib.lynx_cache_trim, TRIM, TRIM, dict(batch=0, keep=None)) == 0


def _many(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*[None if p is None else p.value for p in ptrs])


def _copy(lib, pools=(FAR[0], FAR[1]), size=(4096, 16), n_pools=None, blocks=9, src=FAR[2],
          dst=FAR[3], n=4, count=FAR[4]):
    return lib.lynx_cache_copy_pages(_many(pools), (ctypes.c_int64 * len(size))(*size),
                                     len(pools) if n_pools is None else n_pools, blocks, src, dst, n,
                                     count, None)


def test_copy_pages_rejects(lynx_lib):
    lib = lynx_lib.lib()
    inside = ctypes.c_void_p((1 << 40) + 4096)
    for over, code in (
            (dict(n=-1), -2), (dict(n_pools=-1), -2), (dict(n_pools=257), -3), (dict(blocks=0), -2),
            (dict(blocks=1 << 31), -3), (dict(n=1 << 31), -3), (dict(src=None), -1),
            (dict(dst=BAD), -1), (dict(count=BAD), -1), (dict(pools=(FAR[0], None)), -1),
            (dict(pools=(FAR[0], ctypes.c_void_p(0x100008))), -1), (dict(size=(4096, 24)), -2),
            (dict(size=(0, 16)), -2), (dict(size=((1 << 36) + 16, 16)), -3),
            (dict(pools=(FAR[0], FAR[0])), -1), (dict(pools=(FAR[0], inside)), -1),
            (dict(pools=(inside, FAR[0]), size=(16, 4096)), -1), (dict(src=inside), -1), (dict(count=FAR[1]), -1)):
        assert _copy(lib, **over) == code, (over, lynx_lib.lynx_last_error())
    assert _copy(lib, n=0, src=None) == 0
    assert _copy(lib, pools=(), size=(), src=None) == 0
    assert lib.lynx_cache_copy_pages(None, None, 2, 9, FAR[2], FAR[3], 4, None, None) == -1


def _keep(lib, nodes=(FAR[0], FAR[1]), pools=(FAR[2], FAR[3]), n_pools=2, path=FAR[4],
          granted=FAR[5], kv=FAR[6], table=FAR[7], max_pages=4, blocks=9, batch=2, T=8, H_kv=2,
          D=128, page=64):
    return lib.lynx_cache_keep(_many(nodes), _many(pools), n_pools, path, granted, kv, table,
                               max_pages, blocks, batch, T, H_kv, D, page, None)


def test_keep_rejects(lynx_lib):
    lib = lynx_lib.lib()
    for over, code in (
            (dict(D=64), -3), (dict(page=96), -3), (dict(H_kv=0), -2), (dict(batch=-1), -2),
            (dict(T=0), -2), (dict(T=65), -3), (dict(blocks=0), -2), (dict(max_pages=0), -2),
            (dict(blocks=1 << 25), -3), (dict(n_pools=-1), -2), (dict(n_pools=257), -3),
            (dict(path=None), -1), (dict(granted=BAD), -1), (dict(kv=None), -1),
            (dict(table=None), -1), (dict(nodes=(FAR[0], None)), -1),
            (dict(pools=(ctypes.c_void_p(0x100008), FAR[3])), -1), (dict(pools=(FAR[2], FAR[2])), -1),
            (dict(pools=(FAR[0], FAR[3])), -1), (dict(nodes=(FAR[3], FAR[1])), -1),
            (dict(path=FAR[2]), -1), (dict(table=FAR[3]), -1)):
        assert _keep(lib, **over) == code, (over, lynx_lib.lynx_last_error())
    assert _keep(lib, batch=0, path=None) == 0
    assert _keep(lib, n_pools=0, path=None) == 0
    # what is only read may be shared: keys and values of one buffer are the caller's affair
    assert _keep(lib, nodes=(FAR[0], FAR[0]), pools=(FAR[2], FAR[2])) == -1


def test_binding_rejects_what_the_pointers_would_hide(lynx_lib):
    """CPU tensors and other shapes are refused before anything is launched."""
    import torch
    lynx = lynx_lib
    i = torch.zeros((2, 4), dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    refs = torch.zeros(9, dtype=torch.int32)
    for call in (lambda: lynx.lynx_token_logprobs(torch.zeros((2, 9))),
                 lambda: lynx.lynx_tree_plan(i, one), lambda: lynx.lynx_tree_verify(i, i, i),
                 lambda: lynx.lynx_cache_fork(i, one, refs, one, 64),
                 lambda: lynx.lynx_cache_reserve(i, one, refs, one, 64),
                 lambda: lynx.lynx_cache_trim(i, one, refs, one, 64),
                 lambda: lynx.lynx_cache_compact(i, one, refs, 64),
                 lambda: lynx.lynx_cache_copy_pages([refs], one, one),
                 lambda: lynx.lynx_cache_keep([refs], [refs], i, one, one, i),
                 lambda: lynx.lynx_cache_keep([], [refs], i, one, one, i)):
        with pytest.raises(ValueError):
            call()


TREE = dict(q=FAR[0], q_stride=4096, batch=2, T=3, H_q=32, kn=FAR[1], vn=FAR[2], mask=FAR[3],
            k_pool=FAR[4], v_pool=FAR[5], table=FAR[6], max_pages=4, blocks=9, kv=FAR[7], H_kv=8,
            D=128, page=64, score=None, out=FAR[8], lse=FAR[9], ws=FAR[10], ws_bytes=1 << 40)


@pytest.mark.parametrize("over,code", [
    (dict(T=0), -2), (dict(T=65), -3), (dict(batch=-1), -2), (dict(batch=1 << 26), -3),
    (dict(D=64), -3), (dict(page=96), -3), (dict(H_q=30), -2), (dict(H_kv=0), -2),
    (dict(q_stride=2048), -2), (dict(blocks=1 << 25), -3), (dict(max_pages=0), -2),
    (dict(mask=None), -1), (dict(mask=ctypes.c_void_p(0x100004)), -1), (dict(kn=None), -1),
    (dict(vn=ctypes.c_void_p(0x100008)), -1), (dict(q=None), -1), (dict(kv=BAD), -1),
    (dict(out=FAR[1]), -1), (dict(out=FAR[3]), -1), (dict(lse=FAR[2]), -1), (dict(lse=FAR[8]), -1),
    (dict(ws=None, max_pages=99), -1), (dict(ws_bytes=0, max_pages=99), -5),
    (dict(ws=FAR[3], max_pages=99), -1)])
def test_tree_attention_rejects(lynx_lib, over, code):
    assert _call(lynx_lib.lib().lynx_cache_attn_tree, TREE, TREE, over) == code, \
        lynx_lib.lynx_last_error()


def test_tree_attention_takes_nothing_without_looking(lynx_lib):
    assert _call(lynx_lib.lib().lynx_cache_attn_tree, TREE, TREE, dict(batch=0, mask=None)) == 0
    n = lynx_lib.lynx_cache_attn_tree_workspace_bytes(2, 3, 32, 8, 128, 64, 99)
    assert n == lynx_lib.lynx_cache_attn_decode_workspace_bytes(2, 3, 32, 8, 128, 64, 99) > 0
    with pytest.raises(lynx_lib.LynxError):
        lynx_lib.lynx_cache_attn_tree_workspace_bytes(2, 65, 32, 8, 128, 64, 99)


def test_what_smoke_holds_against_a_tree():
    """Right outputs pass; wrong masks, tokens and probabilities do not."""
    import numpy as np
    import torch

    import __graft_entry__ as entry
    rng = np.random.default_rng(1)
    bf = lambda *s: torch.tensor(rng.standard_normal(s)).to(torch.bfloat16).float().numpy()  # noqa: E731
    q, k, v, kn, vn = bf(3, 4, 128), bf(70, 2, 128), bf(70, 2, 128), bf(3, 2, 128), bf(3, 2, 128)
    masks, x = [1, 3, 5], rng.standard_normal(500).astype(np.float32)
    z = x - np.log(np.exp(x.astype(np.float64)).sum())
    order = np.argsort(-z)[:2]

    def attend(masks):
        rows = []
        for t, m in enumerate(masks):
            seen = [i for i in range(3) if m >> i & 1]
            for h in range(4):
                K = torch.tensor(np.concatenate((k[:, h // 2], kn[seen, h // 2]))).double()
                V = torch.tensor(np.concatenate((v[:, h // 2], vn[seen, h // 2]))).double()
                rows.append((K @ torch.tensor(q[t, h]).double() / 128 ** 0.5).softmax(0) @ V)
        return torch.stack(rows).view(3, 4, 128).to(torch.bfloat16).float().numpy()

    top = (-(np.exp(z) * z).sum(), z[order], list(order))
    entry.check_tree_outputs(x, top, masks, q, k, v, kn, vn, attend(masks))
    for bad, m in (((top[0] + 1e-3, *top[1:]), masks), ((top[0], top[1] + 1e-3, top[2]), masks),
                   ((*top[:2], top[2][::-1]), masks), (top, [1, 3, 7]), (top, [1, 2, 5])):
        with pytest.raises(AssertionError):
            entry.check_tree_outputs(x, bad, m, q, k, v, kn, vn, attend(masks))
