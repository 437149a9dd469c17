"""The BF16 paged cache on the GPU: append, decode and prefill attention against
the definitions in 64 bits (tests/cache_plain.py has them and the bounds), and
a run of them together with the codec."""
import functools
import math
import os
import subprocess
import sys

import pytest
import torch

from . import cache_plain as plain

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN = float("nan")


def own_process(fn):
    """Runs a test in a process of its own: the error words it sets are never
    reset, and other tests look for them."""
    @functools.wraps(fn)
    def run(lynx_lib, cuda_dev):
        if os.environ.get("LYNX_TEST_CHILD"):
            return fn(lynx_lib, cuda_dev)
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
                            f"{os.path.abspath(__file__)}::{fn.__name__}"],
                           env=dict(os.environ, LYNX_TEST_CHILD="1"), capture_output=True,
                           text=True, timeout=600)
        assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
    return run


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x[..., 3::29] *= 4.0                      # a few channels are large
    return x.to(BF)


def _cache(kv, page, H_kv, seed, spare=3, max_pages=None):
    """Pools that hold NaN wherever no token lies, table, lengths (CPU)."""
    table, blocks = plain.table_for(kv, page, spare, seed, max_pages)
    pools = []
    for i in range(2):
        p = torch.full((blocks, page, H_kv, 128), NAN, dtype=BF)
        for b, n in enumerate(kv):
            if n > 0:
                at = torch.arange(n)
                p[table[b].long()[at // page], at % page] = _rand((n, H_kv, 128), seed + 7 * b + i)
        pools.append(p)
    return pools[0], pools[1], table, torch.tensor(kv, dtype=torch.int32)


# ----------------------------------------------------------------- append

APPEND = [
    # counts, kv, H_q, H_kv, page, rot, axes, interleaved
    ([1], [1], 1, 1, 64, 128, 1, False),
    ([1], [777], 32, 8, 64, 128, 1, False),
    ([0, 3, 0, 130, 1, 0], [0, 3, 9, 131, 65, 0], 8, 2, 64, 64, 1, True),
    ([513, 7], [513, 600], 6, 3, 512, 96, 3, True),
    ([100, 29], [229, 29], 5, 5, 128, 112, 2, False),
    ([17], [300], 40, 8, 256, 0, 1, False),
    ([1] * 70, [37 * i + 1 for i in range(70)], 4, 2, 128, 16, 4, False),
]


@pytest.mark.parametrize("counts,kv,H_q,H_kv,page,rot,axes,inter", APPEND)
def test_append_matches_the_definition(lynx_lib, cuda_dev, counts, kv, H_q, H_kv, page, rot, axes,
                                       inter):
    n = sum(counts)
    kp, vp, table, lens = _cache(kv, page, H_kv, seed=n)
    fused = _rand((n + 3, H_q + 2 * H_kv, 128), n + 1)       # three rows of padding
    q, k, v = fused[:, :H_q], fused[:, H_q:H_q + H_kv], fused[:, H_q + H_kv:]
    f = lynx_lib.rope_frequencies(1e4, rot)
    axis = [i % axes for i in range(rot // 2)] if axes > 1 else None
    pos = None
    if axes > 1:
        g = torch.Generator().manual_seed(n)
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (axes, n + 3), generator=g).to(torch.int32)
    want = plain.append(k[:n], v[:n], counts, kv, table, kp, vp, q[:n], f, axis, inter,
                        None if pos is None else pos[:, :n])
    d = fused.to(cuda_dev)
    dk, dv = kp.to(cuda_dev), vp.to(cuda_dev)
    qo = torch.full((n + 3, H_q, 128), 7.0, dtype=BF, device=cuda_dev)
    got = lynx_lib.lynx_cache_append(
        d[:, H_q:H_q + H_kv], d[:, H_q + H_kv:], plain.offsets_of(counts).to(cuda_dev),
        lens.to(cuda_dev), table.to(cuda_dev), dk, dv, q=d[:, :H_q], q_out=qo,
        rope=lynx_lib.Rope(f, axis, inter), positions=None if pos is None else pos.to(cuda_dev))
    assert got is qo
    plain.assert_close(qo[:n], want[2], want[4], "q")
    assert (qo[n:] == 7.0).all(), "padding rows were written"
    plain.assert_close(dk, want[0], want[3], "k pool")
    # what no new token wrote stays bit for bit, the values are copied bit for bit
    old = want[3] == 0
    assert torch.equal(dk.cpu()[old].view(torch.int16), want[0].to(BF)[old].view(torch.int16))
    assert torch.equal(dv.cpu().view(torch.int16), want[1].to(BF).view(torch.int16))


def test_append_in_place_without_queries_and_without_rotation(lynx_lib, cuda_dev):
    kp, vp, table, lens = _cache([70], 64, 2, seed=5)
    k, v, q = (_rand((70, h, 128), s).to(cuda_dev) for h, s in ((2, 1), (2, 2), (4, 3)))
    off = plain.offsets_of([70]).to(cuda_dev)
    args = (off, lens.to(cuda_dev), table.to(cuda_dev))
    a, b = kp.to(cuda_dev), vp.to(cuda_dev)
    assert lynx_lib.lynx_cache_append(k, v, *args, a, b) is None
    at = torch.arange(70)
    where = table[0].long()[at // 64], at % 64
    assert torch.equal(a.cpu()[where], k.cpu()) and torch.equal(b.cpu()[where], v.cpu())
    rope = lynx_lib.Rope(lynx_lib.rope_frequencies(1e6, 128))
    apart = lynx_lib.lynx_cache_append(k, v, *args, a, b, q=q, rope=rope)
    lynx_lib.lynx_cache_append(k, v, *args, a, b, q=q, q_out=q, rope=rope)
    assert torch.equal(q, apart)


@own_process
def test_append_leaves_out_what_has_no_slot(lynx_lib, cuda_dev):
    """Tokens at negative positions, beyond the table, or behind a bad entry are
    left out (the last two reported); the others arrive."""
    errors = lynx_lib.lynx_device_errors() & ~2
    counts, kv, page = [5, 4, 3], [3, 130, 66], 64
    table = torch.tensor([[0, -7], [1, 2], [3, 9]], dtype=torch.int32)   # 6 blocks
    k, v = _rand((12, 1, 128), 1), _rand((12, 1, 128), 2)
    pool = torch.zeros((6, page, 1, 128), dtype=BF)
    want = plain.append(k, v, counts, kv, table, pool, pool)
    a, b = pool.to(cuda_dev), pool.to(cuda_dev)
    lynx_lib.lynx_cache_append(k.to(cuda_dev), v.to(cuda_dev),
                               plain.offsets_of(counts).to(cuda_dev),
                               torch.tensor(kv, dtype=torch.int32).to(cuda_dev),
                               table.to(cuda_dev), a, b)
    assert torch.equal(a.cpu().double(), want[0]) and torch.equal(b.cpu().double(), want[1])
    assert lynx_lib.lynx_device_errors() == errors | 2


# ----------------------------------------------------------------- attention

def _attend(lynx, dev, q, counts, kv, page, H_kv, seed, decode, max_pages=None, **kw):
    """Runs the call and compares; q [n_tokens][H_q][D] on the CPU."""
    kp, vp, table, lens = _cache(kv, page, H_kv, seed, max_pages=max_pages)
    want = plain.attention(q, counts, kv, table, kp, vp, **kw)
    on = {k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in kw.items()}
    pad = 0 if decode else 2
    shape = (len(counts), counts[0]) + q.shape[1:] if decode else (len(q) + pad,) + q.shape[1:]
    dq = torch.cat((q, torch.ones((pad,) + q.shape[1:], dtype=BF))).to(dev).view(shape)
    out = torch.full(shape, 7.0, dtype=BF, device=dev)
    lse = torch.full(shape[:-1], 7.0, device=dev)
    args = (kp.to(dev), vp.to(dev), table.to(dev), lens.to(dev))
    if decode:
        lynx.lynx_cache_attn_decode(dq, *args, out=out, lse=lse, **on)
    else:
        lynx.lynx_cache_attn_prefill(dq, plain.offsets_of(counts).to(dev), *args, out=out,
                                     lse=lse, **on)
        assert (out[len(q):] == 7.0).all() and (lse[len(q):] == 7.0).all()
    plain.assert_close(lse.view(-1, q.shape[1])[:len(q)], want[1], want[3], "lse")
    plain.assert_close(out.view(-1, *q.shape[1:])[:len(q)], want[0], want[2], "out")
    return out, lse


DECODE = [
    # kv, T, H_q, H_kv, page
    ([1], 1, 1, 1, 64),
    ([0], 1, 4, 1, 64),
    ([63, 64, 65, 0, 1, 128, 129], 1, 8, 2, 64),
    ([3, 0, 700], 5, 8, 2, 64),                 # fewer cached tokens than new ones
    ([1000], 1, 32, 8, 64),
    ([4097, 511], 1, 40, 8, 512),               # five query heads a KV head
    ([300, 2049], 3, 14, 2, 256),               # 21 rows
    ([900, 901], 8, 8, 2, 128),                 # 32 rows
    ([777, 64, 1500], 8, 16, 2, 128),           # 64 rows
    ([650, 90], 64, 4, 2, 64),                  # 128 rows: two units a head
    ([500], 33, 3, 1, 64),                      # 99 rows
    ([90] * 161, 1, 2, 1, 64),                  # more sequences than a CTA has threads
    ([20000, 1], 1, 4, 1, 64),                  # long against short
    ([7000, 0, 2, 300], 48, 8, 1, 128),         # 384 rows on the many-row kernel
    ([300] * 45, 5, 8, 1, 64),                  # 40 rows, more units than clusters
]


def _table_pages(kv, page, wide):
    """A table with room for just the lengths (short contexts run as clusters), or
    for 8192 tokens at least (the split and its join)."""
    return max(8192, max(kv)) // page + 1 if wide else None


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kv,T,H_q,H_kv,page", DECODE)
def test_decode_matches_the_definition(lynx_lib, cuda_dev, kv, T, H_q, H_kv, page, wide):
    q = _rand((len(kv) * T, H_q, 128), 11, 2.0)
    _attend(lynx_lib, cuda_dev, q, [T] * len(kv), kv, page, H_kv, seed=3, decode=True,
            max_pages=_table_pages(kv, page, wide))


SCORES = [
    dict(softcap=20.0), dict(softcap=1e-7), dict(softcap=1e30), dict(window=1), dict(window=64), dict(window=200, prefix=5),
    dict(prefix=70), dict(slopes=True), dict(softcap=5.0, window=130, prefix=64, slopes=True),
    dict(scale=0.5), dict(window=10 ** 12), dict(prefix=10 ** 6),
]


def _score_args(kw, batch, H_q):
    kw = dict(kw)
    if kw.pop("slopes", None):
        kw["slopes"] = torch.tensor([2.0 ** -(1 + h % 8) for h in range(H_q)])
    if "prefix" in kw:
        # one of the sequences has none, one a negative one
        kw["prefix"] = torch.tensor([kw["prefix"] if b % 3 == 0 else -(b % 3 == 1)
                                     for b in range(batch)], dtype=torch.int32)
    return kw


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", SCORES)
@pytest.mark.parametrize("T,H_q,H_kv", [(1, 4, 2), (7, 6, 2)])
def test_decode_scores(lynx_lib, cuda_dev, kw, T, H_q, H_kv, wide):
    kv = [1, 130, 640, 4, 333, 1000]
    q = _rand((len(kv) * T, H_q, 128), 12, 2.0)
    _attend(lynx_lib, cuda_dev, q, [T] * len(kv), kv, 64, H_kv, seed=4, decode=True,
            max_pages=_table_pages(kv, 64, wide), **_score_args(kw, len(kv), H_q))


PREFILL = [
    # counts, kv, H_q, H_kv, page
    ([1], [1], 1, 1, 64),
    ([5, 0, 1, 64, 0, 130], [5, 9, 700, 64, 0, 131], 8, 2, 64),
    ([301, 33, 1], [301, 33, 1], 8, 8, 128),
    ([257], [1300], 10, 2, 256),
    ([40, 300], [20, 513], 5, 1, 512),          # twenty tokens at negative positions
    ([1000], [1000], 4, 1, 64),
    ([513, 700], [2000, 900], 16, 2, 128),
    ([3, 70, 0, 1], [9000, 5000, 20, 2500], 8, 2, 256),   # few rows, long caches
    ([1] * 40, [100 * i for i in range(40)], 4, 1, 64),
    ([i % 3 for i in range(700)], [i % 3 + i % 40 for i in range(700)], 4, 2, 64),
    ([1, 2, 1], [40000, 1, 3], 2, 1, 512),
    ([130], [4000], 4, 1, 64),
    ([30, 1, 50, 7], [2500, 700, 3000, 40], 40, 40, 256),  # the last units cut in parts
    ([30, 0, 50, 7], [3000, 5, 2100, 2], 40, 40, 512),     # of which some are not there
]


@pytest.mark.parametrize("counts,kv,H_q,H_kv,page", PREFILL)
def test_prefill_matches_the_definition(lynx_lib, cuda_dev, counts, kv, H_q, H_kv, page):
    q = _rand((sum(counts), H_q, 128), 13, 2.0)
    _attend(lynx_lib, cuda_dev, q, counts, kv, page, H_kv, seed=5, decode=False)


@pytest.mark.parametrize("kw", SCORES)
@pytest.mark.parametrize("counts,kv,H_q,H_kv", [
    ([60, 1, 131, 3], [60, 500, 200, 3], 8, 2), ([600, 290], [600, 700], 6, 2),
    ([2, 90], [4000, 1500], 8, 2),              # cut over the CTAs
    ([1, 7, 0, 33], [2300, 2500, 0, 130], 4, 1),
    ([9, 0, 20, 1], [2300, 5, 130, 900], 40, 40)])
def test_prefill_scores(lynx_lib, cuda_dev, kw, counts, kv, H_q, H_kv):
    q = _rand((sum(counts), H_q, 128), 14, 2.0)
    _attend(lynx_lib, cuda_dev, q, counts, kv, 64, H_kv, seed=6, decode=False,
            **_score_args(kw, len(counts), H_q))


def test_large_scores_and_rising_maxima(lynx_lib, cuda_dev):
    """Scores in the hundreds, the largest key last: every tile raises the
    maximum, and early weights vanish."""
    kv, page, H_kv, H_q = [640], 64, 1, 4
    kp, vp, table, lens = _cache(kv, page, H_kv, seed=8)
    at = torch.arange(640)
    where = table[0].long()[at // page], at % page
    kp[where] = (torch.ones(640, 1, 128) * (at / 640.0).view(-1, 1, 1)).to(BF)
    for T, call in ((1, "decode"), (300, "prefill")):
        q = torch.full((T, H_q, 128), 40.0, dtype=BF)
        want = plain.attention(q, [T], kv, table, kp, vp)
        args = [t.to(cuda_dev) for t in (kp, vp, table, lens)]
        lse = torch.empty((T, H_q), device=cuda_dev)
        if call == "decode":
            out = lynx_lib.lynx_cache_attn_decode(q.to(cuda_dev).view(1, T, H_q, 128), *args,
                                                  lse=lse.view(1, T, H_q))
        else:
            out = lynx_lib.lynx_cache_attn_prefill(q.to(cuda_dev),
                                                   plain.offsets_of([T]).to(cuda_dev), *args,
                                                   lse=lse)
        plain.assert_close(lse, want[1], want[3], call)
        plain.assert_close(out.view(T, H_q, 128), want[0], want[2], call)


@pytest.mark.parametrize("cap,reach", [(30.0, 0.3), (30.0, 0.495), (30.0, 0.51), (30.0, 20.0),
                                       (2.0, 0.7)])
def test_caps_below_and_above_their_polynomial(lynx_lib, cuda_dev, cap, reach):
    """Scores that reach `reach` caps: 0.5 is where the prefill kernel leaves the
    polynomial of the tanh for the exponential form."""
    kv, page, H_kv, H_q = [200, 130], 64, 1, 4
    kp, vp, table, lens = _cache(kv, page, H_kv, seed=22)
    q = _rand((330, H_q, 128), 6)
    top = 0.0
    for b, (n, t0) in enumerate(((200, 0), (130, 200))):
        k = plain.rows_of(kp, table, b, n, page)[:, 0]
        top = max(top, float((q[t0:t0 + n].double() @ k.T).abs().max()) / math.sqrt(128.0))
    scale = reach * cap / top / math.sqrt(128.0)
    kw = dict(scale=scale, softcap=cap)
    want = plain.attention(q, kv, kv, table, kp, vp, **kw)
    lse = torch.empty((330, H_q), device=cuda_dev)
    out = lynx_lib.lynx_cache_attn_prefill(
        q.to(cuda_dev), plain.offsets_of(kv).to(cuda_dev),
        *(t.to(cuda_dev) for t in (kp, vp, table, lens)), lse=lse, **kw)
    plain.assert_close(lse, want[1], want[3], "lse")
    plain.assert_close(out, want[0], want[2], "out")


@own_process
def test_strided_queries_bad_pages_and_pages_out_of_sight(lynx_lib, cuda_dev):
    kv, page, H_kv, H_q = [700, 256], 64, 2, 8
    kp, vp, table, lens = _cache(kv, page, H_kv, seed=9)
    fused = _rand((2, 1, H_q + 2 * H_kv, 128), 3, 2.0)
    want = plain.attention(fused[:, 0, :H_q], [1, 1], kv, table, kp, vp, window=100)
    # entries of pages that the window has left, and of pages behind the end
    table[0, :8] = -5
    table[1, :1] = 10 ** 6
    before = lynx_lib.lynx_device_errors()
    args = [t.to(cuda_dev) for t in (kp, vp, table, lens)]
    out = lynx_lib.lynx_cache_attn_decode(fused.to(cuda_dev)[:, :, :H_q], *args, window=100)
    plain.assert_close(out.view(2, H_q, 128), want[0], want[2], "out")
    assert lynx_lib.lynx_device_errors() == before
    # an entry that is needed and no page: page 0 is read and the call says so
    table[0, 10] = 10 ** 6
    broken = table.clone()
    broken[0, 10] = 0
    args[2] = table.to(cuda_dev)
    a = lynx_lib.lynx_cache_attn_decode(fused.to(cuda_dev)[:, :, :H_q], *args, window=100)
    args[2] = broken.to(cuda_dev)
    b = lynx_lib.lynx_cache_attn_decode(fused.to(cuda_dev)[:, :, :H_q], *args, window=100)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert lynx_lib.lynx_device_errors() == before | 2


def test_outputs_on_any_16_bytes(lynx_lib, cuda_dev):
    """Inputs and outputs that start 16 bytes past a larger alignment."""
    kv, page, H_kv, H_q, T = [300, 70], 64, 2, 6, 40
    kp, vp, table, lens = (t.to(cuda_dev) for t in _cache(kv, page, H_kv, seed=21))
    off = plain.offsets_of([T, T]).to(cuda_dev)
    q = _rand((2 * T, H_q, 128), 4).to(cuda_dev)

    def shifted(n):
        return torch.empty(n + 8, dtype=BF, device=cuda_dev)[8:]

    q2, o2 = (shifted(q.numel()).view(q.shape) for _ in range(2))
    q2.copy_(q)
    want = lynx_lib.lynx_cache_attn_prefill(q, off, kp, vp, table, lens)
    lynx_lib.lynx_cache_attn_prefill(q2, off, kp, vp, table, lens, out=o2)
    assert torch.equal(o2, want)
    q4 = q.view(2, T, H_q, 128)
    o2.zero_()
    want = lynx_lib.lynx_cache_attn_decode(q4, kp, vp, table, lens)
    lynx_lib.lynx_cache_attn_decode(q2.view(q4.shape), kp, vp, table, lens, out=o2.view(q4.shape))
    assert torch.equal(o2, want.view(q.shape))
    p2 = shifted(kp.numel()).view(kp.shape), shifted(kp.numel()).view(kp.shape)
    for a, b in zip(p2, (kp, vp)):
        a.copy_(b)
    got = lynx_lib.lynx_cache_attn_decode(q4, *p2, table, lens)
    assert torch.equal(got, want)
    n = 2 * T
    k = shifted(n * H_kv * 128).view(n, H_kv, 128)
    k.copy_(_rand((n, H_kv, 128), 9))
    lynx_lib.lynx_cache_append(k, k, off, lens, table, *p2, q=q2, q_out=o2)
    assert torch.equal(o2, q)


def test_lengths_beyond_the_table(lynx_lib, cuda_dev):
    """kv_len past the table's end counts as the table's end."""
    kv, page = [128], 64
    kp, vp, table, lens = _cache(kv, page, 1, seed=10)
    q = _rand((1, 2, 4, 128), 1)
    args = [t.to(cuda_dev) for t in (kp, vp, table)]
    a = lynx_lib.lynx_cache_attn_decode(q.to(cuda_dev), *args, lens.to(cuda_dev))
    far = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=cuda_dev)
    b = lynx_lib.lynx_cache_attn_decode(q.to(cuda_dev), *args, far)
    assert torch.equal(a, b)


def test_same_result_twice_on_streams_and_in_graphs(lynx_lib, cuda_dev):
    """Bit for bit: again, on another stream, and replayed by a graph whose
    lengths, tables and values changed after the capture."""
    kv, page, H_kv, H_q, T = [900, 70, 2300], 64, 2, 8, 2
    kp, vp, table, lens = (t.to(cuda_dev) for t in _cache(kv, page, H_kv, seed=20, max_pages=80))
    q = _rand((3, T, H_q, 128), 2, 2.0).to(cuda_dev)
    off = plain.offsets_of([T] * 3).to(cuda_dev)
    rope = lynx_lib.Rope(lynx_lib.rope_frequencies(1e6, 128))
    k, v = (_rand((3 * T, H_kv, 128), s).to(cuda_dev) for s in (3, 4))
    ws = torch.empty(max(lynx_lib.lynx_cache_attn_decode_workspace_bytes(3, T, H_q, H_kv, 128, page,
                                                                         table.shape[1]),
                         lynx_lib.lynx_cache_attn_prefill_workspace_bytes(3 * T, 3, H_q, H_kv, 128,
                                                                          page, table.shape[1])),
                     dtype=torch.uint8, device=cuda_dev)
    assert ws.numel() > 0
    qr, out, pre = (torch.empty_like(q) for _ in range(3))

    def step():
        lynx_lib.lynx_cache_append(k, v, off, lens, table, kp, vp, q=q.view(-1, H_q, 128),
                                   q_out=qr.view(-1, H_q, 128), rope=rope)
        lynx_lib.lynx_cache_attn_decode(qr, kp, vp, table, lens, out=out, workspace=ws)
        lynx_lib.lynx_cache_attn_prefill(qr.view(-1, H_q, 128), off, kp, vp, table, lens,
                                         out=pre.view(-1, H_q, 128), workspace=ws)

    step()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # the next tokens, and a page that has moved (within the table of 80)
    blocks = kp.shape[0]
    lens.copy_(torch.tensor([902, 72, 2302], dtype=torch.int32))
    for pool in (kp, vp):
        pool[blocks - 1] = pool[table[1, 0].long()]
    table[1, 0] = blocks - 1
    q.mul_(0.5)
    graph.replay()
    replayed = out.clone(), pre.clone()
    out.zero_()
    pre.zero_()
    step()
    assert torch.equal(out, replayed[0]) and torch.equal(pre, replayed[1])
    assert torch.isfinite(out).all() and torch.isfinite(pre).all()
    assert not torch.equal(out, first)


def test_behind_copies_and_other_streams_in_a_graph(lynx_lib, cuda_dev):
    """The calls are launched as programmatic dependents: captured right behind a
    copy, a memset, or work of another stream, they must see what it wrote, and
    what follows must see theirs."""
    kv, page, H_kv, H_q = [900, 70, 2300], 64, 2, 8
    kp, vp, table, lens = (t.to(cuda_dev) for t in _cache(kv, page, H_kv, seed=40))
    q = _rand((3, 1, H_q, 128), 2, 2.0).to(cuda_dev)
    off = plain.offsets_of([1] * 3).to(cuda_dev)
    want = lynx_lib.lynx_cache_attn_decode(q, kp, vp, table, lens)
    packed = lynx_lib.lynx_cache_attn_prefill(q[:, 0], off, kp, vp, table, lens)[:, None]
    host = lens.cpu().pin_memory()
    big = torch.empty(1 << 26, device=cuda_dev)
    q2, kp2, lens2 = torch.zeros_like(q), torch.zeros_like(kp), torch.zeros_like(lens)
    results = []
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in range(3):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):        # slow work first, the inputs last
                big.normal_()
                kp2.copy_(kp)
            lens2.zero_()
            q2.copy_(q)
            main.wait_stream(side)
            lens2.copy_(host, non_blocking=True)
            if call < 2:
                out = lynx_lib.lynx_cache_attn_decode(q2, kp2, vp, table, lens2)
            else:
                out = lynx_lib.lynx_cache_attn_prefill(q2[:, 0], off, kp2, vp, table, lens2)[:, None]
            results.append(out.clone())
            kp2.zero_()                          # nothing may still be reading
    for _ in range(3):
        for r in results:
            r.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(results[0], want) and torch.equal(results[1], want)
        assert torch.equal(results[2], packed)


@pytest.mark.parametrize("max_pages", [None, 99])
def test_guards_around_every_output(lynx_lib, cuda_dev, max_pages):
    """Canaries around what the calls write, the workspace included, and the same
    bits twice."""
    from .test_guards_gpu import twice
    counts, kv, page, H_kv, H_q = [9, 0, 30], [800, 5, 130], 64, 2, 6
    kp, vp, table, lens = (t.to(cuda_dev)
                           for t in _cache(kv, page, H_kv, seed=31, max_pages=max_pages))
    off = plain.offsets_of(counts).to(cuda_dev)
    q, k, v = (_rand((39, h, 128), h).to(cuda_dev) for h in (H_q, H_kv, H_kv))
    rope = lynx_lib.Rope(lynx_lib.rope_frequencies(1e4, 64))

    def append(o):
        o[1].copy_(kp)
        o[2].copy_(vp)
        lynx_lib.lynx_cache_append(k, v, off, lens, table, o[1], o[2], q=q, q_out=o[0], rope=rope)

    qr, kp2, vp2 = twice(append, [(q.shape, BF, cuda_dev), (kp.shape, BF, cuda_dev),
                                  (vp.shape, BF, cuda_dev)])

    def attend(call, shape, need):
        def run(o):
            o[2].zero_()
            call(o[0].view(shape), o[1].view(shape[:-1]), o[2] if need else None)
            o[2].zero_()
        twice(run, [(shape, BF, cuda_dev), (shape[:-1], torch.float32, cuda_dev),
                    ((max(need, 16),), torch.uint8, cuda_dev)])

    pages = table.shape[1]
    attend(lambda o, l, w: lynx_lib.lynx_cache_attn_prefill(qr, off, kp2, vp2, table, lens, out=o,
                                                            lse=l, workspace=w), q.shape,
           lynx_lib.lynx_cache_attn_prefill_workspace_bytes(39, 3, H_q, H_kv, 128, page, pages))
    q3 = q.view(3, 13, H_q, 128)
    attend(lambda o, l, w: lynx_lib.lynx_cache_attn_decode(q3, kp2, vp2, table, lens, out=o, lse=l,
                                                           workspace=w), q3.shape,
           lynx_lib.lynx_cache_attn_decode_workspace_bytes(3, 13, H_q, H_kv, 128, page, pages))


def test_a_far_pool(lynx_lib, cuda_dev):
    """Pages whose elements lie past 2^31 and bytes past 2^32."""
    page, H_kv, H_q = 512, 8, 8
    blocks = 4400                               # 2.3e9 elements a pool
    kp = torch.zeros((blocks, page, H_kv, 128), dtype=BF, device=cuda_dev)
    vp = torch.zeros_like(kp)
    counts, kv = [600], [600]
    table = torch.tensor([[blocks - 1, blocks - 2]], dtype=torch.int32)
    k, v, q = (_rand((600, 8, 128), s) for s in (1, 2, 3))
    lens = torch.tensor(kv, dtype=torch.int32, device=cuda_dev)
    off = plain.offsets_of(counts).to(cuda_dev)
    lynx_lib.lynx_cache_append(k.to(cuda_dev), v.to(cuda_dev), off, lens, table.to(cuda_dev), kp, vp)
    assert torch.equal(kp[-1].cpu(), k[:512]) and torch.equal(vp[-2, :88].cpu(), v[512:])
    small = (kp[-2:].cpu(), vp[-2:].cpu())
    near = torch.tensor([[1, 0]], dtype=torch.int32)
    want = plain.attention(q, counts, kv, near, *small)
    got = lynx_lib.lynx_cache_attn_prefill(q.to(cuda_dev), off, kp, vp, table.to(cuda_dev), lens)
    plain.assert_close(got, want[0], want[2], "prefill")
    got = lynx_lib.lynx_cache_attn_decode(q[-1:].to(cuda_dev)[None], kp, vp, table.to(cuda_dev), lens)
    plain.assert_close(got[0], want[0][-1:], want[2][-1:], "decode")


def test_a_request_from_prefill_to_packed_pages(lynx_lib, cuda_dev):
    """The three calls and the codec in the order of a request: two prompts are
    appended chunk by chunk and attended, one token at a time follows, the
    finished pages are packed by lynx_encode and read by the packed attention
    through the same block table."""
    page, H_kv, H_q, C, alpha = 64, 2, 8, 32, 255.0
    total = [256, 256]
    table, blocks = plain.table_for(total, page, 2, seed=1)
    kp = torch.full((blocks, page, H_kv, 128), NAN, dtype=BF, device=cuda_dev)
    vp = torch.full_like(kp, NAN)
    tab = table.to(cuda_dev)
    f = lynx_lib.rope_frequencies(1e6, 128)
    rope = lynx_lib.Rope(f)
    q, k, v = (_rand((2, 256, h, 128), s) for h, s in ((H_q, 1), (H_kv, 2), (H_kv, 3)))
    done, out_of = [0, 0], {}
    for counts in ([100, 0], [91, 250], [60, 1], [1, 1], [1, 1], [1, 1], [1, 1], [1, 1]):
        after = [min(256, d + c) for d, c in zip(done, counts)]
        counts = [a - d for a, d in zip(after, done)]
        take = lambda x: torch.cat([x[b, done[b]:after[b]] for b in range(2)]).to(cuda_dev)
        off = plain.offsets_of(counts).to(cuda_dev)
        lens = torch.tensor(after, dtype=torch.int32, device=cuda_dev)
        qr = lynx_lib.lynx_cache_append(take(k), take(v), off, lens, tab, kp, vp, q=take(q),
                                        rope=rope)
        if counts == [1, 1]:
            o = lynx_lib.lynx_cache_attn_decode(qr.view(2, 1, H_q, 128), kp, vp, tab, lens)
            o = o.view(2, H_q, 128)
        else:
            o = lynx_lib.lynx_cache_attn_prefill(qr, off, kp, vp, tab, lens)
        at = 0
        for b in range(2):
            for t in range(done[b], after[b]):
                out_of[b, t] = o[at]
                at += 1
        done = after
    assert done == [256, 256]
    # the same from the definitions: rotate everything, attend over everything
    kv = [256, 256]
    zero = torch.zeros((blocks, page, H_kv, 128), dtype=BF)
    a = plain.append(k.flatten(0, 1), v.flatten(0, 1), kv, kv, table, zero, zero,
                     q.flatten(0, 1), f)
    used = table.flatten().long()
    plain.assert_close(kp[used], a[0][used], a[3][used], "keys")
    assert torch.equal(vp.cpu()[used].double(), a[1][used])
    qr = lynx_lib.lynx_cache_append(k.flatten(0, 1).to(cuda_dev), v.flatten(0, 1).to(cuda_dev),
                                    plain.offsets_of(kv).to(cuda_dev),
                                    torch.tensor(kv, dtype=torch.int32, device=cuda_dev), tab, kp,
                                    vp, q=q.flatten(0, 1).to(cuda_dev), rope=rope).cpu()
    want = plain.attention(qr, kv, kv, table, kp.cpu(), vp.cpu())
    got = torch.stack([out_of[b, t] for b in range(2) for t in range(256)])
    plain.assert_close(got, want[0], want[2], "step by step")
    # pack the pools as they stand; read them through the same table
    clean = torch.nan_to_num(kp), torch.nan_to_num(vp)
    packed = [tuple(t[:, 0] for t in lynx_lib.lynx_encode(p, page, C, alpha)) for p in clean]
    last = qr.view(2, 256, H_q, 128)[:, -1:].to(cuda_dev)
    full = lynx_lib.lynx_attn_decode_paged(last, packed[0], packed[1], tab, 256, page, C, alpha,
                                           lynx_lib.LYNX_FULL)
    dense = [lynx_lib.lynx_decode_paged(*p, tab, 256, page, C, alpha, lynx_lib.LYNX_FULL)
             for p in packed]
    back = [torch.zeros_like(kp) for _ in range(2)]
    back_table = torch.arange(8, dtype=torch.int32, device=cuda_dev).view(2, 4)
    lynx_lib.lynx_cache_append(dense[0].flatten(0, 1), dense[1].flatten(0, 1),
                               plain.offsets_of(kv).to(cuda_dev),
                               torch.tensor(kv, dtype=torch.int32, device=cuda_dev), back_table,
                               *back)
    again = lynx_lib.lynx_cache_attn_decode(
        last, *back, back_table, torch.tensor(kv, dtype=torch.int32, device=cuda_dev))
    # both read the same BF16 values; the packed attention's bound is 2e-3, the
    # other's two roundings to BF16 of an output below 4
    assert (full - again.float()).abs().max().item() <= 2e-3 + 4 * 2 ** -7


@pytest.mark.parametrize("max_pages", [None, 99])
def test_two_at_once(lynx_lib, cuda_dev, max_pages):
    """Calls on two streams with a workspace each, and no waits between."""
    jobs = []
    for i, kv in enumerate(([3000, 11], [17, 2500])):
        kp, vp, table, lens = (t.to(cuda_dev) for t in _cache(kv, 64, 2, seed=30 + i, max_pages=max_pages))
        q = _rand((2, 3, 8, 128), i, 2.0).to(cuda_dev)
        jobs.append((q, kp, vp, table, lens))
    alone = [lynx_lib.lynx_cache_attn_decode(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lynx_lib.lynx_cache_attn_decode(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, alone[i]) for x in got[i])
    assert lynx_lib.lynx_wait_timeouts() == 0
    assert math.isfinite(float(alone[0].float().sum()))


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(lynx_lib, cuda_dev, seed):
    """Seeded random calls of both attention entry points."""
    import random
    rng = random.Random(1000 + seed)
    decode = rng.random() < 0.5
    H_kv = rng.choice((1, 2, 3, 5))
    H_q = H_kv * rng.choice((1, 2, 3, 4, 6, 8))
    page = rng.choice((64, 128, 256, 512))
    batch = rng.choice((1, 2, 3, 7, 12))
    longest = rng.choice((70, 300, 900, 2600))
    kv = [rng.choice((0, 1, page, rng.randint(0, longest), longest)) for _ in range(batch)]
    kv[rng.randrange(batch)] = longest
    if decode:
        counts = [rng.choice((1, 1, 2, 5, 8, 17))] * batch
    else:
        counts = [rng.choice((0, 1, rng.randint(0, max(1, n)), min(n, 260))) for n in kv]
        counts[0] = max(1, counts[0])
    kw = {}
    if rng.random() < 0.4:
        kw["softcap"] = rng.choice((2.0, 30.0, 100.0))
    if rng.random() < 0.4:
        kw["window"] = rng.choice((1, 2, 63, 64, 65, 127, 128, 129, 500))
    if rng.random() < 0.4:
        kw["prefix"] = torch.tensor([rng.choice((0, 1, 64, 100, 128, 200)) for _ in kv],
                                    dtype=torch.int32)
    if rng.random() < 0.3:
        kw["slopes"] = torch.tensor([rng.uniform(0, 0.5) for _ in range(H_q)])
    if rng.random() < 0.2:
        kw["scale"] = rng.choice((0.02, 0.3))
    q = _rand((sum(counts), H_q, 128), seed, 2.0)
    _attend(lynx_lib, cuda_dev, q, counts, kv, page, H_kv, seed=seed, decode=decode,
            max_pages=rng.choice((None, max(kv) // page + 3, 5000 // page)) if max(kv) < 4900 else None,
            **kw)
