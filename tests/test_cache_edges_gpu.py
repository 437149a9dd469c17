"""The BF16 paged cache where its results are easy to get wrong: queries that are
not numbers, on every way the work is shared out."""
import math

import pytest
import torch

from . import cache_plain as plain
from .test_cache_gpu import BF, _cache, _rand

pytestmark = pytest.mark.gpu


# counts, kv, H_q, H_kv, page, decode, least pages of the table (on 152 SMs: how
# the work is shared out)
FORMS = {
    "decode clusters": ([2, 2, 2], [700, 65, 1], 8, 2, 64, True, None),
    "decode shares": ([1, 1, 1], [9000, 3, 130], 8, 2, 64, True, None),
    "decode short shares": ([2] * 40, [3 * i + 1 for i in range(40)], 8, 2, 64, True, 99),
    "decode many rows": ([12, 12], [5000, 7], 8, 2, 128, True, None),
    "prefill whole": ([70, 0, 301], [70, 9, 500], 4, 2, 128, False, None),
    "prefill shares": ([40, 3], [9000, 2500], 4, 1, 256, False, None),
    "prefill parts": ([300, 301], [2600, 301], 40, 40, 64, False, None),
}
SCORES = {"plain": {}, "cap": dict(softcap=15.0), "bias": dict(slopes=0.03),
          "window": dict(window=90), "all": dict(softcap=15.0, slopes=0.03, window=90)}


def _run(lynx, dev, form, q, kw, seed=50):
    """(out, lse) on the CPU and the definitions' (out, lse, bounds)."""
    counts, kv, H_q, H_kv, page, decode, pages = FORMS[form]
    kp, vp, table, lens = _cache(kv, page, H_kv, seed, max_pages=pages)
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = torch.linspace(0.0, kw["slopes"], H_q)
    want = plain.attention(q, counts, kv, table, kp, vp, **kw)
    on = {k: v.to(dev) if torch.is_tensor(v) else v for k, v in kw.items()}
    args = [t.to(dev) for t in (kp, vp, table, lens)]
    lse = torch.empty(q.shape[:2], device=dev)
    if decode:
        shape = (len(counts), counts[0]) + tuple(q.shape[1:])
        out = lynx.lynx_cache_attn_decode(q.to(dev).view(shape), *args, lse=lse.view(shape[:-1]), **on)
    else:
        out = lynx.lynx_cache_attn_prefill(q.to(dev), plain.offsets_of(counts).to(dev), *args,
                                           lse=lse, **on)
    return out.view(q.shape).cpu(), lse.cpu(), want


def _largest_value(form, seed=50):
    counts, kv, _, H_kv, page, _, pages = FORMS[form]
    return float(_cache(kv, page, H_kv, seed, max_pages=pages)[1].nan_to_num().abs().max())


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("form", FORMS)
def test_a_query_that_is_not_a_number(lynx_lib, cuda_dev, form, score):
    """Its row is NaN, in the output and in the log-sum, not the zeros and -inf of a
    row that sees nothing; the other rows are what they are without it."""
    counts, _, H_q = FORMS[form][:3]
    q = _rand((sum(counts), H_q, 128), 51, 2.0)
    for row in range(0, len(q), 7):
        q[row, row % H_q, (5 * row) % 128] = math.nan
    out, lse, want = _run(lynx_lib, cuda_dev, form, q, SCORES[score])
    assert torch.isnan(want[1]).any() and not torch.isnan(want[1]).all()
    assert torch.equal(torch.isnan(lse), torch.isnan(want[1]))
    assert torch.equal(torch.isnan(out), torch.isnan(want[0]))
    # (a bound that is NaN beside a number is that of a row which sees nothing: the
    # error counted for its NaN scores, times weights of zero.  Such a row is exact.)
    plain.assert_close(lse, want[1], want[3].nan_to_num(0.0), "lse")
    plain.assert_close(out, want[0], want[2].nan_to_num(0.0), "out")


@pytest.mark.parametrize("form", FORMS)
def test_an_infinite_query(lynx_lib, cuda_dev, form):
    """A score of +inf leaves no weights to speak of: NaN.  Where all scores are -inf
    no key has any weight: the row is one that sees nothing.  A cap makes both finite."""
    counts, _, H_q = FORMS[form][:3]
    q = _rand((sum(counts), H_q, 128), 52, 2.0)
    q[::5, 0, 9] = math.inf
    out, lse, want = _run(lynx_lib, cuda_dev, form, q, {})
    none = want[1] == -math.inf
    must = want[0].masked_fill(none[..., None], 0.0)
    assert torch.isnan(must).any()
    assert torch.equal(torch.isnan(out), torch.isnan(must))
    assert (lse[none] == -math.inf).all()
    assert torch.equal(torch.isnan(lse), torch.isnan(must).all(-1))
    plain.assert_close(out, must, want[2].nan_to_num(0.0), "out")
    out, lse, want = _run(lynx_lib, cuda_dev, form, q, SCORES["cap"])
    assert not torch.isnan(want[0]).any()
    # (the definitions' bound counts sum |q k|, here infinite.  Of such scores only the
    # cap's own error is left: delta = 2^-20 cap; the largest value of the cache bounds
    # every output, and 15 + ln 9000 < 2^5 every log-sum.)
    fin = torch.isfinite(q.float()).all(-1)
    delta, top = 2.0 ** -20 * 15, _largest_value(form)
    tol = (2 * delta + 2.0 ** -19 + 2.0 ** -8 + 2.0 ** -8) * top + 2.0 ** -30
    plain.assert_close(out, want[0], torch.where(fin[..., None], want[2], tol), "capped out")
    tol = delta + 2.0 ** -20 + 2.0 ** -22 * 2 ** 5
    plain.assert_close(lse, want[1], torch.where(fin, want[3], tol), "capped lse")


def test_a_wait_that_is_given_up_leaves_nothing_in_flight(lynx_lib, cuda_dev):
    """A CTA of these kernels that gives up a wait still drains its copies and
    products before its shared and tensor memory go; the error words stay clear."""
    before = lynx_lib.lynx_device_errors()
    assert lynx_lib.lynx_wait_selftest(1_000_000, 3, cuda_dev) == 5
    assert lynx_lib.lynx_device_errors() == before
    assert lynx_lib.lynx_wait_timeouts() == 0


@pytest.mark.parametrize("kw", [dict(softcap=1e-40), dict(softcap=1e-44), dict(softcap=3e38),
                                dict(scale=3e38), dict(scale=3e38, softcap=2.0),
                                dict(scale=1e-44), dict(scale=1e-44, softcap=1e-44),
                                dict(slopes=3e38), dict(slopes=3e38, softcap=2.0)])
@pytest.mark.parametrize("form", FORMS)
def test_scales_and_caps_at_the_ends_of_their_type(lynx_lib, cuda_dev, form, kw):
    """Accepted values whose products with log2(e) or with each other leave float32.
    Queries of zeros have scores of zero whatever the scale and the cap; others are
    tried where the scores are small."""
    counts, _, H_q = FORMS[form][:3]
    queries = [torch.zeros((sum(counts), H_q, 128), dtype=BF)]
    if kw.get("scale", 0) < 1 and kw.get("softcap", 0) < 1:
        queries.append(_rand(queries[0].shape, 53))
    for q in queries:
        out, lse, want = _run(lynx_lib, cuda_dev, form, q, kw)
        assert torch.isfinite(want[0]).all()
        plain.assert_close(lse, want[1], want[3], "lse")
        plain.assert_close(out, want[0], want[2], "out")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("freq", [1.0, -3.0, 1000003.0, 16777213.0, 2.0 ** 40, 1.7976931348623157e308])
def test_angles_of_far_positions_and_high_frequencies(lynx_lib, cuda_dev, freq, inter):
    """The angle of any 32-bit position at any frequency.  The reference is exact: the
    product with the position is made with integers, and reduced by 1200 bits of pi."""
    pos = [0, 1, 2, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31, 1234567890]
    n, half = len(pos), 64
    from fractions import Fraction
    turn = 2 * _pi(1200)
    want = torch.empty((n, 2), dtype=torch.float64)
    for i, p in enumerate(pos):
        a = Fraction(freq) * p / turn
        a = float((a - math.floor(a + Fraction(1, 2))) * turn)
        want[i] = torch.tensor([math.cos(a), math.sin(a)], dtype=torch.float64)
    k = torch.zeros((n, 1, 128), dtype=BF)
    first = slice(0, 128, 2) if inter else slice(0, half)
    second = slice(1, 128, 2) if inter else slice(half, 128)
    k[..., first] = 1.0
    kp, vp = (torch.zeros((1, 64, 1, 128), dtype=BF, device=cuda_dev) for _ in range(2))
    lens = torch.tensor([n], dtype=torch.int32, device=cuda_dev)
    lynx_lib.lynx_cache_append(
        k.to(cuda_dev), k.to(cuda_dev), plain.offsets_of([n]).to(cuda_dev), lens,
        torch.zeros((1, 1), dtype=torch.int32, device=cuda_dev), kp, vp,
        rope=lynx_lib.Rope([freq] * half, None, inter),
        positions=torch.tensor(pos, dtype=torch.int32, device=cuda_dev))
    got = kp[0, :n, 0].cpu().double()
    # one rounding to BF16, sin.approx and cos.approx, as for the other rotations
    for c, part in ((0, first), (1, second)):
        y = want[:, c:c + 1].expand(n, half)
        plain.assert_close(got[:, part], y, 2.0 ** -8 * y.abs() + 2.0 ** -19, ("cos", "sin")[c])


def _pi(bits):
    """pi as a fraction, by Machin's formula."""
    from fractions import Fraction
    one = 1 << (bits + 16)

    def arctan_inv(x):
        total, term, k = 0, one // x, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= x * x
            k += 2
        return total

    return Fraction(4 * (4 * arctan_inv(5) - arctan_inv(239)), one)
