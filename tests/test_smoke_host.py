"""What smoke() holds against the BF16 paged cache's outputs: right ones pass, and a
mistake that both readers share does not.  No GPU."""
import math

import pytest
import torch

import __graft_entry__ as entry

N, H_Q, H_KV, D, THETA = 100, 4, 2, 128, 1e6


def _rotate(x, shift=0, pairs=False, theta=THETA):
    half = D // 2
    a = (torch.arange(N) + shift)[:, None] * theta ** (-torch.arange(half, dtype=torch.float64) / half)
    i = torch.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    y, c, s = x.double(), a.cos()[:, None], a.sin()[:, None]
    z = y.clone()
    z[..., lo], z[..., hi] = y[..., lo] * c - y[..., hi] * s, y[..., hi] * c + y[..., lo] * s
    return z.to(torch.bfloat16)


def _attend(q, k, v, scale=1.0 / math.sqrt(D), ahead=0, heads=None):
    kv = [h // (H_Q // H_KV) for h in range(H_Q)] if heads is None else heads
    s = torch.einsum("qhd,khd->hqk", q.double(), k.double()[:, kv]) * scale
    i = torch.arange(N)
    s = s.masked_fill(i[None, :] > i[:, None] + ahead, -math.inf)
    return torch.einsum("hqk,khd->qhd", s.softmax(-1), v.double()[:, kv]).to(torch.bfloat16)


def _check(rotate={}, attend={}):
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn((N, h, D), generator=g).to(torch.bfloat16) for h in (H_KV, H_KV, H_Q))
    kr, qr = _rotate(k, **rotate), _rotate(q, **rotate)
    out = _attend(qr, kr, v, **attend)
    entry.check_cache_outputs(*(x.float().numpy() for x in (k, v, q)), THETA,
                              *(x.float().numpy() for x in (kr, qr, out, out[-1])))


def test_right_outputs_pass():
    _check()


@pytest.mark.parametrize("rotate,attend", [
    ({}, dict(scale=1.0 / D)), ({}, dict(scale=0.09)), ({}, dict(ahead=1)), ({}, dict(ahead=-1)),
    ({}, dict(heads=[0, 1, 0, 1])), (dict(shift=1), {}), (dict(pairs=True), {}),
    (dict(theta=1e4), {})])
def test_a_mistake_that_both_readers_share(rotate, attend):
    with pytest.raises(AssertionError):
        _check(rotate, attend)
