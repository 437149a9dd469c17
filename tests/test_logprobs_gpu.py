"""lynx_token_logprobs on the GPU against the definition in 64 bits (tests/tree_plain.py has
it and the bounds): types, sizes, strides, ties, masks, and rows that are no distribution."""
import math

import pytest
import torch

from . import tree_plain as plain

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _rows(rows, V, seed, dtype, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, V), generator=g) * spread
    hot = torch.randint(0, V, (rows, 5), generator=g)
    x.scatter_add_(1, hot, torch.rand((rows, 5), generator=g) * 10)
    return x.to(dtype)


def _close(got, want, tol, what):
    got, want = got.cpu().double(), want.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    fin = ~nan & ~inf
    off = ((got - want).abs() - tol)[fin]
    assert not off.numel() or off.max() <= 0, f"{what}: off by {off.max()} too much"


def _check(lynx, dev, x, tokens=None, top=0, scale=1.0, on_gpu=None):
    """x on the CPU; on_gpu: the same rows there, laid out otherwise."""
    want = plain.logprobs(x, tokens, top, scale)
    d = x.to(dev) if on_gpu is None else on_gpu
    got = lynx.lynx_token_logprobs(d, None if tokens is None else tokens.to(dev), top=top,
                                   scale=scale)
    if tokens is not None:
        _close(got[0], want[0], want[4], "logprob")
    else:
        assert got[0] is None
    _close(got[1], want[1], want[5], "entropy")
    _close(got[2], want[2], want[6], "top_logprob")
    assert torch.equal(got[3].cpu(), want[3]), "top_token"
    return got


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,V,top,given,scale", [
    (1, 1, 1, 1, 1.0), (3, 2, 2, 3, 0.5), (5, 31, 31, 1, 2.0), (2, 33, 32, 64, 1.0),
    (4, 4095, 8, 2, 1.0), (4, 4096, 32, 2, 0.7), (4, 4097, 1, 2, 1.0), (1, 8192, 5, 1, 1.0),
    (19, 16385, 20, 4, 1.0), (40, 40001, 8, 1, 1.3), (1, 128256, 32, 7, 1.0),
    (77, 32000, 4, 1, 1.0), (2, 200003, 8, 1, 1.0), (700, 3001, 3, 1, 1e-3), (1300, 97, 0, 2, 9.0)])
def test_matches_the_definition(lynx_lib, cuda_dev, kind, rows, V, top, given, scale):
    x = _rows(rows, V, rows + V, TYPES[kind])
    g = torch.Generator().manual_seed(V)
    tokens = torch.randint(0, V, (rows, given), generator=g, dtype=torch.int32)
    _check(lynx_lib, cuda_dev, x, tokens, top, scale)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("first,gap", [(0, 1), (1, 0), (3, 5), (7, 9)])
def test_rows_at_any_address(lynx_lib, cuda_dev, kind, first, gap):
    """Rows that begin at every element of a 16-byte vector, with NaN around them."""
    rows, V = 9, 8229
    x = _rows(rows, V, 5, TYPES[kind])
    buf = torch.full((first + rows * (V + gap) + 8,), math.nan, dtype=x.dtype, device=cuda_dev)
    view = buf[first:first + rows * (V + gap)].view(rows, V + gap)[:, :V]
    view.copy_(x)
    tokens = torch.tensor([[0, V - 1]] * rows, dtype=torch.int32)
    _check(lynx_lib, cuda_dev, x, tokens, 6, on_gpu=view)
    one = view[4:5]                       # a single row: its stride means nothing
    _check(lynx_lib, cuda_dev, x[4:5], tokens[4:5], 6, on_gpu=one)


def _shapes(V, dtype):
    """Rows of every kind that the selection could trip over."""
    lowest = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    ramp = torch.linspace(-20.0, 20.0, V)
    some = torch.randn(V, generator=g)
    few = torch.full((V,), -math.inf)
    few[torch.randperm(V, generator=g)[:3]] = torch.tensor([1.0, 1.0, 0.5])[:min(3, V)]
    low = torch.full((V,), lowest)
    low[V // 2] = 2.0
    last = torch.full((V,), -5.0)
    last[-1] = 5.0
    steps = (torch.arange(V) // 700).float()          # rising, in long runs of equals
    spike = some.clone()
    spike[0] = 60.0                                   # 2^y of all others is nearly nothing
    late = some.clone()
    late[-3:] = torch.tensor([50.0, 51.0, 80.0])[-min(3, V):]
    zeros = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    rows = [ramp, ramp.flip(0), torch.zeros(V), zeros, torch.full((V,), 3.0), steps, steps.flip(0),
            few, low, torch.full((V,), lowest), torch.full((V,), -math.inf), last, spike, late,
            some * 0.01, torch.where(torch.rand(V, generator=g) < 0.97, -math.inf, some)]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("V", [1, 5, 70, 5000, 33001])
@pytest.mark.parametrize("top", [1, 8, 32])
def test_rows_of_every_shape(lynx_lib, cuda_dev, kind, V, top):
    x = _shapes(V, TYPES[kind])
    tokens = torch.tensor([[0, V // 2, V - 1]] * len(x), dtype=torch.int32)
    _check(lynx_lib, cuda_dev, x, tokens, min(top, V))
    # many rows at once (a CTA each), and each alone (a cluster each)
    many = x.repeat(45, 1)
    _check(lynx_lib, cuda_dev, many, tokens.repeat(45, 1), min(top, V))
    for i in range(len(x)):
        _check(lynx_lib, cuda_dev, x[i:i + 1], tokens[i:i + 1], min(top, V))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("V", [3, 9001])
def test_nan_and_infinite_logits(lynx_lib, cuda_dev, kind, V):
    x = _rows(6, V, 3, TYPES[kind])
    x[0, V // 2] = math.nan
    x[1, :] = math.nan
    x[2, 0] = math.inf
    x[3, :2] = math.inf
    x[4, 0], x[4, 1] = math.nan, math.inf
    x[5, 0] = -math.inf
    tokens = torch.tensor([[0, V - 1]] * 6, dtype=torch.int32)
    _check(lynx_lib, cuda_dev, x, tokens, 2)


def test_given_tokens_that_are_none(lynx_lib, cuda_dev):
    x = _rows(2, 300, 1, torch.float32)
    tokens = torch.tensor([[-1, 5, -7], [299, -2 ** 31, 0]], dtype=torch.int32)
    before = lynx_lib.lynx_device_errors()
    _check(lynx_lib, cuda_dev, x, tokens, 1)
    assert lynx_lib.lynx_device_errors() == before


def test_outputs_of_the_caller_graphs_and_streams(lynx_lib, cuda_dev):
    """One graph over logits that change, and calls on other streams at once, give bit for
    bit what a call alone gives."""
    x = _rows(64, 20011, 9, torch.bfloat16).to(cuda_dev)
    tokens = torch.randint(0, 20011, (64,), dtype=torch.int32).to(cuda_dev)
    out = (torch.empty(64, device=cuda_dev), torch.empty(64, device=cuda_dev),
           torch.empty((64, 8), device=cuda_dev),
           torch.empty((64, 8), dtype=torch.int32, device=cuda_dev))
    lynx_lib.lynx_token_logprobs(x, tokens, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = lynx_lib.lynx_token_logprobs(x, tokens, 8, 1.0, *out)
    assert all(a is b for a, b in zip(got, out))
    for seed in (1, 2):
        x.copy_(_rows(64, 20011, seed, torch.bfloat16))
        g.replay()
        alone = lynx_lib.lynx_token_logprobs(x, tokens, 8)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        more = []
        for s in streams:
            with torch.cuda.stream(s):
                more += [lynx_lib.lynx_token_logprobs(x, tokens, 8) for _ in range(4)]
        torch.cuda.synchronize()
        for m in [out] + more:
            assert all(torch.equal(a.view(torch.int32), b.view(torch.int32))
                       for a, b in zip(m, alone))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("scale", [1e-6, 1e6])
def test_scales_at_the_ends(lynx_lib, cuda_dev, kind, scale):
    x = _rows(5, 20003, 4, TYPES[kind], spread=1e4 if scale < 1 and kind != "f16" else 3.0)
    tokens = torch.tensor([[0, 20002]] * 5, dtype=torch.int32)
    _check(lynx_lib, cuda_dev, x, tokens, 4, scale)


@pytest.mark.parametrize("apart", [1_500_000_000, 1_500_000_005])
def test_rows_beyond_32_bits(lynx_lib, cuda_dev, apart):
    """Rows whose first bytes, and values, lie beyond 2^32."""
    V = 9001
    x = _rows(4, V, 2, torch.bfloat16)
    buf = torch.empty(3 * apart + V, dtype=torch.bfloat16, device=cuda_dev)
    view = buf.as_strided((4, V), (apart, 1))
    view.copy_(x)
    _check(lynx_lib, cuda_dev, x, torch.tensor([[0, V - 1]] * 4, dtype=torch.int32), 4, on_gpu=view)


def test_no_rows(lynx_lib, cuda_dev):
    x = torch.empty((0, 50), device=cuda_dev)
    lp, h, tl, tt = lynx_lib.lynx_token_logprobs(x, torch.empty(0, dtype=torch.int32,
                                                                device=cuda_dev), 3)
    assert lp.shape == (0,) and h.shape == (0,) and tl.shape == tt.shape == (0, 3)


def _tall(V, dtype, high):
    """Rows with logits so large that the others' distance from them, times the scale, is
    beyond float32: in the first place, in the middle, in the last, in several and in all."""
    g = torch.Generator().manual_seed(V)
    some = torch.randn(V, generator=g)
    rows = []
    for at in (0, V // 2, V - 1):
        x = some.clone()
        x[at] = high
        rows.append(x)
    several = some.clone()
    several[::3] = high
    masked = torch.full((V,), -math.inf)
    masked[V // 3] = high
    masked[V // 2] = 1.0
    low = torch.full((V,), -6e4 if dtype == torch.float16 else -1e29)
    low[V // 2] = high
    rows += [several, torch.full((V,), high), masked, low]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("kind,scale,high", [
    ("f32", 1.0, None), ("bf16", 1.0, None), ("f16", 1.0, None), ("f32", 1e6, 1e33),
    ("bf16", 1e6, 1e33), ("f32", 1e-6, None), ("bf16", 2.0, 2e38), ("f32", 1.0, 2.3e38),
    ("f32", 1.0, 2.4e38), ("f32", 1e6, 2e29)])
@pytest.mark.parametrize("V", [5, 70, 5000, 33001])
def test_logits_near_the_types_highest(lynx_lib, cuda_dev, kind, scale, high, V):
    """Entropies of finite logits are numbers, wherever the large ones stand.  (A log
    probability beyond float32 is -inf: what is wanted is rounded.)"""
    x = _tall(V, TYPES[kind], torch.finfo(TYPES[kind]).max if high is None else high)
    tokens = torch.tensor([[0, V // 2, V - 1]] * len(x), dtype=torch.int32)
    want = plain.logprobs(x, tokens, 4, scale)
    n = len(x)
    for rows, times in ([slice(0, n), 45], *([slice(i, i + 1), 1] for i in range(n))):
        d, t = x[rows].repeat(times, 1), tokens[rows].repeat(times, 1)
        lp, h, tl, tt = lynx_lib.lynx_token_logprobs(d.to(cuda_dev), t.to(cuda_dev), top=4,
                                                     scale=scale)
        w = [None if a is None else a[rows].repeat(times, *[1] * (a.dim() - 1)) for a in want]
        assert not torch.isnan(h).any()
        _close(h, w[1], w[5], "entropy")
        _close(lp, w[0].float(), w[4], "logprob")
        _close(tl, w[2].float(), w[6], "top_logprob")
        assert torch.equal(tt.cpu(), w[3])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.25, 1e-6])
def test_log_probabilities_of_logits_far_apart(lynx_lib, cuda_dev, kind, scale):
    """Logits whose difference is beyond float32, and scaled is not: from the type's lowest
    value to its highest."""
    V, top = 4001, 6
    f = torch.finfo(TYPES[kind])
    x = torch.full((3, V), f.min)
    x[0, 1000] = f.max
    x[1, :5] = torch.tensor([f.max, 0.9 * f.min, 0.5 * f.max, 0.0, f.max])
    x[2, ::2] = f.max
    x = x.to(TYPES[kind])
    _check(lynx_lib, cuda_dev, x, torch.tensor([[0, 1, 4, V - 1]] * 3, dtype=torch.int32), top, scale)
    for i in range(3):
        _check(lynx_lib, cuda_dev, x[i:i + 1], None, top, scale)
