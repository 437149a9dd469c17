"""lynx_cache_attn_tree on the GPU against the definition in 64 bits (tests/tree_plain.py, the
bounds of tests/cache_plain.py), and a drafting step from logits to pages with it."""
import random

import pytest
import torch

from . import cache_plain
from . import tree_plain as plain
from .test_cache_gpu import _cache, _rand
from .test_tree_pages_gpu import ints, parents_of

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN = float("nan")


def _words(masks, dev):
    return torch.tensor([[plain.signed(m) for m in r] for r in masks], dtype=torch.int64, device=dev)


def _nodes(batch, T, H_kv, seed):
    """Node buffers with NaN behind the T nodes."""
    bufs = []
    for i in range(2):
        x = torch.full((batch, 64, H_kv, 128), NAN, dtype=BF)
        x[:, :T] = _rand((batch, T, H_kv, 128), seed + i)
        bufs.append(x)
    return bufs


def _trees(rng, batch, T):
    """Masks of trees of several kinds: full, small, none, a chain."""
    rows = []
    for b in range(batch):
        kind = rng.choice(("full", "full", "small", "chain", "none")) if batch > 1 else "full"
        if kind == "chain":
            rows.append(list(range(-1, T - 1)))
        elif kind == "none":
            rows.append([-3] * T)
        else:
            rows.append(parents_of(rng, T if kind == "full" else rng.randrange(1, T + 1), T, 5))
    return [plain.masks(r) for r in rows]


def _attend(lynx, dev, batch, T, kv, H_q, H_kv, page, seed, masks=None, max_pages=None, stride=0, **kw):
    rng = random.Random(seed)
    masks = _trees(rng, batch, T) if masks is None else masks
    kp, vp, table, lens = _cache(kv, page, H_kv, seed, max_pages=max_pages)
    kn, vn = _nodes(batch, T, H_kv, seed + 50)
    q = _rand((batch, T, H_q, 128), seed + 90, 2.0)
    want = plain.attention(q, masks, kv, table, kp, vp, kn, vn, **kw)
    on = {k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in kw.items()}
    dq = q.to(dev)
    if stride:                                # queries as a view of a wider projection
        wide = torch.full((batch, T, H_q + stride, 128), NAN, dtype=BF, device=dev)
        wide[:, :, :H_q] = dq
        dq = wide[:, :, :H_q]
    for b, m in enumerate(masks):             # what no node sees may be anything
        for t in range(T):
            if not any(x >> t & 1 for x in m):
                kn[b, t], vn[b, t] = NAN, NAN
    lse = torch.full((batch, T, H_q), 7.0, device=dev)
    out = torch.full((batch, T, H_q, 128), 7.0, dtype=BF, device=dev)
    got = lynx.lynx_cache_attn_tree(dq, kn.to(dev), vn.to(dev), _words(masks, dev), kp.to(dev),
                                    vp.to(dev), table.to(dev), lens.to(dev), lse=lse, out=out, **on)
    assert got is out
    cache_plain.assert_close(lse, want[1], want[3], "lse")
    cache_plain.assert_close(out, want[0], want[2], "out")


KV = [0, 1, 63, 64, 65, 127, 128, 129, 700]


@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 64])
@pytest.mark.parametrize("H_q,H_kv,page", [(4, 4, 64), (8, 2, 128), (8, 1, 256), (6, 2, 512)])
def test_matches_the_definition(lynx_lib, cuda_dev, T, H_q, H_kv, page):
    _attend(lynx_lib, cuda_dev, len(KV), T, KV, H_q, H_kv, page, seed=T)
    # a table with room for long contexts takes other forms
    _attend(lynx_lib, cuda_dev, len(KV), T, KV, H_q, H_kv, page, seed=T + 1, max_pages=80)


@pytest.mark.parametrize("batch,T,kv,H_q,H_kv,page", [
    (1, 16, [9000], 32, 8, 64), (3, 1, [5000, 1, 2300], 8, 1, 128), (2, 64, [3001, 2000], 16, 1, 256),
    (2, 64, [4500, 0], 8, 2, 64), (9, 8, [2100 + 37 * i for i in range(9)], 16, 4, 64),
    (40, 20, [(i * 71) % 900 for i in range(40)], 10, 2, 64)])
def test_long_and_ragged_contexts(lynx_lib, cuda_dev, batch, T, kv, H_q, H_kv, page):
    _attend(lynx_lib, cuda_dev, batch, T, kv, H_q, H_kv, page, seed=batch + T, stride=3)


@pytest.mark.parametrize("kv,T,H_q,H_kv,kw", [
    ([(i * 1999) % 8000 for i in range(15)], 40, 16, 8, {}),
    ([6200, 100, 3000, 50, 60, 0, 1], 64, 64, 4, {}),
    ([5000, 0, 4100, 64, 129, 4999, 300, 0, 2500, 4600, 5, 77, 1, 2], 19, 32, 8,
     dict(window=8400, prefix=4)),
    ([6100] + [17] * 13, 12, 32, 8, dict(softcap=9.0)),
    ([6100] + [400] * 13, 13, 40, 8, dict(slopes=True))])
def test_units_that_lend_a_hand(lynx_lib, cuda_dev, kv, T, H_q, H_kv, kw):
    """Fewer units than SMs, or short ones: CTAs take parts of the long ones."""
    kw = dict(kw)
    if "prefix" in kw:
        kw["prefix"] = torch.full((len(kv),), kw["prefix"], dtype=torch.int32)
    if "slopes" in kw:
        kw["slopes"] = torch.linspace(0.001, 0.1, H_q)
    _attend(lynx_lib, cuda_dev, len(kv), T, kv, H_q, H_kv, 64, seed=T, max_pages=130, **kw)


@pytest.mark.parametrize("extra", [1, 20, 60, 100])
def test_more_units_than_sms(lynx_lib, cuda_dev, extra):
    """A unit per sequence and KV head: one round and a part of the next, whole and (where
    the table has room for long contexts) cut in parts."""
    sms = torch.cuda.get_device_properties(cuda_dev).multi_processor_count
    batch = (sms + extra) // 2
    kv = [(i * 83) % 400 for i in range(batch)]
    kv[1], kv[-1] = 2300, 1900
    _attend(lynx_lib, cuda_dev, batch, 17, kv, 4, 2, 64, seed=extra)
    _attend(lynx_lib, cuda_dev, batch, 17, [min(n, 600) for n in kv], 4, 2, 64, seed=extra)


@pytest.mark.parametrize("T,H_q", [(3, 2), (20, 4)])
def test_many_short_sequences(lynx_lib, cuda_dev, T, H_q):
    _attend(lynx_lib, cuda_dev, 1300, T, [(7 * i) % 40 for i in range(1300)], H_q, 1, 64, seed=T)


@pytest.mark.parametrize("max_pages", [None, 60])
@pytest.mark.parametrize("T,H_q,H_kv", [(5, 4, 2), (12, 8, 2), (64, 8, 1)])
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(window=1), dict(window=3), dict(window=63), dict(window=64),
    dict(window=200), dict(prefix=70), dict(window=40, prefix=5), dict(window=130, prefix=200),
    dict(slopes=True), dict(softcap=5.0, window=100, prefix=3, slopes=True), dict(scale=0.3)])
def test_scores_windows_prefixes(lynx_lib, cuda_dev, T, H_q, H_kv, kw, max_pages):
    kv = [0, 50, 128, 333, 1000]
    kw = dict(kw)
    if "prefix" in kw:
        kw["prefix"] = torch.full((len(kv),), kw["prefix"], dtype=torch.int32)
    if "slopes" in kw:
        kw["slopes"] = torch.linspace(0.01, 0.6, H_q)
    _attend(lynx_lib, cuda_dev, len(kv), T, kv, H_q, H_kv, 64, seed=T, max_pages=max_pages, **kw)


@pytest.mark.parametrize("max_pages", [None, 60])
@pytest.mark.parametrize("T,H_q", [(9, 2), (40, 8)])
def test_masks_that_are_no_trees(lynx_lib, cuda_dev, T, H_q, max_pages):
    """Any bits: nodes that see later ones, not themselves, nothing, and bits behind the last
    node, which are ignored."""
    rng = random.Random(T)
    kv = [0, 77, 640]
    masks = [[rng.getrandbits(64) if rng.random() < 0.8 else 0 for _ in range(T)] for _ in kv]
    masks[1] = [((1 << 64) - 1) ^ ((1 << T) - 1)] * T           # nothing but such bits
    _attend(lynx_lib, cuda_dev, 3, T, kv, H_q, 1, 64, seed=T, masks=masks, max_pages=max_pages)
    _attend(lynx_lib, cuda_dev, 3, T, kv, H_q, 1, 64, seed=T, masks=masks, max_pages=max_pages,
            window=20, slopes=torch.linspace(0.1, 0.4, H_q))


@pytest.mark.parametrize("T,kv,H_q,H_kv,max_pages", [
    (8, [700, 33], 8, 2, None), (8, [700, 33], 8, 2, 80), (64, [2500, 0], 8, 1, None),
    (33, [300, 129], 16, 2, None)])
def test_a_chain_is_what_decode_gives(lynx_lib, cuda_dev, T, kv, H_q, H_kv, max_pages):
    """A tree that is a chain over n tokens, and the same tokens appended and decoded."""
    page, batch = 64, len(kv)
    table, blocks = cache_plain.table_for([n + T for n in kv], page, 2, 5, max_pages)
    kp, vp = (_rand((blocks, page, H_kv, 128), s).to(cuda_dev) for s in (1, 2))
    kn, vn = (_rand((batch, 64, H_kv, 128), s).to(cuda_dev) for s in (3, 4))
    q = _rand((batch, T, H_q, 128), 6, 2.0).to(cuda_dev)
    dt = table.to(cuda_dev)
    masks = [[(2 << t) - 1 for t in range(T)]] * batch
    lse = [torch.empty((batch, T, H_q), device=cuda_dev) for _ in range(2)]
    tree = lynx_lib.lynx_cache_attn_tree(q, kn, vn, _words(masks, cuda_dev), kp, vp, dt,
                                         ints(kv, cuda_dev), lse=lse[0])
    lens = ints([n + T for n in kv], cuda_dev)
    off = torch.arange(batch + 1, dtype=torch.int32, device=cuda_dev) * T
    lynx_lib.lynx_cache_append(kn[:, :T].reshape(-1, H_kv, 128).contiguous(),
                               vn[:, :T].reshape(-1, H_kv, 128).contiguous(), off, lens, dt, kp, vp)
    chain = lynx_lib.lynx_cache_attn_decode(q, kp, vp, dt, lens, lse=lse[1])
    # both are within their bounds of the same value: weights once rounded to BF16, and
    # the outputs; values are below 16 in size
    assert (lse[0] - lse[1]).abs().max() < 2.0 ** -14
    off_by = (tree.double() - chain.double()).abs()
    assert (off_by <= 2.0 ** -6 * chain.double().abs().amax() + 2.0 ** -7).all()
    assert off_by.mean() < 2.0 ** -9


def test_captured_and_at_once(lynx_lib, cuda_dev):
    """Graphs replayed over other lengths and trees, and calls on several streams, give bit
    for bit what a call alone gives."""
    for T, H_q, H_kv, pages in ((6, 8, 2, 16), (6, 8, 2, 80), (64, 16, 2, 16), (64, 16, 2, 80)):
        batch, page = 4, 64
        kv = [700, 64, 0, 911]
        kp, vp, table, lens = (t.to(cuda_dev) for t in _cache(kv, page, H_kv, T, max_pages=pages))
        kp, vp = kp.nan_to_num(0.5), vp.nan_to_num(0.5)
        table = table.clamp(min=0)
        kn, vn = (t.to(cuda_dev) for t in _nodes(batch, T, H_kv, 9))
        q = _rand((batch, T, H_q, 128), 3, 2.0).to(cuda_dev)
        mask = _words(_trees(random.Random(1), batch, T), cuda_dev)
        need = lynx_lib.lynx_cache_attn_tree_workspace_bytes(batch, T, H_q, H_kv, 128, page, pages)

        def call(out=None, lse=None):
            lse = torch.empty((batch, T, H_q), device=cuda_dev) if lse is None else lse
            ws = torch.empty(need, dtype=torch.uint8, device=cuda_dev) if need else None
            return lynx_lib.lynx_cache_attn_tree(q, kn, vn, mask, kp, vp, table, lens, lse=lse,
                                                 out=out, workspace=ws), lse

        call()
        out = torch.empty_like(q), torch.empty((batch, T, H_q), device=cuda_dev)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*out)
        for seed, n in enumerate((kv, [0, 0, 0, 0], [1, 1000, 129, 300])):
            lens.copy_(ints(n, cuda_dev))
            mask.copy_(_words(_trees(random.Random(seed), batch, T), cuda_dev))
            g.replay()
            want = call()
            torch.cuda.synchronize()
            more = []
            for s in [torch.cuda.Stream() for _ in range(3)]:
                with torch.cuda.stream(s):
                    more += [call() for _ in range(3)]
            torch.cuda.synchronize()
            for got in [out] + more:
                assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
                assert torch.equal(got[1], want[1])
    assert lynx_lib.lynx_wait_timeouts() == 0


def test_units_that_lend_a_hand_in_a_graph(lynx_lib, cuda_dev):
    """One graph over lengths that change what is lent, and calls at once on other streams,
    give bit for bit what a call alone gives."""
    batch, T, H_q, H_kv, page, pages = 14, 17, 16, 8, 64, 130
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    kp, vp = (torch.randn((batch * pages, page, H_kv, 128), generator=g, device=cuda_dev).to(BF)
              for _ in "kv")
    table = torch.randperm(batch * pages, generator=g, device=cuda_dev).to(torch.int32)
    table = table.view(batch, pages)
    kn, vn = (t.to(cuda_dev) for t in _nodes(batch, T, H_kv, 9))
    q = _rand((batch, T, H_q, 128), 3, 2.0).to(cuda_dev)
    mask = _words(_trees(random.Random(2), batch, T), cuda_dev)
    for b in range(batch):
        kn[b].nan_to_num_(0.5), vn[b].nan_to_num_(0.5)
    lens = ints([0] * batch, cuda_dev)

    def call(out=None):
        lse = torch.empty((batch, T, H_q), device=cuda_dev)
        return lynx_lib.lynx_cache_attn_tree(q, kn, vn, mask, kp, vp, table, lens, lse=lse,
                                             out=out), lse

    call()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = call(out)
    for n in ([8000] + [100] * 13, [8320] * 14, [(i * 1999) % 8000 for i in range(14)], [0] * 14,
              [10] * 7 + [7000] * 7):
        lens.copy_(ints(n, cuda_dev))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        more = [(out, lse)]
        for s in [torch.cuda.Stream() for _ in range(2)]:
            with torch.cuda.stream(s):
                more += [call() for _ in range(2)]
        torch.cuda.synchronize()
        for got in more:
            assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
            assert torch.equal(got[1], want[1])
        # and each sequence by itself, which takes another form, within the outputs' rounding
        for b in (0, 5, 13):
            one = lynx_lib.lynx_cache_attn_tree(q[b:b + 1], kn[b:b + 1], vn[b:b + 1], mask[b:b + 1],
                                                kp, vp, table[b:b + 1], lens[b:b + 1])
            off = (one.double() - want[0][b:b + 1].double()).abs()
            assert off.max() <= 2.0 ** -6 * one.double().abs().max() + 2.0 ** -7


def test_a_drafting_step_from_logits_to_pages(lynx_lib, cuda_dev):
    """Two layers, three sequences of one prompt that share its pages: alternatives from
    logits, a tree, its attention, the walk along the answers, pages and tokens kept; and
    decode over the result gives what a cache filled token by token gives."""
    lynx, dev = lynx_lib, cuda_dev
    rng = random.Random(3)
    layers, batch, H_q, H_kv, page, V, prompt = 2, 3, 8, 2, 64, 5003, 90
    num_blocks, max_pages = 24, 4
    rope = lynx.Rope(lynx.rope_frequencies(1e4, 128))
    kvs = torch.zeros((2 * layers, num_blocks, page, H_kv, 128), dtype=BF, device=dev)
    pools = list(kvs)
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device=dev)
    kv, refs = ints([0], dev), torch.zeros(num_blocks, dtype=torch.int32, device=dev)
    lynx.lynx_cache_reserve(table, kv, refs, ints([prompt], dev), page)
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(BF).to(dev)

    told = [[(rand(prompt, H_kv, 128), rand(prompt, H_kv, 128)) for _ in range(layers)]
            for _ in range(batch)]
    told = [told[0] if b else told[0] for b in range(batch)]          # one prompt
    for i in range(layers):
        lynx.lynx_cache_append(*told[0][i], ints([0, prompt], dev), kv, table, pools[2 * i],
                               pools[2 * i + 1], rope=rope)
    table, kv = lynx.lynx_cache_fork(table, kv, refs, ints([0, 0, 0], dev), page)
    assert refs.max() == batch
    kept = [[] for _ in range(batch)]                                 # per sequence: rows
    for step in range(4):
        # a tree of two levels: the root and four alternatives, two more below the first
        logits = torch.randn((batch, V), generator=g).to(BF).to(dev)
        lp, entropy, top_lp, top = lynx.lynx_token_logprobs(logits, top=4)
        assert (top_lp[:, :-1] >= top_lp[:, 1:]).all() and (entropy > 0).all()
        T = 7
        parents = ints([[-1, 0, 0, 0, 0, 1, 1]] * batch, dev)
        tokens = torch.cat((torch.zeros((batch, 1), dtype=torch.int32, device=dev), top,
                            ints([[11, 12]] * batch, dev)), 1).contiguous()
        mask, positions = lynx.lynx_tree_plan(parents, kv)
        nodes = [torch.zeros((batch, 64, H_kv, 128), dtype=BF, device=dev) for _ in range(2 * layers)]
        own = ints([[b] for b in range(batch)], dev)
        off = ints([T * b for b in range(batch + 1)], dev)
        rows = [(rand(batch * T, H_kv, 128), rand(batch * T, H_kv, 128)) for _ in range(layers)]
        for i in range(layers):
            q = lynx.lynx_cache_append(*rows[i], off, ints([T] * batch, dev), own, nodes[2 * i],
                                       nodes[2 * i + 1], q=rand(batch * T, H_q, 128), rope=rope,
                                       positions=positions)
            lynx.lynx_cache_attn_tree(q.view(batch, T, H_q, 128), nodes[2 * i], nodes[2 * i + 1],
                                      mask, pools[2 * i], pools[2 * i + 1], table, kv)
        # each sequence is answered otherwise: a node of depth 2, of depth 1, none
        pick = [int(tokens[0, 1]), int(tokens[1, 3]), -7]
        answers = ints([[pick[b], 12, 5, 6, 7, 8, 9] for b in range(batch)], dev)
        path, n, token = lynx.lynx_tree_verify(parents, tokens, answers)
        want = [[0, 1, 6], [0, 3], [0]]
        assert n.tolist() == [3, 2, 1] and token.tolist() == [9, 6, -7]
        assert [p[:len(w)] for p, w in zip(path.tolist(), want)] == want
        granted, src, dst = lynx.lynx_cache_reserve(table, kv, refs, n, page)
        assert granted.tolist() == n.tolist()
        assert (step == 0) == (max(src.tolist()) >= 0)               # the prompt's page was shared
        lynx.lynx_cache_copy_pages(pools, src, dst)
        lynx.lynx_cache_keep(nodes, pools, path, granted, kv, table)
        for b in range(batch):
            kept[b] += [[(k[T * b + t], v[T * b + t]) for k, v in rows] for t in want[b]]
        if step == 2:                                                # in between, pages move
            src, dst, count = lynx.lynx_cache_compact(table, kv, refs, page)
            lynx.lynx_cache_copy_pages(pools, src, dst, count)
            assert (refs > 0).nonzero().max() < (refs > 0).sum()
    # a cache filled with the prompt and the kept tokens, one after the other
    lens = [prompt + len(k) for k in kept]
    assert kv.tolist() == lens
    t2, blocks = cache_plain.table_for(lens, page, 1, 7, max_pages)
    t2 = t2.to(dev)
    for i in range(layers):
        k2, v2 = (torch.zeros((blocks, page, H_kv, 128), dtype=BF, device=dev) for _ in "kv")
        k = torch.cat([torch.cat((told[b][i][0], torch.stack([r[i][0] for r in kept[b]])))
                       for b in range(batch)])
        v = torch.cat([torch.cat((told[b][i][1], torch.stack([r[i][1] for r in kept[b]])))
                       for b in range(batch)])
        lynx.lynx_cache_append(k, v, cache_plain.offsets_of(lens).to(dev), kv, t2, k2, v2, rope=rope)
        q = rand(batch, 1, H_q, 128)
        a = lynx.lynx_cache_attn_decode(q, pools[2 * i], pools[2 * i + 1], table, kv)
        z = lynx.lynx_cache_attn_decode(q, k2, v2, t2, kv)
        assert torch.equal(a.view(torch.int16), z.view(torch.int16))
