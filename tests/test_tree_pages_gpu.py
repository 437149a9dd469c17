"""Trees of drafted tokens and the paged cache's books on the GPU, against Python integers
(tests/tree_plain.py): plan, verify, fork, reserve, trim, compact, the copies they ask for,
and the nodes kept."""
import functools
import os
import random
import subprocess
import sys

import pytest
import torch

from . import tree_plain as plain

pytestmark = pytest.mark.gpu

I32 = torch.int32


def own_process(fn):
    """Runs a test in a process of its own: the error words it sets are never reset."""
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


def ints(v, dev):
    return torch.tensor(v, dtype=I32, device=dev)


def parents_of(rng, n, T, wide):
    return [-1] + [rng.randrange(max(0, t - wide), t) for t in range(1, n)] + [-1] * (T - n)


# ----------------------------------------------------------------- trees

@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64])
def test_plan_and_verify_match_the_definition(lynx_lib, cuda_dev, T):
    rng = random.Random(T)
    rows = [parents_of(rng, T, T, w) for w in (1, 2, 5, 64)]
    rows += [parents_of(rng, rng.randrange(1, T + 1), T, 3) for _ in range(5)]
    rows += [[0] + [0] * (T - 1), [-1] * T, [-1] + [t for t in range(1, T)],
             [-1] + [2 ** 31 - 1] * (T - 1), [-1] + [-7] * (T - 1), [-2] + [0] * (T - 1)]
    odd = parents_of(rng, T, T, 4)
    odd[T // 2] = -1                                   # nothing there, nor below
    rows.append(odd)
    kv = [rng.randrange(0, 5000) for _ in rows]
    mask, pos = lynx_lib.lynx_tree_plan(ints(rows, cuda_dev), ints(kv, cuda_dev))
    want = [plain.masks(r) for r in rows]
    assert mask.cpu().tolist() == [[plain.signed(m) for m in r] for r in want]
    assert pos.cpu().tolist() == [n + bin(m).count("1") - 1 if m else -1
                                  for n, r in zip(kv, want) for m in r]
    # few tokens, so that siblings have the same ones
    tokens = [[rng.randrange(0, 3) for _ in range(T)] for _ in rows]
    answers = [[rng.randrange(0, 3) for _ in range(T)] for _ in rows]
    path, n, nxt = lynx_lib.lynx_tree_verify(*(ints(v, cuda_dev) for v in (rows, tokens, answers)))
    for b, r in enumerate(rows):
        p, token = plain.verify(r, tokens[b], answers[b])
        assert path[b].tolist() == p + [-1] * (T - len(p))
        assert (int(n[b]), int(nxt[b])) == (len(p), token)


def test_a_chain_is_accepted_whole(lynx_lib, cuda_dev):
    T = 64
    parents = ints([list(range(-1, T - 1))] * 3, cuda_dev)
    tokens = ints([list(range(T))] * 3, cuda_dev)
    answers = ints([list(range(1, T + 1))] * 3, cuda_dev)
    path, n, nxt = lynx_lib.lynx_tree_verify(parents, tokens, answers)
    assert path.tolist() == [list(range(T))] * 3 and n.tolist() == [T] * 3 and nxt.tolist() == [T] * 3
    mask, pos = lynx_lib.lynx_tree_plan(parents, ints([0, 5, -3], cuda_dev))
    assert mask[0].tolist() == [plain.signed((2 << t) - 1) for t in range(T)]
    assert pos.view(3, T)[:, -1].tolist() == [63, 68, 63]


# ----------------------------------------------------------------- books

class Cache:
    """The same books on the GPU and in Python, and a pool whose pages hold their tokens'
    names, so that copies can be followed."""

    def __init__(self, lynx, dev, batch, max_pages, num_blocks, page, seed):
        self.lynx, self.dev, self.page = lynx, dev, page
        self.rng = random.Random(seed)
        self.b = plain.Books(batch, max_pages, num_blocks, page)
        self.put()
        self.pools = [torch.zeros((num_blocks, page, 4), dtype=I32, device=dev),
                      torch.zeros((num_blocks, page, 2), dtype=torch.float64, device=dev)]
        self.told = [[] for _ in range(batch)]      # what each sequence has been told

    def put(self):
        self.table, self.kv, self.refs = (ints(v, self.dev) for v in
                                          (self.b.table, self.b.kv, self.b.refs))

    def same(self):
        assert self.table.tolist() == self.b.table
        assert self.kv.tolist() == self.b.kv
        assert self.refs.tolist() == self.b.refs

    def copy(self, src, dst, count=None):
        self.lynx.lynx_cache_copy_pages(self.pools, src, dst, count)

    def grow(self, n):
        got = self.lynx.lynx_cache_reserve(self.table, self.kv, self.refs, ints(n, self.dev),
                                           self.page)
        want = self.b.reserve(n)
        assert tuple(t.tolist() for t in got) == want
        self.same()
        self.copy(got[1], got[2])
        host = self.pools[0].cpu()
        for b, m in enumerate(want[0]):
            for i in range(self.b.kv[b] - m, self.b.kv[b]):
                name = self.rng.randrange(1, 2 ** 31)
                self.told[b].append(name)
                host[self.b.table[b][i // self.page], i % self.page] = name
        self.pools[0].copy_(host)
        self.pools[1].copy_(host[:, :, :2].double())

    def fork(self, source):
        self.table, self.kv = self.lynx.lynx_cache_fork(self.table, self.kv, self.refs,
                                                        ints(source, self.dev), self.page)
        self.b.fork(source)
        self.told = [list(self.told[s]) if 0 <= s < len(self.told) else [] for s in source]
        self.same()

    def trim(self, keep):
        self.lynx.lynx_cache_trim(self.table, self.kv, self.refs, ints(keep, self.dev), self.page)
        self.b.trim(keep)
        self.told = [t[:n] for t, n in zip(self.told, self.b.kv)]
        self.same()

    def compact(self):
        got = self.lynx.lynx_cache_compact(self.table, self.kv, self.refs, self.page)
        src, dst, count = self.b.compact()
        assert (got[0].tolist(), got[1].tolist(), got[2].tolist()) == (src, dst, [count])
        self.same()
        self.copy(*got)

    def read(self):
        """Every sequence reads what it has been told."""
        self.b.check()
        host, more = self.pools[0].cpu(), self.pools[1].cpu()
        for row, n, told in zip(self.b.table, self.b.kv, self.told):
            for i in range(n):
                where = row[i // self.page], i % self.page
                assert host[where].tolist() == [told[i]] * 4 and more[where].tolist() == [told[i]] * 2


@pytest.mark.parametrize("batch,max_pages,num_blocks,page", [
    (1, 3, 4, 64), (5, 6, 24, 64), (7, 4, 20, 128), (12, 3, 64, 256), (3, 2, 5, 512)])
def test_a_life_of_a_cache(lynx_lib, cuda_dev, batch, max_pages, num_blocks, page):
    """Sequences that grow, share, write, are cut back, freed and moved, pages running out
    on the way: books and contents as in Python after every call."""
    before = lynx_lib.lynx_device_errors()    # (other tests plant bad entries)
    c = Cache(lynx_lib, cuda_dev, batch, max_pages, num_blocks, page, batch)
    rng = c.rng
    for step in range(24):
        k = len(c.b.kv)
        do = rng.choice(("grow", "grow", "grow", "fork", "trim", "compact"))
        if do == "grow":
            c.grow([rng.choice((0, 1, 3, page - 1, page, rng.randrange(0, 2 * page), -2))
                    for _ in range(k)])
        elif do == "fork":
            c.fork([rng.choice((-1, rng.randrange(0, k), rng.randrange(0, k)))
                    for _ in range(rng.choice((batch, max(1, batch - 2), batch + 1)))])
        elif do == "trim":
            c.trim([rng.choice((0, n, n + 5, -1, rng.randrange(0, n + 1))) for n in c.b.kv])
        else:
            c.compact()
        c.read()
    assert lynx_lib.lynx_device_errors() == before


@pytest.mark.parametrize("num_blocks", [1, 31, 1024, 1025, 16384, 16385, 20011, 300007])
@pytest.mark.parametrize("batch", [1, 33, 1024, 1025, 2500])
def test_many_pages_and_sequences(lynx_lib, cuda_dev, num_blocks, batch):
    """Free pages anywhere among many, for more sequences than a block has threads."""
    rng = random.Random(num_blocks + batch)
    page, max_pages = 64, 4
    b = plain.Books(batch, max_pages, num_blocks, page)
    pinned = [p for p in range(num_blocks) if rng.random() < (0.97 if num_blocks > 9000 else 0.3)]
    for p in pinned:                                   # pages kept without a sequence
        b.refs[p] = 1
    table, kv, refs = (ints(v, cuda_dev) for v in (b.table, b.kv, b.refs))
    for grow in ([rng.randrange(0, 100) for _ in range(batch)],
                 [rng.randrange(0, 200) for _ in range(batch)]):
        got = lynx_lib.lynx_cache_reserve(table, kv, refs, ints(grow, cuda_dev), page)
        want = b.reserve(grow)
        assert tuple(t.tolist() for t in got) == want
        assert table.tolist() == b.table and kv.tolist() == b.kv and refs.tolist() == b.refs
    keep = [rng.choice((0, n)) for n in b.kv]
    lynx_lib.lynx_cache_trim(table, kv, refs, ints(keep, cuda_dev), page)
    b.trim(keep)
    b.check(pinned)
    got = lynx_lib.lynx_cache_compact(table, kv, refs, page)
    want = b.compact()
    assert (got[0].tolist(), got[1].tolist(), got[2].tolist()) == (want[0], want[1], [want[2]])
    assert table.tolist() == b.table and kv.tolist() == b.kv and refs.tolist() == b.refs


def test_compaction_of_nothing_and_of_all(lynx_lib, cuda_dev):
    for refs in ([0] * 9, [1] * 9, [0, 0, 0, 0, 0, 0, 0, 0, 5], [3, 0, 0, 0, 0, 0, 0, 0, 0], [2], [0]):
        b = plain.Books(1, 2, len(refs), 64)
        b.refs = list(refs)
        args = [ints(v, cuda_dev) for v in (b.table, b.kv, b.refs)]
        got = lynx_lib.lynx_cache_compact(*args, 64)
        want = b.compact()
        assert (got[0].tolist(), got[1].tolist(), int(got[2])) == want
        assert args[2].tolist() == b.refs


def test_captured_steps_follow_the_books(lynx_lib, cuda_dev):
    """Reserve and copy in a graph, replayed while the books change between replays."""
    page = 64
    b = plain.Books(3, 5, 16, page)
    table, kv, refs = (ints(v, cuda_dev) for v in (b.table, b.kv, b.refs))
    grow = ints([1, 1, 1], cuda_dev)
    pool = torch.arange(16 * page, device=cuda_dev, dtype=I32).view(16, page, 1).repeat(1, 1, 4)
    start = [t.clone() for t in (table, kv, refs)]
    lynx_lib.lynx_cache_copy_pages([pool], *lynx_lib.lynx_cache_reserve(table, kv, refs, grow, page)[1:])
    for t, s in zip((table, kv, refs), start):
        t.copy_(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lynx_lib.lynx_cache_reserve(table, kv, refs, grow, page)
        lynx_lib.lynx_cache_copy_pages([pool], out[1], out[2])
    for n in ([70, 3, 0], [5, 62, 64], [1, 1, 1], [200, 1, 1]):
        grow.copy_(ints(n, cuda_dev))
        g.replay()
        assert tuple(t.tolist() for t in out) == b.reserve(n)
        assert table.tolist() == b.table and refs.tolist() == b.refs and kv.tolist() == b.kv


@pytest.mark.parametrize("shapes", [[(16,)], [(4096, 4)], [(3, 64, 2, 128), (4, 7), (1,)],
                                    [(64, 1, 128)] * 70])
def test_copies_of_any_pools(lynx_lib, cuda_dev, shapes):
    n = 37
    kinds = (torch.float64, torch.bfloat16, torch.uint8, torch.int32)
    pools, want = [], []
    g = torch.Generator().manual_seed(len(shapes))
    for i, s in enumerate(shapes):
        kind = kinds[i % 4]
        words = torch.Size(s).numel() * torch.empty(0, dtype=kind).element_size()
        if words % 16:
            s, kind = (*s, 2), torch.float64
        raw = torch.randint(0, 200, (n, *s), generator=g).to(kind)
        pools.append(raw.to(cuda_dev))
        want.append(raw)
    src = [3, -1, 36, 3, 0, 9, 30]
    dst = [4, 5, 7, 1, -1, 8, 31]
    for count in (None, 0, 3, 5, 99, -4):
        m = len(src) if count is None else max(0, min(count, len(src)))
        lynx_lib.lynx_cache_copy_pages(pools, ints(src, cuda_dev), ints(dst, cuda_dev),
                                       None if count is None else ints([count], cuda_dev))
        for a, z in list(zip(src, dst))[:m]:
            if a >= 0 and z >= 0:
                for w in want:
                    w[z] = w[a]
        assert all(torch.equal(p.cpu(), w) for p, w in zip(pools, want))
    lynx_lib.lynx_cache_copy_pages(pools, ints([], cuda_dev), ints([], cuda_dev))
    lynx_lib.lynx_cache_copy_pages([], ints([1], cuda_dev), ints([2], cuda_dev))


# ----------------------------------------------------------------- nodes kept

@pytest.mark.parametrize("batch,T,H_kv,page,layers", [
    (1, 1, 1, 64, 1), (3, 16, 2, 64, 2), (5, 64, 3, 128, 1), (2, 33, 8, 512, 5), (40, 7, 1, 64, 1),
    (2, 9, 4, 256, 64)])
def test_kept_nodes_go_to_their_pages(lynx_lib, cuda_dev, batch, T, H_kv, page, layers):
    rng = random.Random(batch * T)
    b = plain.Books(batch, 4, 4 * batch + 2, page)
    b.reserve([rng.randrange(0, 3 * page) for _ in range(batch)])
    paths = []
    for _ in range(batch):
        n = rng.choice((0, 1, T, rng.randrange(0, T + 1)))
        paths.append(sorted(rng.sample(range(T), n)))
    if batch > 1:
        b.kv[1] = len(paths[1])                        # a sequence that begins with its nodes
    granted = [len(p) if 3 * i % 5 != 4 else 0 for i, p in enumerate(paths)]
    kv = [max(n, g) for n, g in zip(b.kv, granted)]
    b.table = [[rng.randrange(0, 4 * batch + 2) for _ in range(4)] for _ in range(batch)]
    order = list(range(4 * batch + 2))
    rng.shuffle(order)
    b.table = [order[4 * i:4 * i + 4] for i in range(batch)]
    g = torch.Generator().manual_seed(T)
    nodes = [torch.randn((batch, 64, H_kv, 128), generator=g).to(torch.bfloat16)
             for _ in range(2 * layers)]
    pools = [torch.randn((4 * batch + 2, page, H_kv, 128), generator=g).to(torch.bfloat16)
             for _ in range(2 * layers)]
    d_pools = [p.to(cuda_dev) for p in pools]
    path = ints([p + [-1] * (T - len(p)) for p in paths], cuda_dev)
    lynx_lib.lynx_cache_keep([t.to(cuda_dev) for t in nodes], d_pools, path,
                             ints(granted, cuda_dev), ints(kv, cuda_dev), ints(b.table, cuda_dev))
    for s in range(batch):
        for i in range(granted[s]):
            at = kv[s] - granted[s] + i
            for x, p in zip(nodes, pools):
                p[b.table[s][at // page], at % page] = x[s, paths[s][i]]
    assert all(torch.equal(p.cpu().view(torch.int16), w.view(torch.int16))
               for p, w in zip(d_pools, pools))


def test_as_many_pools_as_a_call_takes(lynx_lib, cuda_dev):
    n, page = 256, 64
    g = torch.Generator().manual_seed(2)
    both = torch.randn((2, n, 3, page, 1, 128), generator=g).to(torch.bfloat16)
    pools, nodes = both[0].to(cuda_dev), both[1, :, :2].contiguous().to(cuda_dev)
    lynx_lib.lynx_cache_copy_pages(list(pools), ints([2], cuda_dev), ints([0], cuda_dev))
    lynx_lib.lynx_cache_keep(list(nodes), list(pools), ints([[5], [0]], cuda_dev),
                             ints([1, 1], cuda_dev), ints([64, 1], cuda_dev),
                             ints([[1], [2]], cuda_dev))
    want = both[0].clone()
    want[:, 0] = want[:, 2]
    want[:, 1, 63], want[:, 2, 0] = both[1, :, 0, 5], both[1, :, 1, 0]
    assert torch.equal(pools.cpu().view(torch.int16), want.view(torch.int16))


def test_more_room_than_nodes(lynx_lib, cuda_dev):
    """granted above what the path holds, and above T: the nodes go to the first of the new
    positions, the others are left as they are, and nothing is reported."""
    page = 64
    pool = torch.full((4, page, 1, 128), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    nodes = torch.arange(2 * 64, device=cuda_dev).view(2, 64, 1, 1).expand(2, 64, 1, 128)
    nodes = nodes.to(torch.bfloat16).contiguous()
    table, kv = ints([[2, 0], [3, 1]], cuda_dev), ints([66, 10], cuda_dev)
    errors = lynx_lib.lynx_device_errors()
    lynx_lib.lynx_cache_keep([nodes], [pool], ints([[0, 2, -1], [0, 1, 2]], cuda_dev),
                             ints([4, 6], cuda_dev), kv, table)
    want = torch.full((4, page), 7.0)
    want[2, 62], want[2, 63] = 0.0, 2.0
    want[3, 4:7] = torch.tensor([64.0, 65.0, 66.0])
    assert torch.equal(pool.float().cpu(), want.view(4, page, 1, 1).expand(4, page, 1, 128))
    assert lynx_lib.lynx_device_errors() == errors


def test_pools_beyond_32_bits(lynx_lib, cuda_dev):
    """Pages whose bytes, and whose values, lie beyond 2^32."""
    page, H_kv, blocks = 64, 8, 66_000                 # 4.3e9 values, 8.7 GB
    pool = torch.empty((blocks, page, H_kv, 128), dtype=torch.bfloat16, device=cuda_dev)
    low, high = 5, blocks - 1
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    for p in (low, high, high - 1):
        pool[p] = torch.randn((page, H_kv, 128), generator=g, device=cuda_dev).to(torch.bfloat16)
    want = pool[high - 1].clone()
    lynx_lib.lynx_cache_copy_pages([pool], ints([high - 1, low], cuda_dev), ints([6, high], cuda_dev))
    assert torch.equal(pool[6], want) and torch.equal(pool[high], pool[low])
    nodes = torch.randn((1, 64, H_kv, 128), generator=g, device=cuda_dev).to(torch.bfloat16)
    before = pool[high].clone()
    lynx_lib.lynx_cache_keep([nodes], [pool], ints([[0, 3]], cuda_dev), ints([2], cuda_dev),
                             ints([12], cuda_dev), ints([[high]], cuda_dev))
    assert torch.equal(pool[high, 10], nodes[0, 0]) and torch.equal(pool[high, 11], nodes[0, 3])
    assert torch.equal(pool[high, :10], before[:10]) and torch.equal(pool[high, 12:], before[12:])


@own_process
def test_bad_entries_are_reported_and_touch_nothing(lynx_lib, cuda_dev):
    errors = lynx_lib.lynx_device_errors()
    assert errors & 6 == 0                    # (a process of its own)
    page = 64

    def reported(bit):
        nonlocal errors
        new = lynx_lib.lynx_device_errors()
        assert new & bit, "not reported"
        errors = new

    # a row that names what is no page, and a length beyond the table's room
    table = ints([[7, 99], [-1, 3], [1, 2]], cuda_dev)
    kv = ints([100, 65, 5000], cuda_dev)
    refs = ints([0, 1, 1, 1, 0, 0, 0, 1], cuda_dev)
    out, n = lynx_lib.lynx_cache_fork(table, kv, refs, ints([0, 1, 2, 3, -5], cuda_dev), page)
    assert out.tolist() == [[7, -1], [-1, 3], [1, 2], [-1, -1], [-1, -1]]
    assert n.tolist() == [100, 65, 128, 0, 0]
    assert refs.tolist() == [0, 1, 1, 1, 0, 0, 0, 1]
    reported(2)
    granted, src, dst = lynx_lib.lynx_cache_reserve(out, n, refs, ints([1, 63, 1, 0, 64], cuda_dev),
                                                    page)
    assert granted.tolist() == [1, 63, 0, 0, 64] and src.tolist() == dst.tolist() == [-1] * 5
    assert out[4].tolist() == [0, -1] and refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 1]
    lynx_lib.lynx_cache_trim(out, n, refs, ints([0] * 5, cuda_dev), page)
    assert refs.tolist() == [0] * 8 and n.tolist() == [0] * 5 and (out == -1).all()
    # copies and nodes to and from where nothing is
    pool = torch.arange(8 * 64 * 128, device=cuda_dev, dtype=torch.float32).view(8, 64, 1, 128)
    pool = pool.to(torch.bfloat16)
    before = pool.clone()
    lynx_lib.lynx_cache_copy_pages([pool], ints([8, 2 ** 31 - 1, 0], cuda_dev),
                                   ints([1, 2, 8], cuda_dev))
    nodes = torch.zeros((2, 64, 1, 128), dtype=torch.bfloat16, device=cuda_dev)
    lynx_lib.lynx_cache_keep([nodes], [pool], ints([[64, -1, 5], [0, 1, 2]], cuda_dev),
                             ints([2, 3], cuda_dev), ints([2, 3], cuda_dev),
                             ints([[0], [8]], cuda_dev))
    assert torch.equal(pool, before)
    # a given token behind the vocabulary
    x = torch.zeros((1, 4), device=cuda_dev)
    lp = lynx_lib.lynx_token_logprobs(x, ints([[4, 3]], cuda_dev))[0]
    assert lp[0, 0] == -float("inf") and abs(float(lp[0, 1]) + 1.3862943611198906) < 1e-6
    reported(4)


def test_a_page_held_without_a_sequence_is_followed_through_a_compaction(lynx_lib, cuda_dev):
    """A caller's own page moves as the others do, and is found where copy_dst says."""
    page, held = 64, 6
    pool = torch.arange(8, device=cuda_dev).view(8, 1, 1, 1).expand(8, page, 1, 128)
    pool = pool.to(torch.bfloat16).contiguous()
    table, kv = ints([[7, 3]], cuda_dev), ints([100], cuda_dev)
    refs = ints([0, 0, 0, 1, 0, 0, 1, 1], cuda_dev)
    src, dst, count = lynx_lib.lynx_cache_compact(table, kv, refs, page)
    lynx_lib.lynx_cache_copy_pages([pool], src, dst, count)
    moves = dict(zip(src.tolist()[:int(count)], dst.tolist()[:int(count)]))
    assert moves == {3: 0, 6: 1, 7: 2} and table.tolist() == [[2, 0]]
    assert refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    assert pool[moves[held]].eq(held).all() and pool[2].eq(7).all() and pool[0].eq(3).all()
    # a sequence that begins with it, and grows on a page of its own
    table, kv = ints([[moves[held], -1]], cuda_dev), ints([page], cuda_dev)
    refs[moves[held]] += 1
    granted, src, dst = lynx_lib.lynx_cache_reserve(table, kv, refs, ints([1], cuda_dev), page)
    assert granted.tolist() == [1] and table.tolist() == [[1, 3]] and src.tolist() == [-1]
