"""What the books' calls do with entries that are no pages: each reports them
(lynx_device_errors bit 2) and touches nothing else.  The error words are never reset, so
every call has a process of its own, six at a time."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PAGE = 64


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda:0")


def _pool():
    import torch
    pool = torch.arange(8 * PAGE * 128, device="cuda:0", dtype=torch.float32)
    return pool.view(8, PAGE, 1, 128).to(torch.bfloat16)


def fork(lynx, bad):
    """A row names block 9 of 8; or a source from the batch on."""
    table, kv = _ints([[7, 9 if bad == "entry" else 1], [-1, 3]]), _ints([100, 0])
    refs = _ints([0, 1, 0, 0, 0, 0, 0, 1])
    out, n = lynx.lynx_cache_fork(table, kv, refs, _ints([0, 2 if bad == "source" else -1, -5]),
                                  PAGE)
    assert out.tolist() == [[7, -1 if bad == "entry" else 1], [-1, -1], [-1, -1]]
    assert n.tolist() == [100, 0, 0]
    assert refs.tolist() == [0, 1, 0, 0, 0, 0, 0, 1]


def reserve(lynx, bad, batch=1, num_blocks=8):
    """The last page, which has room, is none."""
    table = _ints([[{"above": num_blocks, "below": -1}.get(bad, 3), -1]] * batch)
    kv = _ints([10] * batch)
    refs = _ints([0, 0, 0, batch] + [0] * (num_blocks - 4))
    granted, src, dst = lynx.lynx_cache_reserve(table, kv, refs, _ints([0] * (batch - 1) + [20]),
                                                PAGE)
    assert granted.tolist() == [0] * (batch - 1) + [20]
    assert kv.tolist() == [10] * (batch - 1) + [30]
    if bad or batch == 1:
        assert src.tolist() == dst.tolist() == [-1] * batch
        assert refs.tolist() == [0, 0, 0, batch] + [0] * (num_blocks - 4)


def reserve_cluster(lynx, bad):
    reserve(lynx, bad, 1030, 20000)


def trim(lynx, bad):
    """What is cut off holds an entry that is no page."""
    table = _ints([[2, {"above": 8, "below": -1}.get(bad, 5), 6]])
    kv, refs = _ints([3 * PAGE]), _ints([0, 0, 1, 0, 0, 1, 1, 0])
    lynx.lynx_cache_trim(table, kv, refs, _ints([5]), PAGE)
    assert table.tolist() == [[2, -1, -1]] and kv.tolist() == [5]
    assert refs.tolist() == [0, 0, 1, 0, 0, 1 if bad else 0, 0, 0]


def copy_pages(lynx, bad):
    pool = _pool()
    want = pool.clone()
    want[2] = want[1]
    src, dst = [1, -1, -1], [2, 5, -7]
    if bad == "source":
        src[1] = 8
    elif bad == "destination":
        src[1], dst[1] = 0, 2 ** 31 - 1
    lynx.lynx_cache_copy_pages([pool], _ints(src), _ints(dst))
    assert (pool == want).all()


def keep(lynx, bad):
    import torch
    pool = _pool()
    want = pool.clone()
    nodes = torch.zeros((2, 64, 1, 128), dtype=torch.bfloat16, device="cuda:0")
    path, table = [[63, -1, 5], [0, 1, 2]], [[0, 1], [4, 3]]
    want[0, 0] = 0
    if bad == "node":
        path[0][1] = 64
    if bad == "block":
        table[1][0] = 8
    elif bad == "none":
        table[1][0] = -1
    elif bad != "room":
        want[4, :3] = 0
    kv = [2, 3]
    if bad == "room":                      # a length beyond the table's room
        kv[1] = 2 * PAGE + 3
    lynx.lynx_cache_keep([nodes], [pool], _ints(path), _ints([2, 3]), _ints(kv), _ints(table))
    assert (pool == want).all()


def compact(lynx, bad, batch=2, max_pages=3, moves=True):
    """A row of 2 pages holds an entry that is none; what is behind it may be -1."""
    num_blocks = 8
    rows = [[-1] * max_pages for _ in range(batch)]
    rows[batch - 1][:2] = [6 if moves else 0, {"above": 8, "below": -2, "none": -1}.get(bad, 1)]
    lens = [0] * (batch - 1) + [PAGE + 1]
    refs = [0] * num_blocks
    for p in rows[batch - 1][:2]:
        if 0 <= p < num_blocks:
            refs[p] = 1
    table, kv, counts = _ints(rows), _ints(lens), _ints(refs)
    src, dst, count = lynx.lynx_cache_compact(table, kv, counts, PAGE)
    at = {6: 0} if moves else {}
    assert count.tolist() == [len(at)]
    assert src.tolist() == ([6] if moves else []) + [-1] * (num_blocks // 2 - len(at))
    assert dst.tolist() == ([0] if moves else []) + [-1] * (num_blocks // 2 - len(at))
    assert table.tolist() == [[at.get(p, p) for p in row] for row in rows]
    assert counts.tolist() == [1, 0 if bad else 1] + [0] * 6 and kv.tolist() == lens


def compact_in_place(lynx, bad):
    compact(lynx, bad, moves=False)


def compact_large(lynx, bad):
    compact(lynx, bad, 30, 1001)


def compact_large_in_place(lynx, bad):
    compact(lynx, bad, 30, 1001, moves=False)


CASES = {fork: ["entry", "source"], reserve: ["above"], reserve_cluster: ["below"],
         trim: ["above", "below"], copy_pages: ["source", "destination"],
         keep: ["node", "block", "none", "room"], compact: ["above", "below", "none"],
         compact_in_place: ["none"], compact_large: ["above", "none"],
         compact_large_in_place: ["above", "none"]}
NAMES = [f"{fn.__name__}-{bad}" for fn, kinds in CASES.items() for bad in kinds]


def child(name):
    """The right call first, which reports nothing, then the bad one."""
    from split_stream_kv_gb300 import lynx
    fn, bad = name.split("-")
    call = {f.__name__: f for f in CASES}[fn]
    call(lynx, "")
    assert lynx.lynx_device_errors() == 0, "reported without a cause"
    call(lynx, bad)
    assert lynx.lynx_device_errors() == 2, "not reported"


@pytest.fixture(scope="module")
def children(lynx_lib, cuda_dev):
    def run(name):
        code = f"from tests import test_tree_reports_gpu as t; t.child({name!r})"
        return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True,
                              text=True, timeout=300)
    with ThreadPoolExecutor(6) as pool:
        return dict(zip(NAMES, pool.map(run, NAMES)))


@pytest.mark.parametrize("name", NAMES)
def test_an_entry_that_is_no_page_is_reported(children, name):
    assert children[name].returncode == 0, children[name].stderr[-2000:]
