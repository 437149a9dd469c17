"""The checked build (liblynx_checked.so: every kernel verifies its index arithmetic and
records a failed check in lynx_device_errors bit 8) on tree drafting and the paged
cache's books: the outputs equal the regular build's bit for bit, and no check fires.
The checked build runs in a child process."""
import os
import random
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def run_cases():
    """{name: bytes of the outputs}."""
    import torch

    from split_stream_kv_gb300 import lynx
    from tests import cache_plain, tree_plain
    dev, out = torch.device("cuda:0"), {}
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def keep(name, *tensors):
        for i, t in enumerate(tensors):
            out[f"{name} {i}"] = t.contiguous().view(torch.uint8).cpu().numpy()

    for rows, V, top in ((3, 5001, 8), (500, 9000, 3), (40, 70001, 32)):
        x = rand(rows, V)
        keep(f"logprobs {rows}", *lynx.lynx_token_logprobs(x, ints([[0, V - 1]] * rows), top))
    for name, T, kv, H_q, H_kv, page, wide, kw in (
            ("clusters", 5, [700, 65], 8, 2, 64, None, {}),
            ("split", 3, [9000, 0, 130], 16, 2, 256, None, dict(softcap=30.0)),
            ("whole", 40, [70, 0, 501], 10, 2, 128, None, dict(window=100)),
            ("shares", 64, [5000, 2500], 16, 1, 512, None, {}),
            ("parts", 17, [(i * 97) % 300 for i in range(85)], 4, 2, 64, 40, {}),
            ("lent", 12, [6100] + [17] * 13, 32, 8, 64, 130, {})):
        table, blocks = cache_plain.table_for(kv, page, 2, len(name), wide)
        batch = len(kv)
        rng = random.Random(T)
        parents = ints([[-1] + [rng.randrange(max(0, t - 4), t) for t in range(1, T)]] * batch)
        lens = ints(kv)
        mask, pos = lynx.lynx_tree_plan(parents, lens)
        lse = torch.empty((batch, T, H_q), device=dev)
        o = lynx.lynx_cache_attn_tree(rand(batch, T, H_q, 128), rand(batch, 64, H_kv, 128),
                                      rand(batch, 64, H_kv, 128), mask,
                                      rand(blocks, page, H_kv, 128), rand(blocks, page, H_kv, 128),
                                      table.to(dev), lens, lse=lse, **kw)
        keep(name, mask, pos, o, lse)
    for num_blocks in (60, 20000):
        b = tree_plain.Books(9, 4, num_blocks, 64)
        table, kv, refs = (ints(v) for v in (b.table, b.kv, b.refs))
        pool = rand(num_blocks, 64, 1, 128)
        lynx.lynx_cache_reserve(table, kv, refs, ints([30 * i for i in range(9)]), 64)
        table, kv = lynx.lynx_cache_fork(table, kv, refs, ints([1, 1, 3, 3, 8, 8, 8, -1, 0]), 64)
        got = lynx.lynx_cache_reserve(table, kv, refs, ints([3] * 9), 64)
        lynx.lynx_cache_copy_pages([pool], got[1], got[2])
        lynx.lynx_cache_keep([rand(9, 64, 1, 128)], [pool], ints([[0, 4, 63]] * 9), got[0], kv, table)
        lynx.lynx_cache_trim(table, kv, refs, ints([0, 70, 5, 500, 100, 0, 1, 9, 0]), 64)
        moves = lynx.lynx_cache_compact(table, kv, refs, 64)
        lynx.lynx_cache_copy_pages([pool], *moves)
        keep(f"books {num_blocks}", table, kv, refs, pool, *got, *moves)
    torch.cuda.synchronize()
    out["errors"] = np.array([lynx.lynx_device_errors()])
    out["library"] = np.frombuffer(os.path.basename(lynx.LIB_PATH).encode(), dtype="uint8")
    return out


def test_checked_build_matches_and_no_check_fires(lynx_lib, cuda_dev, tmp_path):
    before = lynx_lib.lynx_device_errors()
    path = tmp_path / "checked.npz"
    r = subprocess.run([sys.executable, "-m", "tests.test_tree_checked_gpu", str(path)], cwd=ROOT,
                       env=dict(os.environ, LYNX_LIBRARY="checked"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    checked = dict(np.load(path))
    assert bytes(checked["library"]).decode() == "liblynx_checked.so"
    assert int(checked["errors"][0]) == 0, "an index check fired"
    plain = run_cases()
    assert int(plain["errors"][0]) == before
    assert sorted(plain) == sorted(checked)
    for k in plain:
        if k not in ("library", "errors"):
            assert np.array_equal(plain[k], checked[k]), k


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_cases())
