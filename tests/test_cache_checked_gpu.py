"""The checked build (liblynx_checked.so: every kernel verifies its index arithmetic
and records a failed check in lynx_device_errors bit 8) on the BF16 paged
cache: the outputs equal the regular build's bit for bit, and no check fires.
The checked build runs in a child process."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def run_cases():
    """{name: bytes of the outputs}: append, decode as clusters, split and joined,
    prefill whole, cut in shares and with its last units in parts."""
    import torch

    from split_stream_kv_gb300 import lynx
    from tests import cache_plain as plain
    dev, out = torch.device("cuda:0"), {}
    for name, counts, kv, H_q, H_kv, page, wide, kw in (
            ("clusters", [3, 3], [700, 65], 8, 2, 64, 0, {}),
            ("split", [1, 1, 1], [9000, 0, 130], 16, 2, 256, 0, dict(softcap=30.0)),
            ("split rows", [8, 8], [5000, 2], 16, 2, 64, 0, dict(window=300, prefix=True)),
            ("whole", [70, 0, 301], [70, 9, 500], 10, 2, 128, 0, dict(slopes=True)),
            ("shares", [40, 3], [9000, 2500], 8, 1, 512, 0, {}),
            ("parts", [30, 1, 0, 7], [2500, 700, 5, 40], 40, 40, 256, 0, dict(softcap=20.0))):
        table, blocks = plain.table_for(kv, page, 2, seed=len(name))
        g = torch.Generator().manual_seed(len(name))
        n = sum(counts)

        def rand(*shape):
            return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)

        kp, vp = rand(blocks, page, H_kv, 128), rand(blocks, page, H_kv, 128)
        lens = torch.tensor(kv, dtype=torch.int32, device=dev)
        off = plain.offsets_of(counts).to(dev)
        tab = table.to(dev)
        q = lynx.lynx_cache_append(rand(n, H_kv, 128), rand(n, H_kv, 128), off, lens, tab, kp, vp,
                                   q=rand(n, H_q, 128),
                                   rope=lynx.Rope(lynx.rope_frequencies(1e6, 96)))
        kw = dict(kw)
        if kw.pop("slopes", None):
            kw["slopes"] = torch.linspace(0.01, 0.5, H_q, device=dev)
        if kw.pop("prefix", None):
            kw["prefix"] = torch.full((len(kv),), 70, dtype=torch.int32, device=dev)
        if len(set(counts)) == 1:
            o = lynx.lynx_cache_attn_decode(q.view(len(kv), counts[0], H_q, 128), kp, vp, tab, lens,
                                            **kw)
        else:
            o = lynx.lynx_cache_attn_prefill(q, off, kp, vp, tab, lens, **kw)
        for k, t in (("q", q), ("k", kp), ("v", vp), ("out", o)):
            out[f"{name} {k}"] = t.contiguous().view(torch.uint8).cpu().numpy()
    torch.cuda.synchronize()
    out["errors"] = np.array([lynx.lynx_device_errors()])
    out["library"] = np.frombuffer(os.path.basename(lynx.LIB_PATH).encode(), dtype="uint8")
    return out


def test_checked_build_matches_and_no_check_fires(lynx_lib, cuda_dev, tmp_path):
    before = lynx_lib.lynx_device_errors()
    path = tmp_path / "checked.npz"
    r = subprocess.run([sys.executable, "-m", "tests.test_cache_checked_gpu", str(path)], cwd=ROOT,
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
