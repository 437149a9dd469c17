"""Refusals and host-only parts of the BF16 paged cache that test_cache_host.py does
not reach: no GPU."""
import pytest

from .test_cache_host import FAR, _append


@pytest.mark.parametrize("over", [
    dict(k=FAR[2]), dict(v=FAR[2]), dict(off=FAR[2]), dict(kv=FAR[2]), dict(table=FAR[2]),
    dict(k=FAR[2], k_stride=4096), dict(v=FAR[2], v_stride=4096, n=1)])
def test_queries_in_place_over_another_input(lynx_lib, over):
    """q_out may be q; what else lies at the address of q is not exempt."""
    a = dict(q_out=FAR[2], H_q=32, q_stride=4096)
    a.update(over)
    assert _append(lynx_lib.lib(), lynx_lib, **a) == -1, lynx_lib.lynx_last_error()
    assert "q_out overlaps" in lynx_lib.lynx_last_error()


def test_queries_in_place_over_the_positions(lynx_lib):
    import ctypes
    f = (ctypes.c_double * 8)(*([1.0] * 8))
    rope = lynx_lib.LynxRope(16, 0, 1, 0, ctypes.addressof(f), None, FAR[2].value)
    assert _append(lynx_lib.lib(), lynx_lib, q_out=FAR[2], rope=rope) == -1
    assert "q_out overlaps positions" in lynx_lib.lynx_last_error()


def test_dependent_kernels_read_with_coherent_loads():
    """The cache's kernels may be resident while the kernel before them still writes
    their inputs (they start as programmatic dependents).  ld.global.nc, which __ldg
    and the streaming helpers are, is for data that nobody writes as long as a kernel
    lives: no ordering makes it right there, so no source of theirs may use it."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "split_stream_kv_gb300", "csrc")
    found = glob.glob(os.path.join(csrc, "cache*"))
    assert len(found) >= 6
    for path in found:
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        hits = re.findall(r"__ldg\w*|ldg_stream\w*|ld\.global\.nc|__restrict__|LDG", code)
        assert not hits, f"{os.path.basename(path)}: {hits}"


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(batch=(1 << 23) + 1, H_kv=8, T=1, n=1), -3), (dict(batch=1 << 27, H_kv=1, H_q=1, T=1, n=1), -3),
    (dict(batch=1 << 23, H_kv=8, T=1, n=1, kv=None), -1)])
def test_attention_rejects_batches_it_could_not_walk(lynx_lib, prefill, over, code):
    """The largest batch gets as far as the next check, a larger one is refused."""
    from .test_cache_host import _attn
    over = dict(dict(H_q=8, ws_bytes=1 << 50), **over)
    assert _attn(lynx_lib.lib(), prefill, **over) == code, lynx_lib.lynx_last_error()
