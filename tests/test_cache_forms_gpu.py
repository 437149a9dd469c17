"""Prefill over the BF16 paged cache where its work is shared out in ways that few shapes
reach: the last units cut in parts, and CTAs that take over several units of one and
of both row halves.  Against the definitions in 64 bits, and in the checked build."""
import functools
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from . import cache_forms as forms
from . import cache_plain as plain
from .test_cache_gpu import BF, _cache, _rand

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
PARTS = ("long", "short last", "negative", "nothing", "absent", "heads")
SCORES = {"plain": {}, "cap": dict(softcap=20.0), "bias": dict(slopes=0.05),
          "masks": dict(window=700, prefix=90), "all": dict(softcap=20.0, slopes=0.05, window=150,
                                                            prefix=200)}
DISTINCT = 7        # KV heads that differ: the others repeat them, so that 64 bits stay cheap


def _sms(dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count


@functools.lru_cache(maxsize=None)
def _inputs(case, seed):
    """q, k_pool, v_pool of the DISTINCT heads, table, lengths (CPU)."""
    counts, kv, H_q, H_kv, page, _, pages = case
    kp, vp, table, lens = _cache(list(kv), page, DISTINCT, seed, max_pages=pages)
    return _rand((sum(counts), DISTINCT * (H_q // H_kv), 128), seed + 1, 2.0), kp, vp, table, lens


def _frozen(case):
    return (tuple(case[0]), tuple(case[1])) + tuple(case[2:])


def _spread(case):
    """Indexes of the distinct KV heads and query heads that the call's heads repeat."""
    _, _, H_q, H_kv = case[:4]
    G = H_q // H_kv
    kvh = torch.arange(H_kv) % DISTINCT
    return kvh, (kvh[:, None] * G + torch.arange(G)).flatten()


def _score_args(kw, case):
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = torch.linspace(0.0, kw["slopes"], DISTINCT * (case[2] // case[3]))
    if "prefix" in kw:
        kw["prefix"] = torch.tensor([kw["prefix"] if b % 2 == 0 else 0 for b in range(len(case[0]))],
                                    dtype=torch.int32)
    return kw


def _call(lynx, dev, case, q, kp, vp, table, lens, kw):
    """(out, lse) of one call on all heads."""
    kvh, qh = _spread(case)
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"][qh]
    on = {k: v.to(dev) if torch.is_tensor(v) else v for k, v in kw.items()}
    pools = [p.to(dev)[:, :, kvh.to(dev)].contiguous() for p in (kp, vp)]
    qd = q.to(dev)[:, qh.to(dev)].contiguous()
    out, lse = torch.full_like(qd, 7.0), torch.full(qd.shape[:2], 7.0, device=dev)
    lynx.lynx_cache_attn_prefill(qd, plain.offsets_of(case[0]).to(dev), *pools, table.to(dev),
                                 lens.to(dev), out=out, lse=lse, **on)
    return out, lse


def _compare(lynx, dev, case, score):
    case = _frozen(case)
    q, kp, vp, table, lens = _inputs(case, 60)
    kw = _score_args(SCORES[score], case)
    want = plain.attention(q, list(case[0]), list(case[1]), table, kp, vp, **kw)
    out, lse = _call(lynx, dev, case, q, kp, vp, table, lens, kw)
    qh = _spread(case)[1]
    plain.assert_close(lse, want[1][:, qh], want[3][:, qh], "lse")
    plain.assert_close(out, want[0][:, qh], want[2][:, qh], "out")
    again = _call(lynx, dev, case, q, kp, vp, table, lens, kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    return out, lse


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("name", PARTS)
def test_last_units_in_parts(lynx_lib, cuda_dev, name, score):
    case = forms.parts_cases(lynx_lib, _sms(cuda_dev))[name]
    assert forms.form_of(lynx_lib, *case, _sms(cuda_dev)) == lynx_lib.LYNX_CACHE_PARTS
    _compare(lynx_lib, cuda_dev, case, score)


@pytest.mark.parametrize("score", SCORES)
def test_several_units_to_a_cta(lynx_lib, cuda_dev, score):
    """And bit for bit what the same sequences give in a call of their own."""
    case = forms.TAKEOVER
    assert forms.form_of(lynx_lib, *case, _sms(cuda_dev)) == lynx_lib.LYNX_CACHE_WHOLE
    out, lse = _compare(lynx_lib, cuda_dev, case, score)
    q, kp, vp, table, lens = _inputs(_frozen(case), 60)
    kw = _score_args(SCORES[score], case)
    at = 0
    for b, (n, kv) in enumerate(zip(*case[:2])):
        one = ([n], [kv]) + case[2:]
        if n:
            assert forms.form_of(lynx_lib, *one, _sms(cuda_dev)) == lynx_lib.LYNX_CACHE_WHOLE
            own = dict(kw)
            if "prefix" in own:
                own["prefix"] = own["prefix"][b:b + 1]
            o, l = _call(lynx_lib, cuda_dev, one, q[at:at + n], kp, vp, table[b:b + 1].contiguous(),
                         lens[b:b + 1], own)
            assert torch.equal(o, out[at:at + n]) and torch.equal(l, lse[at:at + n]), b
        at += n


def run_cases():
    """{name: outputs' bits} of every form here, for the checked build."""
    from split_stream_kv_gb300 import lynx
    dev, found = torch.device("cuda:0"), {}
    cases = dict(forms.parts_cases(lynx, _sms(dev)), takeover=forms.TAKEOVER)
    for name, case in cases.items():
        case = _frozen(case)
        for score in ("plain", "all"):
            out, lse = _call(lynx, dev, case, *_inputs(case, 61), _score_args(SCORES[score], case))
            found[f"{name} {score} out"] = out.view(torch.int16).cpu().numpy()
            found[f"{name} {score} lse"] = lse.cpu().numpy()
    torch.cuda.synchronize()
    found["errors"] = np.array([lynx.lynx_device_errors()])
    found["library"] = np.frombuffer(os.path.basename(lynx.LIB_PATH).encode(), dtype="uint8")
    return found


def test_checked_build_matches_and_no_check_fires(lynx_lib, cuda_dev, tmp_path):
    before = lynx_lib.lynx_device_errors()
    path = tmp_path / "checked.npz"
    r = subprocess.run([sys.executable, "-m", "tests.test_cache_forms_gpu", str(path)],
                       cwd=os.path.dirname(HERE), env=dict(os.environ, LYNX_LIBRARY="checked"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    checked = dict(np.load(path))
    assert bytes(checked["library"]).decode() == "liblynx_checked.so"
    assert int(checked["errors"][0]) == 0, "an index check fired"
    here = run_cases()
    assert int(here["errors"][0]) == before
    assert sorted(here) == sorted(checked)
    for k in here:
        if k not in ("library", "errors"):
            assert np.array_equal(here[k], checked[k], equal_nan="lse" in k), k


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_cases())
