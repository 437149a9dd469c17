"""Attention over the BF16 paged cache in company: every way its work is shared out, on
several streams and from several threads at once, and captured into graphs that are
replayed over other lengths.  A call's result does not depend on what runs beside it,
so all are compared bit for bit with the call alone."""
import threading

import pytest
import torch

from . import cache_forms as forms
from . import cache_plain as plain
from .test_cache_edges_gpu import FORMS
from .test_cache_gpu import _cache, _rand

pytestmark = pytest.mark.gpu


def _cases(lynx, dev):
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    found = dict(FORMS, takeover=forms.TAKEOVER)
    found["prefill parts"] = forms.parts_cases(lynx, sms)["short last"]
    return found


class _Call:
    """One call's inputs on the device; run() makes it with a workspace of its own."""

    def __init__(self, lynx, dev, case, seed):
        counts, kv, H_q, H_kv, page, self.decode, pages = case
        self.lynx, self.kv = lynx, kv
        args = _cache(list(kv), page, H_kv, seed, max_pages=pages)
        self.pools = [p.nan_to_num(0.25).to(dev) for p in args[:2]]
        self.table, self.lens = args[2].clamp(min=0).to(dev), args[3].to(dev)
        q = _rand((sum(counts), H_q, 128), seed + 1, 2.0).to(dev)
        self.q = q.view((len(counts), counts[0]) + tuple(q.shape[1:])) if self.decode else q
        self.off = plain.offsets_of(counts).to(dev)
        shape = (len(counts), H_q, H_kv, 128, page, self.table.shape[1])
        need = lynx.lynx_cache_attn_decode_workspace_bytes(shape[0], counts[0], *shape[1:]) \
            if self.decode else lynx.lynx_cache_attn_prefill_workspace_bytes(
                sum(counts), *shape)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None

    def run(self, out=None, lse=None):
        lse = torch.empty(self.q.shape[:-1], device=self.q.device) if lse is None else lse
        kw = dict(lse=lse, workspace=self.ws, softcap=25.0, out=out)
        rest = (*self.pools, self.table, self.lens)
        if self.decode:
            return self.lynx.lynx_cache_attn_decode(self.q, *rest, **kw), lse
        return self.lynx.lynx_cache_attn_prefill(self.q, self.off, *rest, **kw), lse


def _same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


def test_every_form_at_once_on_streams(lynx_lib, cuda_dev):
    calls = {n: _Call(lynx_lib, cuda_dev, c, 70) for n, c in _cases(lynx_lib, cuda_dev).items()}
    alone = {n: c.run() for n, c in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(12):
        for i, (n, c) in enumerate(calls.items()):
            # each call stays on one stream (its workspace is its own), in changing company
            with torch.cuda.stream(streams[i % 4]):
                if (i + r) % 3:
                    got.append((n, c.run()))
    torch.cuda.synchronize()
    assert all(_same(x, alone[n]) for n, x in got)
    assert lynx_lib.lynx_wait_timeouts() == 0


def test_every_form_from_threads(lynx_lib, cuda_dev):
    cases = _cases(lynx_lib, cuda_dev)
    alone = {n: _Call(lynx_lib, cuda_dev, c, 71).run() for n, c in cases.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(order):
        with torch.cuda.stream(torch.cuda.Stream()):
            calls = [(n, _Call(lynx_lib, cuda_dev, cases[n], 71)) for n in order]
            for _ in range(4):
                got = [(n, c.run()) for n, c in calls]
                torch.cuda.current_stream().synchronize()
                wrong.extend(n for n, x in got if not _same(x, alone[n]))

    names = list(cases)
    threads = [threading.Thread(target=work, args=(names[i:] + names[:i],)) for i in (0, 3, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert lynx_lib.lynx_wait_timeouts() == 0


def test_every_form_replayed_over_other_lengths(lynx_lib, cuda_dev):
    """Two graphs of each call, captured over other lengths than they are replayed
    with, and replayed on two streams at once with workspaces and outputs of their own."""
    for n, case in _cases(lynx_lib, cuda_dev).items():
        pair = [_Call(lynx_lib, cuda_dev, case, 72) for _ in range(2)]
        graphs, outs = [], []
        for c in pair:
            c.run()
            out = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:-1], 7.0, device=cuda_dev)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.run(*out)
            graphs.append(g)
            outs.append(out)
        for kv in ([max(0, k - 1 - 67 * (i % 2)) for i, k in enumerate(case[1])],
                   [0] * len(case[1]), list(case[1]), [k // 3 for k in case[1]]):
            for c in pair:
                c.lens.copy_(torch.tensor(kv, dtype=torch.int32))
            want = pair[0].run()
            torch.cuda.synchronize()
            streams = [torch.cuda.Stream() for _ in graphs]
            for o in outs:
                o[0].fill_(9.0)
                o[1].fill_(9.0)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
                    g.replay()
            torch.cuda.synchronize()
            assert _same(outs[0], want) and _same(outs[1], want), (n, kv)
    assert lynx_lib.lynx_wait_timeouts() == 0
    assert lynx_lib.lynx_device_errors() & ~2 == 0
