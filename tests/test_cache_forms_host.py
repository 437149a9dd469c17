"""How attention over the BF16 paged cache shares out its work: the rules as the library
gives them, and that the tests' calls reach each form.  No GPU."""
import pytest

from . import cache_forms as forms
from .test_cache_edges_gpu import FORMS


@pytest.mark.parametrize("sms", [132, 148, 152, 160])
def test_the_tests_reach_every_form(lynx_lib, sms):
    want = {"decode clusters": 1, "decode shares": 2, "decode short shares": 2,
            "decode many rows": 4, "prefill whole": 3, "prefill shares": 4}
    for name, form in want.items():
        assert forms.form_of(lynx_lib, *FORMS[name], sms) == form, name
    cases = forms.parts_cases(lynx_lib, sms)
    for name, case in cases.items():
        assert forms.form_of(lynx_lib, *case, sms) == lynx_lib.LYNX_CACHE_PARTS, name
    assert forms.form_of(lynx_lib, *forms.TAKEOVER, sms) == lynx_lib.LYNX_CACHE_WHOLE
    counts, _, H_q, H_kv = forms.TAKEOVER[:4]
    units = sum(-(-n * (H_q // H_kv) // 256) for n in counts) * H_kv
    assert units >= 3 * sms


def test_parts_on_the_present_gpu(lynx_lib):
    assert forms.form_of(lynx_lib, *FORMS["prefill parts"], 152) == lynx_lib.LYNX_CACHE_PARTS


def test_rules(lynx_lib):
    form = lynx_lib.lynx_cache_attn_form
    L = lynx_lib
    assert form(0, 1, 0, 8, 2, 128, 64, 4, 152) == 0
    assert form(0, 0, 1, 8, 2, 128, 64, 4, 152) == 0
    # a table wider than 2048 tokens: no clusters
    assert form(1, 1, 1, 32, 8, 128, 64, 32, 152) == L.LYNX_CACHE_CLUSTERS
    assert form(1, 1, 1, 32, 8, 128, 64, 33, 152) == L.LYNX_CACHE_SPLIT
    # more than 32 rows
    assert form(64, 8, 8, 64, 8, 128, 64, 512, 152) == L.LYNX_CACHE_SHARES
    assert form(16384, 2, 0, 32, 8, 128, 256, 32, 152) == L.LYNX_CACHE_WHOLE
    assert form(100, 1, 0, 32, 8, 128, 64, 512, 152) == L.LYNX_CACHE_SHARES
    assert form(2046, 2, 0, 64, 4, 128, 128, 128, 152) == L.LYNX_CACHE_PARTS


@pytest.mark.parametrize("bad", [
    dict(sms=0), dict(sms=-1), dict(T=-1), dict(T=65), dict(H_q=7), dict(H_kv=0), dict(D=64),
    dict(page=32), dict(max_pages=0), dict(batch=-1), dict(n_tokens=-1), dict(n_tokens=5)])
def test_refusals(lynx_lib, bad):
    a = dict(n_tokens=4, batch=2, T=2, H_q=8, H_kv=2, D=128, page=64, max_pages=9, sms=152)
    a.update(bad)
    with pytest.raises(lynx_lib.LynxError):
        lynx_lib.lynx_cache_attn_form(**a)
    assert lynx_lib.lib().lynx_cache_attn_form(4, 2, 2, 8, 2, 128, 64, 9, 152, None) == -1


def test_a_workspace_for_every_form_that_needs_one(lynx_lib):
    """The workspace is sized for any number of SMs; a form that needs none on this
    one must not find one missing."""
    import random
    rng = random.Random(7)
    L = lynx_lib
    for _ in range(4000):
        H_kv = rng.choice((1, 2, 4, 8, 16, 40))
        H_q = H_kv * rng.choice((1, 2, 4, 5, 8, 16))
        batch, T = rng.choice((1, 2, 3, 8, 40, 300)), rng.choice((0, 0, 1, 2, 8, 33, 64))
        n = batch * T if T else rng.choice((1, 7, 100, 1000, 9000, 60000))
        pages, page = rng.choice((1, 8, 16, 17, 32, 33, 100, 2000)), rng.choice((64, 128, 512))
        a = (H_q, H_kv, 128, page, pages)
        need = L.lynx_cache_attn_decode_workspace_bytes(batch, T, *a) if T else \
            L.lynx_cache_attn_prefill_workspace_bytes(n, batch, *a)
        for sms in (1, 100, 132, 148, 152, 160, 200):
            form = L.lynx_cache_attn_form(n, batch, T, *a, sms)
            if form in (L.LYNX_CACHE_SPLIT, L.LYNX_CACHE_SHARES, L.LYNX_CACHE_PARTS):
                assert need > 0, (n, batch, T, a, sms)
