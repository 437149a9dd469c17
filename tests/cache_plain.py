"""The BF16 paged cache in 64 bits on the CPU, from the definitions: what the
tests of lynx_cache_append, lynx_cache_attn_decode and lynx_cache_attn_prefill
compare with, and the bounds they may be off by.

Bounds, per element.  A value rounded to BF16 is off by at most 2^-8 of itself.
 * append: one rounding, and sin.approx / cos.approx within 2^-21 (the angle
   itself within 2^-24 of pi): 2^-8 |y| + 2^-19 (|x1| + |x2|).
 * scores: a float32 sum of 128 exact products is off by at most 2^-23 * 130
   of sum |q k| (truncating adders included); cap and bias add 2^-20 of the cap
   and 2^-22 of the bias: delta.
 * lse: delta, the sum's own 2^-20 and 2^-22 |lse|.
 * out: weights off by 2 delta + 2^-19 and once rounded to BF16 for the second
   product, all relative: (2 delta + 2^-19 + 2^-8) sum w |v|, then one rounding
   of the result to BF16.
"""
import math

import torch

D = 128


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def table_for(kv, page, spare, seed, max_pages=None):
    """Distinct physical pages in scattered order; -1 where no token lies."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in kv]
    blocks = sum(need) + spare
    order = torch.randperm(blocks, generator=g)
    table = torch.full((len(kv), max_pages or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(need):
        table[b, :p] = order[at:at + p].to(torch.int32)
        at += p
    return table, blocks


def rows_of(pool, table, b, n, page):
    """Positions 0 .. n-1 of sequence b, [n][H_kv][D] float64."""
    p = torch.arange(n)
    slot = table[b].long()[p // page] * page + p % page
    return pool.reshape(-1, *pool.shape[2:])[slot].double()


def rotate(x, pos, inv_freq, axis, interleaved):
    """x [n][H][D] float64, pos [n_axes][n]: (rotated, bound's second term)."""
    half = len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64)
    ax = torch.tensor(axis if axis is not None else [0] * half, dtype=torch.long)
    a = (pos.double()[ax] * f[:, None]).T[:, None]          # [n][1][half]
    i = torch.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., lo] = x[..., lo] * a.cos() - x[..., hi] * a.sin()
    y[..., hi] = x[..., hi] * a.cos() + x[..., lo] * a.sin()
    m = x[..., lo].abs() + x[..., hi].abs()
    mag[..., lo], mag[..., hi] = m, m
    return y, mag


def append(k, v, counts, kv, table, k_pool, v_pool, q=None, inv_freq=(), axis=None,
           interleaved=False, positions=None):
    """CPU tensors; the pools and q_out after the call, and the bounds of keys and
    queries.  q_out rows of no sequence hold NaN."""
    page = k_pool.shape[1]
    kp, vp = k_pool.double(), v_pool.double()
    k_tol = torch.zeros_like(kp)
    qo = None if q is None else torch.full(q.shape, math.nan, dtype=torch.float64)
    q_tol = None if q is None else torch.zeros(q.shape, dtype=torch.float64)
    t0 = 0
    for b, n in enumerate(counts):
        if n:
            t = slice(t0, t0 + n)
            at = torch.arange(kv[b] - n, kv[b])
            pos = at[None] if positions is None else positions[:, t]
            fits = (at >= 0) & (at < table.shape[1] * page)
            pg = table[b].long()[(at // page).clamp(0, table.shape[1] - 1)]
            fits &= (pg >= 0) & (pg < k_pool.shape[0])
            slot = (pg * page + at % page)[fits]
            y, mag = rotate(k[t].double(), pos, inv_freq, axis, interleaved)
            kp.view(-1, *kp.shape[2:])[slot] = y[fits]
            k_tol.view(-1, *kp.shape[2:])[slot] = (2.0 ** -8 * y.abs() + 2.0 ** -19 * mag)[fits]
            vp.view(-1, *vp.shape[2:])[slot] = v[t].double()[fits]
            if q is not None:
                y, mag = rotate(q[t].double(), pos, inv_freq, axis, interleaved)
                qo[t] = y
                q_tol[t] = 2.0 ** -8 * y.abs() + 2.0 ** -19 * mag
        t0 += n
    return kp, vp, qo, k_tol, q_tol


def attention(q, counts, kv, table, k_pool, v_pool, scale=None, softcap=0.0, window=0,
              slopes=None, prefix=None):
    """q [n_tokens][H_q][D]; (out, lse, out's bound, lse's bound) in float64.  Rows
    of no sequence hold NaN."""
    page, H_kv = k_pool.shape[1], k_pool.shape[2]
    H_q = q.shape[1]
    G = H_q // H_kv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    o_tol, l_tol = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for b, n in enumerate(counts):
        t = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        L = max(0, min(kv[b], table.shape[1] * page))
        i = torch.arange(L - n, L)[:, None]
        j = torch.arange(L)[None]
        see = j <= i
        if window:
            see = see & (i - j < window)
        if prefix is not None:
            see = see | (j < prefix[b])
        see = see & (i >= 0)
        # pages that nothing sees need not be there
        seen = see.any(0)
        if L:
            K, V = (torch.zeros((L, H_kv, D), dtype=torch.float64) for _ in range(2))
            where = seen.nonzero()[:, 0]
            slot = table[b].long()[where // page] * page + where % page
            K[where] = k_pool.reshape(-1, H_kv, D)[slot].double()
            V[where] = v_pool.reshape(-1, H_kv, D)[slot].double()
        else:
            K = V = torch.zeros((0, H_kv, D), dtype=torch.float64)
        for hq in range(H_q):
            k, v, x = K[:, hq // G], V[:, hq // G], q[t, hq].double()
            s = scale * (x @ k.T)
            delta = 2.0 ** -23 * 130 * scale * (x.abs() @ k.abs().T)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                delta = delta + 2.0 ** -20 * softcap
            if slopes is not None:
                bias = float(slopes[hq]) * (i - j).abs().double()
                s = s - bias
                delta = delta + 2.0 ** -22 * bias
            s = s.masked_fill(~see, -math.inf)
            some = see.any(1)
            z = torch.logsumexp(s, 1) if L else torch.full((n,), -math.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(some, z, 0.0)[:, None]).masked_fill(~see, 0.0)
            # rows are as far off as their worst score that carries weight
            d = (delta * (w > 2.0 ** -40)).amax(1) if L else torch.zeros(n, dtype=torch.float64)
            lse[t, hq] = z
            l_tol[t, hq] = d + 2.0 ** -20 + 2.0 ** -22 * torch.where(some, z, 0.0).abs()
            out[t, hq] = w @ v
            o_tol[t, hq] = (2 * d + 2.0 ** -19 + 2.0 ** -8)[:, None] * (w @ v.abs()) + \
                2.0 ** -8 * (w @ v).abs() + 2.0 ** -30
    return out, lse, o_tol, l_tol


def assert_close(got, want, tol, what):
    """Everywhere that `want` is a number; infinities have to be equal."""
    got = got.cpu().double()
    here = ~torch.isnan(want)
    fin = here & torch.isfinite(want)
    inf = here & ~torch.isfinite(want)
    assert torch.equal(got[inf], want[inf]), what
    assert torch.isfinite(got[fin]).all(), f"{what}: not finite"
    off = (got - want).abs()[fin] - tol[fin]
    if off.numel():
        worst = off.argmax()
        assert off[worst] <= 0, (f"{what}: {got[fin][worst]} for {want[fin][worst]}, "
                                 f"may be off by {tol[fin][worst]}")
