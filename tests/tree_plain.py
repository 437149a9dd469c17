"""Log probabilities, trees of drafted tokens and the paged cache's books on the CPU, from
their definitions (float64, Python integers): what the tests compare with, and the
bounds that float32 sums may be off by.

Bounds of the log probabilities.  With y = (x - r) scale log2 e and r within 8 / (scale log2 e) of
the row's maximum, a thread's y is off by 3 roundings, 2^-22.4 |y|, its 2^y by that and
2^-22 more; a sum of V values is V / 512 additions in a row in each of two lanes of 256 threads
(V / 512 2^-24, for a cluster less) and the joins of 14 levels, each two roundings and a
factor 2^d.  So s is off by eps = 2^-21 (1 + E) + (V / 512 + 64) 2^-24 relative, E the mean of
|y| under p, at most the mean of (max - x) scale log2 e, plus 8.
 * logprob = (x - r) scale - ln s: eps, and 2^-22 of |logprob| + 8 + ln V.
 * entropy = ln s - ln 2 t / s: t's terms carry |y| too: 2 eps (1 + E), and 2^-22 (16 + ln V).
"""
import math

import torch


def logprobs(x, tokens, top, scale):
    """x [rows][V] CPU; (logprob, entropy, top_logprob, top_token, bounds of the first
    two and of the third) in float64."""
    x = x.double()
    rows, V = x.shape
    scale = float(torch.tensor(scale, dtype=torch.float32))
    z = x * scale
    bad = torch.isnan(x).any(1) | (x == math.inf).any(1)
    none = (x == -math.inf).all(1)
    m = z.nan_to_num(nan=-math.inf).amax(1, keepdim=True)
    d = torch.where(z > -math.inf, z - torch.where(m > -math.inf, m, 0.0), -math.inf)
    e = d.exp()
    s = e.sum(1, keepdim=True)
    ln = torch.where(none[:, None], 0.0, s.log())
    lp = torch.where(z > -math.inf, d - ln, -math.inf)
    lp[bad] = math.nan
    p = e / torch.where(none[:, None], 1.0, s)
    ent = torch.where(p > 0, -p * (d - ln), 0.0).sum(1)
    ent[bad] = math.nan
    E = torch.where(p > 0, -p * d, 0.0).sum(1) * 1.4426950408889634 + 8
    eps = 2.0 ** -21 * (1 + E) + (V / 512 + 64) * 2.0 ** -24
    l_tol = eps[:, None] + 2.0 ** -22 * (lp.abs().nan_to_num(posinf=0.0) + 8 + math.log(V))
    h_tol = 2 * eps * (1 + E) + 2.0 ** -22 * (16 + math.log(V))
    # the likeliest: by value, the lowest first among equals; a NaN or -inf is none
    order = torch.where(torch.isnan(x), -math.inf, x).sort(dim=1, descending=True, stable=True)
    tt = order.indices[:, :top].clone()
    gone = order.values[:, :top] == -math.inf
    tl = lp.gather(1, tt)
    tl_tol = l_tol.gather(1, tt)
    tt[gone] = -1
    tl[gone] = -math.inf
    out = None
    g_tol = None
    if tokens is not None:
        t = tokens.long()
        ok = (t >= 0) & (t < V)
        out = torch.where(ok, lp.gather(1, t.clamp(0, V - 1)), -math.inf)
        g_tol = l_tol.gather(1, t.clamp(0, V - 1))
    return out, ent, tl, tt.to(torch.int32), g_tol, h_tol, tl_tol


def chains(parents):
    """For each place its chain of nodes up to the root, itself first; [] without a node."""
    got = []
    for t, p in enumerate(parents):
        if t == 0:
            got.append([0] if p == -1 else [])
        elif 0 <= p < t and got[p]:
            got.append([t] + got[p])
        else:
            got.append([])
    return got


def masks(parents):
    return [sum(1 << a for a in c) for c in chains(parents)]


def signed(m):
    """A 64-bit word as an int64 holds it."""
    return m - (1 << 64) if m >> 63 else m


def verify(parents, tokens, answers):
    c = chains(parents)
    path = [0] if c[0] else []
    while path:
        below = [t for t in range(1, len(parents))
                 if c[t][1:2] == path[-1:] and tokens[t] == answers[path[-1]]]
        if not below:
            break
        path.append(below[0])
    return path, answers[path[-1]] if path else -1


class Books:
    """A cache's books and what its pages hold, as Python lists."""

    def __init__(self, batch, max_pages, num_blocks, page):
        self.table = [[-1] * max_pages for _ in range(batch)]
        self.kv = [0] * batch
        self.refs = [0] * num_blocks
        self.page = page

    def pages(self, n):
        return -(-n // self.page)

    def check(self, pinned=()):
        """Rows name what their lengths need, refs counts it."""
        refs = [0] * len(self.refs)
        for p in pinned:
            refs[p] += 1
        for row, n in zip(self.table, self.kv):
            have = self.pages(n)
            assert all(p >= 0 for p in row[:have]) and all(p == -1 for p in row[have:])
            for p in row[:have]:
                refs[p] += 1
        assert refs == self.refs

    def fork(self, source):
        new = [list(self.table[s]) if 0 <= s < len(self.kv) else [-1] * len(self.table[0])
               for s in source]
        kv = [self.kv[s] if 0 <= s < len(self.kv) else 0 for s in source]
        for rows, d in ((new, 1), (self.table, -1)):
            for row in rows:
                for p in row:
                    if p >= 0:
                        self.refs[p] += d
        self.table, self.kv = new, kv

    def reserve(self, grow):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        shared = list(self.refs)
        at = asked = 0
        there = len(free)
        granted, src, dst = [], [], []
        for b, n in enumerate(grow):
            n = max(n, 0)
            row, kv = self.table[b], self.kv[b]
            have, want = self.pages(kv), self.pages(kv + n)
            copy = n > 0 and kv % self.page > 0 and shared[row[have - 1]] > 1
            granted.append(0)
            src.append(-1)
            dst.append(-1)
            if want > len(row):
                continue
            need = want - have + copy
            asked += need
            if need and asked > there:
                continue
            if copy:
                src[b], dst[b] = row[have - 1], free[at]
                at += 1
                self.refs[src[b]] -= 1
                self.refs[dst[b]] = 1
                row[have - 1] = dst[b]
            for m in range(have, want):
                row[m] = free[at]
                at += 1
                self.refs[row[m]] = 1
            granted[b] = n
            self.kv[b] += n
        return granted, src, dst

    def trim(self, keep):
        for b, k in enumerate(keep):
            n = min(self.kv[b], max(k, 0))
            for m in range(self.pages(n), self.pages(self.kv[b])):
                self.refs[self.table[b][m]] -= 1
                self.table[b][m] = -1
            self.kv[b] = n

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        dst = [p for p in range(n) if self.refs[p] == 0]
        src = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        for a, z in zip(src, dst):
            self.refs[z], self.refs[a] = self.refs[a], 0
        at = dict(zip(src, dst))
        self.table = [[at.get(p, p) for p in row] for row in self.table]
        blank = [-1] * (len(self.refs) // 2 - len(src))
        return src + blank, dst + blank, len(src)


def attention(q, masks, kv, table, k_pool, v_pool, k_nodes, v_nodes, scale=None, softcap=0.0,
              window=0, slopes=None, prefix=None):
    """q [batch][T][H_q][D], masks a list of T integers a sequence; (out, lse, out's bound,
    lse's bound) in float64, the bounds of cache_plain."""
    D = q.shape[-1]
    page, H_kv = k_pool.shape[1], k_pool.shape[2]
    batch, T, H_q = q.shape[:3]
    G = H_q // H_kv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64)
    o_tol, l_tol = torch.full_like(out, 2.0 ** -30), torch.full_like(lse, 2.0 ** -20)
    for b in range(batch):
        L = max(0, min(kv[b], table.shape[1] * page))
        words = [m & ((1 << T) - 1) for m in masks[b]]
        depth = torch.tensor([bin(m).count("1") - 1 for m in words])
        p = (L + depth)[:, None]
        j = torch.arange(L)[None]
        see = torch.ones((T, L), dtype=torch.bool)
        sees = torch.tensor([[bool(m >> a & 1) for a in range(T)] for m in words])
        if window:
            see = see & (p - j < window)
            sees = sees & (depth[:, None] - depth[None] < window)
        if prefix is not None:
            see = see | (j < prefix[b])
        see = see.expand(T, L) & (depth >= 0)[:, None]
        sees = sees & (depth >= 0)[:, None]
        where = see.any(0).nonzero()[:, 0]
        K = torch.zeros((L + T, H_kv, D), dtype=torch.float64)
        V = torch.zeros_like(K)
        if len(where):
            slot = table[b].long()[where // page] * page + where % page
            K[where] = k_pool.reshape(-1, H_kv, D)[slot].double()
            V[where] = v_pool.reshape(-1, H_kv, D)[slot].double()
        K[L:], V[L:] = k_nodes[b, :T].double(), v_nodes[b, :T].double()
        ok = torch.cat((see, sees), 1)
        K[~ok.any(0)] = 0.0
        V[~ok.any(0)] = 0.0
        away = torch.cat((p - j, depth[:, None] - depth[None]), 1).abs().double()
        for hq in range(H_q):
            k, v, x = K[:, hq // G], V[:, hq // G], q[b, :, hq].double()
            s = scale * (x @ k.T)
            delta = 2.0 ** -23 * 130 * scale * (x.abs() @ k.abs().T)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                delta = delta + 2.0 ** -20 * softcap
            if slopes is not None:
                s = s - float(slopes[hq]) * away
                delta = delta + 2.0 ** -22 * float(slopes[hq]) * away
            s = s.masked_fill(~ok, -math.inf)
            some = ok.any(1)
            z = torch.logsumexp(s, 1)
            w = torch.exp(s - torch.where(some, z, 0.0)[:, None]).masked_fill(~ok, 0.0)
            d = (delta * (w > 2.0 ** -40)).amax(1)
            lse[b, :, hq] = z
            l_tol[b, :, hq] = d + 2.0 ** -20 + 2.0 ** -22 * torch.where(some, z, 0.0).abs()
            out[b, :, hq] = w @ v
            o_tol[b, :, hq] = (2 * d + 2.0 ** -19 + 2.0 ** -8)[:, None] * (w @ v.abs()) + \
                2.0 ** -8 * (w @ v).abs() + 2.0 ** -30
    return out, lse, o_tol, l_tol
