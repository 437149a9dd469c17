"""Drafting with trees over the BF16 paged cache: what is measured of its operators.

A draft model proposes a tree of tokens.  `logprobs` reads a step's logits: the alternatives that
become a node's children, the log probabilities of given tokens, the entropy that says how far to
draft.  `tree` is the one pass over the cache that verifies all nodes of a tree.  `keep` walks down
the tree along what the model answered, finds pages for the nodes kept and writes their keys and
values behind the context, in all layers.  `fork` lets sequences share pages (the beams or
samples of one prompt) and gives each its own last page before it writes; `compact` drops what
sequences no longer need and moves the pages in use to the front of the pools.

Nodes 0 .. T-1 of a sequence are numbered parents first, node 0 being the root; keys and values of
the nodes lie beside the cache, [batch][64][H_kv][128].  A table row names the pages that its kv_len
tokens need, refs counts in how many places each page is named.
"""
import math
import random

import torch

own = False

D = 128
ROOM = 64              # nodes of a tree, at most


# ------------------------------------------------------------------ cases

def _logprobs(name, rows, V, dtype, top, given=1, scale=1.0, masked=False):
    c = {"op": "logprobs", "rows": rows, "V": V, "dtype": dtype, "top": top, "given": given,
         "scale": scale, "masked": masked}
    return dict(c, name=name) if name else c


def _tree(name, batch, nodes, context, H_q, H_kv, page, ragged=False, softcap=0.0, window=0,
          prefix=0, slopes=False):
    c = {"op": "tree", "batch": batch, "nodes": nodes, "context": context, "H_q": H_q,
         "H_kv": H_kv, "page": page, "ragged": ragged, "softcap": softcap, "window": window,
         "prefix": prefix, "slopes": slopes}
    return dict(c, name=name) if name else c


def _pages(name, op, batch, context, H_kv, page, layers, nodes=0):
    c = {"op": op, "batch": batch, "context": context, "H_kv": H_kv, "page": page,
         "layers": layers}
    if op == "keep":
        c["nodes"] = nodes
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's draft step: the four likeliest next tokens; latency
        _logprobs("logprobs-1", 1, 128256, "float32", 4),
        # the nodes of eight trees, an odd vocabulary, a grammar that rules most tokens out
        _logprobs("logprobs-nodes", 128, 100003, "bfloat16", 8, given=3, scale=1.25, masked=True),
        # the log probabilities of a prompt's own tokens
        _logprobs("logprobs-prompt", 4096, 128256, "bfloat16", 5),
        # a small tree over a short chat: latency
        _tree("tree-b1-1k", 1, 16, 1000, 32, 8, 64),
        # a serving batch of every length: capped scores, a window, the first tokens kept visible
        _tree("tree-b16-window", 16, 26, 12001, 40, 8, 64, ragged=True, softcap=50.0, window=4096,
              prefix=4),
        # full trees over long contexts, many query heads to a KV head
        _tree("tree-b8-32k", 8, 64, 32768, 64, 4, 256),
        # one sequence, two layers: nothing but latency
        _pages("keep-1", "keep", 1, 777, 8, 64, 2, nodes=16),
        # a serving batch, all layers of a small model in one call
        _pages("keep-b32", "keep", 32, 600, 4, 64, 16, nodes=64),
        # four samples of one short prompt
        _pages("fork-4", "fork", 4, 777, 8, 64, 2),
        # sixteen groups of four beams
        _pages("fork-b64", "fork", 64, 9001, 2, 256, 4),
        # a few short sequences that are over
        _pages("compact-4", "compact", 4, 700, 8, 64, 2),
        # a batch of which much has been dropped: about half a gigabyte to move
        _pages("compact-b48", "compact", 48, 5003, 4, 128, 8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("logprobs", "logprobs", "tree", "tree", "keep", "fork", "compact"))
    if op == "logprobs":
        rows = _log(rng, 1, 4096)
        V = _log(rng, 40, min(200003, 500000000 // rows))
        return _logprobs(None, rows, V, rng.choice(("float32", "bfloat16", "float16")),
                         rng.choice((0, 1, 4, 8, 20, 32)), rng.choice((1, 1, 2, 7)),
                         rng.choice((1.0, 1.0, 0.5, 1.7)), rng.random() < 0.3)
    if op == "tree":
        H_q, H_kv = rng.choice(((32, 8), (64, 8), (64, 4), (40, 8), (16, 16), (8, 1), (24, 2)))
        batch = _log(rng, 1, 32)
        nodes = rng.choice((1, 2, 7, 16, 25, 48, 63, 64))
        most = min(131072, 1000000 // (batch * H_kv), 800000000 // (batch * nodes * H_q))
        context = _log(rng, 1, most)
        return _tree(None, batch, nodes, context, H_q, H_kv, rng.choice((64, 128, 256, 512)),
                     ragged=rng.random() < 0.5, softcap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                     window=rng.choice((0, 0, _log(rng, 1, context))),
                     prefix=rng.choice((0, 0, rng.randrange(1, 200))), slopes=rng.random() < 0.25)
    page = rng.choice((64, 128, 256, 512))
    H_kv = rng.choice((1, 2, 4, 8))
    layers = rng.choice((1, 2, 3, 5, 8))
    batch = _log(rng, 1, 64)
    room = 800000000 // (batch * layers * H_kv * 512)       # tokens, all K and V in a gigabyte
    context = _log(rng, 1, max(page, min(6000, room)))
    return _pages(None, op, batch, context, H_kv, page, layers,
                  nodes=rng.choice((1, 5, 16, 33, 64)))


def _lengths(c):
    """The sequences' lengths, from the case alone."""
    batch, context = c["batch"], c["context"]
    if not c.get("ragged", True):
        return [context] * batch
    rng = random.Random("%d %d %d" % (batch, context, c["page"]))
    kv = [context] + [rng.randint(0, context) for _ in range(batch - 1)]
    if batch > 2:
        kv[1] = 1
    if batch > 4:
        kv[2] = 0
    return kv


# ------------------------------------------------------------------ inputs

def _tokens(gen, n, heads, boost):
    """n rows of `heads` heads of 128 BF16 values; some channels are large, as in real keys."""
    x = torch.randn((n, heads, D), generator=gen, device="cuda", dtype=torch.float32)
    scale = torch.ones(D, device="cuda")
    scale[torch.randperm(D, generator=gen, device="cuda")[:6]] = boost
    return (x * scale).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _table(kv, page, gen, spare, max_pages):
    """Physical pages in any order; -1 where no token lies.  (table, blocks)"""
    used = sum(-(-n // page) for n in kv)
    order = torch.randperm(used + spare, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(kv), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(kv):
        p = -(-n // page)
        table[b, :p] = order[at:at + p]
        at += p
    return table, used + spare


def _parents(rng, n, T):
    """A tree of n nodes in T places: each node a child of one of the last few, as a draft that
    follows its best leaves gives them.  -1: the root, and places without a node."""
    p = [-1] + [max(0, t - 1 - rng.randrange(0, 5)) for t in range(1, n)]
    return p + [-1] * (T - n)


def _prepare_logprobs(c, gen, seed):
    rows, V = c["rows"], c["V"]
    dtype = getattr(torch, c["dtype"])
    x = torch.empty((rows, V), dtype=dtype, device="cuda")
    for r in range(0, rows, 512):
        n = min(512, rows - r)
        z = torch.randn((n, V), generator=gen, device="cuda") * 2.5
        # a few tokens stand out, in each row others
        hot = torch.randint(0, V, (n, 6), generator=gen, device="cuda")
        z.scatter_add_(1, hot, torch.rand((n, 6), generator=gen, device="cuda") * 12)
        if c["masked"]:
            z.masked_fill_(torch.rand((n, V), generator=gen, device="cuda") < 0.97, -math.inf)
        x[r:r + n] = z.to(dtype)
    return {"logits": x, "tokens": torch.randint(0, V, (rows, c["given"]), generator=gen,
                                                 device="cuda", dtype=torch.int32)}


def _prepare_tree(c, gen, seed):
    rng = random.Random(seed)
    batch, T, page, H_kv = c["batch"], c["nodes"], c["page"], c["H_kv"]
    kv = _lengths(c)
    table, blocks = _table(kv, page, gen, 2, max(1, -(-max(kv) // page)))
    s = {"table": table.cuda(), "kv_len": _ints(kv)}
    s["k_pool"] = _tokens(gen, blocks * page, H_kv, 3.0).view(blocks, page, H_kv, D)
    s["v_pool"] = _tokens(gen, blocks * page, H_kv, 1.0).view(blocks, page, H_kv, D)
    s["k_nodes"] = _tokens(gen, batch * ROOM, H_kv, 3.0).view(batch, ROOM, H_kv, D)
    s["v_nodes"] = _tokens(gen, batch * ROOM, H_kv, 1.0).view(batch, ROOM, H_kv, D)
    s["q"] = _tokens(gen, batch * T, c["H_q"], 3.0).view(batch, T, c["H_q"], D)
    s["parents"] = _ints([_parents(rng, T - (rng.randrange(0, T) if c["ragged"] and b % 2 else 0), T)
                          for b in range(batch)])
    s["slopes"] = s["prefix"] = None
    if c["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["H_q"]) for h in range(c["H_q"])],
                                   dtype=torch.float32).cuda()
    if c["prefix"]:
        s["prefix"] = _ints([c["prefix"]] * batch)
    return s


def _prepare_pages(c, gen, seed):
    rng = random.Random(seed)
    batch, page, H_kv, op = c["batch"], c["page"], c["H_kv"], c["op"]
    kv = _lengths(c)
    max_pages = -(-(c["context"] + ROOM) // page)
    spare = {"keep": 2 * batch, "fork": 2 * batch, "compact": 3}[op]
    table, blocks = _table(kv, page, gen, spare, max_pages)
    n = 2 * c["layers"]
    s = {"pools": torch.empty((n, blocks, page, H_kv, D), dtype=torch.bfloat16, device="cuda")}
    for i in range(n):
        s["pools"][i] = _tokens(gen, blocks * page, H_kv, 3.0).view(blocks, page, H_kv, D)
    refs = torch.zeros(blocks, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    # the cache's books, which a step changes, in one piece: table, lengths, counts
    s["books"] = torch.cat((table.reshape(-1), torch.tensor(kv, dtype=torch.int32), refs)).cuda()
    s["live"] = torch.empty_like(s["books"])
    s["shape"] = (batch, max_pages, blocks)
    if op == "keep":
        T = c["nodes"]
        s["nodes"] = torch.stack([_tokens(gen, batch * ROOM, H_kv, 3.0).view(batch, ROOM, H_kv, D)
                                  for _ in range(n)])
        parents = [_parents(rng, T - (rng.randrange(0, T) if b % 3 == 2 else 0), T)
                   for b in range(batch)]
        tokens = [[rng.randrange(0, 50000) for _ in range(T)] for _ in range(batch)]
        # what the model answers at each node: mostly one of the drafts that follow it
        answers = []
        for p, t in zip(parents, tokens):
            a = [rng.randrange(0, 50000) for _ in range(T)]
            for i in range(1, T):
                if p[i] >= 0 and rng.random() < 0.6:
                    a[p[i]] = t[i]
            answers.append(a)
        s["parents"], s["tokens"], s["answers"] = _ints(parents), _ints(tokens), _ints(answers)
    elif op == "fork":
        # each group of four goes on from one or two of its members; all write one token more
        s["source"] = _ints([b // 4 * 4 + rng.randrange(0, min(4, batch - b // 4 * 4))
                             for b in range(batch)])
        s["grow"] = _ints([1] * batch)
    else:
        # sequences that are over, ones that are cut back, ones that stay
        s["keep"] = _ints([rng.choice((0, 0, rng.randrange(0, m + 1), m)) for m in kv])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"logprobs": _prepare_logprobs, "tree": _prepare_tree}.get(case["op"], _prepare_pages)
    return dict(make(case, gen, seed), case=dict(case))


def _books(s, flat):
    """Views of the table, the lengths and the counts."""
    batch, max_pages, blocks = s["shape"]
    n = batch * max_pages
    return flat[:n].view(batch, max_pages), flat[n:n + batch], flat[n + batch:]


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from split_stream_kv_gb300 import lynx
    c = s["case"]
    if c["op"] == "logprobs":
        lp, entropy, top_lp, top = lynx.lynx_token_logprobs(s["logits"], s["tokens"], top=c["top"],
                                                            scale=c["scale"])
        return {"logprob": lp, "entropy": entropy, "top_logprob": top_lp, "top_token": top}
    if c["op"] == "tree":
        mask, positions = lynx.lynx_tree_plan(s["parents"], s["kv_len"])
        lse = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
        out = lynx.lynx_cache_attn_tree(s["q"], s["k_nodes"], s["v_nodes"], mask, s["k_pool"],
                                        s["v_pool"], s["table"], s["kv_len"], softcap=c["softcap"],
                                        window=c["window"], slopes=s["slopes"], prefix=s["prefix"],
                                        lse=lse)
        return {"positions": positions, "out": out, "lse": lse}
    s["live"].copy_(s["books"])             # the step changes the books: each pass has its own
    table, kv_len, refs = _books(s, s["live"])
    pools, page = list(s["pools"]), c["page"]
    if c["op"] == "keep":
        path, n, token = lynx.lynx_tree_verify(s["parents"], s["tokens"], s["answers"])
        granted, src, dst = lynx.lynx_cache_reserve(table, kv_len, refs, n, page)
        lynx.lynx_cache_copy_pages(pools, src, dst)
        lynx.lynx_cache_keep(list(s["nodes"]), pools, path, granted, kv_len, table)
        return {"path": path, "n": n, "token": token, "granted": granted, "table": table,
                "kv_len": kv_len, "refs": refs, "pools": s["pools"]}
    if c["op"] == "fork":
        table, kv_len = lynx.lynx_cache_fork(table, kv_len, refs, s["source"], page)
        granted, src, dst = lynx.lynx_cache_reserve(table, kv_len, refs, s["grow"], page)
        lynx.lynx_cache_copy_pages(pools, src, dst)
        return {"table": table, "kv_len": kv_len, "refs": refs, "granted": granted, "src": src,
                "dst": dst, "pools": s["pools"]}
    lynx.lynx_cache_trim(table, kv_len, refs, s["keep"], page)
    src, dst, count = lynx.lynx_cache_compact(table, kv_len, refs, page)
    lynx.lynx_cache_copy_pages(pools, src, dst, count)
    return {"table": table, "kv_len": kv_len, "refs": refs, "src": src, "dst": dst, "count": count,
            "pools": s["pools"]}


# ------------------------------------------------------------------ plain forms

def _plain_logprobs(s):
    c, x = s["case"], s["logits"]
    z = x.float() * c["scale"]
    m = z.amax(1, keepdim=True)
    some = m > -math.inf
    z = z - torch.where(some, m, 0.0)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    ln = torch.where(some, total.log(), 0.0)
    lp = torch.where(some, z.gather(1, s["tokens"].long()) - ln, -math.inf)
    mean = torch.where(e > 0, e * z, 0.0).sum(1, keepdim=True)
    entropy = torch.where(some, ln - mean / torch.where(some, total, 1.0), 0.0)[:, 0]
    del e
    # the likeliest tokens, the lowest first among equals: one after the other is taken out
    z.sub_(ln)
    found = []
    left = x.to(torch.float32, copy=True)
    for _ in range(c["top"]):
        i = left.argmax(1, keepdim=True)
        none = left.gather(1, i) == -math.inf
        found.append((torch.where(none, -math.inf, z.gather(1, i)), torch.where(none, -1, i)))
        left.scatter_(1, i, -math.inf)
    blank = torch.empty((x.shape[0], 0), device="cuda")
    return {"logprob": lp, "entropy": entropy,
            "top_logprob": torch.cat([blank] + [f[0] for f in found], 1),
            "top_token": torch.cat([blank.long()] + [f[1] for f in found], 1).to(torch.int32)}


def _ancestors(parents):
    """parents [batch][T] -> [batch][T][T] truth values: column a is node t or one of its
    ancestors; rows of places without a node are all false."""
    T = parents.shape[1]
    t = torch.arange(T, device="cuda")
    step = (parents[:, :, None] == t) & (t[:, None] > t)
    reach = (step | torch.eye(T, dtype=torch.bool, device="cuda")).float()
    for _ in range(6):                       # 2^6 steps up
        reach = (torch.matmul(reach, reach) > 0).float()
    reach = reach > 0
    return reach & (reach[:, :, :1] & (parents[:, :1, None] == -1))    # those that reach the root


def _plain_tree(s):
    c, q = s["case"], s["q"]
    batch, T, H_q, _ = q.shape
    H_kv, G = c["H_kv"], H_q // c["H_kv"]
    anc = _ancestors(s["parents"])
    depth = anc.sum(2) - 1
    kv = s["kv_len"].long()
    here = kv[:, None] + depth.clamp(min=0)                 # [batch][T]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * c["page"]
    j = torch.arange(L, device="cuda")
    k = torch.cat((s["k_pool"][table].reshape(batch, L, H_kv, D), s["k_nodes"][:, :T]), 1).float()
    v = torch.cat((s["v_pool"][table].reshape(batch, L, H_kv, D), s["v_nodes"][:, :T]), 1).float()
    at = torch.cat((j.expand(batch, L), here), 1)           # position of each key
    gap = here[:, :, None] - at[:, None]
    near = (gap < c["window"]) if c["window"] else torch.ones_like(gap, dtype=torch.bool)
    seen = torch.cat(((j < kv[:, None])[:, None].expand(batch, T, L), anc), 2) & near
    if s["prefix"] is not None:
        first = (j < s["prefix"][:, None]) & (j < kv[:, None])
        seen[:, :, :L] |= first[:, None]
    seen &= (depth >= 0)[:, :, None]
    qq = q.float().reshape(batch, T, H_kv, G, D).permute(0, 2, 3, 1, 4)
    a = torch.matmul(qq.reshape(batch, H_kv, G * T, D), k.permute(0, 2, 3, 1))
    a = a.mul_(1.0 / math.sqrt(D)).view(batch, H_kv, G, T, L + T)
    if c["softcap"]:
        a = a.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if s["slopes"] is not None:
        a.sub_(s["slopes"].view(1, H_kv, G, 1, 1) * gap.abs()[:, None, None])
    a.masked_fill_(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    some = m > -math.inf
    a = a.sub_(torch.where(some, m, 0.0)).exp_()
    l = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(batch, H_kv, G * T, L + T), v.permute(0, 2, 1, 3))
    o = o.view(batch, H_kv, G, T, D) / torch.where(some, l, 1.0)
    lse = torch.where(some, m + l.log(), -math.inf)[..., 0]
    return {"positions": torch.where(depth >= 0, here, -1).reshape(-1).to(torch.int32),
            "out": o.permute(0, 3, 1, 2, 4).reshape(batch, T, H_q, D).to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(batch, T, H_q)}


def _plain_verify(parents, tokens, answers):
    """(path [batch][T], its length, the token behind it)"""
    T = parents.shape[1]
    anc = _ancestors(parents)
    up = parents.clamp(min=0).long()
    fits = tokens == answers.gather(1, up)
    fits[:, 0] = True
    # of children of one node with the same token the first counts
    twin = (parents[:, :, None] == parents[:, None]) & (tokens[:, :, None] == tokens[:, None])
    t = torch.arange(T, device="cuda")
    fits &= ~(twin & (t < t[:, None]) & (t > 0)).any(2)
    kept = anc[:, :, 0] & ~(anc & ~fits[:, None]).any(2)
    n = kept.sum(1)
    path = torch.where(kept, t, T).sort(1).values
    last = path.gather(1, (n - 1).clamp(min=0)[:, None])
    token = torch.where(n > 0, answers.gather(1, last.clamp(max=T - 1))[:, 0], -1)
    return torch.where(path < T, path, -1).to(torch.int32), n.to(torch.int32), token.to(torch.int32)


def _plain_reserve(table, kv_len, refs, grow, page):
    """The books changed in place; (granted, src, dst)."""
    batch, max_pages = table.shape
    kv, n = kv_len.long(), grow.long()
    have = (kv + page - 1) // page
    want = (kv + n + page - 1) // page
    old = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    own_copy = (n > 0) & (kv % page > 0) & (refs[old.clamp(min=0)] > 1)
    fits = want <= max_pages
    need = torch.where(fits, want - have + own_copy, 0)
    ok = fits & ((need == 0) | (need.cumsum(0) <= (refs == 0).sum()))
    need = torch.where(ok, need, 0)
    own_copy &= ok
    free = (refs == 0).nonzero()[:, 0]
    b = torch.repeat_interleave(torch.arange(batch, device="cuda"), need)
    i = torch.arange(b.numel(), device="cuda") - (need.cumsum(0) - need)[b]
    free = free[:b.numel()]
    table[b, (have - own_copy.long())[b] + i] = free.to(torch.int32)
    refs.index_add_(0, free, torch.ones_like(free, dtype=torch.int32))
    refs.index_add_(0, old.clamp(min=0), -own_copy.to(torch.int32))
    granted = torch.where(ok, n, 0)
    kv_len += granted.to(torch.int32)
    dst = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    return (granted.to(torch.int32), torch.where(own_copy, old, -1).to(torch.int32),
            torch.where(own_copy, dst, -1).to(torch.int32))


def _plain_copy(pools, src, dst):
    src, dst = src[src >= 0].long(), dst[dst >= 0].long()
    pools[:, dst] = pools[:, src]


def _plain_pages(s):
    c, page, pools = s["case"], s["case"]["page"], s["pools"]
    table, kv_len, refs = (x.clone() for x in _books(s, s["books"]))
    batch, max_pages = table.shape
    m = torch.arange(max_pages, device="cuda")
    if c["op"] == "keep":
        path, n, token = _plain_verify(s["parents"], s["tokens"], s["answers"])
        granted, src, dst = _plain_reserve(table, kv_len, refs, n, page)
        _plain_copy(pools, src, dst)
        b, i = ((torch.arange(path.shape[1], device="cuda") < granted[:, None])).nonzero().T
        at = kv_len[b].long() - granted[b] + i
        where = table[b, at // page].long()
        pools[:, where, at % page] = s["nodes"][:, b, path[b, i].long()]
        return {"path": path, "n": n, "token": token, "granted": granted, "table": table,
                "kv_len": kv_len, "refs": refs, "pools": pools}
    if c["op"] == "fork":
        src = s["source"].long()
        new, new_len = table[src], kv_len[src]
        refs.index_add_(0, new[new >= 0].long(), torch.ones_like(new[new >= 0]))
        refs.index_add_(0, table[table >= 0].long(), -torch.ones_like(table[table >= 0]))
        granted, src, dst = _plain_reserve(new, new_len, refs, s["grow"], page)
        _plain_copy(pools, src, dst)
        return {"table": new, "kv_len": new_len, "refs": refs, "granted": granted, "src": src,
                "dst": dst, "pools": pools}
    kv_len = torch.minimum(kv_len, s["keep"].clamp(min=0))
    gone = (m >= (kv_len[:, None] + page - 1) // page) & (table >= 0)
    refs.index_add_(0, table[gone].long(), -torch.ones_like(table[gone]))
    table[gone] = -1
    used = refs > 0
    n = int(used.sum())
    holes = (~used[:n]).nonzero()[:, 0]
    moved = used[n:].nonzero()[:, 0] + n
    to = torch.arange(refs.numel(), device="cuda", dtype=torch.int32)
    to[moved] = holes.to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    refs[holes] = refs[moved]
    refs[moved] = 0
    pools[:, holes] = pools[:, moved]
    src = torch.full((refs.numel() // 2,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[:len(moved)] = moved.to(torch.int32)
    dst[:len(moved)] = holes.to(torch.int32)
    count = torch.full((1,), len(moved), dtype=torch.int32, device="cuda")
    return {"table": table, "kv_len": kv_len, "refs": refs, "src": src, "dst": dst, "count": count,
            "pools": pools}


def run(state):
    if own:
        return _run_own(state)
    plain = {"logprobs": _plain_logprobs, "tree": _plain_tree}.get(state["case"]["op"], _plain_pages)
    return plain(state)


# ------------------------------------------------------------------ in 64 bits

def _exact_logprobs(s, c):
    got = {"logprob": [], "entropy": [], "top_logprob": [], "top_token": []}
    for r in range(0, c["rows"], 64):
        x = s["logits"][r:r + 64].double()
        z = x * c["scale"]
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        lp = torch.where((x > -math.inf).any(1, keepdim=True), lp, -math.inf)
        got["logprob"].append(torch.gather(lp, 1, s["tokens"][r:r + 64].long()))
        got["entropy"].append(torch.special.entr(lp.exp()).sum(1))
        order = x.sort(dim=1, descending=True, stable=True)
        i = order.indices[:, :c["top"]]
        none = order.values[:, :c["top"]] == -math.inf
        got["top_logprob"].append(lp.gather(1, i).masked_fill(none, -math.inf))
        got["top_token"].append(i.masked_fill(none, -1).to(torch.int32))
    return {k: torch.cat(v) for k, v in got.items()}


def _chains(parents):
    """For each place its chain of nodes up to the root, the node itself first; none without one."""
    chains = []
    for t, p in enumerate(parents):
        if t == 0:
            chains.append([0] if p == -1 else [])
        elif 0 <= p < t and chains[p]:
            chains.append([t] + chains[p])
        else:
            chains.append([])
    return chains


def _slots(row, n, page):
    p = torch.arange(n, device="cuda")
    return row.long()[p // page] * page + p % page


def _exact_tree(s, c):
    T, H_q, H_kv, page = c["nodes"], c["H_q"], c["H_kv"], c["page"]
    kv, G = _lengths(c), H_q // H_kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    positions = []
    for b, (n, parents) in enumerate(zip(kv, s["parents"].tolist())):
        chains = _chains(parents)
        places = [n + len(x) - 1 if x else -1 for x in chains]
        positions += places
        see = torch.zeros((T, n + T), dtype=torch.bool)
        pos = torch.cat((torch.arange(n), torch.tensor(places)))
        for t, chain in enumerate(chains):
            if not chain:
                continue
            see[t, :n] = True
            see[t, [n + a for a in chain]] = True
            if c["window"]:
                see[t] &= pos > places[t] - c["window"]
            if c["prefix"]:
                see[t, :min(n, c["prefix"])] = True
        see = see.cuda()
        dist = (torch.tensor(places)[:, None] - pos[None]).abs().cuda().double()
        where = _slots(s["table"][b], n, page)
        for h in range(H_kv):
            k = torch.cat((s["k_pool"].view(-1, H_kv, D)[where, h], s["k_nodes"][b, :T, h])).double()
            v = torch.cat((s["v_pool"].view(-1, H_kv, D)[where, h], s["v_nodes"][b, :T, h])).double()
            for hq in range(h * G, (h + 1) * G):
                e = s["q"][b, :, hq].double() @ k.T / D ** 0.5
                if c["softcap"]:
                    e = c["softcap"] * torch.tanh(e / c["softcap"])
                if c["slopes"]:
                    e = e - s["slopes"][hq].double() * dist
                e = e.masked_fill(~see, -math.inf)
                z = torch.logsumexp(e, 1)
                lse[b, :, hq] = z
                w = torch.exp(e - torch.where(z > -math.inf, z, 0.0)[:, None]).masked_fill(~see, 0.0)
                out[b, :, hq] = w @ v
    return {"positions": _ints(positions), "out": out, "lse": lse}


def _exact_reserve(table, kv, refs, grow, page):
    free = [p for p, r in enumerate(refs) if r == 0]
    shared, max_pages = list(refs), len(table[0])
    granted, src, dst = [], [], []
    asked, there = 0, len(free)
    for b, n in enumerate(grow):
        have, want = -(-kv[b] // page), -(-(kv[b] + n) // page)
        copy = n > 0 and kv[b] % page > 0 and shared[table[b][have - 1]] > 1
        granted.append(0)
        src.append(-1)
        dst.append(-1)
        if want > max_pages:
            continue
        need = want - have + copy
        asked += need
        if need and asked > there:
            continue
        if copy:
            src[b], dst[b] = table[b][have - 1], free.pop(0)
            refs[src[b]] -= 1
            refs[dst[b]] = 1
            table[b][have - 1] = dst[b]
        for m in range(have, want):
            table[b][m] = free.pop(0)
            refs[table[b][m]] = 1
        granted[b] = n
        kv[b] += n
    return granted, src, dst


def _exact_pages(s, c):
    page = c["page"]
    table, kv, refs = (x.cpu().tolist() for x in _books(s, s["books"]))
    pools = s["pools"].double()
    got = {}
    if c["op"] == "keep":
        paths, tokens = [], []
        for parents, drafts, answers in zip(*(s[k].tolist() for k in ("parents", "tokens", "answers"))):
            chains = _chains(parents)
            path = [0] if chains[0] else []
            while path:
                below = [t for t in range(1, len(parents)) if chains[t][1:2] == path[-1:] and
                         drafts[t] == answers[path[-1]]]
                if not below:
                    break
                path.append(below[0])
            paths.append(path)
            tokens.append(answers[path[-1]] if path else -1)
        granted, src, dst = _exact_reserve(table, kv, refs, [len(p) for p in paths], page)
        got = {"path": _ints([p + [-1] * (c["nodes"] - len(p)) for p in paths]),
               "n": _ints([len(p) for p in paths]), "token": _ints(tokens), "granted": _ints(granted)}
    elif c["op"] == "fork":
        new = [list(table[b]) for b in s["source"].tolist()]
        kv = [kv[b] for b in s["source"].tolist()]
        for rows, d in ((new, 1), (table, -1)):
            for row in rows:
                for p in row:
                    if p >= 0:
                        refs[p] += d
        table = new
        granted, src, dst = _exact_reserve(table, kv, refs, s["grow"].tolist(), page)
        got = {"granted": _ints(granted), "src": _ints(src), "dst": _ints(dst)}
    else:
        for b, k in enumerate(s["keep"].tolist()):
            kv[b] = min(kv[b], max(k, 0))
            for m in range(-(-kv[b] // page), len(table[b])):
                if table[b][m] >= 0:
                    refs[table[b][m]] -= 1
                    table[b][m] = -1
        n = sum(r > 0 for r in refs)
        dst = [p for p in range(n) if refs[p] == 0]
        src = [p for p in range(n, len(refs)) if refs[p] > 0]
        for a, z in zip(src, dst):
            refs[z], refs[a] = refs[a], 0
        at = dict(zip(src, dst))
        table = [[at.get(p, p) for p in row] for row in table]
        blank = [-1] * (len(refs) // 2 - len(src))
        got = {"src": _ints(src + blank), "dst": _ints(dst + blank), "count": _ints([len(src)])}
    for a, z in zip(src, dst):
        if a >= 0:
            pools[:, z] = s["pools"][:, a].double()
    if c["op"] == "keep":
        for b, path in enumerate(paths):
            for i, t in enumerate(path[:granted[b]]):
                at = kv[b] - granted[b] + i
                pools[:, table[b][at // page], at % page] = s["nodes"][:, b, t].double()
    return dict(got, table=_ints(table), kv_len=_ints(kv), refs=_ints(refs), pools=pools)


def exact(case, seed):
    s = prepare(case, seed)
    f = {"logprobs": _exact_logprobs, "tree": _exact_tree}.get(case["op"], _exact_pages)
    return f(s, case)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "logprobs":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["rows"] * (c["V"] * size + 8 * c["given"] + 8 * c["top"] + 4),
                "flops": 5 * c["rows"] * c["V"]}
    kv = _lengths(c)
    row = 2 * D * c["H_kv"]                  # a token's keys (or values) in one layer
    if c["op"] == "tree":
        T = c["nodes"]
        pairs = read = 0
        for n in kv:
            far = max(0, n - c["window"] + 1) if c["window"] else 0   # what the root's window leaves out
            seen = n - far + min(c["prefix"], far)
            read += seen + T
            pairs += T * seen + T * min(T, 8)
        rows = len(kv) * T
        return {"bytes": read * 2 * row + rows * (c["H_q"] * (4 * D + 4) + 8) +
                4 * sum(-(-n // c["page"]) for n in kv), "flops": 4 * D * pairs * c["H_q"]}
    books = 4 * sum(-(-n // c["page"]) for n in kv) + 8 * len(kv)
    n = 2 * c["layers"]
    if c["op"] == "keep":                    # about four nodes of a tree are kept
        return {"bytes": 2 * n * row * len(kv) * min(4, c["nodes"]) + 12 * c["nodes"] * len(kv),
                "flops": 0}
    pages = len(kv)                          # the last page of each beam
    if c["op"] == "compact":                 # a quarter of the pages, about: half are free, half move
        pages = max(1, sum(-(-m // c["page"]) for m in kv) // 4)
    return {"bytes": 2 * n * row * c["page"] * pages + 2 * books, "flops": 0}
