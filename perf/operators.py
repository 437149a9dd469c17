"""The BF16 paged cache: what is measured of its three operators.

A request that has arrived as split streams goes on in BF16: every step writes the new tokens'
keys and values to a paged cache (`append`: positions rotated on the way), and attends over it,
a few tokens per sequence (`decode`) or a whole chunk of a prompt (`prefill`).  Pages hold
[page][H_kv][128] values, so a full page is what lynx_encode packs.

A case is one call.  `context` is the length of the longest sequence in the cache after the
append; with `ragged` the others are spread below it, down to a length of zero or one.  The lengths
follow from the case alone; the values, and which physical page holds what, from the seed.
"""
import math
import random

import torch

own = False

D = 128


# ------------------------------------------------------------------ cases

def _case(name, op, batch, new, context, H_q, H_kv, page, ragged=False, rope="half", rot=128,
          axes=1, fused=False, softcap=0.0, window=0, prefix=0, slopes=False):
    c = {"op": op, "batch": batch, "new": new, "context": context, "H_q": H_q, "H_kv": H_kv,
         "page": page, "ragged": ragged}
    if op == "append":
        c.update(rope=rope, rot=rot, axes=axes, fused=fused)
    else:
        c.update(softcap=softcap, window=window, prefix=prefix, slopes=slopes)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence's next token: nothing but latency
        _case("append-1", "append", 1, 1, 777, 32, 8, 64),
        # a decode step of a full batch, q, k and v being views of one fused projection
        _case("append-b64", "append", 64, 1, 6000, 64, 4, 128, ragged=True, fused=True),
        # prompts: four of them, packed, about 16K tokens in all
        _case("append-16k", "append", 4, 6144, 6144, 64, 8, 256, ragged=True, fused=True),
        # an image's tokens: time, height and width positions, pairs of neighbours, part of the head
        _case("append-axes", "append", 2, 2521, 2700, 40, 8, 512, rope="pairs", rot=96, axes=3),
        # the first answer tokens of a short chat: latency
        _case("decode-b1-1k", "decode", 1, 1, 1000, 32, 8, 64),
        # the draft step over a batch of long contexts
        _case("decode-b8-32k", "decode", 8, 1, 32768, 64, 4, 256, ragged=True),
        # one very long context, the work split over its length
        _case("decode-b1-128k", "decode", 1, 1, 131071, 64, 8, 128),
        # the verification of eight draft tokens in one pass
        _case("decode-verify", "decode", 8, 8, 32767, 32, 8, 128),
        # a serving batch of every length: capped scores, a window, the first tokens kept visible
        _case("decode-b48-window", "decode", 48, 1, 12001, 40, 8, 64, ragged=True, softcap=50.0,
              window=4096, prefix=4),
        # packed short documents with a bidirectional prefix and a distance bias
        _case("prefill-short", "prefill", 6, 301, 301, 32, 8, 64, ragged=True, prefix=70,
              slopes=True),
        # two prompts of 8K, causal
        _case("prefill-8k", "prefill", 2, 8192, 8192, 32, 8, 256),
        # the next chunk of a prompt whose beginning is cached, capped scores
        _case("prefill-chunk", "prefill", 2, 1023, 16384, 64, 4, 128, softcap=30.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    H_q, H_kv = rng.choice(((32, 8), (64, 8), (64, 4), (40, 8), (16, 16), (8, 1), (24, 2)))
    page = rng.choice((64, 128, 256, 512))
    if op == "append":
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, 16384 // batch)
        rot = rng.choice((128, 128, 64, 96, 32))
        axes = rng.choice((1, 1, 2, 3))
        return _case(None, op, batch, new, new + rng.randrange(0, 4000), H_q, H_kv, page,
                     ragged=rng.random() < 0.5, rope=rng.choice(("half", "pairs")), rot=rot,
                     axes=axes, fused=rng.random() < 0.5)
    softcap = rng.choice((0.0, 0.0, 20.0, 50.0))
    slopes = rng.random() < 0.25
    if op == "decode":
        batch = _log(rng, 1, 64)
        new = rng.choice((1, 1, 1, 2, 5, 8))
        context = _log(rng, new, 1800000 // (batch * H_kv * new))
        context = max(new, min(context, 131072))
    else:
        batch = _log(rng, 1, 8)
        new = _log(rng, 2, 6000 // batch)
        context = new + rng.choice((0, 0, _log(rng, 1, 6000 // batch)))
    window = rng.choice((0, 0, _log(rng, 1, context)))
    prefix = rng.choice((0, 0, rng.randrange(1, 200)))
    return _case(None, op, batch, new, context, H_q, H_kv, page, ragged=rng.random() < 0.5,
                 softcap=softcap, window=window, prefix=prefix, slopes=slopes)


def _lengths(c):
    """Per sequence: tokens that are new in this call, and the cache's length with them."""
    batch, new, context = c["batch"], c["new"], c["context"]
    if not c["ragged"]:
        return [new] * batch, [context] * batch
    rng = random.Random("%d %d %d %d" % (batch, new, context, c["page"]))
    kv = [context] + [rng.randint(0, context) for _ in range(batch - 1)]
    if batch > 2:
        kv[1] = 1
    if batch > 4:
        kv[2] = 0
    if c["op"] == "decode":
        return [new] * batch, kv          # a sequence may hold fewer tokens than the step brings
    return [min(new, n) if new == context else min(rng.randint((new + 1) // 2, new) if i else new, n)
            for i, n in enumerate(kv)], kv


# ------------------------------------------------------------------ inputs

def _tokens(gen, n, heads, stride, boost):
    """n rows of `heads` heads of 128 BF16 values, `stride` values apart; some channels are large, as
    in real keys and queries."""
    x = torch.randn((n, stride // D, D), generator=gen, device="cuda", dtype=torch.float32)
    scale = torch.ones(D, device="cuda")
    scale[torch.randperm(D, generator=gen, device="cuda")[:6]] = boost
    return (x * scale).to(torch.bfloat16)[:, :heads]


def _spread(lengths):
    t = torch.zeros(len(lengths) + 1, dtype=torch.int32)
    t[1:] = torch.cumsum(torch.tensor(lengths, dtype=torch.int64), 0).to(torch.int32)
    return t.cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    batch, H_q, H_kv, page = c["batch"], c["H_q"], c["H_kv"], c["page"]
    new, kv = _lengths(c)
    max_pages = max(1, -(-max(kv) // page))
    used = sum(-(-n // page) for n in kv)
    blocks = used + 2
    # physical pages in any order; entries that no token needs are not pages at all
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(kv):
        p = -(-n // page)
        table[b, :p] = order[at:at + p]
        at += p
    s = {"case": dict(c), "table": table, "max_new": max(1, max(new)),
         "kv_len": torch.tensor(kv, dtype=torch.int32).cuda()}
    n = sum(new)
    if c["op"] == "append":
        stride = (H_q + 2 * H_kv) * D
        if c["fused"]:
            qkv = _tokens(gen, n, H_q + 2 * H_kv, stride, 4.0)
            s["q"], s["k"], s["v"] = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
        else:
            s["q"] = _tokens(gen, n, H_q, H_q * D, 4.0)
            s["k"] = _tokens(gen, n, H_kv, H_kv * D, 4.0)
            s["v"] = _tokens(gen, n, H_kv, H_kv * D, 1.0)
        s["k_pool"] = torch.zeros((blocks, page, H_kv, D), dtype=torch.bfloat16, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["offsets"] = _spread(new)
        half = c["rot"] // 2
        s["inv_freq"] = [1e6 ** (-i / half) for i in range(half)]
        s["axis"] = [i * c["axes"] // half for i in range(half)]
        s["inv_freq_gpu"] = torch.tensor(s["inv_freq"], dtype=torch.float64).cuda()
        s["axis_gpu"] = torch.tensor(s["axis"], dtype=torch.int64).cuda()
        s["positions"] = None
        if c["axes"] > 1:      # the axes of images and video: small numbers, and late ones
            s["positions"] = torch.randint(0, 60000, (c["axes"], max(n, 1)), generator=gen, device="cuda",
                                           dtype=torch.int32)[:, :n].contiguous()
        s["rope"] = None
        return s
    pool = _tokens(gen, blocks * page, H_kv, H_kv * D, 3.0).reshape(blocks, page, H_kv, D)
    s["k_pool"] = pool
    s["v_pool"] = torch.randn((blocks, page, H_kv, D), generator=gen, device="cuda",
                              dtype=torch.float32).to(torch.bfloat16)
    q = _tokens(gen, batch * c["new"] if c["op"] == "decode" else n, H_q, H_q * D, 3.0)
    s["q"] = q.reshape(batch, c["new"], H_q, D) if c["op"] == "decode" else q
    s["offsets"] = _spread(new)
    s["slopes"] = s["prefix"] = None
    if c["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H_q) for h in range(H_q)],
                                   dtype=torch.float32).cuda()
    if c["prefix"]:
        s["prefix"] = torch.full((batch,), c["prefix"], dtype=torch.int32).cuda()
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from split_stream_kv_gb300 import lynx
    c = s["case"]
    if c["op"] == "append":
        if s["rope"] is None:       # built once, like a model's own table of frequencies
            s["rope"] = lynx.Rope(s["inv_freq"], s["axis"] if c["axes"] > 1 else None,
                                  interleaved=c["rope"] == "pairs")
        q = lynx.lynx_cache_append(s["k"], s["v"], s["offsets"], s["kv_len"], s["table"],
                                   s["k_pool"], s["v_pool"], q=s["q"], rope=s["rope"],
                                   positions=s["positions"])
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    kw = {"softcap": c["softcap"], "window": c["window"], "slopes": s["slopes"],
          "prefix": s["prefix"]}
    q = s["q"]
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    if c["op"] == "decode":
        out = lynx.lynx_cache_attn_decode(q, s["k_pool"], s["v_pool"], s["table"], s["kv_len"],
                                          lse=lse, **kw)
    else:
        out = lynx.lynx_cache_attn_prefill(q, s["offsets"], s["k_pool"], s["v_pool"], s["table"],
                                           s["kv_len"], lse=lse, **kw)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ plain forms

def _owner(offsets, n):
    """Of n packed tokens: the sequence of each and its index there."""
    t = torch.arange(n, device=offsets.device)
    b = torch.searchsorted(offsets[1:].long().contiguous(), t, right=True)
    return b, t - offsets.long()[b]


def _turn(x, cos, sin, pairs):
    """x [n][heads][D] in 32 bits, its first 2 * cos.shape[-1] channels rotated."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if pairs:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half:]), -1).to(torch.bfloat16)


def _plain_append(s):
    c, k = s["case"], s["k"]
    page = c["page"]
    b, i = _owner(s["offsets"], k.shape[0])
    new = (s["offsets"][1:] - s["offsets"][:-1]).long()
    at = s["kv_len"].long()[b] - new[b] + i
    where = (s["positions"].double() if s["positions"] is not None else at.double()[None])
    angle = where[s["axis_gpu"]].T * s["inv_freq_gpu"]
    cos, sin = angle.cos().float(), angle.sin().float()
    pairs = c["rope"] == "pairs"
    slot = s["table"][b, at // page].long() * page + at % page
    s["k_pool"].view(-1, c["H_kv"], D)[slot] = _turn(k.float(), cos, sin, pairs)
    s["v_pool"].view(-1, c["H_kv"], D)[slot] = s["v"]
    return {"q": _turn(s["q"].float(), cos, sin, pairs), "k_pool": s["k_pool"],
            "v_pool": s["v_pool"]}


def _plain_attention(s, q, first, c):
    """q [batch][T][H_q][D], the token of row t at position first[b] + t; rows of no sequence are
    computed too and dropped by the caller."""
    batch, T, H_q, _ = q.shape
    H_kv, G = c["H_kv"], H_q // c["H_kv"]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * c["page"]
    j = torch.arange(L, device=q.device)
    held = j < s["kv_len"].long()[:, None]
    k = s["k_pool"][table].reshape(batch, L, H_kv, D).float()
    v = s["v_pool"][table].reshape(batch, L, H_kv, D).float()
    v = v.masked_fill_(~held[..., None, None], 0.0)
    qq = q.float().reshape(batch, T, H_kv, G, D).permute(0, 2, 3, 1, 4)
    a = torch.matmul(qq.reshape(batch, H_kv, G * T, D), k.permute(0, 2, 3, 1))
    a = a.mul_(1.0 / math.sqrt(D)).view(batch, H_kv, G, T, L)
    if c["softcap"]:
        a = a.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    i = first[:, None] + torch.arange(T, device=q.device)
    gap = i[:, :, None] - j
    if s["slopes"] is not None:
        a.sub_(s["slopes"].view(1, H_kv, G, 1, 1) * gap.abs()[:, None, None])
    seen = gap >= 0
    if c["window"]:
        seen &= gap < c["window"]
    if s["prefix"] is not None:
        seen |= (j < s["prefix"][:, None])[:, None]
    seen &= held[:, None]
    seen &= (i >= 0)[:, :, None]
    a.masked_fill_(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    some = m > -math.inf
    a = a.sub_(torch.where(some, m, 0.0)).exp_()
    l = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(batch, H_kv, G * T, L), v.permute(0, 2, 1, 3))
    o = o.view(batch, H_kv, G, T, D) / torch.where(some, l, 1.0)
    lse = torch.where(some, m + l.log(), -math.inf)[..., 0]
    return (o.permute(0, 3, 1, 2, 4).reshape(batch, T, H_q, D).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2).reshape(batch, T, H_q))


def _plain(s):
    c = s["case"]
    if c["op"] == "append":
        return _plain_append(s)
    kv = s["kv_len"].long()
    if c["op"] == "decode":
        out, lse = _plain_attention(s, s["q"], kv - c["new"], c)
        return {"out": out, "lse": lse}
    q, offsets = s["q"], s["offsets"].long()
    new = offsets[1:] - offsets[:-1]
    rows = offsets[:-1, None] + torch.arange(s["max_new"], device=q.device)
    out, lse = _plain_attention(s, q[rows.clamp(max=q.shape[0] - 1)], kv - new, c)
    b, i = _owner(s["offsets"], q.shape[0])
    return {"out": out[b, i], "lse": lse[b, i]}


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits

def _place(s, b, n):
    """The physical slots of positions 0 .. n-1 of sequence b."""
    page = s["case"]["page"]
    p = torch.arange(n, device="cuda")
    return s["table"][b].long()[p // page] * page + p % page


def _exact_append(s, c, new, kv):
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    q_out = s["q"].double()
    rot, half = c["rot"], c["rot"] // 2
    ch = torch.arange(half, device="cuda")
    lo, hi = (2 * ch, 2 * ch + 1) if c["rope"] == "pairs" else (ch, ch + half)
    t0 = 0
    for b, (n, total) in enumerate(zip(new, kv)):
        if n == 0:
            continue
        at = torch.arange(total - n, total, device="cuda")
        where = at[:, None].expand(n, half) if s["positions"] is None else \
            s["positions"][:, t0:t0 + n].T[:, s["axis_gpu"]]
        z = torch.polar(torch.ones((n, half), dtype=torch.float64, device="cuda"),
                        where.double() * s["inv_freq_gpu"])[:, None]
        for name in ("q", "k"):
            x = s[name][t0:t0 + n].double()
            w = torch.complex(x[..., lo], x[..., hi]) * z
            y = x.clone()
            y[..., lo], y[..., hi] = w.real, w.imag
            if name == "q":
                q_out[t0:t0 + n] = y
            else:
                k_pool.view(-1, c["H_kv"], D)[_place(s, b, total)[-n:]] = y
        v_pool.view(-1, c["H_kv"], D)[_place(s, b, total)[-n:]] = s["v"][t0:t0 + n].double()
        t0 += n
    return {"q": q_out, "k_pool": k_pool, "v_pool": v_pool}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    new, kv = _lengths(c)
    if c["op"] == "append":
        return _exact_append(s, c, new, kv)
    G = c["H_q"] // c["H_kv"]
    q = s["q"].reshape(-1, c["H_q"], D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, total) in enumerate(zip(new, kv)):
        if n and total:
            slots = _place(s, b, total)
            pos = torch.arange(total - n, total, device="cuda")[:, None]
            key = torch.arange(total, device="cuda")[None]
            ok = key <= pos
            if c["window"]:
                ok = ok & (key > pos - c["window"])
            if c["prefix"]:
                ok = ok | (key < c["prefix"])
            ok = ok & (pos >= 0)
            for h in range(c["H_kv"]):
                kk = s["k_pool"].view(-1, c["H_kv"], D)[slots, h].double()
                vv = s["v_pool"].view(-1, c["H_kv"], D)[slots, h].double()
                for hq in range(h * G, (h + 1) * G):
                    e = q[t0:t0 + n, hq].double() @ kk.T / D ** 0.5
                    if c["softcap"]:
                        e = c["softcap"] * torch.tanh(e / c["softcap"])
                    if c["slopes"]:
                        e = e - s["slopes"][hq].double() * (pos - key).abs()
                    e = torch.where(ok, e, -math.inf)
                    z = torch.logsumexp(e, 1)
                    lse[t0:t0 + n, hq] = z
                    w = torch.where(ok, torch.exp(e - torch.where(z > -math.inf, z, 0.0)[:, None]), 0.0)
                    out[t0:t0 + n, hq] = w @ vv
        t0 += n
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}


# ------------------------------------------------------------------ work

def work(case):
    c = case
    new, kv = _lengths(c)
    n, row = sum(new), 2 * D
    if c["op"] == "append":
        move = n * row * (2 * c["H_q"] + 4 * c["H_kv"])
        where = 4 * n * c["axes"] if c["axes"] > 1 else 0
        return {"bytes": move + where + 4 * (2 * c["batch"] + 1),
                "flops": 3 * n * c["rot"] * (c["H_q"] + c["H_kv"])}
    pairs = read = 0
    for m, total in zip(new, kv):
        read_b = 0
        first = None
        for i in range(max(0, total - m), total):
            lo = max(0, i + 1 - c["window"]) if c["window"] else 0
            pre = min(c["prefix"], total)
            pairs += i + 1 - lo + min(pre, lo) + max(0, pre - (i + 1))
            first = lo if first is None else first
        if first is not None:
            read_b = total - first + min(min(c["prefix"], total), first)
        read += read_b
    rows = n if c["op"] == "prefill" else c["batch"] * c["new"]
    pages = sum(-(-t // c["page"]) for t in kv)
    return {"bytes": read * 2 * row * c["H_kv"] + rows * c["H_q"] * (2 * row + 4) + 4 * pages,
            "flops": 4 * D * pairs * c["H_q"]}
