"""What a model does to its scores besides the product, and the positions under it, as cases to be timed.

Three operators: rotary positions with several axes (ring_attn_rope and its backward),
attention with capped scores, a bias by distance and a prefix that all tokens see
(ring_attn_fwd / _bwd and their varlen forms with `scores`), and the same scores over the
paged 4-bit cache (ring_attn_cache_fwd with `scores`).  `run` computes a case in its plain
form (elementary torch operations) or, with `own` set, by the framework's calls.

Scores: x = scale q.k, y = cap tanh(x / cap), z = y - slope_h |i - j| (i, j: tokens of the
query and the key in their sequence); a key is seen when causal is off, or j <= i, or j lies
in the sequence's prefix.  Rotation: pair f of a token turns by row pos[axis of f] of a table.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16


def listed():
    """rows: packed tokens (q as (rows, h, d)), or with batched (1, h, rows, d); axes: pairs per
    axis in eighths of the rotated half; back: the gradients too.  kind "ring": (seqs, h, new,
    d) in the order of `layout` over `shards`; "packed": documents of new_lo to new_hi tokens;
    "cached": new tokens over kv_lo to kv_hi cached ones.  slopes: a bias by distance; prefix:
    the share of each sequence that all its tokens see."""
    r = dict(op="rope", rot=128, inter=False, back=False, batched=False)
    a = dict(op="attend", kind="ring", layout="contiguous", shards=1, causal=True, cap=0.0, slopes=False, prefix=0.0, back=False, seqs=1,
             new_lo=0, kv_lo=0, kv_hi=0, page=0, mix=1)
    c = dict(a, kind="cached", new_lo=1, new_hi=1, mix=2)
    return [
        # one user's next token of a model that sees images: launch latency
        dict(r, name="rope_one_token", rows=1, h=32, hk=8, d=128, axes="2 3 3"),
        # gradients of a ragged batch of images and text, 64-wide heads, neighbouring pairs, time / height / width
        dict(r, name="rope_back_d64", rows=9001, h=16, hk=16, d=64, rot=64, axes="2 3 3", inter=True, back=True),
        # the benchmark's sequence on its way into attention
        dict(r, name="rope_64k", rows=65536, h=32, hk=8, d=128, axes="2 3 3", batched=True),
        # a short prompt with capped scores: launch latency
        dict(a, name="capped_small", new_hi=257, h=4, hk=4, d=64, cap=50.0),
        # capped scores over a long sequence, as the ring's shards hold it (the benchmark's 16K sequence)
        dict(a, name="capped_zigzag_16k", new_hi=16384, h=32, hk=32, d=128, layout="zigzag", shards=8, cap=50.0),
        # a training step with a bias by distance, tokens dealt out one by one
        dict(a, name="train_biased_stripe", seqs=2, new_hi=4096, h=16, hk=16, d=64, layout="stripe", shards=4, slopes=True, back=True),
        # a training step with capped scores on prompts that their own tokens see both ways, four query heads to a key head
        dict(a, name="train_capped_prefix", new_hi=8192, h=32, hk=8, d=128, layout="zigzag", shards=4, cap=30.0, prefix=0.3, back=True),
        # both ways, an odd length, both changes of the scores
        dict(a, name="train_both_ways_odd", seqs=3, new_hi=1001, h=8, hk=8, d=64, causal=False, cap=20.0, slopes=True, back=True),
        # a training step on packed documents with a bias by distance
        dict(a, name="train_documents", kind="packed", seqs=12, new_lo=200, new_hi=4000, h=16, hk=4, d=128, slopes=True, back=True),
        # one user's next token over a very long context
        dict(c, name="cached_one_128k", kv_lo=131072, kv_hi=131072, h=32, hk=8, d=128, page=64, cap=50.0),
        # a decoding step of a ragged batch
        dict(c, name="cached_batch_biased", seqs=64, kv_lo=200, kv_hi=16384, h=32, hk=4, d=128, page=64, slopes=True),
        # chunks of prompts over what is cached already, their instructions seen both ways
        dict(c, name="cached_chunks", seqs=3, new_lo=129, new_hi=700, kv_lo=2000, kv_hi=20000, h=32, hk=8, d=128, page=32, cap=30.0, prefix=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice((64, 128))
    hk = rng.choice((1, 2, 4, 8, 16) if d == 64 else (1, 2, 3, 4, 8))
    h = hk * rng.choice((1, 2, 4, 5, 7) if hk <= 4 else (1, 2, 4))
    if rng.random() < 0.25:
        rot = rng.choice((d, d, d // 2))
        return dict(op="rope", rows=_log(rng, 1, 60000), h=h, hk=hk, d=d, rot=rot, axes=rng.choice(("8", "4 4", "2 3 3", "1 1 3 3")),
                    inter=rng.random() < 0.4, back=rng.random() < 0.4, batched=rng.random() < 0.4)
    case = dict(op="attend", h=h, hk=hk, d=d, causal=rng.random() < 0.75, cap=rng.choice((0.0, 0.0, 15.0, 30.0, 50.0)), slopes=rng.random() < 0.5,
                prefix=0.0, layout="contiguous", shards=1, back=False, new_lo=0, kv_lo=0, kv_hi=0, page=0, mix=rng.randrange(1 << 20))
    if case["causal"] and rng.random() < 0.3:
        case["prefix"] = rng.choice((0.1, 0.4, 0.9))
    if not (case["cap"] or case["slopes"] or case["prefix"]):
        case["cap" if rng.random() < 0.5 else "slopes"] = 40.0
    case["slopes"] = bool(case["slopes"])
    kind = case["kind"] = rng.choice(("ring", "ring", "packed", "cached", "cached"))
    if kind == "ring":
        case["back"] = rng.random() < 0.6
        case["seqs"] = rng.choice((1, 1, 2, 3))
        both = 1 if case["causal"] and case["prefix"] < 0.5 else 2  # pairs, in halves of the square
        most = math.sqrt(32 * 8192 ** 2 / (h * case["seqs"] * both))
        n = _log(rng, 50, min(8192, most))
        case["layout"] = rng.choice(("contiguous", "zigzag", "stripe"))
        case["shards"] = rng.choice((1, 2, 4, 8))
        case["new_hi"] = max(1, n // (2 * case["shards"])) * 2 * case["shards"] if case["layout"] == "zigzag" else max(1, n // case["shards"]) * case["shards"]
    elif kind == "packed":
        case["back"] = rng.random() < 0.6
        case["seqs"] = _log(rng, 1, 24)
        n = min(4000, max(2, _log(rng, 100, 24000) // case["seqs"]))
        case.update(new_lo=max(1, n // 8), new_hi=n)
    else:
        case["page"] = rng.choice((16, 32, 64, 128, 256))
        if rng.random() < 0.6:  # single tokens, or a few to be verified
            case["seqs"] = _log(rng, 1, 128)
            new = rng.choice((1, 1, 1, 2, 3, 4, 7))
            kv = _log(rng, 50, min(100000, 600000 // case["seqs"]))
            case.update(new_lo=new, new_hi=new, kv_lo=max(new, kv // 20), kv_hi=max(new, kv))
        else:
            case["seqs"] = rng.choice((1, 1, 2, 3, 5))
            new = _log(rng, 20, 1500 // case["seqs"])
            kv = _log(rng, 2000, 40000 // case["seqs"])
            case.update(new_lo=max(1, new // 4), new_hi=new, kv_lo=kv // 3, kv_hi=kv)
    return case


def _lengths(case):
    """(new tokens, keys, prefix) of every sequence: fixed by the case."""
    rng = random.Random(case["mix"])
    if case["kind"] == "ring":
        new = [case["new_hi"]] * case["seqs"]
        kv = new
    else:
        new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
        kv = [max(n, _log(rng, case["kv_lo"], case["kv_hi"])) for n in new] if case["kind"] == "cached" else new
    return new, kv, [int(m * case["prefix"] * rng.uniform(0.7, 1.0)) for m in kv]


def _seen(case):
    """Pairs of a query and a key that it sees, of one head."""
    total = 0
    for n, m, p in zip(*_lengths(case)):
        if not case["causal"]:
            total += n * m
            continue
        first = m - n  # rows see their own index + 1 keys, or the prefix
        t = min(n, max(0, p - 1 - first))  # rows whose own token lies before the prefix's end
        total += t * p + (first + t + first + n - 1) * (n - t) // 2 + (n - t)
    return total


def work(case):
    h, hk, d = case["h"], case["hk"], case["d"]
    if case["op"] == "rope":
        n_axes = len(case["axes"].split())
        return {"bytes": case["rows"] * ((h + hk) * d * 4 + 4 * case["rot"] + 4 * n_axes), "flops": case["rows"] * (h + hk) * case["rot"] * 3}
    new, kv, _ = _lengths(case)
    total, row = sum(new), d // 2 + d // GROUP  # bytes of one cached row
    pairs = _seen(case)
    if case["kind"] == "cached":
        return {"bytes": total * h * (4 * d + 4) + sum(kv) * 2 * hk * row, "flops": 4 * d * h * pairs}
    if not case["back"]:
        return {"bytes": total * (h * (4 * d + 4) + 4 * hk * d), "flops": 4 * d * h * pairs}
    # q, k, v, dout in; out, lse, dq, dk, dv out; 2 + 5 products
    return {"bytes": total * (h * (8 * d + 4) + 8 * hk * d), "flops": 14 * d * h * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, hk, *shape):
    """Keys as a model has them: some channels carry more than others."""
    return _normal(g, *shape) * torch.exp(0.5 * _normal(g, *(hk if n == -1 else n for n in shape[-1:])))


def _pair_axes(case):
    """The axis of every rotated pair."""
    eighth = case["rot"] // 16
    return [i for i, n in enumerate(case["axes"].split()) for _ in range(int(n) * eighth)]


def _rope_inputs(case, seed):
    g, n, d = _gen(seed), case["rows"], case["d"]
    n_axes = len(case["axes"].split())
    x = {name: (_normal(g, *((1, heads, n, d) if case["batched"] else (n, heads, d)))).bfloat16()
         for name, heads in (("q", case["h"]), ("k", case["hk"]))}
    far = 4096 + n
    freq = 500000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") * 2 / case["rot"])
    angle = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * freq
    x["cos"], x["sin"] = angle.cos().float(), angle.sin().float()
    # time goes on along the sequence, the other axes walk over images of random widths
    start = torch.randint(0, 4096, (1,), generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    width = torch.randint(7, 64, (n_axes, 1), generator=g, device="cuda")
    walk = (t // width ** torch.arange(n_axes, device="cuda")[:, None] % (width * 4)) if n_axes > 1 else t[None].clone()
    walk[0] = start + t
    x["pos"] = walk.to(torch.int32).contiguous()
    return x


def _tokens(case):
    """The token at each place of the ring's order (contiguous: the places themselves)."""
    s, n = case["new_hi"], case["shards"]
    p = torch.arange(s, device="cuda")
    r, i = p // (s // n), p % (s // n)
    if case["layout"] == "stripe":
        return i * n + r
    if case["layout"] == "zigzag":
        c = s // (2 * n)
        return torch.where(i < c, r * c + i, (2 * n - 1 - r) * c + i - c)
    return p


def _inputs(case, seed):
    new, kv, prefix = _lengths(case)
    g, n, h, hk, d = _gen(seed), case["seqs"], case["h"], case["hk"], case["d"]
    total = sum(new)
    x = {}
    if case["kind"] == "ring":
        s = case["new_hi"]
        x["q"] = (2 * _normal(g, n, h, s, d)).bfloat16()
        x["k"] = _keys(g, hk, n, hk, s, d).bfloat16()
        x["v"] = _normal(g, n, hk, s, d).bfloat16()
    else:
        x["q"] = (2 * _normal(g, total, h, d)).bfloat16()
        if case["kind"] == "packed":
            x["k"] = _keys(g, hk, total, hk, d).bfloat16()
            x["v"] = _normal(g, total, hk, d).bfloat16()
    if case["back"]:
        x["do"] = _normal(g, *x["q"].shape).bfloat16()
    x["slopes"] = None
    if case["slopes"]:  # a geometric row of slopes, as such models have
        x["slopes"] = torch.exp2(-8.0 * (torch.arange(h, device="cuda") + torch.rand(h, generator=g, device="cuda")) / h)
    x["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda") if case["prefix"] else None
    x["cu"] = [0]
    for m in new:
        x["cu"].append(x["cu"][-1] + m)
    if case["kind"] == "cached":
        page = case["page"]
        need = [-(-m // page) for m in kv]
        x["n_pages"] = sum(need) + 3
        order = torch.randperm(x["n_pages"], generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + need[:-1], device="cuda").cumsum(0)
        at = first[:, None] + torch.arange(max(need), device="cuda")[None]
        x["page_table"] = order[at.clamp(max=x["n_pages"] - 1)].contiguous()
        x["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        x["cache"] = _fill(case, x["n_pages"], g)
    return x


def _to_4_bits(x):
    """(codes, scales as e4m3 bytes) of (..., d) numbers, two codes per byte."""
    x = x.unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(-1, keepdim=True) / 6).clamp(min=2.0 ** -9, max=448).to(torch.float8_e4m3fn)
    y = (x / s.float()).abs().clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.round(y / step) * step
    code = sum((y >= v).to(torch.uint8) for v in E2M1[1:]) + 8 * (x < 0).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], s.squeeze(-1).view(torch.uint8)


def _fill(case, n, g):
    """A cache that holds tokens already: keys and values quantised some pages at a time."""
    hk, page, d = case["hk"], case["page"], case["d"]
    got = []
    for what in ("k", "v"):
        codes = torch.empty(n, hk, page, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n, hk, page, d // GROUP, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (hk * page * d))
        for p in range(0, n, step):
            m = min(step, n - p)
            codes[p:p + m], scales[p:p + m] = _to_4_bits(_keys(g, hk, m, hk, page, d) if what == "k" else _normal(g, m, hk, page, d))
        got += [codes, scales]
    return got


def prepare(case, seed):
    if case["op"] == "rope":
        state = {"case": dict(case), "x": _rope_inputs(case, seed), "axes": _pair_axes(case)}
        if not own:
            state["axes"] = torch.tensor(state["axes"], device="cuda")
        return state
    x = _inputs(case, seed)
    state = {"case": dict(case), "x": x}
    if own:  # the handles that a program makes once, and the buffers that it keeps
        import ring_attn_gb300 as ra

        state["scores"] = ra.Scores(softcap=case["cap"], slopes=x["slopes"], prefix=x["prefix"])
        if case["kind"] != "ring":
            state["cu"] = ra.CuSeqlens(x["cu"], "cuda")
        if case["kind"] == "cached":
            kc, ks, vc, vs = x["cache"]
            state["handle"] = ra.KVCache(kc, ks.view(torch.float8_e4m3fn), vc, vs.view(torch.float8_e4m3fn))
            state["workspace"] = ra.ring_attn_cache_workspace(x["q"], state["handle"], state["cu"])
        return state
    new, kv, _ = _lengths(case)
    if case["kind"] == "ring":
        state["tok_q"] = state["tok_k"] = _tokens(case).expand(case["seqs"], -1)
    else:  # packed rows at their places in a padded batch
        cu = torch.tensor(x["cu"], device="cuda")
        t = torch.arange(x["cu"][-1], device="cuda")
        state["seq"] = torch.bucketize(t, cu[1:], right=True)
        state["nth"] = t - cu[:-1][state["seq"]]
        before = torch.tensor(kv, device="cuda") - torch.tensor(new, device="cuda")
        state["tok_q"] = before[:, None] + torch.arange(max(new), device="cuda")
        width = x["page_table"].shape[1] * case["page"] if case["kind"] == "cached" else max(kv)
        state["tok_k"] = torch.arange(width, device="cuda").expand(len(kv), -1)
    state["len"] = torch.tensor(kv, device="cuda")
    return state


# ------------------------------------------------------------------ plain form
def _plain_rope(st):
    c, x = st["case"], st["x"]
    pair = torch.arange(c["rot"] // 2, device="cuda")
    row = x["pos"].long()[st["axes"]].t()  # (rows, pairs): the table row of every pair
    cos, sin = x["cos"][row, pair], x["sin"][row, pair]
    if c["back"]:  # the turn's transpose is the turn back
        sin = -sin
    if not c["batched"]:
        cos, sin = cos[:, None], sin[:, None]

    def turn(t):
        t, keep = t[..., :c["rot"]].float(), t[..., c["rot"]:].float()
        a, b = (t[..., 0::2], t[..., 1::2]) if c["inter"] else (t[..., :c["rot"] // 2], t[..., c["rot"] // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        t = torch.stack((a, b), -1).flatten(-2) if c["inter"] else torch.cat((a, b), -1)
        return torch.cat((t, keep), -1).bfloat16()

    return turn(x["q"]), turn(x["k"])


def _of_4_bits(codes, scales):
    """fp32 numbers of codes (..., d / 2) and scales (..., d / 16)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _padded(st, t):
    """(rows, heads, d) packed rows as (seqs, heads, longest, d) in fp32."""
    y = torch.zeros(st["len"].numel(), st["tok_q"].shape[1], *t.shape[1:], device="cuda")
    y[st["seq"], st["nth"]] = t.float()
    return y.transpose(1, 2)


def _plain_attend(st):
    c, x = st["case"], st["x"]
    h, hk, d, cap = c["h"], c["hk"], c["d"], c["cap"]
    scale = 1 / math.sqrt(d)
    if c["kind"] == "ring":
        q, k, v = x["q"].float(), x["k"].float(), x["v"].float()
    elif c["kind"] == "packed":
        q, k, v = _padded(st, x["q"]), _padded(st, x["k"]), _padded(st, x["v"])
    else:
        at = x["page_table"].long()
        kc, ks, vc, vs = x["cache"]
        q = _padded(st, x["q"])
        k = _of_4_bits(kc[at], ks[at]).transpose(1, 2).flatten(2, 3)  # (seqs, hk, keys, d)
        v = _of_4_bits(vc[at], vs[at]).transpose(1, 2).flatten(2, 3)
        v = torch.where(st["tok_k"][:, None, :, None] < st["len"][:, None, None, None], v, 0.0)
    n, mq, mk = q.shape[0], q.shape[2], k.shape[2]

    def by_key_head(t):  # (n, h, rows, ...) -> (n, hk, group * rows, ...)
        return t.unflatten(1, (hk, h // hk)).flatten(2, 3)

    def by_head(t):
        return t.unflatten(2, (h // hk, mq)).flatten(1, 2)

    i, j = st["tok_q"][:, :, None], st["tok_k"][:, None, :]
    see = j < st["len"][:, None, None]
    if c["causal"]:
        last = i if x["prefix"] is None else torch.maximum(i, x["prefix"].long()[:, None, None] - 1)
        see = see & (j <= last)
    z = by_head(by_key_head(q) @ k.transpose(-1, -2)).mul_(scale)
    t = None
    if cap:
        t = z.div_(cap).tanh_()
        z = t * cap
    if x["slopes"] is not None:
        z = z - x["slopes"][:, None, None] * (i - j).abs().float()[:, None]
    z.masked_fill_(~see[:, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    lse = (m + total.log()).squeeze(-1)  # (n, h, rows)
    out = by_head(by_key_head(p) @ v)
    if c["kind"] == "ring":
        whole, whole_lse = (lambda t: t.bfloat16()), (lambda t: t)
    else:
        whole = lambda t: t.transpose(1, 2)[st["seq"], st["nth"]].bfloat16()  # noqa: E731
        whole_lse = lambda t: t.transpose(1, 2)[st["seq"], st["nth"]].t().contiguous()  # noqa: E731
    if not c["back"]:
        return whole(out), whole_lse(lse)
    do = x["do"].float() if c["kind"] == "ring" else _padded(st, x["do"])
    dv = by_key_head(p).transpose(-1, -2) @ by_key_head(do)
    ds = by_head(by_key_head(do) @ v.transpose(-1, -2)).sub_((do * out).sum(-1, keepdim=True)).mul_(p)
    if t is not None:
        ds = ds.mul_(1 - t * t)
    dq = by_head(by_key_head(ds) @ k) * scale
    dk = by_key_head(ds).transpose(-1, -2) @ by_key_head(q) * scale
    return whole(out), whole_lse(lse), whole(dq), whole(dk), whole(dv)


def run(state):
    c, x = state["case"], state["x"]
    if not own:
        return _plain_rope(state) if c["op"] == "rope" else _plain_attend(state)
    import ring_attn_gb300 as ra

    if c["op"] == "rope":
        turn = ra.ring_attn_rope_bwd if c["back"] else ra.ring_attn_rope
        pos = x["pos"][:, None] if c["batched"] else x["pos"]
        return turn(x["q"], x["k"], (x["cos"], x["sin"]), positions=pos, axes=state["axes"], interleaved=c["inter"])
    scores = state["scores"]
    if c["kind"] == "cached":
        return ra.ring_attn_cache_fwd(x["q"], state["handle"], x["page_table"], x["kv_lens"], state["cu"], causal=c["causal"],
                                      workspace=state["workspace"], scores=scores)
    if c["kind"] == "ring":
        how = dict(layout=c["layout"], n_shards=c["shards"], causal=c["causal"], scores=scores)
        out, lse = ra.ring_attn_fwd(x["q"], x["k"], x["v"], **how)
        return (out, lse, *ra.ring_attn_bwd(x["do"], x["q"], x["k"], x["v"], out, lse, **how)) if c["back"] else (out, lse)
    how = dict(causal=c["causal"], scores=scores)
    out, lse = ra.ring_attn_varlen_fwd(x["q"], x["k"], x["v"], state["cu"], **how)
    return (out, lse, *ra.ring_attn_varlen_bwd(x["do"], x["q"], x["k"], x["v"], out, lse, state["cu"], **how)) if c["back"] else (out, lse)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _turned(c, x, name, axes):
    """Each pair as a complex number, turned by its angle."""
    t = x[name].double().clone()
    if c["batched"]:
        t = t[0].transpose(0, 1)  # (rows, heads, d)
    f = torch.arange(c["rot"] // 2, device="cuda")
    a, b = (2 * f, 2 * f + 1) if c["inter"] else (f, f + c["rot"] // 2)
    turn = torch.empty(t.shape[0], c["rot"] // 2, dtype=torch.complex128, device="cuda")
    for i, axis in enumerate(axes):
        row = x["pos"][axis].long()
        turn[:, i] = torch.complex(x["cos"][row, i].double(), x["sin"][row, i].double())
    z = torch.complex(t[..., a], t[..., b]) * (turn.conj() if c["back"] else turn)[:, None]
    t[..., a], t[..., b] = z.real, z.imag
    return t.transpose(0, 1)[None] if c["batched"] else t


def _values(codes, scales):
    """Cached rows as 64-bit numbers, from the bits: sign, two of exponent, one of mantissa; four of exponent, three of mantissa."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).int()
    e, m = n // 2 % 4, n % 2
    v = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2.0), m / 2.0) * (1 - 2.0 * (n // 8))
    s = scales.int()
    e, m = s // 8, s % 8
    s = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8.0), m * 2.0 ** -9)
    return v * s.repeat_interleave(GROUP, -1)


def _head(c, q, k, v, i, j, slope, prefix, do):
    """One head of one sequence: out, lse and, with do, the gradients."""
    scale = c["d"] ** -0.5
    y = q @ k.t() * scale
    slack = torch.ones((), dtype=torch.float64, device="cuda")
    if c["cap"]:
        e = torch.exp(-2 * y.abs() / c["cap"])
        th = torch.sign(y) * (1 - e) / (1 + e)
        slack = 4 * e / (1 + e) ** 2  # of tanh: 1 - tanh^2
        y = c["cap"] * th
    if slope is not None:
        y = y - slope * (i[:, None] - j).abs()
    if c["causal"]:
        see = j <= i[:, None]
        if prefix is not None:
            see = see | (j < prefix)
        y = torch.where(see, y, -math.inf)
    lse = torch.logsumexp(y, 1)
    p = torch.softmax(y, 1)
    out = p @ v
    if do is None:
        return out, lse
    ds = p * (do @ v.t() - (do * out).sum(1, keepdim=True)) * slack * scale
    return out, lse, ds @ k, ds.t() @ q, p.t() @ do


def exact(case, seed):
    c = case
    if c["op"] == "rope":
        x, axes = _rope_inputs(c, seed), _pair_axes(c)
        return _turned(c, x, "q", axes), _turned(c, x, "k", axes)
    x = _inputs(c, seed)
    new, kv, _ = _lengths(c)
    h, hk = c["h"], c["hk"]
    if c["kind"] == "ring":
        rows_of = lambda t, i, head: t[i, head]  # noqa: E731
    else:
        rows_of = lambda t, i, head: t[x["cu"][i]:x["cu"][i + 1], head]  # noqa: E731
    f64 = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros(x["q"].shape, **f64)
    lse = torch.zeros(x["q"].shape[:3] if c["kind"] == "ring" else x["q"].shape[:2], **f64)
    dq, dk, dv = ([torch.zeros(x[n].shape, **f64) for n in "qkv"] if c["back"] else (None,) * 3)
    for i, (n, m) in enumerate(zip(new, kv)):
        j = _tokens(c) if c["kind"] == "ring" else torch.arange(m, device="cuda")
        own_tok = j if c["kind"] == "ring" else torch.arange(m - n, m, device="cuda")
        if c["kind"] == "cached":
            ids = x["page_table"][i, :-(-m // c["page"])].long()
            keys, values = (_values(x["cache"][w][ids], x["cache"][w + 1][ids]).transpose(1, 2).flatten(0, 1)[:m] for w in (0, 2))
        prefix = None if x["prefix"] is None else x["prefix"][i].long()
        for a in range(h):
            b = a // (h // hk)
            k, v = (keys[:, b], values[:, b]) if c["kind"] == "cached" else (rows_of(x["k"], i, b).double(), rows_of(x["v"], i, b).double())
            do = rows_of(x["do"], i, a).double() if c["back"] else None
            got = _head(c, rows_of(x["q"], i, a).double(), k, v, own_tok, j, None if x["slopes"] is None else x["slopes"][a].double(), prefix, do)
            rows_of(out, i, a).copy_(got[0])
            rows_of(lse, i, a).copy_(got[1])
            if c["back"]:
                rows_of(dq, i, a).copy_(got[2])
                rows_of(dk, i, b).add_(got[3])
                rows_of(dv, i, b).add_(got[4])
    lse = lse if c["kind"] == "ring" else lse.t()
    return (out, lse, dq, dk, dv) if c["back"] else (out, lse)
