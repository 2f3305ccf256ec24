"""The operators of the 4-bit paged key / value cache, as cases to be timed.

Three operators: appending rotated keys and values (ring_attn_cache_append),
reading cached tokens back (ring_attn_cache_read) and attention over the cache
(ring_attn_cache_fwd).  `run` computes a case in its plain form (elementary torch
operations) or, with `own` set, by the framework's calls.

A cache page holds `page` tokens of every key / value head: two e2m1 codes per
byte (the even head dim in the low half) and one e4m3 scale per 16 head dims.
A new token j of the n of a sequence sits at cache index len - n + j, where len
is the sequence's length after the append.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16


def listed():
    """Cases of a server that keeps long contexts in 4 bits.

    new_* / kv_*: new tokens and cache length per sequence (after the append),
    drawn log-uniformly on [lo, hi] by `mix`; rot: rotated head dims; inter:
    rotation pairs (2i, 2i + 1) instead of (i, i + rot / 2); far: explicit
    positions (a shard's tokens are not consecutive) instead of cache indices."""
    a = dict(op="append", causal=True, inter=False, far=False, mix=1)
    r = dict(op="read", causal=True, inter=False, far=False, mix=2, rot=0)
    f = dict(op="attend", causal=True, inter=False, far=False, mix=3, rot=0)
    return [
        # one user's next token: launch latency
        dict(a, name="append_one_token", seqs=1, new_lo=1, new_hi=1, kv_lo=1000, kv_hi=1000, h=32, hk=8, d=128, rot=128, page=16),
        # one decoding step of a batch whose contexts differ
        dict(a, name="append_batch_step", seqs=128, new_lo=1, new_hi=1, kv_lo=64, kv_hi=32768, h=32, hk=8, d=128, rot=128, page=64),
        # ragged prompts of a model with 64-wide heads, every head its own keys, half of each head rotated, one ring shard's positions
        dict(a, name="append_ragged_d64", seqs=9, new_lo=1, new_hi=2500, kv_lo=2500, kv_hi=9001, h=16, hk=16, d=64, rot=32, page=32, inter=True, far=True),
        # the benchmark's sequence goes into the cache after its forward
        dict(a, name="append_64k_prompt", seqs=1, new_lo=65536, new_hi=65536, kv_lo=65536, kv_hi=65536, h=32, hk=8, d=128, rot=128, page=64),
        # a short cached prefix taken back for a ring attention call
        dict(r, name="read_short_prefix", seqs=1, new_lo=1001, new_hi=1001, kv_lo=1001, kv_hi=1001, h=8, hk=2, d=64, page=16),
        # a long cached context taken back
        dict(r, name="read_128k", seqs=1, new_lo=131072, new_hi=131072, kv_lo=131072, kv_hi=131072, h=32, hk=8, d=128, page=64),
        # one user's next token over a short context
        dict(f, name="attend_one_short", seqs=1, new_lo=1, new_hi=1, kv_lo=1000, kv_hi=1000, h=32, hk=8, d=128, page=16),
        # one user's next token over a very long context: the keys have to be split
        dict(f, name="attend_one_128k", seqs=1, new_lo=1, new_hi=1, kv_lo=131072, kv_hi=131072, h=32, hk=8, d=128, page=64),
        # a decoding step of a ragged batch, eight query heads to a key head
        dict(f, name="attend_batch_ragged", seqs=64, new_lo=1, new_hi=1, kv_lo=200, kv_hi=16384, h=32, hk=4, d=128, page=64),
        # proposed tokens being verified, 64-wide heads, every head its own keys
        dict(f, name="attend_verify_d64", seqs=16, new_lo=5, new_hi=5, kv_lo=300, kv_hi=9000, h=16, hk=16, d=64, page=32),
        # chunks of prompts over what is cached already
        dict(f, name="attend_chunk_ragged", seqs=3, new_lo=129, new_hi=700, kv_lo=2000, kv_hi=20000, h=32, hk=8, d=128, page=32),
        # a chunk at the end of the benchmark's sequence
        dict(f, name="attend_chunk_64k", seqs=1, new_lo=2048, new_hi=2048, kv_lo=65536, kv_hi=65536, h=32, hk=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend"))
    d = rng.choice((64, 128))
    hk = rng.choice((1, 2, 4, 8, 16) if d == 64 else (1, 2, 3, 4, 8))
    h = hk * rng.choice((1, 2, 4, 5, 7, 8))
    case = dict(op=op, h=h, hk=hk, d=d, page=rng.choice((16, 32, 64, 128, 256)), mix=rng.randrange(1 << 20),
                causal=True, rot=0, inter=False, far=False)
    if op == "append":
        case.update(rot=rng.choice((d, d, d // 2)), inter=rng.random() < 0.3, far=rng.random() < 0.3)
        if rng.random() < 0.4:  # a decoding step
            case.update(seqs=_log(rng, 1, 256), new_lo=1, new_hi=1, kv_lo=1, kv_hi=_log(rng, 100, 32768))
        else:
            total = _log(rng, 50, 40000)
            case.update(seqs=_log(rng, 1, 16))
            n = max(1, total // case["seqs"])
            case.update(new_lo=max(1, n // 8), new_hi=n, kv_lo=n, kv_hi=n + _log(rng, 1, 8000))
    elif op == "read":
        seqs = _log(rng, 1, 32)
        n = max(1, _log(rng, 100, 100000) // seqs)
        case.update(seqs=seqs, new_lo=max(1, n // 8), new_hi=n, kv_lo=n, kv_hi=n)
    else:
        case["causal"] = rng.random() < 0.8
        if rng.random() < 0.6:  # single tokens, or a few to be verified
            seqs = _log(rng, 1, 128)
            new = rng.choice((1, 1, 1, 2, 3, 4, 7))
            kv = _log(rng, 50, min(100000, 600000 // seqs))
            case.update(seqs=seqs, new_lo=new, new_hi=new, kv_lo=max(new, kv // 20), kv_hi=kv)
        else:
            seqs = rng.choice((1, 1, 2, 3, 5))
            new = _log(rng, 20, 1500 // seqs)
            kv = _log(rng, 2000, 40000 // seqs)
            case.update(seqs=seqs, new_lo=max(1, new // 4), new_hi=new, kv_lo=kv // 3, kv_hi=kv)
    return case


def _lengths(case):
    """(new tokens, cache length) of every sequence: fixed by the case."""
    rng = random.Random(case["mix"])
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    kv = [max(n, _log(rng, case["kv_lo"], case["kv_hi"])) for n in new]
    if case["op"] == "read":
        new = [min(n, m) for n, m in zip(new, kv)]
    return new, kv


def work(case):
    new, kv = _lengths(case)
    h, hk, d = case["h"], case["hk"], case["d"]
    total, row = sum(new), d // 2 + d // GROUP  # bytes of one cached row
    if case["op"] == "append":
        # q in and out, k and v in, codes and scales out, table rows, and the appended rows read back as values
        return {"bytes": total * (4 * h * d + 4 * hk * d + 2 * hk * row + 4 * case["rot"] + 2 * hk * row + 4 * hk * d),
                "flops": total * (h + hk) * case["rot"] * 3 + total * hk * d * 2}
    if case["op"] == "read":
        return {"bytes": total * 2 * hk * (row + 2 * d), "flops": total * 2 * hk * d}
    pairs = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(new, kv))
    return {"bytes": total * h * (4 * d + 4) + sum(kv) * 2 * hk * row, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _keys(g, tokens, hk, d):
    """Keys as a model has them: some channels carry more than others."""
    gain = torch.exp(0.5 * torch.randn(hk, d, generator=g, device="cuda"))
    return (torch.randn(tokens, hk, d, generator=g, device="cuda") * gain).bfloat16()


def _inputs(case, seed):
    """What the case's call is given, the cache's contents apart."""
    new, kv = _lengths(case)
    g, page = _gen(seed), case["page"]
    total, h, hk, d = sum(new), case["h"], case["hk"], case["d"]
    x = {"q": torch.randn(total, h, d, generator=g, device="cuda").bfloat16(),
         "k": _keys(g, total, hk, d),
         "v": torch.randn(total, hk, d, generator=g, device="cuda").bfloat16()}
    need = [-(-m // page) for m in kv]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need[:-1], device="cuda").cumsum(0)
    at = first[:, None] + torch.arange(max(need), device="cuda")[None]
    x["page_table"] = order[at.clamp(max=n_pages - 1)].contiguous()
    x["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    x["cu"] = [0]
    for n in new:
        x["cu"].append(x["cu"][-1] + n)
    x["n_pages"] = n_pages
    if case["op"] == "append":
        far = max(kv) * (2 if case["far"] else 1)
        freq = 500000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") * 2 / case["rot"])
        angle = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * freq
        x["cos"], x["sin"] = angle.cos().float(), angle.sin().float()
        x["pos"] = None
        if case["far"]:  # every second token of a longer sequence
            lens, starts = torch.tensor(kv, device="cuda"), torch.tensor(x["cu"][:-1], device="cuda")
            n = torch.tensor(new, device="cuda")
            t = torch.arange(total, device="cuda")
            s = torch.bucketize(t, torch.tensor(x["cu"][1:], device="cuda"), right=True)
            x["pos"] = (2 * (lens[s] - n[s] + t - starts[s]) + 1).to(torch.int32)
    return x, g


def _fill(case, x, g):
    """A cache that holds tokens already: keys and values quantised page by page."""
    n, hk, page, d = x["n_pages"], case["hk"], case["page"], case["d"]
    got = []
    for what in ("k", "v"):
        codes = torch.empty(n, hk, page, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n, hk, page, d // GROUP, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (hk * page * d))
        for p in range(0, n, step):
            m = min(step, n - p)
            t = (_keys if what == "k" else lambda g, *s: torch.randn(*s, generator=g, device="cuda"))(g, m * page, hk, d)
            c, s = _to_4_bits(t.float())
            codes[p:p + m] = c.view(m, page, hk, d // 2).transpose(1, 2)
            scales[p:p + m] = s.view(m, page, hk, d // GROUP).transpose(1, 2)
        got += [codes, scales]
    return got


def _cache(case, x, g):
    if case["op"] != "append":
        return _fill(case, x, g)
    n, hk, page, d = x["n_pages"], case["hk"], case["page"], case["d"]
    return [torch.zeros(n, hk, page, w, dtype=torch.uint8, device="cuda") for w in (d // 2, d // GROUP, d // 2, d // GROUP)]


def prepare(case, seed):
    x, g = _inputs(case, seed)
    kc, ks, vc, vs = _cache(case, x, g)
    state = {"case": dict(case), "x": x, "cache": (kc, ks, vc, vs)}
    if own:  # the handles that a program makes once, and the buffers that it keeps
        import ring_attn_gb300 as ra

        e4m3 = torch.float8_e4m3fn
        state["handle"] = ra.KVCache(kc, ks.view(e4m3), vc, vs.view(e4m3))
        state["cu"] = ra.CuSeqlens(x["cu"], "cuda")
        if case["op"] == "attend":
            state["workspace"] = ra.ring_attn_cache_workspace(x["q"], state["handle"], state["cu"])
    else:
        new, kv = _lengths(case)
        cu = torch.tensor(x["cu"], device="cuda")
        t = torch.arange(x["cu"][-1], device="cuda")
        state["seq"] = torch.bucketize(t, cu[1:], right=True)
        state["slot"] = x["kv_lens"].long()[state["seq"]] - (cu[1:] - cu[:-1])[state["seq"]] + t - cu[:-1][state["seq"]]
        state["nth"] = t - cu[:-1][state["seq"]]
        state["max_new"] = max(new)
    return state


# ------------------------------------------------------------------ plain form
def _to_4_bits(x):
    """(codes, scales as e4m3 bytes) of (..., d) numbers, two codes per byte."""
    x = x.unflatten(-1, (-1, GROUP))
    a = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448)
    step = torch.exp2((torch.frexp(a)[1].clamp(min=-5) - 4).to(a.dtype))  # e4m3: 8 steps to a power of two, 2^-9 the least
    s = (torch.round(a / step) * step).clamp(min=2.0 ** -9, max=448)
    y = (x / s).abs().clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).to(y.dtype)
    y = torch.round(y / step) * step
    code = sum((y >= v).to(torch.uint8) for v in E2M1[1:]) + 8 * (x < 0).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], s.squeeze(-1).float().to(torch.float8_e4m3fn).view(torch.uint8)


def _of_4_bits(codes, scales):
    """fp32 numbers of codes (..., d / 2) and scales (..., d / 16)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _rotated(x, cos, sin, rot, inter):
    """In 64 bits: keys lie next to the 4-bit format's borders."""
    x, keep = x[..., :rot].double(), x[..., rot:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :rot // 2], x[..., rot // 2:])
    c, s = cos[:, None].double(), sin[:, None].double()
    a, b = a * c - b * s, b * c + a * s
    return torch.cat((torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1), keep), -1)


def _plain_append(st):
    c, x, (kc, ks, vc, vs) = st["case"], st["x"], st["cache"]
    pos = st["slot"] if x["pos"] is None else x["pos"].long()
    cos, sin = x["cos"][pos], x["sin"][pos]
    q = _rotated(x["q"], cos, sin, c["rot"], c["inter"]).bfloat16()
    at, row = x["page_table"][st["seq"], st["slot"] // c["page"]].long(), st["slot"] % c["page"]
    kc[at, :, row], ks[at, :, row] = _to_4_bits(_rotated(x["k"], cos, sin, c["rot"], c["inter"]))
    vc[at, :, row], vs[at, :, row] = _to_4_bits(x["v"].double())
    return q, *_plain_read(st)


def _plain_read(st):
    c, x, (kc, ks, vc, vs) = st["case"], st["x"], st["cache"]
    at, row = x["page_table"][st["seq"], st["slot"] // c["page"]].long(), st["slot"] % c["page"]
    return _of_4_bits(kc[at, :, row], ks[at, :, row]).bfloat16(), _of_4_bits(vc[at, :, row], vs[at, :, row]).bfloat16()


def _plain_attend(st):
    c, x, (kc, ks, vc, vs) = st["case"], st["x"], st["cache"]
    n, h, hk, d = c["seqs"], c["h"], c["hk"], c["d"]
    at = x["page_table"].long()
    k = _of_4_bits(kc[at], ks[at]).transpose(1, 2).flatten(2, 3)  # (seqs, hk, keys, d)
    v = _of_4_bits(vc[at], vs[at]).transpose(1, 2).flatten(2, 3)
    q = torch.zeros(n, st["max_new"], hk, h // hk, d, device="cuda")
    q[st["seq"], st["nth"]] = x["q"].float().unflatten(1, (hk, h // hk))
    last = torch.full((n, st["max_new"]), -1, dtype=torch.long, device="cuda")
    last[st["seq"], st["nth"]] = st["slot"] if c["causal"] else x["kv_lens"].long()[st["seq"]] - 1
    rows = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # (seqs, hk, new * group, d)
    s = rows @ k.transpose(-1, -2) * (1 / math.sqrt(d))
    hide = torch.arange(k.shape[2], device="cuda") > last.repeat_interleave(h // hk, 1)[:, None, :, None]
    s = s.masked_fill_(hide, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ torch.where(torch.arange(k.shape[2], device="cuda")[:, None] < x["kv_lens"][:, None, None, None], v, 0.0)
    o = (o / torch.where(total > 0, total, 1.0)).unflatten(2, (st["max_new"], h // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (m + total.log()).squeeze(-1).unflatten(2, (st["max_new"], h // hk)).permute(0, 2, 1, 3).flatten(2)
    return o[st["seq"], st["nth"]].bfloat16(), lse[st["seq"], st["nth"]].t().contiguous()


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[op](state)
    import ring_attn_gb300 as ra

    x, cache, cu = state["x"], state["handle"], state["cu"]
    table, lens = x["page_table"], x["kv_lens"]
    if op == "append":
        # the appended tokens come back through the read call, as the values that the 4 bits stand for
        q = ra.ring_attn_cache_append(x["k"], x["v"], cache, table, lens, cu, q=x["q"], rope=(x["cos"], x["sin"]),
                                      interleaved=state["case"]["inter"], positions=x["pos"])
        return q, *ra.ring_attn_cache_read(cache, table, lens, cu)
    if op == "read":
        return ra.ring_attn_cache_read(cache, table, lens, cu)
    return ra.ring_attn_cache_fwd(x["q"], cache, table, lens, cu, causal=state["case"]["causal"], workspace=state["workspace"])


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _nearest(x, values):
    """The nearest of `values` (ascending; ties to the one of even index), by counting the midpoints passed."""
    mids = (values[1:] + values[:-1]) / 2
    lo = torch.searchsorted(mids, x)               # midpoints < x
    hi = torch.searchsorted(mids, x, right=True)   # midpoints <= x
    return values[torch.where(lo % 2 == 0, lo, hi)]


def _grid8():
    """The e4m3 numbers from 0 to 448, in order."""
    small = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(small + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)],
                        dtype=torch.float64, device="cuda")


def _stored(x):
    """What the cache's 4 bits stand for, of (tokens, heads, d) numbers in 64 bits."""
    t, h, d = x.shape
    x = x.reshape(-1, GROUP)
    scale = _nearest(x.abs().amax(1) / 6, _grid8()).clamp(min=2.0 ** -9)
    y = _nearest((x.abs() / scale[:, None]).contiguous(), torch.tensor(E2M1, dtype=torch.float64, device="cuda"))
    return (torch.sign(x) * y * scale[:, None]).reshape(t, h, d)


def _turned(x, cos, sin, rot, inter):
    """Each pair as a complex number, turned by its angle."""
    x = x.double()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    z = torch.complex(x[..., a], x[..., b]) * torch.complex(cos.double(), sin.double())[:, None]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _values(codes, scales):
    """Cached rows as 64-bit numbers, from the bits: sign, two of exponent, one of mantissa; four of exponent, three of mantissa."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).int()
    e, m = n // 2 % 4, n % 2
    v = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2.0), m / 2.0) * (1 - 2.0 * (n // 8))
    s = scales.int()
    e, m = s // 8, s % 8
    s = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8.0), m * 2.0 ** -9)
    return v * s.repeat_interleave(GROUP, -1)


def exact(case, seed):
    x, g = _inputs(case, seed)
    new, kv = _lengths(case)
    page, h, hk, d = case["page"], case["h"], case["hk"], case["d"]
    if case["op"] == "append":
        pos = x["pos"]
        if pos is None:
            pos = torch.cat([torch.arange(m - n, m) for n, m in zip(new, kv)]).cuda()
        c, s = x["cos"][pos.long()], x["sin"][pos.long()]
        return (_turned(x["q"], c, s, case["rot"], case["inter"]), _stored(_turned(x["k"], c, s, case["rot"], case["inter"])),
                _stored(x["v"].double()))
    kc, ks, vc, vs = _cache(case, x, g)

    def tokens(i, codes, scales, lo, hi):
        ids = x["page_table"][i, lo // page:-(-hi // page)].long()
        rows = _values(codes[ids], scales[ids]).transpose(1, 2).flatten(0, 1)  # (tokens, hk, d)
        return rows[lo - lo // page * page:][:hi - lo]

    if case["op"] == "read":
        return tuple(torch.cat([tokens(i, c, s, m - n, m) for i, (n, m) in enumerate(zip(new, kv))]) for c, s in ((kc, ks), (vc, vs)))
    out = torch.zeros(sum(new), h, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(h, sum(new), dtype=torch.float64, device="cuda")
    for i, (n, m) in enumerate(zip(new, kv)):
        rows = slice(x["cu"][i], x["cu"][i + 1])
        k, v = tokens(i, kc, ks, 0, m), tokens(i, vc, vs, 0, m)
        for j in range(hk):
            heads = slice(j * (h // hk), (j + 1) * (h // hk))
            s = torch.einsum("nhd,md->hnm", x["q"][rows, heads].double(), k[:, j]) / math.sqrt(d)
            if case["causal"]:
                s += torch.full((n, m), -math.inf, dtype=torch.float64, device="cuda").triu(m - n + 1)
            lse[heads, rows] = torch.logsumexp(s, -1)
            out[rows, heads] = torch.einsum("hnm,md->nhd", torch.softmax(s, -1), v[:, j])
    return out, lse
