"""Changed scores at the ends of what the calls take: steep biases, single ring steps, products and values far from 1,
saturated caps, a block's share of a longer row."""
import numpy as np
import pytest
import torch

import oracle
import ring_attn_gb300 as ra
from tests.helpers import check_no_device_error, lse_to_original, to_layout, to_original
from tests.score_case import EPS, assert_within, expect, f64, head_bounds
from tests.test_gpu_scores import inputs, rows_first, scores_of, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_attn_gb300.build import build

    build()
    ra.load()


def steep(h, of):
    return torch.tensor([of * (1.0 - 0.25 * i) for i in range(h)], dtype=torch.float32)


@pytest.mark.parametrize("layout,causal,cap,slopes,prefix", [
    ("contiguous", True, 8.0, "alibi", (150,)), ("zigzag", True, 0.0, "alibi", None), ("stripe", False, 8.0, "mixed", None),
    ("contiguous", False, 0.0, 100.0, None), ("contiguous", True, 90.0, 100.0, (3,)), ("zigzag", True, 0.0, 60.0, None),
    ("zigzag", False, 0.0, -60.0, None), ("stripe", True, 8.0, -100.0, None), ("contiguous", True, 30.0, 80.0, None),
])
def test_every_ring_step_on_its_own(layout, causal, cap, slopes, prefix):
    """out and lse of a step are those of its keys alone: 0 and -inf only for rows that see none of them.  Steep biases put
    the scores of far keys 2^14 to 2^17 (log2 units) below those near."""
    b, h, hk, s, d, n = 1, 2, 1, 544, 64, 4
    x = inputs(b, h, hk, s, d, 9110)
    sl = slopes_of(h, slopes) if not isinstance(slopes, float) else steep(h, slopes)
    z = scores_of(cap, sl, prefix)
    g = {k: to_layout(ra, v.cuda(), layout, n) for k, v in x.items()}
    place = oracle.token_of_position(layout, n, s).reshape(n, -1)  # tokens of every shard
    for step in range(n):
        out, lse = ra.ring_attn_fwd_step(g["q"], g["k"], g["v"], step, layout, n, causal, scores=z)
        check_no_device_error(ra)
        want = {name: (np.zeros(shape), np.zeros(shape)) for name, shape in (("out", (b, h, s, d)), ("lse", (b, h, s)))}
        for r in range(n):
            gq, gk = place[r], place[(r - step) % n]
            for a in range(h):
                e = head_bounds(x["q"][0, a, gq], x["k"][0, 0, gk], x["v"][0, 0, gk], gq, gk, d ** -0.5, cap,
                                0.0 if sl is None else float(sl[a]), causal, prefix[0] if prefix else 0)
                for name, (val, tol) in want.items():
                    val[0, a, gq], tol[0, a, gq] = e[name], e["tol"][name]
        assert_within("out", to_original(ra, out, layout, n), want["out"])
        assert_within("lse", lse_to_original(ra, lse, layout, n), want["lse"])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap,slope,gain", [(0.0, -100.0, 1.0), (0.0, 100.0, 1.0), (90.0, -60.0, 1.0), (0.0, 0.01, 200.0),
                                            (40.0, -100.0, 1.0)])
def test_far_scores_of_whole_calls(causal, cap, slope, gain):
    """Rows whose largest score is 2^14 and more: a bias that rises with the distance, or large products next to one."""
    b, h, hk, s, d = 1, 2, 1, 600, 128
    x = inputs(b, h, hk, s, d, 9120, gain)
    x["k"] = (x["k"].float() * gain).bfloat16()
    sl = steep(h, slope)
    g = {k: v.cuda() for k, v in x.items()}
    z = scores_of(cap, sl, None)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, causal, scores=z)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, causal, None)
    assert_within("lse", lse, want["lse"])
    assert_within("out", out, want["out"])


@pytest.mark.parametrize("d,cap,slope,gain", [(64, 12.0, 0.0, 2.0), (128, 0.0, 0.02, 2.0), (128, 12.0, 0.02, 1.0)])
@pytest.mark.parametrize("share", [0, 1])
def test_a_blocks_share_of_the_gradients(d, cap, slope, gain, share):
    """The keys of a row in two calls with the whole row's out and lse: each gives its share of dq, and dk and dv of its
    keys, with D = rowsum(dout * out) of the out that it was given."""
    b, h, hk, s = 1, 2, 1, 256
    x = inputs(b, h, hk, 2 * s, d, 9150, gain)
    scale, sl = d ** -0.5, None if not slope else steep(h, slope)
    q, do = x["q"][:, :, :s].contiguous(), x["do"][:, :, :s].contiguous()
    t = np.arange(s)
    out, lse = torch.zeros(b, h, s, d), torch.zeros(b, h, s)
    # (both blocks take distances from tokens 0 to s - 1, as a call has them)
    tokens = np.concatenate([t, t])
    heads = [head_bounds(q[0, a], x["k"][0, 0], x["v"][0, 0], t, tokens, scale, cap, 0.0 if sl is None else float(sl[a]),
                         False, 0, do[0, a]) for a in range(h)]
    for a, r in enumerate(heads):
        out[0, a], lse[0, a] = torch.from_numpy(r["out"]).float(), torch.from_numpy(r["lse"]).float()
    out = out.bfloat16()
    here = slice(share * s, (share + 1) * s)
    k, v = (x[n][:, :, here].contiguous() for n in "kv")
    z = scores_of(cap, sl, None)
    dq, dk, dv = ra.ring_attn_bwd(do.cuda(), q.cuda(), k.cuda(), v.cuda(), out.cuda(), lse.cuda(), "contiguous", 1, False,
                                  scale, scores=z)
    check_no_device_error(ra)
    want = {n: np.zeros((s, d)) for n in ("dk", "dv")}
    bound = {n: np.zeros((s, d)) for n in ("dk", "dv")}
    k64, v64 = f64(k[0, 0]), f64(v[0, 0])
    for a, r in enumerate(heads):
        q64, do64, o64 = f64(q[0, a]), f64(do[0, a]), f64(out[0, a])
        P, gr = r["P"][:, here], r["g"][:, here]
        D = (do64 * o64).sum(1)
        dP, ado = do64 @ v64.T, np.abs(do64)
        aw = dP - D[:, None]
        dx = P * aw * gr
        rel = r["tol"]["lse"][:, None] + 2.0 ** -20
        off = np.abs(dx) * (2.0 ** -8 * 1.02 + rel) + P * np.abs(aw) * 2.0 ** -19 * (cap > 0)
        off += P * gr * d * EPS * (ado @ np.abs(v64).T + (ado * np.abs(o64)).sum(1)[:, None])
        # the sum of a row's roundings, at most 2^-8 of its dS, is taken off as P' would share it out
        off_q = off + P * gr * (np.abs(dx) * 2.0 ** -8).sum(1)[:, None]
        dq64 = scale * dx @ k64
        assert_within("dq", dq[0, a], (dq64, scale * off_q @ np.abs(k64) + 2.0 ** -8 * np.abs(dq64)))
        want["dk"] += scale * dx.T @ q64
        bound["dk"] += scale * off.T @ np.abs(q64)
        want["dv"] += P.T @ do64
        bound["dv"] += (P * (2.0 ** -8 * 1.01 + rel)).T @ ado
    for name, got in (("dk", dk), ("dv", dv)):
        assert_within(name, got[0, 0], (want[name], bound[name] + 2.0 ** -8 * np.abs(want[name])))


def test_slopes_and_prefixes_are_read_from_where_they_are_at_the_call():
    """The storage of a handle's tensors is exchanged: every call gives what a new handle gives."""
    b, h, s, d = 2, 2, 200, 64
    x = {k: v.cuda() for k, v in inputs(b, h, h, s, d, 9170).items()}
    p = {k: v[0].transpose(0, 1).contiguous() for k, v in x.items()}
    cu = ra.CuSeqlens([0, 120, 200], "cuda")
    cache = ra.KVCache.empty(8, 64, h, d)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([120, 80], dtype=torch.int32, device="cuda")
    ra.ring_attn_cache_append(p["k"], p["v"], cache, table, lens, cu)

    def calls(z):
        out, lse = ra.ring_attn_fwd(x["q"], x["k"], x["v"], causal=True, scores=z)
        r = [out, lse, *ra.ring_attn_bwd(x["do"], x["q"], x["k"], x["v"], out, lse, causal=True, scores=z)]
        r += ra.ring_attn_fwd_step(x["q"], x["k"], x["v"], 0, causal=True, scores=z)
        out, lse = ra.ring_attn_varlen_fwd(p["q"], p["k"], p["v"], cu, scores=z)
        r += [out, lse, *ra.ring_attn_varlen_bwd(p["do"], p["q"], p["k"], p["v"], out, lse, cu, scores=z)]
        half = [p[n][:100].contiguous() for n in ("q", "do")]
        out, lse = ra.ring_attn_llama3_varlen_fwd(half[0], p["k"], p["v"], cu, 0, 2, scores=z)
        r += [out, lse, *ra.ring_attn_llama3_varlen_bwd(half[1], half[0], p["k"], p["v"], out, lse, cu, 0, 2, scores=z)]
        return r + list(ra.ring_attn_cache_fwd(p["q"], cache, table, lens, cu, scores=z))

    sl, pre = slopes_of(h, "alibi").cuda(), torch.tensor([10, 60], dtype=torch.int32, device="cuda")
    z = ra.Scores(11.0, sl, pre)
    first = calls(z)
    sl.data = slopes_of(h, "mixed").cuda()
    pre.data = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    now, fresh = calls(z), calls(ra.Scores(11.0, slopes_of(h, "mixed").cuda(), torch.tensor([0, 30], dtype=torch.int32, device="cuda")))
    check_no_device_error(ra)
    assert not torch.equal(first[0], now[0]) and all(torch.equal(a, c) for a, c in zip(now, fresh))


@pytest.mark.parametrize("d,causal,slope", [(64, False, 0.0), (128, True, 0.0), (64, True, 0.05)])
@pytest.mark.parametrize("u", [4.0, 7.0, 9.0, -8.0])
def test_gradients_of_saturated_scores(d, causal, slope, u):
    """x / softcap of u: the derivative is 4 e^(-2|u|) and small, and dq and dk have all of its bits that bf16 keeps.
    x is off by d 2^-24 sum |q k|, which the derivative takes twice over (relatively, next to softcap), and its own
    exponential, reciprocal and products by 2^-18 (the exponential's argument, 26 at most, is rounded)."""
    b, h, hk, s, cap = 1, 2, 1, 320, 1.0
    x = inputs(b, h, hk, s, d, 9140)
    x["q"] = (x["q"].float() * 0.2 + u * 0.5).bfloat16()
    x["k"] = (x["k"].float() * 0.1 + 1.0).bfloat16()
    scale = 2.0 * cap / d  # x is about u cap
    sl = None if not slope else steep(h, slope)
    g = {k: v.cuda() for k, v in x.items()}
    z = scores_of(cap, sl, None)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, causal, scale, scores=z)
    dq, dk, dv = ra.ring_attn_bwd(g["do"], g["q"], g["k"], g["v"], out, lse, "contiguous", 1, causal, scale, scores=z)
    check_no_device_error(ra)
    t = np.arange(s)
    want_dk, tol_dk = np.zeros((s, d)), np.zeros((s, d))
    for a in range(h):
        q, k, v, do = (f64(x[n][0, 0 if n in "kv" else a]) for n in ("q", "k", "v", "do"))
        r = head_bounds(q, k, v, t, t, scale, cap, 0.0 if sl is None else float(sl[a]), causal, 0, do)
        xs = scale * (q @ k.T)
        gr = 1.0 / np.cosh(xs / cap) ** 2  # (1 - tanh^2 in 64 bits has but half of them here)
        dx = r["P"] * (r["dP"] - r["D"][:, None]) * gr
        ado = np.abs(do)
        err = 2 * d * EPS * scale * (np.abs(q) @ np.abs(k).T) / cap + 2.0 ** -18
        rel = 2.0 ** -8 * 1.02 + 2.0 ** -17 + err
        dD = (ado * r["tol"]["out"]).sum(1) + d * EPS * (ado * np.abs(r["out"])).sum(1)
        off = np.abs(dx) * rel + r["P"] * gr * (dD[:, None] + d * EPS * (ado @ np.abs(v).T))
        dq64, tol = scale * dx @ k, scale * off @ np.abs(k)
        assert (np.abs(f64(dq[0, a]) - dq64) <= tol + 2.0 ** -8 * np.abs(dq64)).all()
        want_dk += scale * dx.T @ q
        tol_dk += scale * off.T @ np.abs(q)
    assert (np.abs(f64(dk[0, 0]) - want_dk) <= tol_dk + 2.0 ** -8 * np.abs(want_dk)).all()


@pytest.mark.parametrize("power", [80, -60])
@pytest.mark.parametrize("cap", [12.0, 30.0, 50.0, 56.0, 70.0])
@pytest.mark.parametrize("end", [-1.0, 0.0, 1.0])
def test_values_far_from_one(power, cap, end):
    """Rows at an end of the cap, or near 0, over values of 2^80 and 2^-60: weights are those of the row's largest."""
    b, h, hk, s, d = 1, 2, 1, 384, 64
    x = inputs(b, h, hk, s, d, 9130)
    x["q"] = (x["q"].float() + 60.0 * end).bfloat16()
    x["k"] = (x["k"].float() + 20.0).bfloat16() if end else x["k"]
    x["v"] = (x["v"].float() * 2.0 ** power).bfloat16()
    g = {k: v.cuda() for k, v in x.items()}
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, True, scores=ra.Scores(cap))
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, None, True, None)
    assert_within("out", out, want["out"])
    assert_within("lse", lse, want["lse"])


@pytest.mark.parametrize("form", ["contiguous", "zigzag", "stripe", "packed", "packed zigzag", "step"])
@pytest.mark.parametrize("d,slopes,rows", [(64, None, "third"), (128, None, "one"), (128, "alibi", "third")])
def test_blocks_whose_rows_need_offsets_of_their_own(form, d, slopes, rows):
    """A few rows at the cap's negative end among others near 0, in every form of the forward, over values of 2^70."""
    h, hk, n, cap = 2, 1, 2, 50.0
    lens = [256, 640, 128] if form.startswith("packed") else None
    b, s = (1, 1024) if lens else (2, 640)
    if form == "step" and slopes:
        slopes = None
    x = inputs(b, h, hk, s, d, 9180)
    low = torch.arange(s) % 3 == 0 if rows == "third" else torch.arange(s) == s // 2 + 5
    x["k"] = (x["k"].float() + 8.0).bfloat16()
    x["q"] = (x["q"].float() * 0.1 - 20.0 * low[None, None, :, None]).bfloat16()
    x["v"] = (x["v"].float() * 2.0 ** 70).bfloat16()
    sl = slopes_of(h, slopes)
    z = scores_of(cap, sl, None)
    if lens:
        layout = "zigzag" if "zigzag" in form else "contiguous"
        cu = ra.CuSeqlens([0, *np.cumsum(lens)], "cuda")
        g = {k: ra.ring_attn_varlen_permute(rows_first(v), cu, layout, n, seq_dim=0) for k, v in x.items()}
        out, lse = ra.ring_attn_varlen_fwd(g["q"], g["k"], g["v"], cu, None, n, True, layout=layout, scores=z)

        def back(t):
            t = torch.empty(t.shape, dtype=t.dtype, device="cuda").copy_(t)
            return ra.ring_attn_varlen_unpermute(t, cu, layout, n, seq_dim=0).transpose(0, 1).unsqueeze(0)

        out, lse = back(out), back(lse.t().contiguous().unsqueeze(-1)).squeeze(-1)
        want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, True, None, [0, *np.cumsum(lens)])
    else:
        layout = "contiguous" if form == "step" else form
        shards = 1 if form == "step" else n
        g = {k: to_layout(ra, v.cuda(), layout, shards) for k, v in x.items()}
        if form == "step":
            out, lse = ra.ring_attn_fwd_step(g["q"], g["k"], g["v"], 0, causal=True, scores=z)
        else:
            out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], layout, shards, True, scores=z)
        out, lse = to_original(ra, out, layout, shards), lse_to_original(ra, lse, layout, shards)
        want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, True, None)
    check_no_device_error(ra)
    assert float(want["lse"][0].min()) < -25.0 and float(want["lse"][0].max()) > 0.0
    assert_within("lse", lse, want["lse"])
    assert_within("out", out, want["out"])
