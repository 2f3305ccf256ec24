"""Attention with capped scores, a bias by distance and prefixes: forward and backward of every form that takes
`scores`, against the fp64 oracle with bounds from the kernels' roundings (tests/score_case.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import ring_attn_gb300 as ra
from tests.helpers import check_no_device_error, lse_to_original, to_layout, to_original
from tests.score_case import assert_within, expect
from workload import cu_seqlens, make_qkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_attn_gb300.build import build

    build()
    ra.load()


def inputs(b, h, hk, s, d, seed, gain=1.0):
    x, y = make_qkv(b, h, s, d, seed), make_qkv(b, hk, s, d, seed + 1, with_do=False)
    do = (x["do"].float() * (hk / h) ** 0.5).bfloat16()
    return {"q": (x["q"].float() * gain).bfloat16(), "k": y["k"], "v": y["v"], "do": do}


def slopes_of(h, kind):
    s = {None: None, "alibi": [2.0 ** (-8 * (i + 1) / h) for i in range(h)],
         "mixed": [(0.25, 0.0, -0.01, 1.5)[i % 4] for i in range(h)]}[kind]
    return None if s is None else torch.tensor(s, dtype=torch.float32)


def scores_of(cap, slopes, prefix):
    return ra.Scores(cap, None if slopes is None else slopes.cuda(),
                     None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"))


def rows_first(t):
    """(1, h, total, d) -> (total, h, d) with plain strides."""
    t = t[0].transpose(0, 1)
    return torch.empty(t.shape, dtype=t.dtype, device="cuda").copy_(t)


CASES = [
    # b, h, hk, s, d, layout, n, causal, cap, slopes, prefix, gain
    (1, 2, 2, 256, 64, "contiguous", 1, True, 20.0, None, None, 1.0),
    (1, 2, 2, 300, 128, "contiguous", 2, False, 2.0, None, None, 4.0),        # scores beyond the polynomial
    (2, 4, 2, 390, 64, "contiguous", 3, True, 0.0, "alibi", None, 1.0),
    (1, 4, 1, 520, 64, "zigzag", 2, False, 0.0, "mixed", None, 1.0),          # seams and diagonals inside tiles
    (1, 3, 3, 600, 128, "zigzag", 3, True, 0.0, "alibi", None, 1.0),
    (1, 2, 2, 512, 128, "zigzag", 2, True, 30.0, "alibi", None, 2.0),         # whole tiles left and right of the seam
    (2, 2, 1, 387, 128, "stripe", 3, False, 5.0, "mixed", None, 2.0),
    (1, 2, 2, 640, 64, "stripe", 4, True, 50.0, "alibi", None, 1.0),
    (3, 2, 2, 384, 64, "contiguous", 1, True, 0.0, None, (0, 131, 1000), 1.0),
    (2, 4, 2, 512, 128, "zigzag", 4, True, 0.0, None, (200, 1), 1.0),
    (2, 2, 2, 510, 64, "stripe", 3, True, 10.0, "mixed", (129, -3), 1.0),
    (2, 2, 2, 520, 128, "zigzag", 2, True, 15.0, "mixed", (256, 519), 3.0),
    (1, 1, 1, 1, 64, "contiguous", 1, True, 3.0, "mixed", (1,), 1.0),
    (1, 1, 1, 2, 128, "zigzag", 1, True, 3.0, "mixed", (0,), 1.0),
    (1, 2, 1, 129, 128, "contiguous", 1, False, 0.01, "mixed", None, 1.0),     # a cap far below the scores
    (1, 1, 1, 200, 64, "contiguous", 1, True, 1e6, None, None, 1.0),           # and far above
]


@pytest.mark.parametrize("b,h,hk,s,d,layout,n,causal,cap,slopes,prefix,gain", CASES)
def test_batched(b, h, hk, s, d, layout, n, causal, cap, slopes, prefix, gain):
    x = inputs(b, h, hk, s, d, 9000 + s + h, gain)
    sl = slopes_of(h, slopes)
    z = scores_of(cap, sl, prefix)
    g = {k: to_layout(ra, v.cuda(), layout, n) for k, v in x.items()}
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], layout, n, causal, scores=z)
    grads = ra.ring_attn_bwd(g["do"], g["q"], g["k"], g["v"], out, lse, layout, n, causal, scores=z)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], x["do"], d ** -0.5, cap, sl, causal, prefix)
    assert_within("out", to_original(ra, out, layout, n), want["out"])
    assert_within("lse", lse_to_original(ra, lse, layout, n), want["lse"])
    for name, t in zip(("dq", "dk", "dv"), grads):
        assert_within(name, to_original(ra, t, layout, n), want[name])


@pytest.mark.parametrize("scale,cap,gain", [
    (1e-3, 50.0, 45.0),      # scores up to the cap, of products whose sixth powers times the coefficients leave fp32
    (1e-3, 50.0, 30.0),
    (128 ** -0.5, 1000.0, 17.0),
    (2.0 ** 8, 1.0, 0.25),
    (2.0 ** 20, 2.0 ** 10, 0.008),  # and that leave it upwards
    (1e-30, 50.0, 2.0),      # nothing is left of the scores
])
@pytest.mark.parametrize("causal", [True, False])
def test_scale_far_from_the_cap(scale, cap, gain, causal):
    b, h, hk, s, d = 1, 2, 1, 328, 128
    x = inputs(b, h, hk, s, d, 9050, gain)
    x["k"] = (x["k"].float() * gain).bfloat16()
    g = {k: v.cuda() for k, v in x.items()}
    z = scores_of(cap, None, None)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, causal, scale, scores=z)
    grads = ra.ring_attn_bwd(g["do"], g["q"], g["k"], g["v"], out, lse, "contiguous", 1, causal, scale, scores=z)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], x["do"], scale, cap, None, causal, None)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert_within(name, t, want[name])


@pytest.mark.parametrize("d,causal", [(64, True), (128, False)])
def test_a_cap_far_above_the_scores_leaves_them(d, causal):
    """With softcap 2^20 a score of up to 40 changes by less than 2^-24: lse, which sums fp32 numbers, is the plain call's
    but for the roundings of scores (2^-20 of 40) and of lse itself."""
    x = inputs(1, 2, 2, 520, d, 9070, 2.0)
    q, k, v = (x[n].cuda() for n in "qkv")
    plain, capped = (ra.ring_attn_fwd(q, k, v, "contiguous", 1, causal, scores=z)[1].double().cpu()
                     for z in (None, ra.Scores(2.0 ** 20)))
    check_no_device_error(ra)
    assert float(plain.abs().max()) < 40.0
    assert float(((capped - plain).abs() - 40.0 * 2.0 ** -20 - 2.0 ** -21 * plain.abs()).max()) <= 0


@pytest.mark.parametrize("cap", [25.0, 56.0, 57.0])  # one offset for all rows, up to which cap, and above
@pytest.mark.parametrize("slopes", [None, "alibi"])
def test_rows_at_both_ends_of_the_cap(cap, slopes):
    """Rows whose scores are all at the cap, or all at its negative; with a bias, up to 32 below that."""
    b, h, hk, s, d = 1, 2, 1, 512, 64
    x = inputs(b, h, hk, s, d, 9060)
    sign = torch.where(torch.arange(s) % 3 == 0, -1.0, 1.0)[None, None, :, None]
    x["q"] = (x["q"].float() + 60.0 * sign).bfloat16()
    x["k"] = (x["k"].float() + 20.0).bfloat16()
    sl = slopes_of(h, slopes)
    g = {k: v.cuda() for k, v in x.items()}
    z = scores_of(cap, sl, None)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, True, scores=z)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, True, None)
    assert_within("out", out, want["out"])
    assert_within("lse", lse, want["lse"])


@pytest.mark.parametrize("layout,causal,cap,slopes,prefix", [
    ("contiguous", True, 8.0, "alibi", (150,)), ("zigzag", True, 0.0, "alibi", None), ("stripe", False, 8.0, "mixed", None),
    ("zigzag", True, 0.0, None, (300,)), ("contiguous", True, 8.0, None, None), ("zigzag", True, 80.0, None, (9,)),
])
def test_ring_steps_and_merge(layout, causal, cap, slopes, prefix):
    """Every ring step on its own, merged; steps of a causal ring leave rows without keys."""
    b, h, hk, s, d, n = 1, 2, 1, 544, 64, 4
    x = inputs(b, h, hk, s, d, 9100)
    sl = slopes_of(h, slopes)
    z = scores_of(cap, sl, prefix)
    g = {k: to_layout(ra, v.cuda(), layout, n) for k, v in x.items()}
    acc = torch.zeros((b, h, s, d), device="cuda")
    lacc = torch.full((b, h, s), -np.inf, device="cuda")
    for step in range(n):
        ra.lse_merge(acc, lacc, *ra.ring_attn_fwd_step(g["q"], g["k"], g["v"], step, layout, n, causal, scores=z))
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, causal, prefix)
    assert_within("out", to_original(ra, acc, layout, n), want["out"])
    val, tol = want["lse"]
    assert_within("lse", lse_to_original(ra, lacc, layout, n), (val, tol + n * 2.0 ** -21))  # n merges


@pytest.mark.parametrize("layout,lens,n,ws", [
    ("contiguous", [100, 300, 1, 350, 273], 4, True), ("zigzag", [256, 640, 96, 1056], 4, True),
    ("zigzag", [256, 640, 96, 1056], 4, False),
])
@pytest.mark.parametrize("causal,cap,slopes,with_prefix", [
    (True, 0.0, "alibi", False), (False, 6.0, "mixed", False), (True, 0.0, None, True), (True, 6.0, "mixed", True),
])
def test_packed_documents(layout, lens, n, ws, causal, cap, slopes, with_prefix):
    h, hk, d = 2, 1, 64
    cu = cu_seqlens(lens)
    total = int(cu[-1])
    x = inputs(1, h, hk, total, d, 9200 + len(lens))
    sl = slopes_of(h, slopes)
    prefix = [m * (i % 3) // 2 for i, m in enumerate(lens)] if with_prefix else None  # nothing, half, all of a sequence
    z = scores_of(cap, sl, prefix)
    g = {k: ra.ring_attn_varlen_permute(rows_first(v), cu, layout, n, seq_dim=0) for k, v in x.items()}

    def space(op):
        m = ra.ring_attn_varlen_workspace_size(op, total, h, d, layout if ws else "contiguous", n)
        return torch.empty(m, dtype=torch.uint8, device="cuda")

    out, lse = ra.ring_attn_varlen_fwd(g["q"], g["k"], g["v"], cu, None, n, causal, layout=layout,
                                       workspace=space(ra.RA_OP_FWD), scores=z)
    grads = ra.ring_attn_varlen_bwd(g["do"], g["q"], g["k"], g["v"], out, lse, cu, None, n, causal, layout=layout,
                                    workspace=space(ra.RA_OP_BWD), scores=z)
    check_no_device_error(ra)

    def back(t):
        t = torch.empty(t.shape, dtype=t.dtype, device="cuda").copy_(t)
        return ra.ring_attn_varlen_unpermute(t, cu, layout, n, seq_dim=0).transpose(0, 1).unsqueeze(0)

    want = expect(x["q"], x["k"], x["v"], x["do"], d ** -0.5, cap, sl, causal, prefix, cu)
    assert_within("out", back(out), want["out"])
    assert_within("lse", back(lse.t().contiguous().unsqueeze(-1)).squeeze(-1), want["lse"])
    for name, t in zip(("dq", "dk", "dv"), grads):
        assert_within(name, back(t), want[name])


def test_llama3_ranks():
    """The ranks' rows together, and the sum of their gradients of the keys."""
    lens, n, h, hk, d = [300, 500, 224], 4, 2, 1, 64
    cu = cu_seqlens(lens)
    total = int(cu[-1])
    L = total // n
    x = inputs(1, h, hk, total, d, 9300)
    sl, prefix, cap = slopes_of(h, "alibi"), [120, 400, 0], 12.0
    z = scores_of(cap, sl, prefix)
    g = {k: rows_first(v) for k, v in x.items()}
    got = {k: [] for k in ("out", "lse", "dq", "dk", "dv")}
    for r in range(n):
        rows = slice(r * L, (r + 1) * L)
        q, do = g["q"][rows].contiguous(), g["do"][rows].contiguous()
        out, lse = ra.ring_attn_llama3_varlen_fwd(q, g["k"], g["v"], cu, r, n, scores=z)
        grads = ra.ring_attn_llama3_varlen_bwd(do, q, g["k"], g["v"], out, lse, cu, r, n, scores=z)
        for name, t in zip(got, (out, lse, *grads)):
            got[name].append(t)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], x["do"], d ** -0.5, cap, sl, True, prefix, cu)
    assert_within("out", torch.cat(got["out"]).transpose(0, 1)[None], want["out"])
    assert_within("lse", torch.cat(got["lse"], 1)[None], want["lse"])
    assert_within("dq", torch.cat(got["dq"]).transpose(0, 1)[None], want["dq"])
    for name in ("dk", "dv"):
        parts = [t.float() for t in got[name]]
        val, tol = want[name]
        each = sum(t.abs() for t in parts).transpose(0, 1)[None].double().cpu().numpy()
        assert_within(name, sum(parts).transpose(0, 1)[None], (val, tol + 2.0 ** -8 * each))  # each rank's is rounded


def test_packed_tensors():
    """qkv in one tensor, read and written in place through its strides."""
    b, s, h, d = 2, 260, 2, 64
    x = inputs(b, h, h, s, d, 9400)
    sl, prefix, cap = slopes_of(h, "mixed"), (30, 200), 9.0
    z = scores_of(cap, sl, prefix)
    qkv = torch.stack([x[k].transpose(1, 2) for k in "qkv"], 2).cuda()
    do = x["do"].transpose(1, 2).contiguous().cuda()
    out, lse = ra.ring_attn_qkvpacked_fwd(qkv, causal=True, scores=z)
    dqkv = ra.ring_attn_qkvpacked_bwd(do, qkv, out, lse, causal=True, scores=z)
    out2, lse2 = ra.ring_attn_kvpacked_fwd(qkv[:, :, 0], qkv[:, :, 1:], causal=True, scores=z)
    dq2, dkv2 = ra.ring_attn_kvpacked_bwd(do, qkv[:, :, 0], qkv[:, :, 1:], out, lse, causal=True, scores=z)
    check_no_device_error(ra)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(dqkv[:, :, 0], dq2) and torch.equal(dqkv[:, :, 1:], dkv2)
    want = expect(x["q"], x["k"], x["v"], x["do"], d ** -0.5, cap, sl, True, prefix)
    assert_within("out", out.transpose(1, 2), want["out"])
    assert_within("lse", lse, want["lse"])
    for i, name in enumerate(("dq", "dk", "dv")):
        assert_within(name, dqkv[:, :, i].transpose(1, 2), want[name])


def test_without_changes_the_calls_are_the_plain_ones():
    x = {k: v.cuda() for k, v in inputs(1, 2, 2, 384, 128, 9500).items()}
    plain = ra.ring_attn_fwd(x["q"], x["k"], x["v"], "zigzag", 3, True)
    grads = ra.ring_attn_bwd(x["do"], x["q"], x["k"], x["v"], *plain, "zigzag", 3, True)
    for z in (ra.Scores(), scores_of(0.0, None, (0,)), scores_of(0.0, None, (1,))):  # its own token is seen anyway
        got = ra.ring_attn_fwd(x["q"], x["k"], x["v"], "zigzag", 3, True, scores=z)
        back = ra.ring_attn_bwd(x["do"], x["q"], x["k"], x["v"], *got, "zigzag", 3, True, scores=z)
        assert all(torch.equal(a, b) for a, b in zip((*plain, grads[2]), (*got, back[2])))
        # dq and dk: with a prefix D comes from the products (better than from the rounded out), so other bits
        assert z.prefix is not None or all(torch.equal(a, b) for a, b in zip(grads, back))
    # a prefix of everything is no causal mask
    got = ra.ring_attn_fwd(x["q"], x["k"], x["v"], "zigzag", 3, True, scores=scores_of(0.0, None, (384,)))
    both = ra.ring_attn_fwd(x["q"], x["k"], x["v"], "zigzag", 3, False)
    assert all(torch.equal(a, b) for a, b in zip(got, both))
    check_no_device_error(ra)


def test_infinite_scores_meet_the_cap():
    """Huge and infinite products are scores of +-cap."""
    s, d, cap = 160, 64, 7.0
    x = inputs(1, 1, 1, s, d, 9600)
    q, k, v = (x[n].clone() for n in "qkv")
    q[0, 0, 5] = 1e36
    k[0, 0, 3] = 1e36   # row 5's product with it is infinite, the others' are about 1e36
    k[0, 0, 150] = -1e36
    z = ra.Scores(cap)
    out, lse = ra.ring_attn_fwd(q.cuda(), k.cuda(), v.cuda(), causal=True, scores=z)
    check_no_device_error(ra)
    xs = (q[0, 0].double() @ k[0, 0].double().t()) * d ** -0.5
    y = cap * torch.tanh(xs / cap)
    y = y.masked_fill(torch.ones(s, s).triu(1).bool(), -np.inf)
    ref = torch.softmax(y, -1) @ v[0, 0].double()
    # a huge key's score is +-cap, by its sign; the fp32 sum of 64 products has it unless they cancel to 64 2^-24 of
    # their size, about 2e32
    keep = (xs[:, 3].abs() > 1e34) & ((xs[:, 150].abs() > 1e34) | (torch.arange(s) < 150)) | (torch.arange(s) < 3)
    size = torch.softmax(y, -1) @ v[0, 0].double().abs()
    tol = 2.0 ** -8 * ref.abs() + size * (2.0 ** -8 * 1.01 + 4 * cap * 2.0 ** -21 + 2.0 ** -14) + 1e-6
    err = (out[0, 0].double().cpu() - ref).abs()
    assert int(keep.sum()) > 100 and bool((err <= tol)[keep].all())
    assert bool(torch.isfinite(lse).all())


def test_captured_calls_follow_slopes_and_prefix_and_repeat_their_bits():
    b, h, s, d = 2, 2, 400, 64
    x = {k: v.cuda() for k, v in inputs(b, h, h, s, d, 9700).items()}
    sl = slopes_of(h, "alibi").cuda()
    pre = torch.tensor([10, 300], dtype=torch.int32, device="cuda")
    z = ra.Scores(11.0, sl, pre)
    out, lse = torch.empty_like(x["q"]), torch.empty((b, h, s), device="cuda")
    ws = torch.empty(ra.ring_attn_workspace_size(ra.RA_OP_BWD, b, h, s, d), dtype=torch.uint8, device="cuda")
    grads = [torch.empty_like(x["q"]) for _ in range(3)]

    def step(stream=None):
        ra.ring_attn_fwd(x["q"], x["k"], x["v"], causal=True, out=out, lse=lse, scores=z, stream=stream)
        ra.ring_attn_bwd(x["do"], x["q"], x["k"], x["v"], out, lse, causal=True, dq=grads[0], dk=grads[1], dv=grads[2],
                         workspace=ws, scores=z, stream=stream)

    def bits():
        torch.cuda.synchronize()
        return [t.clone() for t in (out, lse, *grads)]

    step()
    first = bits()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(first, bits()))
    sl.mul_(-0.5)
    pre.copy_(torch.tensor([399, 0], dtype=torch.int32))
    graph.replay()
    changed = bits()
    assert not torch.equal(first[0], changed[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(changed, bits()))
    check_no_device_error(ra)


@pytest.mark.parametrize("d,n", [(64, 3), (128, 400)])
def test_calls_that_follow_one_another_wait_for_one_another(d, n):
    """Kernels are set up while the one before still runs: what that one writes (rotated rows, slopes, prefixes, statistics)
    they read behind it.  The same steps with a wait after each give the same bits."""
    b, h = 2, 2
    x = {k: v.cuda() for k, v in inputs(b, h, h, n, d, 9750).items()}
    angle = torch.rand(4 * n, d // 2, device="cuda") * 6.0
    table = (angle.cos(), angle.sin())
    places = torch.arange(b * n, dtype=torch.int32, device="cuda").view(b, n)

    def steps(wait):
        sl, pre = torch.zeros(h, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
        z, got, q = ra.Scores(9.0, sl, pre), [], x["q"].clone()
        for i in range(12):
            sl.add_(0.02)
            wait()
            pre.add_(n // 12)
            wait()
            q, k = ra.ring_attn_rope(q, x["k"], table, places)
            wait()
            out, lse = ra.ring_attn_fwd(q, k, x["v"], causal=True, scores=z)
            wait()
            dq, dk, dv = ra.ring_attn_bwd(x["do"], q, k, x["v"], out, lse, causal=True, scores=z)
            wait()
            dq, dk = ra.ring_attn_rope_bwd(dq, dk, table, places, dq_out=dq, dk_out=dk)
            wait()
            got += [out, lse, dq, dk, dv]
        return got

    first = steps(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(first, steps(lambda: None)))
    check_no_device_error(ra)


@pytest.mark.parametrize("flag", [1, 2, 4], ids=["fwd", "dkdv", "dq"])
@pytest.mark.parametrize("cap,slopes,d", [(20.0, None, 64), (70.0, None, 128), (0.0, "alibi", 64), (20.0, "alibi", 128)])
def test_a_wait_that_runs_out_is_reported_and_the_context_survives(flag, cap, slopes, d):
    """A load that the others wait for is left out (of Q, of K and V, of Q and dO): their waits end after 2 ms, the halves
    of a row let one another go, and the next call is right."""
    h, s = 2, 512
    x = inputs(1, h, h, s, d, 9800)
    sl = slopes_of(h, slopes)
    z = scores_of(cap, sl, None)
    g = {k: v.cuda() for k, v in x.items()}
    how = dict(layout="contiguous", n_shards=2, causal=True, scores=z)

    def call(out, lse):
        return ra.ring_attn_bwd(g["do"], g["q"], g["k"], g["v"], out, lse, **how)

    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], **how)
    check_no_device_error(ra)
    try:
        ra.ring_attn_set_knob(ra.RA_KNOB_WAIT_LIMIT_NS, 2_000_000)
        ra.ring_attn_set_knob(ra.RA_KNOB_DEBUG_FLAGS, flag)
        if flag == 1:
            ra.ring_attn_fwd(g["q"], g["k"], g["v"], **how)
        else:
            call(out, lse)
        st, info = ra.ring_attn_check_device_error()
    finally:
        ra.ring_attn_set_knob(ra.RA_KNOB_DEBUG_FLAGS, 0)
        ra.ring_attn_set_knob(ra.RA_KNOB_WAIT_LIMIT_NS, int(os.environ.get("RA_TEST_WAIT_LIMIT_NS", 4_000_000_000)))
    assert st == 6, (st, info)
    assert ra.ring_attn_check_device_error() == (0, 0)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], **how)
    grads = call(out, lse)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], x["do"], d ** -0.5, cap, sl, True, None)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert_within(name, t, want[name])


def test_the_sweep_passes_under_the_bounds_checks():
    """The tests above once more, in a child process on the library whose kernels check every tiled copy and row store."""
    from ring_attn_gb300.build import build

    build(debug_bounds=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", __file__,
                        "-k", "not bounds_checks"], env=dict(os.environ, RA_LIB_VARIANT="debug_bounds"),
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, "\n".join(r.stdout.splitlines()[-30:])
