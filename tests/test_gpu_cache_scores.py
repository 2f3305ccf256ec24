"""Attention over the paged 4-bit cache with capped scores, a bias by distance and prefixes, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import ring_attn_gb300 as ra
from oracle import scores as osc
from tests.cache_case import Case, assert_within
from tests.helpers import check_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_attn_gb300.build import build

    build()
    ra.load()


def expect(c, q, causal, cap, slopes, prefix):
    """(out, lse, their bounds): the bounds of Case.expect, and for the changes of a score cap 2^-21
    (exponential, reciprocal, three roundings) and 4 roundings of numbers up to slope * distance or |z|."""
    scale, total = c.d ** -0.5, int(c.cu[-1])
    out, lse = np.zeros((total, c.h, c.d)), np.zeros((c.h, total))
    to, tl = np.zeros_like(out), np.zeros_like(lse)
    qf = q.float().cpu().numpy().astype(np.float64)
    for i, (n, m) in enumerate(zip(c.n_new, c.kv)):
        rows = slice(c.cu[i], c.cu[i + 1])
        gq, gk = np.arange(m - n, m), np.arange(m)
        big = np.abs(c.v[i]).max(initial=0.0)
        for a in range(c.h):
            b, sl = a * c.hk // c.h, 0.0 if slopes is None else float(slopes[a])
            k, v = c.k[i][:, b], c.v[i][:, b]
            r = osc.head(qf[rows, a], k, v, gq, gk, scale, cap, sl, causal, 0 if prefix is None else prefix[i])
            see = np.isfinite(r["z"])
            s_err = (c.d * 2.0 ** -24 * scale * (np.abs(qf[rows, a]) @ np.abs(k).T) + cap * 2.0 ** -21
                     + 2.0 ** -22 * abs(sl) * np.abs(gq[:, None] - gk) + 2.0 ** -22 * np.where(see, np.abs(r["z"]), 0.0))
            e = np.where(see & (r["P"] > 2.0 ** -30), s_err, 0.0).max(1, initial=0.0)
            rel = 2 * e + 2.0 ** -21 + max(m, 1) * 2.0 ** -24
            size = r["P"] @ np.abs(v)
            out[rows, a], lse[a, rows] = r["out"], r["lse"]
            to[rows, a] = 2.0 ** -8 * np.abs(r["out"]) + size * (2.0 ** -11 * 1.01 + rel[:, None]) + max(m, 1) * 2.0 ** -29 * big + 1e-30
            tl[a, rows] = rel + 2.0 ** -21 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0)) + 1e-6
    return out, lse, to, tl


def run(c, causal, cap, slopes, prefix, gain=2.0, **kw):
    cache = c.fill(ra)
    q = c.queries(gain)
    sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32)
    z = ra.Scores(cap, None if sl is None else sl.cuda(),
                  None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"))
    cu = ra.CuSeqlens(c.cu, "cuda")
    out = torch.full((c.rows, c.h, c.d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.h, c.rows), 3.0, device="cuda")
    ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, causal=causal, out=out, lse=lse, scores=z, **kw)
    check_no_device_error(ra)
    total = int(c.cu[-1])
    o, ls, to, tl = expect(c, q, causal, cap, sl, prefix)
    assert_within("out", out[:total], o, to)
    assert_within("lse", lse[:, :total], ls, tl)
    assert bool((out[total:] == 3.0).all()) and bool((lse[:, total:] == 3.0).all())  # padded rows stay
    return q, cache, cu, z, out, lse


def alibi(h):
    return [2.0 ** (-8 * (i + 1) / h) for i in range(h)]


def mixed(h):
    return [(0.25, 0.0, -0.01, 1.5)[i % 4] for i in range(h)]


KINDS = [(8.0, None, None), (0.0, alibi, None), (0.0, None, "some"), (6.0, mixed, "some"), (0.02, alibi, None)]


@pytest.mark.parametrize("cap,slopes,prefix", KINDS)
@pytest.mark.parametrize("n_new,kv,h,hk,d,page", [
    ([1], [1], 4, 1, 64, 16),
    ([1], [4099], 8, 1, 128, 64),                      # split over the keys
    ([1, 1, 1], [300, 17, 1025], 6, 2, 128, 16),
    ([5, 2, 1], [129, 2, 700], 4, 2, 64, 32),          # 16 rows
    ([7, 1, 0, 3], [1500, 40, 9, 3], 8, 2, 64, 128),   # 28 rows, a sequence without new tokens
    ([40, 3], [300, 900], 4, 2, 128, 32),              # the tensor-core kernel: twins
    ([300, 1, 150], [800, 5, 150], 4, 1, 64, 64),      # several tiles
])
def test_against_the_definition(n_new, kv, h, hk, d, page, cap, slopes, prefix):
    c = Case(n_new, kv, h, hk, d, page, seed=sum(kv) + d, pad_rows=3)
    pre = None if prefix is None else [(m * (i + 1)) // 3 if i % 4 < 3 else m + 100 for i, m in enumerate(kv)]
    run(c, True, cap, None if slopes is None else slopes(h), pre)


@pytest.mark.parametrize("n_new,kv,cap,slopes", [([2, 1], [700, 33], 5.0, mixed), ([90, 70], [91, 500], 0.0, mixed)])
def test_both_ways(n_new, kv, cap, slopes):
    """Without causal every token of the sequence is seen, those after the query's own too."""
    run(Case(n_new, kv, 4, 2, 64, 32, seed=3), False, cap, slopes(4), None)


def test_prefixes_of_any_kind_and_rows_before_the_cache():
    """Prefixes below 0, within the new tokens, beyond the sequence; new tokens whose index is negative see the
    prefix if there is one, else nothing."""
    c = Case([40, 40, 40, 40], [200, 200, 200, 40], 4, 2, 64, 16, seed=8)
    run(c, True, 0.0, None, [-5, 170, 100000, 1])
    c = Case([4, 3], [2, 2], 4, 2, 64, 16, seed=9)
    run(c, True, 4.0, alibi(4), [0, 1])


def test_plain_when_nothing_changes():
    for n_new in ([1, 1], [50, 20]):
        c = Case(n_new, [500, 260], 4, 2, 128, 32, seed=4)
        cache, q, cu = c.fill(ra), c.queries(), ra.CuSeqlens(c.cu, "cuda")
        a = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu)
        for z in (ra.Scores(), ra.Scores(prefix=torch.zeros(2, dtype=torch.int32, device="cuda"))):
            b = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, scores=z)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_steps_follow_lengths_slopes_and_prefix():
    """Two captured graphs that share a workspace, replayed in turn; a replay follows the arrays."""
    c = Case([1, 1], [900, 900], 4, 2, 64, 32, seed=6)
    cache, q, cu = c.fill(ra), c.queries(), ra.CuSeqlens(c.cu, "cuda")
    sl = torch.tensor(alibi(4), device="cuda")
    pre = torch.tensor([5, 800], dtype=torch.int32, device="cuda")
    z = ra.Scores(7.0, sl, pre)
    ws = ra.ring_attn_cache_workspace(q, cache, cu)

    def call(scores):
        return ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, workspace=ws, scores=scores)

    call(z)
    graphs, outs = [], []
    for s in (z, ra.Scores(3.0)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(s))
        graphs.append(g)
    c.kv_lens.copy_(torch.tensor([333, 70], dtype=torch.int32))
    c.kv = [333, 70]
    c.k, c.v = [k[:m] for k, m in zip(c.k, c.kv)], [v[:m] for v, m in zip(c.v, c.kv)]
    sl.mul_(2.0)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    check_no_device_error(ra)
    for (out, lse), cap, slopes, prefix in zip(outs, (7.0, 3.0), (sl.cpu(), None), ([5, 800], None)):
        o, ls, to, tl = expect(c, q, True, cap, slopes, prefix)
        assert_within("out", out, o, to)
        assert_within("lse", lse, ls, tl)


def test_a_prompt_and_its_next_token():
    """Training-side and cached attention of one sequence agree on rotated, capped and biased scores: a prompt goes
    through rotation, the cache and attention, then a token more."""
    n, h, hk, d = 150, 4, 2, 64
    g = torch.Generator().manual_seed(21)
    q, k, v = (torch.randn(n + 1, m, d, generator=g).bfloat16().cuda() for m in (h, hk, hk))
    angle = torch.arange(n + 1, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(d // 2) * 2.0 / d)
    rope = angle.cos().float().cuda(), angle.sin().float().cuda()
    z = ra.Scores(9.0, torch.tensor(alibi(h), device="cuda"))
    pos = torch.stack([torch.arange(n + 1), torch.arange(n + 1) // 7]).to(torch.int32).cuda()
    axes = [0] * 20 + [1] * 12
    qr, kr = ra.ring_attn_rope(q, k, rope, pos, axes)
    cache = ra.KVCache.empty(4, 64, hk, d)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ra.ring_attn_cache_append(kr[:n], v[:n], cache, table, lens, [0, n])
    out, lse = ra.ring_attn_cache_fwd(qr[:n].contiguous(), cache, table, lens, [0, n], scores=z)
    lens += 1
    ra.ring_attn_cache_append(kr[n:], v[n:], cache, table, lens, [0, 1])
    one, one_lse = ra.ring_attn_cache_fwd(qr[n:].contiguous(), cache, table, lens, [0, 1], scores=z)
    kc, vc = ra.ring_attn_cache_read(cache, table, lens, [0, n + 1])
    ref, ref_lse = ra.ring_attn_varlen_fwd(qr, kc, vc, [0, n + 1], scores=z)
    check_no_device_error(ra)
    got, got_lse = torch.cat([out, one]).float(), torch.cat([lse, one_lse], 1)
    # both round their weights (2^-11 and 2^-8) and their result (2^-8 each); weights sum to 1 and |v| is at most vmax
    vmax = float(vc.float().abs().max())
    assert float((got - ref.float()).abs().max()) <= (3 * 2.0 ** -8 + 2.0 ** -11 + 1e-4) * vmax
    assert float((got_lse - ref_lse).abs().max()) <= 1e-4


@pytest.mark.parametrize("n_new", [1, 5, 200])  # few rows, and the tensor cores' kernel
@pytest.mark.parametrize("cap", [200.0, 1000.0, 2.0 ** 20])
def test_a_cap_far_above_the_scores_leaves_them(n_new, cap):
    """x - softcap tanh(x / softcap) <= |x|^3 / (3 softcap^2): with scores below 40, 0.54, 0.022 and nothing; lse sums fp32
    numbers, so it shows what the cap's evaluation adds: |x| 2^-20 for the scores, 2^-21 |lse| for lse."""
    c = Case((n_new, n_new), (900, 333), 4, 2, 64, 32, seed=77)
    cache, q, cu = c.fill(ra), c.queries(2.0), ra.CuSeqlens(c.cu, "cuda")
    total = int(c.cu[-1])
    plain, capped = (ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, scores=z)[1][:, :total].double().cpu()
                     for z in (None, ra.Scores(cap)))
    check_no_device_error(ra)
    assert float(plain.abs().max()) < 40.0
    change = (40.0 ** 3 / (3 * cap ** 2)) if cap < 2.0 ** 20 else 0.0
    over = (capped - plain).abs() - (change + 40.0 * 2.0 ** -20 + 2.0 ** -21 * plain.abs())
    assert float(over.max()) <= 0
