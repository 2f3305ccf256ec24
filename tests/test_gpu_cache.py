"""The paged 4-bit cache on the GPU against the fp64 oracle: the stored bits are
equal, read values are equal, attention is within a bound derived from the
roundings (tests/cache_case.py)."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_case import Case, assert_within
from tests.helpers import check_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import ring_attn_gb300
    from ring_attn_gb300.build import build

    build()
    ring_attn_gb300.load()
    return ring_attn_gb300


def f64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def tables(positions, rot, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / rot)
    t = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    return t(np.cos(a)), t(np.sin(a))


APPEND = [
    # n_new, kv, h, hk, d, page, rot, interleaved, order
    ((1,), (1,), 4, 2, 128, 16, 128, False, (0, 1, 2)),
    ((1,), (1000,), 32, 8, 128, 64, 128, False, (0, 1, 2)),
    ((1, 1, 1, 1, 1), (1, 17, 256, 300, 33), 8, 8, 64, 32, 64, True, (0, 1, 2)),
    ((37, 0, 1, 130), (37, 5, 64, 200), 6, 3, 128, 16, 64, False, (0, 2, 1)),
    ((70, 3), (71, 1030), 5, 1, 64, 256, 32, True, (1, 0, 2)),
    ((70, 3), (71, 1030), 14, 2, 128, 128, 16, False, (2, 1, 0)),
    ((600,), (613,), 2, 2, 64, 64, 32, False, (0, 2, 1)),
    ((9, 20), (9, 33), 3, 3, 128, 32, 96, False, (0, 1, 2)),
    ((9, 20), (9, 33), 10, 5, 128, 32, 16, True, (0, 1, 2)),
    ((12,), (12,), 5, 5, 64, 16, 64, False, (0, 1, 2)),
]


@pytest.mark.parametrize("n_new,kv,h,hk,d,page,rot,inter,order", APPEND)
def test_append_stores_the_nearest_numbers(ra, n_new, kv, h, hk, d, page, rot, inter, order):
    c = Case(n_new, kv, h, hk, d, page, seed=1 + d + rot, order=order, pad_rows=3)
    cache = c.cache(ra)
    # one packed (rows, h + 2 hk, d) tensor, as a projection gives it
    x = torch.tensor(c.rng.standard_normal((c.rows, h + 2 * hk, d))).bfloat16().cuda()
    x[:, h] *= 1e-3  # small groups: the least scale
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
    cos, sin = tables(max(kv), rot)
    q_out = torch.full((c.rows, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = ra.ring_attn_cache_append(k, v, cache, c.page_table, c.kv_lens, c.cu.tolist(), q=q, rope=(cos, sin),
                                    interleaved=inter, q_out=q_out)
    assert got is q_out
    check_no_device_error(ra)
    host = [b.cpu().numpy() for b in c.bytes]
    owned = np.zeros((c.n_pages, page), bool)
    for i, (n, m) in enumerate(zip(n_new, kv)):
        r = slice(c.cu[i], c.cu[i + 1])
        pos = np.arange(m - n, m)
        cs, sn = cos.cpu().numpy()[pos], sin.cpu().numpy()[pos]
        pg, row = c.where(i, m - n, m)
        owned[pg, row] = True
        for j, want in ((0, oc.rotate(f64(k)[r], cs, sn, inter)), (2, f64(v)[r])):
            codes, scales = oc.quantise(want)
            assert np.array_equal(host[j + 1][pg, :, row], scales)
            assert np.array_equal(host[j][pg, :, row], codes)
        # fp32 rotation (two products and a sum: 3 half steps of the larger terms), then bf16
        ref = oc.rotate(f64(q)[r], cs, sn, inter)
        assert_within("q_out", q_out[r], ref, 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -24 * 8.0)
    assert bool((q_out[c.cu[-1]:] == 7.0).all())  # rows behind the last sequence
    for b in host:  # nothing else was written
        assert (np.moveaxis(b, 1, 2)[~owned] == 0xff).all()


def test_append_positions_in_place_and_padding(ra):
    """Explicit positions; q rotated in place; tokens before the cache's start are padding."""
    c = Case((4, 6, 2), (50, 3, 2), 4, 2, 64, 16, seed=5)
    cache = c.cache(ra)
    q, k, v = c.queries(), *(torch.tensor(c.rng.standard_normal((c.rows, 2, 64))).bfloat16().cuda() for _ in range(2))
    before = q.clone()
    cos, sin = tables(1000, 64)
    pos = torch.tensor(c.rng.integers(0, 1000, c.rows), dtype=torch.int32, device="cuda")
    out = ra.ring_attn_cache_append(k, v, cache, c.page_table, c.kv_lens, c.cu.tolist(), q=q, rope=(cos, sin),
                                    positions=pos, q_out=q)
    assert out is q
    check_no_device_error(ra)
    host = [b.cpu().numpy() for b in c.bytes]
    p = pos.cpu().numpy()
    cs, sn = cos.cpu().numpy()[p], sin.cpu().numpy()[p]
    ref_q, ref_k = oc.rotate(f64(before), cs, sn, False), oc.rotate(f64(k), cs, sn, False)
    written = np.ones(c.rows, bool)
    written[4:7] = False  # sequence 1 has 6 new tokens and 3 places
    assert_within("q", q[torch.tensor(written)], ref_q[written], (2.0 ** -8 * np.abs(ref_q) + 2e-6)[written])
    assert torch.equal(q[4:7], before[4:7])
    for i, lo, hi, r in ((0, 46, 50, slice(0, 4)), (1, 0, 3, slice(7, 10)), (2, 0, 2, slice(10, 12))):
        pg, row = c.where(i, lo, hi)
        for j, x in ((0, ref_k), (2, f64(v))):
            codes, scales = oc.quantise(x[r])
            assert np.array_equal(host[j][pg, :, row], codes) and np.array_equal(host[j + 1][pg, :, row], scales)


def test_negative_lengths_are_empty_sequences(ra):
    """Also one so low that a token's index would not fit 32 bits: nothing is written, read or seen."""
    c = Case((3, 40, 2), (-2 ** 31, -2 ** 31 + 7, 2), 2, 1, 64, 16, seed=3, spare=4)
    cache = c.cache(ra)
    before = [b.clone() for b in c.bytes]
    x = c.queries()
    cu = ra.CuSeqlens(c.cu, "cuda")
    qo = torch.full_like(x, 5.0)
    ra.ring_attn_cache_append(x[:, :1], x[:, 1:], cache, c.page_table, c.kv_lens, cu, q=x, q_out=qo, rope=tables(64, 64))
    ko, vo = (torch.full((c.rows, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, cu, k_out=ko, v_out=vo)
    for seqs in (1, 2):  # few and many rows
        out, lse = ra.ring_attn_cache_fwd(x[:c.cu[seqs]], cache, c.page_table[:seqs], c.kv_lens[:seqs], c.cu[:seqs + 1].tolist())
        assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    check_no_device_error(ra)
    assert bool((qo[:43] == 5.0).all()) and bool((ko[:43] == 5.0).all()) and bool((vo[:43] == 5.0).all())
    pg, row = c.where(2, 0, 2)
    for b, a in zip(before, c.bytes):
        changed = (a != b).any(-1).nonzero().cpu().numpy()  # only the third sequence's two tokens
        assert {(p, r) for p, _, r in changed.tolist()} <= set(zip(pg.tolist(), row.tolist()))


def test_append_ties_and_extremes(ra):
    """Values on the format's borders go to the even number; infinities and NaN are stored as finite numbers."""
    d, hk = 64, 1
    c = Case((40,), (40,), 1, hk, d, 16, seed=6)
    cache = c.cache(ra)
    x = np.zeros((40, 1, d))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for t in range(32):
        s = oc.E4M3[40 + 2 * t]  # 6 s is the group's maximum, so s is its scale
        x[t, 0] = np.tile(np.concatenate([[6 * s, 0.0], mids * s, -mids * s]), 4)
    # maxima halfway between two scales
    for t in range(32, 40):
        i = 20 + 3 * (t - 32)
        x[t, 0, ::16] = 6 * (oc.E4M3[i] + oc.E4M3[i + 1]) / 2
    v = torch.tensor(x).bfloat16()
    assert np.array_equal(f64(v), x)
    k = v.clone()
    k[3, 0, 5], k[4, 0, 20], k[5, 0, 40] = float("inf"), float("-inf"), float("nan")
    ra.ring_attn_cache_append(k.cuda(), v.cuda(), cache, c.page_table, c.kv_lens, c.cu.tolist())
    pg, row = c.where(0, 0, 40)
    host = [b.cpu().numpy() for b in c.bytes]
    codes, scales = oc.quantise(x)
    assert np.array_equal(host[2][pg, :, row], codes) and np.array_equal(host[3][pg, :, row], scales)
    kk, _ = ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, c.cu.tolist())
    assert bool(torch.isfinite(kk).all())
    assert kk[3, 0, 5].item() == 2688.0 and kk[4, 0, 20].item() == -2688.0
    check_no_device_error(ra)


@pytest.mark.parametrize("n_new,kv,hk,d,page,order", [
    ((1,), (1,), 1, 64, 16, (0, 1, 2)), ((1001,), (1001,), 8, 128, 64, (0, 1, 2)),
    ((5, 0, 90, 33), (70, 4, 90, 1000), 3, 64, 32, (2, 0, 1)), ((257, 1), (257, 40), 5, 128, 256, (0, 2, 1)),
])
def test_read_gives_the_stored_values(ra, n_new, kv, hk, d, page, order):
    c = Case(n_new, kv, hk, hk, d, page, seed=3, order=order)
    cache = c.fill(ra)
    # outputs inside larger tensors, with rows behind the last one
    kv_out = torch.full((c.rows + 2, 2, hk, d), 5.0, dtype=torch.bfloat16, device="cuda")
    ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, c.cu.tolist(), k_out=kv_out[:, 0], v_out=kv_out[:, 1])
    check_no_device_error(ra)
    for i, (n, m) in enumerate(zip(n_new, kv)):
        r = slice(c.cu[i], c.cu[i + 1])
        assert np.array_equal(f64(kv_out[r, 0]), c.k[i][m - n:]) and np.array_equal(f64(kv_out[r, 1]), c.v[i][m - n:])
    assert bool((kv_out[c.cu[-1]:] == 5.0).all())


ATTEND = [
    # n_new, kv, h, hk, d, page, causal, order
    ((1,), (1,), 4, 2, 128, 16, True, (0, 1, 2)),
    ((1,), (1000,), 32, 8, 128, 16, True, (0, 1, 2)),
    ((1,), (20011,), 8, 1, 128, 64, True, (0, 1, 2)),
    ((1,) * 9, (1, 31, 32, 33, 127, 128, 129, 255, 4097), 6, 2, 64, 32, True, (0, 2, 1)),
    ((1, 0, 1, 1), (0, 9, 700, 64), 5, 5, 64, 16, True, (0, 1, 2)),        # an empty sequence, one without a query
    ((5, 3, 1, 7), (5, 2000, 90, 4), 8, 1, 64, 128, True, (1, 2, 0)),      # rows before the cache's start
    ((4, 2), (333, 64), 7, 1, 128, 256, False, (0, 1, 2)),
    ((2, 2, 2), (515, 130, 17), 16, 1, 128, 16, True, (0, 1, 2)),
    ((20, 9), (700, 9), 12, 2, 128, 64, True, (0, 1, 2)),
    ((40,), (3000,), 16, 4, 64, 64, True, (0, 1, 2)),
    ((129, 300, 1), (700, 301, 2100), 8, 2, 128, 32, True, (0, 2, 1)),
    ((300, 77), (1500, 401), 3, 3, 64, 64, False, (0, 1, 2)),
    ((513,), (513,), 9, 1, 128, 128, True, (0, 1, 2)),
    ((150,), (100,), 4, 2, 64, 16, True, (0, 1, 2)),                       # 50 rows see nothing
]


@pytest.mark.parametrize("n_new,kv,h,hk,d,page,causal,order", ATTEND)
def test_attention_over_the_cache(ra, n_new, kv, h, hk, d, page, causal, order):
    c = Case(n_new, kv, h, hk, d, page, seed=11 + h + page, order=order, pad_rows=2)
    cache = c.fill(ra)
    q = c.queries()
    total = int(c.cu[-1])
    out = torch.full((c.rows, h, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.rows, h), 4.0, device="cuda").t()
    ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist(), causal=causal, out=out, lse=lse)
    check_no_device_error(ra)
    ref, ref_l, tol, tol_l = c.expect(q, causal)
    assert_within("lse", lse[:, :total], ref_l, tol_l)
    assert_within("out", out[:total], ref, tol)
    assert bool((out[total:] == 3.0).all()) and bool((lse[:, total:] == 4.0).all())
    # fp32 output, a length bound, a scale of its own
    o32, l32 = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist(), causal=causal, out_dtype=torch.float32,
                                      max_kv_len=max(max(kv), 1), softmax_scale=0.03)
    ref, ref_l, tol, tol_l = c.expect(q, causal, scale=0.03)
    assert_within("lse", l32[:, :total], ref_l, tol_l)
    assert_within("out", o32[:total], ref, tol)


@pytest.mark.parametrize("seqs,lo,hi,new,h,hk,d,page", [
    (60, 1, 400, 1, 16, 8, 64, 32),      # many short items: a block works on several, runs begin and end inside them
    (60, 1, 3000, 1, 12, 4, 128, 64),
    (23, 100, 1500, 3, 16, 8, 64, 16),
    (40, 1, 700, 4, 16, 4, 128, 16),     # 16 rows an item
    (30, 5, 2500, 5, 24, 6, 64, 64),     # 20 rows
    (160, 1, 90, 1, 2, 1, 128, 16),      # more sequences than a block has threads
    (3, 3000, 9000, 1, 8, 8, 128, 64),   # few long items, cut into pieces
    (2, 2100, 4200, 2, 8, 2, 64, 32),
    (1, 30000, 30000, 1, 6, 3, 64, 128),
    (20, 30, 2000, 90, 8, 2, 64, 32),    # many row tiles, tensor-core kernel
    (150, 1, 300, 40, 4, 2, 64, 16),
])
def test_attention_over_many_ragged_sequences(ra, seqs, lo, hi, new, h, hk, d, page):
    """How the work line is cut: every run of items, pieces and turns has to give the same rows."""
    g = np.random.default_rng(seqs + hi)
    kv = np.exp(g.uniform(np.log(lo), np.log(hi), seqs)).astype(int).tolist()
    n_new = g.integers(0 if seqs > 2 else new, new + 1, seqs).tolist()
    n_new[0] = new
    c = Case(n_new, kv, h, hk, d, page, seed=seqs)
    cache = c.fill(ra)
    q = c.queries()
    out, lse = torch.full((c.rows, h, d), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((h, c.rows), float("nan"), device="cuda")
    ws = ra.ring_attn_cache_workspace(q, cache, ra.CuSeqlens(c.cu, "cuda")).fill_(0xff)
    ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist(), out=out, lse=lse, workspace=ws)
    check_no_device_error(ra)
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("lse", lse, ref_l, tol_l)
    assert_within("out", out, ref, tol)


@pytest.mark.parametrize("h,hk,new", [(4, 1, 1), (8, 2, 60)])
def test_attention_with_large_and_small_queries(ra, h, hk, new):
    """Scores far apart (one key takes all), queries beyond fp16's range, all-zero queries."""
    c = Case((new, new), (900, 310), h, hk, 128, 32, seed=2)
    cache = c.fill(ra)
    q = c.queries()
    q[0] *= 1e30
    q[1] *= 1e-30
    q[new] = 0
    out, lse = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist(), softmax_scale=1.0)
    check_no_device_error(ra)
    keep = np.ones(c.rows, bool)
    keep[0] = False  # 1e30: exp of differences of 1e30; only that nothing breaks
    ref, ref_l, tol, tol_l = c.expect(q, True, scale=1.0)
    assert_within("lse", lse[:, torch.tensor(keep)], ref_l[:, keep], tol_l[:, keep])
    assert_within("out", out[torch.tensor(keep)], ref[keep], tol[keep])
    assert bool(torch.isfinite(out).all())


def test_a_step_of_a_server(ra):
    """Prompt: the varlen forward and the append; then tokens are appended and attend; the cache
    read back and given to the varlen forward agrees; two half caches merge to the whole."""
    h, hk, d, page = 8, 2, 64, 16
    c = Case((100, 33), (100, 33), h, hk, d, page, seed=8, spare=8)
    # pages for the tokens to come
    c.table = np.concatenate([c.table, np.full((2, 2), -7, np.int32)], 1)
    free = [p for p in range(c.n_pages) if p not in c.table]
    c.table[0, 7:9], c.table[1, 3:5] = free[:2], free[2:4]
    c.page_table = torch.tensor(c.table, device="cuda")
    cache = c.cache(ra)
    cos, sin = tables(256, d)
    q, k, v = c.queries(), *(torch.tensor(c.rng.standard_normal((133, hk, d))).bfloat16().cuda() for _ in range(2))
    cu = ra.CuSeqlens(c.cu, "cuda")
    qr = ra.ring_attn_cache_append(k, v, cache, c.page_table, c.kv_lens, cu, q=q, rope=(cos, sin))
    kq, vq = ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, cu)
    a, la = ra.ring_attn_cache_fwd(qr, cache, c.page_table, c.kv_lens, cu)
    b, lb = ra.ring_attn_varlen_fwd(qr, kq, vq, cu)  # the same keys and values, through the ring forward
    # each is within its own bound of the exact result; the ring forward rounds p to bf16 (2^-8) and out (2^-8)
    assert (a.float() - b.float()).abs().max().item() < 2.0 ** -5
    assert (la - lb).abs().max().item() < 1e-4
    steps = ra.CuSeqlens([0, 1, 2], "cuda")
    c.k = [f64(kq)[:100], f64(kq)[100:]]
    c.v = [f64(vq)[:100], f64(vq)[100:]]
    for n in range(3):
        c.kv_lens += 1
        x = torch.tensor(c.rng.standard_normal((2, h + 2 * hk, d))).bfloat16().cuda()
        qn = ra.ring_attn_cache_append(x[:, h:h + hk], x[:, h + hk:], cache, c.page_table, c.kv_lens, steps, q=x[:, :h],
                                       rope=(cos, sin))
        out, lse = ra.ring_attn_cache_fwd(qn, cache, c.page_table, c.kv_lens, steps)
        p = np.array([100 + n, 33 + n])
        cs, sn = cos.cpu().numpy()[p], sin.cpu().numpy()[p]
        kn = oc.dequantise(*oc.quantise(oc.rotate(f64(x[:, h:h + hk]), cs, sn, False)))
        vn = oc.dequantise(*oc.quantise(f64(x[:, h + hk:])))
        c.k = [np.concatenate([c.k[i], kn[i:i + 1]]) for i in range(2)]
        c.v = [np.concatenate([c.v[i], vn[i:i + 1]]) for i in range(2)]
        c.n_new, c.kv, c.cu = [1, 1], [101 + n, 34 + n], np.array([0, 1, 2])
        ref, ref_l, tol, tol_l = c.expect(qn, True)
        assert_within("out", out, ref, tol)
        assert_within("lse", lse, ref_l, tol_l)
    # the same tokens as two caches: pages [0, 2) and the rest, not causal, merged
    acc, l_acc = ra.ring_attn_cache_fwd(qn, cache, c.page_table[:, :2].contiguous(), c.kv_lens.clamp(max=32), steps,
                                        causal=False, out_dtype=torch.float32)
    blk, l_blk = ra.ring_attn_cache_fwd(qn, cache, c.page_table[:, 2:], c.kv_lens - 32, steps, causal=False)
    l_acc = l_acc.contiguous()
    ra.lse_merge(acc.transpose(0, 1), l_acc, blk.transpose(0, 1), l_blk)
    assert_within("merged lse", l_acc, ref_l, 2 * tol_l + 1e-6)
    assert_within("merged out", acc, ref, 2 * tol)
    check_no_device_error(ra)


def test_captured_step_follows_lengths_and_pages(ra):
    """A decoding step captured once and replayed with other lengths, pages and inputs, on a stream of its own."""
    h, hk, d, page = 8, 2, 128, 16
    c = Case((1, 1, 1), (600, 31, 200), h, hk, d, page, seed=9)
    cache = c.fill(ra)
    cos, sin = tables(700, d)
    x = torch.zeros(3, h + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    lens, table = torch.ones(3, dtype=torch.int32, device="cuda"), c.page_table.clone()
    cu = ra.CuSeqlens([0, 1, 2, 3], "cuda")
    out, lse = torch.empty(3, h, d, dtype=torch.bfloat16, device="cuda"), torch.empty(h, 3, device="cuda")
    ws = ra.ring_attn_cache_workspace(x[:, :h], cache, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream):
        ra.ring_attn_cache_append(x[:, h:h + hk], x[:, h + hk:], cache, table, lens, cu, q=x[:, :h], rope=(cos, sin),
                                  q_out=x[:, :h], stream=stream)
        ra.ring_attn_cache_fwd(x[:, :h], cache, table, lens, cu, out=out, lse=lse, workspace=ws, stream=stream)

    step(side)  # puts a token of zeros at index 0 of every sequence
    side.synchronize()
    for i in range(3):
        c.k[i][0] = c.v[i][0] = 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(side)
    for kv in ((600, 31, 200), (1, 30, 199), (577, 5, 16)):
        y = torch.tensor(c.rng.standard_normal((3, h + 2 * hk, d))).bfloat16().cuda()
        x.copy_(y)
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        p = np.array(kv) - 1
        cs, sn = cos.cpu().numpy()[p], sin.cpu().numpy()[p]
        kn = oc.dequantise(*oc.quantise(oc.rotate(f64(y[:, h:h + hk]), cs, sn, False)))
        vn = oc.dequantise(*oc.quantise(f64(y[:, h + hk:])))
        e = Case((1, 1, 1), kv, h, hk, d, page)
        for i, m in enumerate(kv):
            c.k[i][m - 1], c.v[i][m - 1] = kn[i], vn[i]
        e.k, e.v = [c.k[i][:m] for i, m in enumerate(kv)], [c.v[i][:m] for i, m in enumerate(kv)]
        ref, ref_l, tol, tol_l = e.expect(x[:, :h], True)
        assert_within("out", out, ref, tol)
        assert_within("lse", lse, ref_l, tol_l)
    check_no_device_error(ra)


@pytest.mark.parametrize("new", [1, 90])
def test_same_bits_again(ra, new):
    c = Case((new,) * 5, (4000, 90, 1203, 333, 2222), 8, 2, 128, 64, seed=4)
    cache = c.fill(ra)
    q = c.queries()
    a, la = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist())
    for _ in range(3):
        b, lb = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist())
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("new", [1, 70])
def test_bad_pages_lengths_and_positions_are_reported(ra, new):
    """Checked in the kernels: never used, reported, and other sequences are right."""
    c = Case((new, new), (200, 150), 4, 2, 64, 16, seed=7)
    cache = c.fill(ra)
    q = c.queries()
    ref, ref_l, tol, tol_l = c.expect(q, True)
    bad = c.page_table.clone()
    for value in (c.n_pages, -1, 2 ** 31 - 1):
        bad[0, 3] = value
        out, lse = ra.ring_attn_cache_fwd(q, cache, bad, c.kv_lens, c.cu.tolist())
        st, info = ra.ring_attn_check_device_error()
        assert st == 7 and info & 0xff == 0x62
        assert_within("out", out[new:], ref[new:], tol[new:])
    long = c.kv_lens.clone()
    long[0] = 100000
    out, lse = ra.ring_attn_cache_fwd(q, cache, c.page_table, long, c.cu.tolist())
    st, info = ra.ring_attn_check_device_error()
    assert st == 7 and info & 0xff in (0x61, 0x62)
    assert_within("out", out[new:], ref[new:], tol[new:])
    k = torch.zeros(c.rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = [b.clone() for b in c.bytes]
    # (tokens of sequence 1 are placed in sequence 0's table row below: use one bad row for both)
    ra.ring_attn_cache_append(k, k, cache, torch.full_like(c.page_table, c.n_pages), c.kv_lens, c.cu.tolist())
    assert ra.ring_attn_check_device_error()[1] & 0xff == 0x62
    ra.ring_attn_cache_append(k, k, cache, c.page_table, c.kv_lens, c.cu.tolist(), rope=tables(10, 64),
                              positions=torch.full((c.rows,), 10, dtype=torch.int32, device="cuda"))
    assert ra.ring_attn_check_device_error()[1] & 0xff == 0x63
    for b, a in zip(before, c.bytes):
        assert torch.equal(a, b)
    kk = torch.full((c.rows, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    ra.ring_attn_cache_read(cache, torch.full_like(c.page_table, -1), c.kv_lens, c.cu.tolist(), k_out=kk, v_out=kk.clone())
    assert ra.ring_attn_check_device_error()[0] == 7 and bool((kk == 9.0).all())
    check_no_device_error(ra)


@pytest.mark.parametrize("new", [1, 70])
def test_graphs_share_a_workspace(ra, new):
    """Two calls captured with one workspace, replayed behind one another without a wait; and
    two streams at once, each with a workspace of its own."""
    calls = []
    for seed, kv in ((31, (9000, 300)), (32, (77, 5001))):
        c = Case((new, new), kv, 8, 2, 128, 32, seed=seed)
        cache = c.fill(ra)
        q = c.queries()
        calls.append((c, cache, q, ra.CuSeqlens(c.cu, "cuda"), torch.empty_like(q), torch.empty(8, c.rows, device="cuda"),
                      c.expect(q, True)))

    def run(x, ws):
        c, cache, q, cu, out, lse, _ = x
        ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, out=out, lse=lse, workspace=ws)

    def check():
        torch.cuda.synchronize()
        for c, _, _, _, out, lse, (ref, ref_l, tol, tol_l) in calls:
            assert_within("lse", lse, ref_l, tol_l)
            assert_within("out", out, ref, tol)
            out.fill_(9.0)
            lse.fill_(9.0)
        torch.cuda.synchronize()

    one = ra.ring_attn_cache_workspace(calls[0][2], calls[0][1], calls[0][3])
    two = torch.empty_like(one)
    graphs = []
    for x in calls:
        run(x, one)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(x, one)
        graphs.append(g)
    check()
    for _ in range(20):
        for g in graphs:
            g.replay()
    check()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for x, ws, st in zip(calls, (one, two), streams):
            with torch.cuda.stream(st):
                run(x, ws)
    check()
    check_no_device_error(ra)


def test_binding_refusals(ra):
    """What only the binding can see; the library's refusals come up as errors, too."""
    c = Case((1, 2), (5, 9), 4, 2, 64, 16, seed=6)
    cache, q, cu = c.fill(ra), c.queries(), ra.CuSeqlens(c.cu, "cuda")
    n = ra.ring_attn_cache_workspace(q, cache, cu).numel()

    def fwd(q=q, cache=cache, page_table=c.page_table, kv_lens=c.kv_lens, cu=cu, **k):
        return ra.ring_attn_cache_fwd(q, cache, page_table, kv_lens, cu, **k)

    for bad in (dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)),  # fewer bytes than it says
                dict(q=q.half()), dict(q=q[0]), dict(q=q.cpu()), dict(kv_lens=c.kv_lens.long()), dict(kv_lens=c.kv_lens[:1]),
                dict(page_table=c.page_table[:1]), dict(kv_lens=c.kv_lens.cpu()), dict(max_kv_len=-1), dict(out=q.cpu()), dict(out_dtype=torch.float16),
                dict(cache=c.bytes)):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in (dict(workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda")), dict(q=q[:2]), dict(q=q[:, :3]),
                dict(q=q.float()), dict(softmax_scale=-1.0), dict(out=torch.empty_like(q[:, :2]))):
        with pytest.raises(RuntimeError):
            fwd(**bad)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    app = lambda **k: ra.ring_attn_cache_append(x, x, cache, c.page_table, c.kv_lens, cu, **k)  # noqa: E731
    cos, sin = tables(16, 64)
    for bad in (dict(q_out=q), dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(q=q, rope=(cos, sin.cpu())),
                dict(q=q, positions=c.kv_lens.float())):
        with pytest.raises(ValueError):
            app(**bad)
    for bad in (dict(q=q, rope=(cos, sin[:, :16])), dict(q=q, rope=(cos[:, ::2], sin[:, ::2])), dict(q=q, q_out=q.flip(0)[:2])):
        with pytest.raises(RuntimeError):
            app(**bad)
    out, _ = fwd()
    ref, _, tol, _ = c.expect(q, True)
    assert_within("out", out, ref, tol)
    check_no_device_error(ra)


def test_steps_from_an_empty_cache(ra):
    """KVCache.empty, one page list shared by value and key, tokens one by one; q and rope left out."""
    g = np.random.default_rng(12)
    hk, d, n = 2, 64, 3
    cache = ra.KVCache.empty(n * 3, 16, hk, d)
    table = torch.arange(n * 3, dtype=torch.int32, device="cuda").flip(0).view(n, 3).contiguous()
    cu = ra.CuSeqlens(range(n + 1), "cuda")
    lens = torch.tensor([0, 5, 30], dtype=torch.int32, device="cuda")  # (zeros so far)
    ks, vs = [np.zeros((m, hk, d)) for m in (0, 5, 30)], [np.zeros((m, hk, d)) for m in (0, 5, 30)]
    for _ in range(4):
        lens += 1
        k, v = (torch.tensor(g.standard_normal((n, hk, d))).bfloat16().cuda() for _ in range(2))
        assert ra.ring_attn_cache_append(k, v, cache, table, lens, cu) is None
        q = torch.tensor(g.standard_normal((n, 4, d))).bfloat16().cuda()
        out, lse = ra.ring_attn_cache_fwd(q, cache, table, lens, cu)
        for i in range(n):
            ks[i] = np.concatenate([ks[i], oc.dequantise(*oc.quantise(f64(k[i:i + 1])))])
            vs[i] = np.concatenate([vs[i], oc.dequantise(*oc.quantise(f64(v[i:i + 1])))])
    c = Case((1,) * n, lens.tolist(), 4, hk, d, 16)
    c.k, c.v = ks, vs
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("out", out, ref, tol)
    assert_within("lse", lse, ref_l, tol_l)
    check_no_device_error(ra)


@pytest.mark.parametrize("new", [2, 40])
def test_attention_under_a_very_wide_page_table(ra, new):
    """2^30 tokens could be there: the work line counts in coarser places (its length has to fit 32 bits)."""
    c = Case((new,), (700,), 130, 130, 64, 256, seed=15)
    cache = c.fill(ra)
    wide = torch.full((1, 2 ** 22), -7, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.page_table
    q = c.queries()
    ref, ref_l, tol, tol_l = c.expect(q, True)
    for bound in (0, 2 ** 30 - 1, 700):
        out, lse = ra.ring_attn_cache_fwd(q, cache, wide, c.kv_lens, c.cu.tolist(), max_kv_len=bound)
        assert_within("lse", lse, ref_l, tol_l)
        assert_within("out", out, ref, tol)
    check_no_device_error(ra)


@pytest.mark.parametrize("new", [1, 50])
def test_offsets_beyond_32_bits(ra, new):
    """The last pages of a cache of more than 2^32 bytes an array: the same bits as in a small cache."""
    hk, d, page, far = 2, 128, 256, 135000
    c = Case((new, new), (300, 777), 4, hk, d, page, seed=16)
    small = c.fill(ra)
    q, x = c.queries(), torch.tensor(c.rng.standard_normal((c.rows, 2, hk, d))).bfloat16().cuda()
    code = lambda w: torch.empty((far + c.n_pages, hk, page, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    b = [code(w) for w in (d // 2, d // 16) * 2]
    assert b[0].numel() > 2 ** 32
    for y, z in zip(b, c.bytes):
        y[far:] = z
    big = ra.KVCache(b[0], b[1].view(torch.float8_e4m3fn), b[2], b[3].view(torch.float8_e4m3fn))
    cu = ra.CuSeqlens(c.cu, "cuda")
    got = []
    for cache, table in ((small, c.page_table), (big, c.page_table + far)):
        qr = ra.ring_attn_cache_append(x[:, 0], x[:, 1], cache, table, c.kv_lens, cu, q=q, rope=tables(800, d))
        got.append((qr, *ra.ring_attn_cache_read(cache, table, c.kv_lens, cu),
                    *ra.ring_attn_cache_fwd(qr, cache, table, c.kv_lens, cu)))
    for y, z in zip(*got):
        assert torch.equal(y, z)
    for y, z in zip(b, c.bytes):
        assert torch.equal(y[far:], z)
    check_no_device_error(ra)
