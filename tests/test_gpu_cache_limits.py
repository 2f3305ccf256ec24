"""The paged 4-bit cache at the ends of its ranges: lengths beyond the page table, tensors between others."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_case import Case, assert_within
from tests.helpers import check_no_device_error
from tests.test_gpu_cache import f64, ra, tables  # noqa: F401 (ra: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,page,rot", [(64, 16, 0), (128, 32, 128)])
@pytest.mark.parametrize("new,over", [(1, 1), (3, 1), (3, 3), (40, 7), (2, 1000000), (2, 2 ** 31 - 1 - 64)])
def test_tokens_past_the_page_table_have_no_place(ra, d, page, rot, new, over):  # noqa: F811
    """A length past the table: its tokens that lie in it are stored at their own places, the
    others nowhere, and cached tokens and the call's other sequences are as they should be."""
    c = Case((new, 2), (64, 40), 4, 2, d, page, seed=new + d)
    cache = c.fill(ra)
    lens = c.kv_lens.clone()
    lens[0] = 64 + over
    q, k, v = c.queries(), *(torch.tensor(c.rng.standard_normal((c.rows, 2, d))).bfloat16().cuda() for _ in range(2))
    cos, sin = tables(64 + 7, d)
    want = [b.cpu().numpy() for b in c.bytes]
    tok = np.concatenate([64 + over - new + np.arange(new, dtype=np.int64), [38, 39]])
    placed = tok < 64
    for r in np.flatnonzero(placed):
        pg, row = c.where(0 if r < new else 1, tok[r], tok[r] + 1)
        at = slice(tok[r], tok[r] + 1)
        x = oc.rotate(f64(k)[r:r + 1], cos.cpu().numpy()[at], sin.cpu().numpy()[at], False) if rot else f64(k)[r:r + 1]
        for j, y in ((0, x), (2, f64(v)[r:r + 1])):
            want[j][pg, :, row], want[j + 1][pg, :, row] = oc.quantise(y)
    q_out = torch.full_like(q, 5.0)
    ra.ring_attn_cache_append(k, v, cache, c.page_table, lens, c.cu.tolist(), q=q, rope=(cos, sin) if rot else None, q_out=q_out)
    st, info = ra.ring_attn_check_device_error()
    assert st == 7 and info & 0xff == 0x61
    for b, w in zip(c.bytes, want):
        assert np.array_equal(b.cpu().numpy(), w)
    lost = torch.tensor(~placed)
    assert bool((q_out[lost] == 5.0).all()) and not bool((q_out[~lost] == 5.0).any(-1).any())
    ko, vo = (torch.full((c.rows, 2, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ra.ring_attn_cache_read(cache, c.page_table, lens, c.cu.tolist(), k_out=ko, v_out=vo)
    st, info = ra.ring_attn_check_device_error()
    assert st == 7 and info & 0xff == 0x61
    assert bool((ko[lost] == 5.0).all()) and bool((vo[lost] == 5.0).all())
    for r in np.flatnonzero(placed):
        pg, row = c.where(0 if r < new else 1, tok[r], tok[r] + 1)
        for got, j in ((ko, 0), (vo, 2)):
            assert np.array_equal(f64(got)[r:r + 1], oc.dequantise(want[j][pg, :, row], want[j + 1][pg, :, row]))
    check_no_device_error(ra)


@pytest.mark.parametrize("new", [1, 60])
def test_slices_of_one_tensor_are_no_overlap(ra, new):  # noqa: F811
    """q, k, v, their outputs and the results as interleaved slices of one allocation."""
    h, hk, d = 4, 2, 64
    c = Case((new, 1), (200, 70), h, hk, d, 16, seed=17)
    cache, rows = c.fill(ra), c.rows
    x = torch.tensor(c.rng.standard_normal((rows, 32, d))).bfloat16().cuda()
    q, k, v, qo, ko, vo, out = (x[:, a:b] for a, b in ((0, 4), (4, 6), (6, 8), (8, 12), (12, 14), (14, 16), (16, 20)))
    lse = x.view(torch.float32)[:, 20:24, 0].t()  # (h, rows), fp32
    kept = x[:, :8].clone()
    cu = ra.CuSeqlens(c.cu, "cuda")
    ra.ring_attn_cache_append(k, v, cache, c.page_table, c.kv_lens, cu, q=q, q_out=qo)
    ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, cu, k_out=ko, v_out=vo)
    ra.ring_attn_cache_fwd(qo, cache, c.page_table, c.kv_lens, cu, out=out, lse=lse)
    check_no_device_error(ra)
    assert torch.equal(x[:, :8], kept) and torch.equal(qo, q)
    for i, m in enumerate(c.kv):
        r = slice(c.cu[i], c.cu[i + 1])
        c.k[i][m - c.n_new[i]:], c.v[i][m - c.n_new[i]:] = (oc.dequantise(*oc.quantise(f64(y)[r])) for y in (k, v))
        assert np.array_equal(f64(ko)[r], c.k[i][m - c.n_new[i]:]) and np.array_equal(f64(vo)[r], c.v[i][m - c.n_new[i]:])
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("out", out, ref, tol)
    assert_within("lse", lse, ref_l, tol_l)


@pytest.mark.parametrize("d", [64, 128])
def test_runs_of_items_of_one_and_two_query_tiles(ra, d):  # noqa: F811
    """Blocks that work through many items of one tile and one unit (one of the softmax warpgroups has no
    part in them), with items of two tiles and of one tile over several units between them."""
    g = np.random.default_rng(d)
    n_new = g.integers(1, 100, 600)
    kv = np.minimum(n_new + g.integers(0, 30, 600), 128)
    n_new[11::37], kv[11::37] = 150, 200   # two tiles
    n_new[5::53], kv[5::53] = 60, 700      # one tile, several units
    n_new[-1], kv[-1] = 200, 230
    c = Case(n_new.tolist(), kv.tolist(), 2, 2, d, 32, seed=d)
    cache, q, cu = c.fill(ra), c.queries(), ra.CuSeqlens(c.cu, "cuda")
    a, la = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu)
    for _ in range(50):
        b, lb = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu)
    check_no_device_error(ra)
    assert torch.equal(a, b) and torch.equal(la, lb)
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("out", a, ref, tol)
    assert_within("lse", la, ref_l, tol_l)


@pytest.mark.parametrize("new", [2, 90])
@pytest.mark.parametrize("scale", [1e-11, 1e-20, 1e-38])
def test_tiny_scales_and_queries(ra, new, scale):  # noqa: F811
    """Scores that vanish next to 1: the mean of what a row sees, the mask included."""
    c = Case((new, new), (300, 200), 4, 2, 64, 64, seed=1)
    cache, q = c.fill(ra), c.queries()
    q[:, 1] = 0
    q[0] *= 1e-30
    for causal in (True, False):
        out, lse = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist(), causal=causal, softmax_scale=scale)
        ref, ref_l, tol, tol_l = c.expect(q, causal, scale=scale)
        assert_within("lse", lse, ref_l, tol_l)
        assert_within("out", out, ref, tol)
    check_no_device_error(ra)


def test_calls_without_new_tokens(ra):  # noqa: F811
    """They give empty results, and refuse what any call refuses."""
    c = Case((0, 0), (30, 5), 4, 2, 64, 64, seed=1)
    cache, x = c.fill(ra), torch.zeros(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    lists = (c.page_table, c.kv_lens, [0, 0, 0])
    out, lse = ra.ring_attn_cache_fwd(q, cache, *lists)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert all(y.shape == (0, 2, 64) for y in ra.ring_attn_cache_read(cache, *lists))
    assert ra.ring_attn_cache_append(k, v, cache, *lists, q=q, rope=tables(9, 64)).shape == (0, 4, 64)
    odd = [b[:, :, :48].contiguous() for b in c.bytes]  # pages of 48 tokens
    odd = ra.KVCache(odd[0], odd[1].view(torch.float8_e4m3fn), odd[2], odd[3].view(torch.float8_e4m3fn))
    for call in (lambda: ra.ring_attn_cache_fwd(q, odd, *lists), lambda: ra.ring_attn_cache_read(odd, *lists),
                 lambda: ra.ring_attn_cache_append(k, v, odd, *lists), lambda: ra.ring_attn_cache_fwd(q.float(), cache, *lists),
                 lambda: ra.ring_attn_cache_append(k, v.float(), cache, *lists)):
        with pytest.raises(RuntimeError):
            call()
    check_no_device_error(ra)
