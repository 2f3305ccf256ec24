"""Every kernel kind that ring_attn_timing_read offers is recorded by the calls that launch it."""
import pytest
import torch

from tests.cache_case import Case
from tests.helpers import check_no_device_error
from tests.test_gpu_cache import ra  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def recorded(ra, call):  # noqa: F811
    """Launches of each kind that `call` makes."""
    ra.ring_attn_timing_enable(True)
    try:
        call()
        got = {}
        for kind in ra.KERNELS:
            ms, n = ra.ring_attn_timing_read(kind)
            assert (ms > 0) == (n > 0)
            if n:
                got[kind] = n
        return got
    finally:
        ra.ring_attn_timing_enable(False)


@pytest.mark.parametrize("new,kv,joins", [(1, 900, 0), (1, 30000, 1), (1, 3000, 1), (12, 3000, 1), (30, 5000, 1), (90, 700, 1)])
def test_cache_attention_and_its_join(ra, new, kv, joins):  # noqa: F811
    c = Case((new,), (kv,), 4, 4, 64, 64, seed=1)
    cache, q, cu = c.fill(ra), c.queries(), ra.CuSeqlens(c.cu, "cuda")
    got = recorded(ra, lambda: ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu, max_kv_len=kv))
    assert got == dict({"cache_fwd": 1}, **({"cache_join": joins} if joins else {}))
    check_no_device_error(ra)


def test_every_kind_is_recorded(ra):  # noqa: F811
    c = Case((1,), (30000,), 4, 4, 64, 64, seed=1)
    cache, cu = c.fill(ra), ra.CuSeqlens(c.cu, "cuda")
    x = c.queries()
    q, k, v = (torch.randn(1, 2, 256, 64, device="cuda").bfloat16() for _ in range(3))

    def call():
        ra.ring_attn_cache_append(x, x, cache, c.page_table, c.kv_lens, cu)
        ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, cu)
        ra.ring_attn_cache_fwd(x, cache, c.page_table, c.kv_lens, cu)
        out, lse = ra.ring_attn_fwd(q, k, v, causal=True)
        ra.ring_attn_bwd(out, q, k, v, out, lse, causal=True)
        ra.ring_attn_permute(q, "zigzag", 2, seq_dim=2)
        ra.lse_merge(out.float()[0], lse.clone()[0], out[0], lse[0])

    got = recorded(ra, call)
    assert set(got) == set(ra.KERNELS) and all(got.values())
    check_no_device_error(ra)
