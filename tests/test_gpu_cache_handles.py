"""Copies of the handles that the paged cache's calls take, on the GPU."""
import copy
import gc
import pickle

import pytest
import torch

from tests.cache_case import Case, assert_within
from tests.helpers import check_no_device_error
from tests.test_gpu_cache import ra  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

COPIES = [copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x)), copy.copy]


@pytest.mark.parametrize("duplicate", COPIES)
@pytest.mark.parametrize("new", [2, 70])
def test_a_copied_cu_seqlens_outlives_the_first(ra, duplicate, new):  # noqa: F811
    c = Case((new, 0, new), (300, 9, 41), 4, 2, 64, 16, seed=21)
    cache, q = c.fill(ra), c.queries()
    first = ra.CuSeqlens(c.cu, "cuda")
    cu = duplicate(first)
    del first
    gc.collect()
    other = [torch.full((c.cu.size,), -9, dtype=torch.int32, device="cuda") for _ in range(8)]  # freed memory's next users
    out, lse = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu)
    k, v = ra.ring_attn_cache_read(cache, c.page_table, c.kv_lens, cu)
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("out", out, ref, tol)
    assert_within("lse", lse, ref_l, tol_l)
    m = min(new, 41)  # (rows before the cache's start are left as they were)
    assert torch.equal(k[-m:].double().cpu(), torch.tensor(c.k[2][-m:]))
    assert torch.equal(v[:new].double().cpu(), torch.tensor(c.v[0][-new:]))
    assert len(other) == 8
    check_no_device_error(ra)


def test_a_cu_seqlens_that_does_not_fit_is_refused(ra):  # noqa: F811
    c = Case((2, 3), (30, 41), 4, 2, 64, 16, seed=22)
    cache, q = c.fill(ra), c.queries()
    for what, bad in (("dev", lambda x: x.cpu()), ("dev", lambda x: x.long()), ("dev", lambda x: x[:2]), ("dev", lambda x: None),
                      ("host", lambda x: x.cuda()), ("host", lambda x: x.long()), ("host", lambda x: x[:1])):
        cu = ra.CuSeqlens(c.cu, "cuda")
        setattr(cu, what, bad(getattr(cu, what)))
        with pytest.raises(ValueError):
            ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, cu)
    check_no_device_error(ra)


@pytest.mark.parametrize("duplicate", COPIES)
def test_a_copied_kv_cache_is_one_of_its_own(ra, duplicate):  # noqa: F811
    """Calls on the copy use its tensors (copy.copy: the same ones), also when the first is gone."""
    c = Case((2, 3), (30, 41), 4, 2, 64, 16, seed=23, order=(0, 2, 1))
    first, q = c.fill(ra), c.queries()
    before = [b.clone() for b in c.bytes]
    cache = duplicate(first)
    del first
    gc.collect()
    out, lse = ra.ring_attn_cache_fwd(q, cache, c.page_table, c.kv_lens, c.cu.tolist())
    ref, ref_l, tol, tol_l = c.expect(q, True)
    assert_within("out", out, ref, tol)
    assert_within("lse", lse, ref_l, tol_l)
    x = c.queries()
    ra.ring_attn_cache_append(x[:, :2], x[:, 2:], cache, c.page_table, c.kv_lens, c.cu.tolist())
    same = all(torch.equal(a, b) for a, b in zip(before, c.bytes))
    assert same == (duplicate is not copy.copy)
    check_no_device_error(ra)
