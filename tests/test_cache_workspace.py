"""CPU checks of ring_attn_cache_workspace_size: bytes for calls of AT MOST max_new new tokens a sequence."""
import pytest

from tests.test_cache import lib  # noqa: F401 (the fixture)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hk", [(1, 1), (8, 8), (16, 8), (12, 4), (32, 8), (7, 1), (8, 1), (16, 2), (40, 1)])
def test_a_size_serves_every_shorter_call(lib, d, h, hk):  # noqa: F811
    sizes = [lib.ring_attn_cache_workspace_size(300, n, h, hk, d, 4) for n in range(1, 101)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
