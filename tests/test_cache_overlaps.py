"""CPU checks, before any launch: which overlaps of a cache call's tensors are refused, and tensors without rows."""
import numpy as np
import pytest

import ring_attn_gb300 as ra
from tests.test_cache import FAR, append, attend, cache, fake, lib, read, seqs  # noqa: F401 (lib: the fixture)

ODD = 0x1002  # positions there are refused (3) behind the overlaps (1)


def part(heads, first, rows=10, d=64, packed=8, base=0x100000, row_of=None):
    """Heads [first, first + heads) of a packed (rows, packed, d) tensor."""
    return fake((rows, heads, d), data=base + 2 * d * first, stride=(packed * d, row_of or d, 1))


@pytest.mark.parametrize("q,out,k,v,refused", [
    # in place: keys or values that are some of the queries' own elements
    (part(4, 0), part(4, 0), part(2, 0), part(2, 6), True),
    (part(4, 0), part(4, 0), part(2, 2), part(2, 6), True),
    (part(4, 0), part(4, 0), part(2, 4), part(2, 3), True),
    (part(4, 4), part(4, 4), part(2, 0), part(2, 3), True),
    (part(4, 0), part(4, 0), part(2, 4), part(2, 6), False),
    # slices of one packed tensor that share no element, q elsewhere or another slice
    (part(4, 0, base=FAR), part(4, 0), part(2, 4), part(2, 6), False),
    (part(4, 0, base=FAR), part(4, 4), part(2, 0), part(2, 2), False),
    (part(4, 0, packed=12), part(4, 8, packed=12), part(2, 4, packed=12), part(2, 6, packed=12), False),
    (part(4, 0, packed=12), part(4, 7, packed=12), part(2, 4, packed=12), part(2, 6, packed=12), True),
    (part(4, 0, packed=12), part(4, 3, packed=12), part(2, 8, packed=12), part(2, 10, packed=12), True),
    # a row further on is the same slice again
    (part(4, 0, base=FAR), part(4, 12), part(2, 4), part(2, 6), True),
    (part(4, 0, base=FAR), part(4, 8), part(2, 4), part(2, 6), False),
    # heads that lie apart, between another tensor's
    (part(4, 0, base=FAR), part(4, 0, row_of=128), part(2, 1, row_of=128), part(2, 5, row_of=128), False),
    (part(4, 0, base=FAR), part(4, 0, row_of=128), part(2, 1, row_of=128), part(2, 4, row_of=128), True),
    # apart altogether
    (part(4, 0), part(4, 0, base=FAR), part(2, 0), part(2, 0), False),
])
def test_append_overlaps(lib, q, out, k, v, refused):  # noqa: F811
    def elements(t):
        i = np.indices(tuple(t.shape)[:3]).reshape(3, -1)
        return set((t.data // 2 + np.array(list(t.stride)[:3]) @ i).tolist())

    shared = lambda a, b: bool(elements(a) & elements(b))  # noqa: E731
    in_place = q.data == out.data and list(q.stride) == list(out.stride)
    assert refused == (shared(k, out) or shared(v, out) or (not in_place and shared(q, out)))
    assert append(lib, q=q, out=out, k=k, v=v, pos=ODD) == (1 if refused else 3)


def test_read_overlaps(lib):  # noqa: F811
    assert read(lib, k=part(2, 0), v=part(2, 0)) == 1
    assert read(lib, k=part(2, 0), v=part(2, 1)) == 1
    assert read(lib, k=fake((10, 2, 64)), v=fake((10, 2, 64), data=0x100000 + 9 * 256)) == 1


def test_attention_overlaps(lib):  # noqa: F811
    far = dict(q=fake((10, 4, 64)), out=fake((10, 4, 64), data=FAR), lse=fake((4, 10), ra.RA_FP32, data=2 * FAR))
    f = lambda **k: attend(lib, **dict(far, **k))  # noqa: E731
    assert f(out=far["q"]) == 1 and f(out=part(4, 1), q=part(4, 0)) == 1
    assert f(out=fake((10, 4, 64), ra.RA_FP32, data=0x100000 + 5120 - 16)) == 1   # q's last bytes
    assert f(lse=fake((4, 10), ra.RA_FP32, data=0x100000 + 512)) == 1             # in q
    assert f(lse=fake((4, 10), ra.RA_FP32, data=FAR + 5120 - 4)) == 1             # in out
    assert f(lse=fake((4, 10), ra.RA_FP32, data=FAR + 128, stride=(64, 128))) == 1


def test_tensors_without_rows(lib):  # noqa: F811
    """A call without new tokens is checked like any other; its tensors may be empty (and have no address)."""
    none = lambda heads, dtype=ra.RA_BF16: fake((0, heads, 64), dtype, data=0, stride=(heads * 64, 64, 1))  # noqa: E731
    s = seqs((0, 0, 0))
    assert append(lib, s=s, k=none(2), v=none(2)) == 0
    assert append(lib, s=s, k=none(2), v=none(2), q=none(4), out=none(4)) == 0
    assert append(lib, s=s, k=none(2), v=none(3)) == 1
    assert read(lib, s=s, k=none(2), v=none(2)) == 0 and read(lib, s=s, k=none(2), v=none(1)) == 1
    lse = fake((4, 0), ra.RA_FP32, data=0, stride=(1, 1))
    assert attend(lib, s=s, q=none(4), out=none(4), lse=lse, ws=None, wb=0) == 0
    assert attend(lib, s=s, q=none(4), out=none(3), lse=lse, ws=None, wb=0) == 1
    assert attend(lib, s=s, c=cache(page=48), q=none(4), out=none(4), lse=lse, ws=None, wb=0) == 2
    assert append(lib, k=none(2)) == 1 and read(lib, v=none(2)) == 1 and attend(lib, q=none(4)) == 1
