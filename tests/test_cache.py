"""CPU checks of the paged 4-bit cache calls: refusals before any launch, and pins of the oracle."""
import ctypes

import numpy as np
import pytest

import ring_attn_gb300 as ra
from oracle import cache as oc


@pytest.fixture(scope="module")
def lib():
    from ring_attn_gb300.build import build

    build()
    return ra.load()


def fake(shape, dtype=ra.RA_BF16, data=0x100000, stride=None):
    if stride is None:
        stride, acc = [], 1
        for n in reversed(shape):
            stride.insert(0, acc)
            acc *= n
    pad = [0] * (4 - len(shape))
    return ra._Tensor(data, dtype, len(shape), ra._I64x4(*shape, *pad), ra._I64x4(*stride, *pad))


def cache(n=9, hk=2, page=32, d=64, **over):
    a = dict(k=fake((n, hk, page, d // 2), ra.RA_E2M1X2), k_scale=fake((n, hk, page, d // 16), ra.RA_E4M3),
             v=fake((n, hk, page, d // 2), ra.RA_E2M1X2), v_scale=fake((n, hk, page, d // 16), ra.RA_E4M3))
    a.update(over)
    return ra._KVCache(a["k"], a["k_scale"], a["v"], a["v_scale"])


def seqs(cu=(0, 3, 10), **over):
    host = (ctypes.c_int32 * len(cu))(*cu)
    a = dict(page_table=0x1000, page_table_stride=4, kv_lens=0x2000, cu_seqlens_dev=0x3000,
             cu_seqlens_host=ctypes.cast(host, ctypes.c_void_p), max_pages=4, n_seqs=len(cu) - 1)
    a.update(over)
    s = ra._KVSeqs(*(a[f] for f, _ in ra._KVSeqs._fields_))
    s._keep = host
    return s


FAR = 0x9000000


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(lib, c=None, s=None, q=None, k=None, v=None, cos=None, sin=None, rope=0, pos=None, out=None):
    r = [ref(x) for x in (q, k or fake((10, 2, 64)), v or fake((10, 2, 64)), cos, sin, c or cache(), s or seqs(), out)]
    return lib.ring_attn_cache_append(*r[:5], rope, pos, *r[5:], None)


def attend(lib, c=None, s=None, q=None, out=None, lse=None, causal=1, scale=0.1, mx=0, ws=0x100000, wb=1 << 40):
    r = [ref(x) for x in (q or fake((10, 4, 64)), c or cache(), s or seqs(), out or fake((10, 4, 64)),
                          lse or fake((4, 10), ra.RA_FP32))]
    return lib.ring_attn_cache_fwd(*r[:3], causal, scale, mx, *r[3:], ws, wb, None)


def read(lib, c=None, s=None, k=None, v=None):
    r = [ref(x) for x in (c or cache(), s or seqs(), k or fake((10, 2, 64)), v or fake((10, 2, 64)))]
    return lib.ring_attn_cache_read(*r, None)


BAD_CACHE = [
    (cache(k=fake((9, 2, 32, 32), ra.RA_BF16)), 1),
    (cache(k=fake((9, 2, 32, 32), ra.RA_E2M1X2, data=0)), 1),
    (cache(k_scale=fake((9, 2, 32, 8), ra.RA_E4M3)), 1),
    (cache(v=fake((8, 2, 32, 32), ra.RA_E2M1X2)), 1),
    (cache(v_scale=fake((9, 2, 32, 4), ra.RA_E2M1X2)), 1),
    (cache(d=96), 2), (cache(page=48), 2), (cache(page=8), 2), (cache(page=512), 2),
    (cache(k=fake((9, 2, 32, 32), ra.RA_E2M1X2, data=0x100008)), 3),
    (cache(v=fake((9, 2, 32, 32), ra.RA_E2M1X2, stride=(4096, 2048, 40, 1))), 3),
    (cache(v=fake((9, 2, 32, 32), ra.RA_E2M1X2, stride=(4096, 2048, 64, 2))), 3),
    (cache(v_scale=fake((9, 2, 32, 4), ra.RA_E4M3, stride=(256, 128, 6, 1))), 3),
    (cache(k_scale=fake((9, 2, 32, 4), ra.RA_E4M3, data=0x100004)), 3),
    (cache(v=fake((9, 2, 32, 32), ra.RA_E2M1X2, stride=(4096, 2048, 64, 1))), 2),  # not k's strides
    (cache(k_scale=fake((9, 2, 32, 4), ra.RA_E4M3, stride=(512, 128, 4, 1))), 2),
]
BAD_SEQS = [
    (seqs(page_table=None), 1), (seqs(kv_lens=None), 1), (seqs(cu_seqlens_dev=None), 1), (seqs(cu_seqlens_host=None), 1),
    (seqs(n_seqs=0), 1), (seqs(max_pages=0), 1), (seqs(page_table_stride=3), 1), (seqs((1, 3, 10)), 1),
    (seqs((0, 11, 10)), 1), (seqs((0, 3, 11)), 1), (seqs(kv_lens=0x2002), 3), (seqs(max_pages=1 << 30, page_table_stride=1 << 30), 2),
]


@pytest.mark.parametrize("c,status", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(lib, c, status):
    assert append(lib, c=c) == status and read(lib, c=c) == status and attend(lib, c=c) == status


@pytest.mark.parametrize("s,status", BAD_SEQS)
def test_every_call_refuses_bad_sequences(lib, s, status):
    assert append(lib, s=s) == status and read(lib, s=s) == status and attend(lib, s=s) == status


def test_append_refuses(lib):
    q, out = fake((10, 4, 64)), fake((10, 4, 64), data=FAR)
    t = lambda n=100, r=32, **k: fake((n, r), ra.RA_FP32, **k)  # noqa: E731
    assert append(lib, k=fake((9, 2, 64))) == 1                      # fewer rows than new tokens
    assert append(lib, v=fake((10, 3, 64))) == 1
    assert append(lib, k=fake((10, 2, 128))) == 1
    assert append(lib, k=fake((10, 2, 64), ra.RA_FP32)) == 1
    assert append(lib, k=fake((10, 2, 64), stride=(128, 68, 1))) == 3
    assert append(lib, k=fake((10, 2, 64), data=0x100008)) == 3
    assert append(lib, q=q) == 1 and append(lib, out=out) == 1       # one without the other
    assert append(lib, q=fake((10, 3, 64)), out=fake((10, 3, 64), data=FAR)) == 1  # 3 heads over 2
    assert append(lib, q=q, out=fake((10, 2, 64), data=FAR)) == 1
    far_k = dict(k=fake((10, 2, 64), data=2 * FAR), v=fake((10, 2, 64), data=3 * FAR))
    assert append(lib, q=q, out=fake((10, 4, 64), data=0x100000 + 512), **far_k) == 1   # overlaps q
    assert append(lib, q=q, out=fake((10, 4, 64), data=2 * FAR + 512), **far_k) == 1    # overlaps k
    assert append(lib, cos=t()) == 1 and append(lib, sin=t()) == 1
    assert append(lib, cos=t(), sin=t(99)) == 1 and append(lib, cos=t(), sin=t(100, 16)) == 1
    assert append(lib, cos=t(r=40), sin=t(r=40)) == 1                # more than d head dims
    assert append(lib, cos=t(r=12), sin=t(r=12)) == 1                # 24 head dims: not 16, not a multiple of 32
    assert append(lib, cos=t(r=24), sin=t(r=24)) == 1
    assert append(lib, cos=fake((100, 32)), sin=t()) == 1            # bf16 table
    assert append(lib, cos=t(data=0x100004), sin=t()) == 3
    assert append(lib, cos=t(stride=(33, 1)), sin=t()) == 3
    assert append(lib, rope=2) == 1
    assert append(lib, pos=0x1002) == 3
    assert append(lib, s=seqs((0, 0, 0))) == 0                       # nothing new: nothing launched


def test_read_refuses(lib):
    assert read(lib, k=fake((9, 2, 64))) == 1
    assert read(lib, v=fake((10, 2, 64), ra.RA_FP32)) == 1
    assert read(lib, v=fake((10, 4, 64))) == 1
    assert read(lib, v=fake((10, 2, 64), stride=(128, 64, 2))) == 3
    assert read(lib, s=seqs((0, 0, 0))) == 0


def test_attention_refuses(lib):
    assert attend(lib, q=fake((9, 4, 64))) == 1
    assert attend(lib, q=fake((10, 3, 64)), out=fake((10, 3, 64)), lse=fake((3, 10), ra.RA_FP32)) == 1
    assert attend(lib, out=fake((10, 2, 64))) == 1
    assert attend(lib, out=fake((10, 4, 64), ra.RA_E4M3)) == 1
    assert attend(lib, out=fake((10, 4, 64), ra.RA_FP32, stride=(256, 66, 1))) == 3
    assert attend(lib, lse=fake((4, 9), ra.RA_FP32)) == 1
    assert attend(lib, lse=fake((4, 10))) == 1
    assert attend(lib, lse=fake((4, 10), ra.RA_FP32, data=0x100002)) == 1
    assert attend(lib, causal=2) == 1 and attend(lib, mx=-1) == 1
    assert attend(lib, scale=0.0) == 1 and attend(lib, scale=float("inf")) == 1
    many = 1 << 26  # 2^26 tokens of 32 heads over one: more than 2^30 rows
    big = (many, 32, 64)
    assert attend(lib, c=cache(hk=1), s=seqs((0, many)), q=fake(big), out=fake(big), lse=fake((32, many), ra.RA_FP32)) == 2
    n, hk = 65535, 10000  # more items than a line of 32 bits holds
    big = (n, hk, 64)
    assert attend(lib, c=cache(hk=hk), s=seqs(range(n + 1)), q=fake(big), out=fake(big), lse=fake((hk, n), ra.RA_FP32)) == 2
    need = lib.ring_attn_cache_workspace_size(10, 7, 4, 2, 64, 2)
    assert need > 0
    assert attend(lib, ws=None) == 4 and attend(lib, wb=need - 1) == 4 and attend(lib, ws=0x100010) == 4
    assert attend(lib, s=seqs((0, 0, 0))) == 0


def test_workspace_size(lib):
    f = lib.ring_attn_cache_workspace_size
    assert f(10, 11, 4, 2, 64, 2) == 0 and f(10, 7, 4, 3, 64, 2) == 0 and f(10, 7, 4, 2, 96, 2) == 0
    assert f(-1, 0, 4, 2, 64, 2) == 0 and f(10, 7, 4, 2, 64, 0) == 0
    assert ra.ring_attn_cache_workspace_size(10, 7, 4, 2, 64, 2) == f(10, 7, 4, 2, 64, 2)


def test_binding_refuses_cpu_tensors():
    import torch

    u8, f8 = torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 16, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        ra.KVCache(u8, f8, u8, f8)
    with pytest.raises(ValueError):
        ra.ring_attn_cache_read(None, None, None, [0, 1])


def test_oracle_numbers():
    """The oracle's grids and roundings against torch's e4m3 and hand-made cases."""
    import torch

    assert np.array_equal(oc.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    x = np.linspace(0, 460, 100001)
    assert np.array_equal(oc.E4M3[oc.nearest(x, oc.E4M3)], torch.tensor(np.minimum(x, 448)).to(torch.float8_e4m3fn).double().numpy())
    got = oc.E2M1[oc.nearest([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.2500001, 9], oc.E2M1)]
    assert got.tolist() == [0, 1, 1, 2, 2, 4, 4, 0.5, 6]
    codes, scales = oc.quantise(np.array([[6.0, -0.5, 0, -0.0] + [3.0] * 12]))
    assert oc.E4M3[scales[0, 0]] == 1 and codes[0, 0] == 7 | (9 << 4) and codes[0, 2] == 5 | (5 << 4)
    assert oc.dequantise(codes, scales)[0, :3].tolist() == [6, -0.5, 0]
    assert oc.quantise(np.zeros((1, 16)))[1][0, 0] == 1  # the least scale


def test_oracle_attention_is_the_softmax():
    import torch

    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((5, 4, 16)), g.standard_normal((9, 2, 16)), g.standard_normal((9, 2, 16))
    out, lse, _, _ = oc.attention(q, k, v, 0.25, [5, 6, 7, 8, 9])
    t = lambda x: torch.tensor(x).transpose(0, 1)  # noqa: E731
    s = t(q) @ t(k).repeat_interleave(2, 0).transpose(1, 2) * 0.25
    s = s.masked_fill(torch.ones(5, 9, dtype=torch.bool).triu(5), -torch.inf)
    assert np.allclose(out, (s.softmax(-1) @ t(v).repeat_interleave(2, 0)).transpose(0, 1).numpy(), atol=1e-12)
    assert np.allclose(lse, s.logsumexp(-1).numpy(), atol=1e-12)
    z = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    assert np.allclose(oc.rotate(z, np.array([[0.0]]), np.array([[1.0]]), True)[0, 0], [-4, 3, 1, 2])
    assert np.allclose(oc.rotate(z, np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]]), False)[0, 0], [-1, 4, 3, 2])
