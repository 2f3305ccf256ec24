"""Changed scores and rotary positions without a GPU: the oracle's own gradients, and what the calls refuse."""
import ctypes

import numpy as np
import pytest
import torch

import ring_attn_gb300 as ra
from oracle import scores as osc
from tests.test_abi import _fake


@pytest.fixture(scope="module")
def lib():
    from ring_attn_gb300.build import build

    build()
    return ra.load()


@pytest.mark.parametrize("cap,slope,causal,prefix", [(1.5, 0.0, True, 0), (0.0, 0.3, False, 0), (0.7, -0.2, True, 4), (0.0, 0.0, True, 5)])
def test_the_oracles_gradients_are_its_differences(cap, slope, causal, prefix):
    rng = np.random.default_rng(0)
    m, n, d, scale = 6, 7, 4, 0.6
    x = {k: rng.standard_normal((r, d)) for k, r in (("q", m), ("k", n), ("v", n), ("do", m))}
    gq, gk = np.arange(m), np.arange(n)

    def value():
        return (osc.head(x["q"], x["k"], x["v"], gq, gk, scale, cap, slope, causal, prefix)["out"] * x["do"]).sum()

    r = osc.head(x["q"], x["k"], x["v"], gq, gk, scale, cap, slope, causal, prefix, x["do"])
    h = 1e-5
    for name in "qkv":
        for at in np.ndindex(x[name].shape):
            keep = x[name][at]
            x[name][at] = keep + h
            up = value()
            x[name][at] = keep - h
            down = value()
            x[name][at] = keep
            # central differences: h^2 / 6 of a third derivative of size 100 at most here, and 1e-16 / h
            assert abs((up - down) / (2 * h) - r["d" + name][at]) < 1e-8


def test_the_turn_back_is_the_transpose():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 5, 3, 16))
    a = rng.uniform(-3, 3, (9, 6))
    pos, axes = rng.integers(0, 9, (2, 5)), [0, 1, 1, 0, 1, 0]
    for inter in (False, True):
        turned = osc.rotate(x, np.cos(a), np.sin(a), pos, axes, inter)
        back = osc.rotate(y, np.cos(a), np.sin(a), pos, axes, inter, inverse=True)
        assert abs((turned * y).sum() - (x * back).sum()) < 1e-12
        assert np.allclose(osc.rotate(turned, np.cos(a), np.sin(a), pos, axes, inter, inverse=True), x)


def _scores(softcap=0.0, slopes=None, prefix=None):
    return ctypes.byref(ra._Scores(softcap, slopes, prefix))


def _ok(shape=(1, 2, 256, 64)):
    return [ctypes.byref(_fake(shape)) for _ in range(4)], ctypes.byref(_fake(shape[:3], ra.RA_FP32))


@pytest.mark.parametrize("grad,other", [(g, o) for g in ("dq", "dk", "dv") for o in ("do", "q", "k", "v", "dq", "dk", "dv")
                                        if g != o])
def test_gradients_on_one_another_or_on_inputs_are_refused(lib, grad, other):
    names = ("do", "q", "k", "v", "out", "dq", "dk", "dv")
    at = {n: 0x1000000 * (i + 1) for i, n in enumerate(names)}
    odd = ctypes.c_void_p(0x20000008)  # a workspace that is refused last: nothing is launched

    def status(at, shape, call):
        t = {n: ctypes.byref(_fake(shape, data=a)) for n, a in at.items()}
        return call(*(t[n] for n in ("do", "q", "k", "v", "out")), *(t[n] for n in ("dq", "dk", "dv")))

    cu = (ctypes.c_int32 * 2)(0, 256)
    host, dev, lse = ctypes.cast(cu, ctypes.c_void_p), ctypes.c_void_p(0x2000), ctypes.byref(_fake((1, 2, 256), ra.RA_FP32))
    l2, z = ctypes.byref(_fake((2, 256), ra.RA_FP32)), _scores(5.0)
    calls = [
        ((1, 2, 256, 64), lambda do, q, k, v, out, dq, dk, dv: lib.ring_attn_scored_bwd(
            do, q, k, v, out, lse, 0, 2, 1, 0.125, z, dq, dk, dv, odd, 1 << 24, None)),
        ((256, 2, 64), lambda do, q, k, v, out, dq, dk, dv: lib.ring_attn_scored_varlen_bwd(
            do, q, k, v, out, l2, dev, host, 1, 256, 0, 1, 1, 0.125, z, dq, dk, dv, odd, 1 << 24, None)),
        ((256, 2, 64), lambda do, q, k, v, out, dq, dk, dv: lib.ring_attn_scored_llama3_varlen_bwd(
            do, q, k, v, out, l2, dev, host, 1, 256, 0, 1, 1, 0.125, z, dq, dk, dv, odd, 1 << 24, None)),
    ]
    for shape, call in calls:
        assert status(at, shape, call) == 4  # the workspace
        assert status(dict(at, **{grad: at[other] + 128}), shape, call) == 1
        assert status(dict(at, **{grad: at[other] + 2 * 256 * 64 * 2}), shape, call) == 4  # right behind it


@pytest.mark.parametrize("z,causal,scale,status", [
    (None, 1, 0.125, 1), (_scores(-1.0), 1, 0.125, 1), (_scores(float("nan")), 1, 0.125, 1), (_scores(float("inf")), 1, 0.125, 1),
    (_scores(1e-4), 1, 0.125, 2), (_scores(1e7), 1, 0.125, 2), (_scores(0.001), 1, 2.0, 2),
    (_scores(prefix=0x1000), 0, 0.125, 1), (_scores(slopes=0x1002), 1, 0.125, 3), (_scores(prefix=0x1001), 1, 0.125, 3),
    (_scores(5.0), 2, 0.125, 1), (_scores(5.0), 1, 0.0, 1), (_scores(5.0), 1, float("nan"), 1),
])
def test_bad_scores_are_refused_before_any_launch(lib, z, causal, scale, status):
    (q, k, v, out), lse = _ok()
    assert lib.ring_attn_scored_fwd(q, k, v, 0, 2, causal, scale, z, out, lse, None) == status
    assert lib.ring_attn_scored_fwd_step(q, k, v, 0, 2, causal, scale, z, 0, out, lse, None) == status
    ws = ctypes.c_void_p(0x100000)
    assert lib.ring_attn_scored_bwd(out, q, k, v, out, lse, 0, 2, causal, scale, z, q, k, v, ws, 1 << 20, None) == status
    cu = (ctypes.c_int32 * 2)(0, 256)
    host = ctypes.cast(cu, ctypes.c_void_p)
    t = [ctypes.byref(_fake((256, 2, 64))) for _ in range(4)]
    l2 = ctypes.byref(_fake((2, 256), ra.RA_FP32))
    dev = ctypes.c_void_p(0x2000)
    for layout in (0, 1):
        assert lib.ring_attn_scored_varlen_fwd(t[0], t[1], t[2], dev, host, 1, 256, layout, 1, causal, scale, z, t[3], l2,
                                               ws, 1 << 30, None) == status
        assert lib.ring_attn_scored_varlen_bwd(t[3], t[0], t[1], t[2], t[3], l2, dev, host, 1, 256, layout, 1, causal, scale,
                                               z, t[0], t[1], t[2], ws, 1 << 30, None) == status
    assert lib.ring_attn_scored_llama3_varlen_fwd(t[0], t[1], t[2], dev, host, 1, 256, 0, 1, causal, scale, z, t[3], l2,
                                                  None) == status
    assert lib.ring_attn_scored_llama3_varlen_bwd(t[3], t[0], t[1], t[2], t[3], l2, dev, host, 1, 256, 0, 1, causal, scale, z,
                                                  t[0], t[1], t[2], ws, 1 << 20, None) == status


@pytest.mark.parametrize("z,causal,scale,status", [
    (None, 1, 0.125, 1), (_scores(-1.0), 1, 0.125, 1), (_scores(1e-4), 1, 0.125, 2), (_scores(prefix=0x1000), 0, 0.125, 1),
    (_scores(slopes=0x1002), 1, 0.125, 3), (_scores(5.0), 1, 0.0, 1),
])
def test_bad_scores_of_a_cache_call(lib, z, causal, scale, status):
    code, sc = (4, 2, 16, 32), (4, 2, 16, 4)
    c = ra._KVCache(_fake(code, ra.RA_E2M1X2), _fake(sc, ra.RA_E4M3), _fake(code, ra.RA_E2M1X2, 0x20000), _fake(sc, ra.RA_E4M3, 0x30000))
    cu = (ctypes.c_int32 * 2)(0, 1)
    s = ra._KVSeqs(0x4000, 4, 0x5000, 0x6000, ctypes.cast(cu, ctypes.c_void_p), 4, 1)
    q, out = ctypes.byref(_fake((1, 4, 64))), ctypes.byref(_fake((1, 4, 64), data=0x40000))
    lse = ctypes.byref(_fake((4, 1), ra.RA_FP32, 0x50000))
    assert lib.ring_attn_scored_cache_fwd(q, ctypes.byref(c), ctypes.byref(s), causal, scale, z, 0, out, lse, None, 0,
                                          None) == status


def test_the_handle_refuses_what_is_not_on_a_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        ra.Scores(slopes=torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        ra.Scores(prefix=[3])
    z = ra.Scores(2.0)
    assert z.softcap == 2.0 and z.slopes is None and z.prefix is None
    with pytest.raises(AttributeError):
        z.softcap = 3.0
    x = torch.zeros(1, 1, 8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ring_attn_fwd(x, x, x, scores=z)
    with pytest.raises(ValueError, match="Scores"):
        ra.ring_attn_fwd(x, x, x, scores=2.0)


def _rope(lib, q=None, k=None, cos=None, sin=None, style=0, pos=None, layout=0, n=1, inverse=0, q_out=None, k_out=None):
    t = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    q = _fake((1, 2, 64, 64)) if q is None else q
    q_out = _fake(tuple(q.shape[:4]), q.dtype, 0x900000) if q_out is None else q_out
    cos = _fake((100, 32), ra.RA_FP32, 0x200000) if cos is None else cos
    sin = _fake((100, 32), ra.RA_FP32, 0x300000) if sin is None else sin
    return lib.ring_attn_rope(t(q), t(k), t(cos), t(sin), style, t(pos), layout, n, inverse, t(q_out), t(k_out), None)


def _positions(pair_axis=None, n_axes=1, data=0x1000):
    buf = None if pair_axis is None else (ctypes.c_uint8 * len(pair_axis))(*pair_axis)
    p = ra._RopePositions(data, 64, 0, 1, ctypes.cast(buf, ctypes.c_void_p) if buf is not None else None, n_axes)
    p.keep = buf
    return p


def test_bad_rotations_are_refused_before_any_launch(lib):
    f = _fake
    assert _rope(lib, q=f((1, 2, 64, 64), data=0)) == 1
    assert _rope(lib, q=f((1, 2, 0, 64))) == 1
    assert _rope(lib, q=f((1, 2, 64, 96)), q_out=f((1, 2, 64, 96), data=0x900000)) == 2
    assert _rope(lib, q=f((1, 2, 64, 64), ra.RA_E4M3)) == 1
    assert _rope(lib, q_out=f((1, 2, 32, 64), data=0x900000)) == 1          # shape
    assert _rope(lib, q_out=f((1, 2, 64, 64), ra.RA_FP32, 0x900000)) == 1   # type
    assert _rope(lib, q=f((1, 2, 64, 64), data=0x10008)) == 3
    assert _rope(lib, q=f((1, 2, 64, 64), strides=(8192, 4096, 68, 1))) == 3
    assert _rope(lib, q=f((1, 2, 64, 64), strides=(8192, 4096, 64, 2))) == 3
    assert _rope(lib, q=f((1, 2, 64, 64), strides=(8192, 0, 64, 1))) == 3   # a broadcast dimension
    assert _rope(lib, k=f((1, 2, 64, 64), data=0x50000)) == 1               # k without k_out
    assert _rope(lib, k=f((1, 2, 32, 64), data=0x50000), k_out=f((1, 2, 32, 64), data=0x60000)) == 1
    assert _rope(lib, k=f((1, 2, 64, 64), ra.RA_FP32, 0x50000), k_out=f((1, 2, 64, 64), ra.RA_FP32, 0x70000)) == 1
    # outputs that share elements with something else than their own input
    assert _rope(lib, q_out=f((1, 2, 64, 64), data=0x10080)) == 1
    assert _rope(lib, k=f((1, 2, 64, 64), data=0x50000), k_out=f((1, 2, 64, 64))) == 1
    assert _rope(lib, k=f((1, 2, 64, 64), data=0x50000), q_out=f((1, 2, 64, 64), data=0x50000),
                 k_out=f((1, 2, 64, 64), data=0x60000)) == 1
    assert _rope(lib, k=f((1, 2, 64, 64), data=0x50000), k_out=f((1, 2, 64, 64), data=0x900000)) == 1
    # tables
    assert _rope(lib, cos=f((100, 33), ra.RA_FP32)) == 1
    assert _rope(lib, cos=f((100, 24), ra.RA_FP32), sin=f((100, 24), ra.RA_FP32)) == 1
    assert _rope(lib, cos=f((100, 64), ra.RA_FP32), sin=f((100, 64), ra.RA_FP32)) == 1  # more than d
    assert _rope(lib, sin=f((99, 32), ra.RA_FP32)) == 1
    assert _rope(lib, sin=f((100, 32), ra.RA_BF16)) == 1
    assert _rope(lib, sin=f((100, 32), ra.RA_FP32, strides=(33, 1))) == 3
    assert _rope(lib, style=2) == 1
    assert _rope(lib, inverse=2) == 1
    # layouts and positions
    assert _rope(lib, layout=3) == 1
    assert _rope(lib, n=3) == 1
    assert _rope(lib, layout=1, n=64) == 1
    assert _rope(lib, pos=_positions(data=0)) == 1
    assert _rope(lib, pos=_positions(data=0x1002)) == 3
    assert _rope(lib, pos=_positions(n_axes=0)) == 1
    assert _rope(lib, pos=_positions(n_axes=3)) == 1                        # which axis?
    assert _rope(lib, pos=_positions([0] * 31 + [2], n_axes=2)) == 1


def test_rotation_takes_cuda_tensors_only(lib):
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ring_attn_rope(x, None, (x, x))


@pytest.fixture(scope="module")
def marshaller(lib):
    """The compiled marshaller, and a maker of tensors that say they are on a GPU and have no memory."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    mode = FakeTensorMode()

    def tensor(*shape, dtype=torch.bfloat16):
        with mode:
            return torch.empty(shape, dtype=dtype, device="cuda")

    return ra._ext(), tensor


@pytest.mark.parametrize("bad", [(), (1, 1, 2, 64, 64), (1,) * 9])
@pytest.mark.parametrize("at", range(9))
def test_tensors_of_other_ranks_are_refused(marshaller, at, bad):
    """A C tensor has four dimensions: what has none or more is refused before any tensor is described, inputs and results."""
    ext, tensor = marshaller
    z = ra.Scores(5.0)
    names = ["dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv"]

    def args(shape):
        t = [tensor(*shape) for _ in names]
        t[5] = tensor(*shape[:-1], dtype=torch.float32)
        t[at] = tensor(*bad)
        return t

    if bad == () and at == 1:
        return  # (no head dim to take the scale from: an IndexError)
    message = "1 to 4 dimensions|expected a [34]-D"
    t = args((1, 2, 64, 64))
    with pytest.raises(ValueError, match=message):
        ra.ring_attn_bwd(*t[:6], dq=t[6], dk=t[7], dv=t[8], scores=z)
    if 1 <= at <= 5:
        with pytest.raises(ValueError, match=message):
            ra.ring_attn_fwd(*t[1:4], out=t[4], lse=t[5], scores=z)
    t, cu = args((64, 2, 64)), torch.tensor([0, 64], dtype=torch.int32)
    with pytest.raises(ValueError, match=message):
        ext.scored_varlen_bwd(*t[:6], cu, cu, None, 0, 1, True, 0.125, ra._of(z), *t[6:], None)
    if 1 <= at <= 5:
        with pytest.raises(ValueError, match=message):
            ext.scored_varlen_fwd(*t[1:4], cu, cu, None, 0, 1, True, 0.125, ra._of(z), *t[4:6], None)


def test_a_handles_tensors_are_taken_as_they_are_at_the_call(marshaller):
    """Storage that was exchanged (x.data = y, x.resize_, x.set_) is described anew: lengths are those of now."""
    _, tensor = marshaller
    slopes, prefix = tensor(2, dtype=torch.float32), tensor(1, dtype=torch.int32)
    x = [tensor(1, 2, 64, 64) for _ in range(3)]
    for z, held, other, message in ((ra.Scores(0.0, slopes), slopes, tensor(3, dtype=torch.float32), "2 query heads"),
                                    (ra.Scores(0.0, None, prefix), prefix, tensor(2, dtype=torch.int32), "1 sequences")):
        held.data = other
        with pytest.raises(ValueError, match=message):
            z._arg(x[0].device, 2, 1)
        with pytest.raises(ValueError, match=message):
            ra.ring_attn_fwd(*x, causal=True, scores=z)


def test_axes_are_a_row_of_numbers(lib):
    """A number is no row (bytes(32) would be 32 pairs on axis 0), and an array means its numbers, not its memory."""
    x = torch.zeros(3, 2, 64)
    for axes in (32, 2.0, torch.tensor(32), np.int64(32)):
        for call in (ra.ring_attn_rope, ra.ring_attn_rope_bwd):
            with pytest.raises(ValueError, match="axes"):
                call(x, None, (x, x), x, axes)
    with pytest.raises(ValueError):
        ra.ring_attn_rope(x, None, (x, x), x, [0, 256])
    want = bytes([0, 1, 2, 1])
    for axes in (want, [0, 1, 2, 1], (0, 1, 2, 1), np.array([0, 1, 2, 1]), torch.tensor([0, 1, 2, 1]), iter([0, 1, 2, 1])):
        assert ra._axes(axes) == want
