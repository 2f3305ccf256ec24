"""ring_attn_rope and its backward against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
import ring_attn_gb300 as ra
from oracle import scores as osc
from tests.helpers import check_no_device_error, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_attn_gb300.build import build

    build()
    ra.load()


def tables(n, r, seed=0):
    angle = np.random.default_rng(seed).uniform(-np.pi, np.pi, (n, r // 2))
    return torch.tensor(np.cos(angle), dtype=torch.float32).cuda(), torch.tensor(np.sin(angle), dtype=torch.float32).cuda()


def check(name, got, x, cos, sin, pos, axes, inter, inverse):
    """got, x: (rows, heads, d).  Two products and a sum in fp32 (2^-24 of a c and b s each, twice), then one rounding
    to the output's type; what is not turned is copied."""
    want = osc.rotate(f64(x), f64(cos), f64(sin), pos, axes, inter, inverse)
    half = torch.finfo(got.dtype).eps / 2
    r = 2 * len(axes)
    mag = np.abs(f64(x))
    pair = np.zeros_like(mag)
    a, b = (mag[..., 0:r:2], mag[..., 1:r:2]) if inter else (mag[..., :r // 2], mag[..., r // 2:r])
    both = a + b
    if inter:
        pair[..., 0:r:2] = pair[..., 1:r:2] = both
    else:
        pair[..., :r // 2] = pair[..., r // 2:r] = both
    tol = half * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -23 * pair
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), f"{name}: off by {err.max():.3e}"
    assert np.array_equal(f64(got)[..., r:], f64(x)[..., r:])


@pytest.mark.parametrize("rows,h,hk,d,r,sections,inter,dtype", [
    (1, 32, 8, 128, 128, (16, 24, 24), False, torch.bfloat16),
    (3, 5, 2, 64, 64, (8, 12, 12), True, torch.bfloat16),
    (1001, 4, 1, 128, 64, (5, 13, 14), False, torch.bfloat16),     # sections that split groups of four pairs
    (257, 3, 3, 64, 32, (16,), True, torch.float32),
    (70, 7, 1, 128, 16, (2, 6), False, torch.float32),
    (9, 1, 1, 64, 64, (1,) * 32, False, torch.bfloat16),           # an axis of its own for every pair
    (4099, 2, 2, 128, 128, (64,), True, torch.float32),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_packed_rows(rows, h, hk, d, r, sections, inter, dtype, inverse):
    g = torch.Generator().manual_seed(rows + d)
    q = (torch.randn(rows, h, d, generator=g) * 3).to(dtype).cuda()
    k = torch.randn(rows, hk, d, generator=g).to(dtype).cuda()
    cos, sin = tables(300, r)
    pos = torch.randint(0, 300, (len(sections), rows), generator=g, dtype=torch.int32)
    axes = [i for i, n in enumerate(sections) for _ in range(n)]
    turn = ra.ring_attn_rope_bwd if inverse else ra.ring_attn_rope
    qo, ko = turn(q, k, (cos, sin), pos.cuda(), axes, inter)
    check_no_device_error(ra)
    check("q", qo, q, cos, sin, pos.numpy(), axes, inter, inverse)
    check("k", ko, k, cos, sin, pos.numpy(), axes, inter, inverse)
    # in place, and q alone
    only, none = turn(q, None, (cos, sin), pos.cuda(), axes, inter)
    q2, k2 = q.clone(), k.clone()
    turn(q2, k2, (cos, sin), pos.cuda(), axes, inter, **({"dq_out": q2, "dk_out": k2} if inverse else {"q_out": q2, "k_out": k2}))
    assert none is None and torch.equal(only, qo) and torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("layout,n", [("contiguous", 1), ("zigzag", 3), ("stripe", 4)])
def test_positions_of_a_layout(layout, n):
    """Without positions a row goes by its original token."""
    b, h, hk, s, d = 2, 3, 1, 24 * n, 64
    g = torch.Generator().manual_seed(n)
    q, k = torch.randn(b, h, s, d, generator=g).bfloat16().cuda(), torch.randn(b, hk, s, d, generator=g).bfloat16().cuda()
    cos, sin = tables(s, d)
    qo, ko = ra.ring_attn_rope(q, k, (cos, sin), layout=layout, n_shards=n)
    check_no_device_error(ra)
    pos = oracle.token_of_position(layout, n, s)[None]
    for i in range(b):
        check("q", qo[i].transpose(0, 1), q[i].transpose(0, 1), cos, sin, pos, [0] * 32, False, False)
        check("k", ko[i].transpose(0, 1), k[i].transpose(0, 1), cos, sin, pos, [0] * 32, False, False)


def test_strides_and_broadcast_positions():
    """Heads of one packed tensor in place, positions shared by the batches and given as a transposed view."""
    b, s, h, d, r = 3, 50, 4, 128, 128
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(b, s, 3, h, d, generator=g).bfloat16().cuda()
    old = qkv.clone()
    cos, sin = tables(64, r)
    pos = torch.randint(0, 64, (s, 2), generator=g, dtype=torch.int32)
    axes = [f % 2 for f in range(64)]
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    got = ra.ring_attn_rope(q, k, (cos, sin), pos.cuda().t()[:, None].expand(2, b, s), axes, q_out=q, k_out=k)
    check_no_device_error(ra)
    assert got[0] is q and got[1] is k and torch.equal(qkv[:, :, 2], old[:, :, 2])
    for i in range(b):
        check("q", qkv[i, :, 0], old[i, :, 0], cos, sin, pos.t().numpy(), axes, False, False)
        check("k", qkv[i, :, 1], old[i, :, 1], cos, sin, pos.t().numpy(), axes, False, False)


def test_rows_with_a_bad_position_stay():
    s, h, d = 40, 3, 64
    q = torch.randn(s, h, d, device="cuda").bfloat16()
    cos, sin = tables(10, d)
    pos = torch.randint(0, 10, (2, s), dtype=torch.int32)
    pos[0, 7], pos[1, 20], pos[1, 39] = 10, -1, 2 ** 31 - 1
    axes = [0] * 20 + [1] * 12
    out = torch.full_like(q, 5.0)
    ra.ring_attn_rope(q, None, (cos, sin), pos.cuda(), axes, q_out=out)
    assert ra.ring_attn_check_device_error()[0] == 7
    check_no_device_error(ra)
    bad = [7, 20, 39]
    good = [i for i in range(s) if i not in bad]
    assert bool((out[bad] == 5.0).all())
    check("q", out[good], q[good], cos, sin, pos.numpy()[:, good], axes, False, False)


def test_captured_call_follows_positions_and_another_stream_agrees():
    s, h, hk, d = 130, 4, 2, 128
    q, k = torch.randn(s, h, d, device="cuda").bfloat16(), torch.randn(s, hk, d, device="cuda").bfloat16()
    cos, sin = tables(500, d)
    pos = torch.arange(s, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    ra.ring_attn_rope(q, k, (cos, sin), pos, q_out=qo, k_out=ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.ring_attn_rope(q, k, (cos, sin), pos, q_out=qo, k_out=ko)
    pos.add_(300)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2, k2 = ra.ring_attn_rope(q, k, (cos, sin), pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    check("q", qo, q, cos, sin, pos.cpu().numpy()[None], [0] * 64, False, False)
    check_no_device_error(ra)


def test_rotated_attention_is_its_own_gradient_chain():
    """Rotation, attention and both backwards together, against the oracle's gradient of the whole."""
    from tests.score_case import assert_within, expect

    h, hk, s, d = 2, 1, 96, 64
    g = torch.Generator().manual_seed(11)
    q, k, v, do = (torch.randn(1, n, s, d, generator=g).bfloat16().cuda() for n in (h, hk, hk, h))
    cos, sin = tables(s, d)
    z = ra.Scores(softcap=10.0)
    qr, kr = ra.ring_attn_rope(q, k, (cos, sin))
    out, lse = ra.ring_attn_fwd(qr, kr, v, causal=True, scores=z)
    dqr, dkr, dv = ra.ring_attn_bwd(do, qr, kr, v, out, lse, causal=True, scores=z)
    dq, dk = ra.ring_attn_rope_bwd(dqr, dkr, (cos, sin))
    check_no_device_error(ra)
    want = expect(qr, kr, v, do, d ** -0.5, 10.0, None, True, None)
    pos = np.arange(s)[None]
    for name, got, t in (("dq", dq, dqr), ("dk", dk, dkr)):
        assert_within(name, t, want[name])
        check(name, got[0].transpose(0, 1), t[0].transpose(0, 1), cos, sin, pos, [0] * 32, False, True)


def test_launches_are_recorded():
    q = torch.randn(1, 2, 40, 64, device="cuda").bfloat16()
    table = torch.rand(40, 32, device="cuda")
    ra.ring_attn_timing_enable(True)
    try:
        ra.ring_attn_rope(q, None, (table, table))
        ra.ring_attn_rope_bwd(q, None, (table, table))
        ms, n = ra.ring_attn_timing_read("rope")
    finally:
        ra.ring_attn_timing_enable(False)
    assert n == 2 and ms > 0
