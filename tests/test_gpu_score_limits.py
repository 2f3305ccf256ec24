"""Changed scores at the ends of what the calls take: steep biases, single ring steps, products and values far from 1,
saturated caps, a block's share of a longer row."""
import numpy as np
import pytest
import torch

import oracle
import ring_attn_gb300 as ra
from tests.helpers import check_no_device_error, lse_to_original, to_layout, to_original
from tests.score_case import EPS, assert_within, expect, f64, head_bounds
from tests.test_gpu_scores import inputs, scores_of, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_attn_gb300.build import build

    build()
    ra.load()


def steep(h, of):
    return torch.tensor([of * (1.0 - 0.25 * i) for i in range(h)], dtype=torch.float32)


@pytest.mark.parametrize("layout,causal,cap,slopes,prefix", [
    ("contiguous", True, 8.0, "alibi", (150,)), ("zigzag", True, 0.0, "alibi", None), ("stripe", False, 8.0, "mixed", None),
    ("contiguous", False, 0.0, 100.0, None), ("contiguous", True, 90.0, 100.0, (3,)), ("zigzag", True, 0.0, 60.0, None),
    ("zigzag", False, 0.0, -60.0, None), ("stripe", True, 8.0, -100.0, None), ("contiguous", True, 30.0, 80.0, None),
])
def test_every_ring_step_on_its_own(layout, causal, cap, slopes, prefix):
    """out and lse of a step are those of its keys alone: 0 and -inf only for rows that see none of them.  Steep biases put
    the scores of far keys 2^14 to 2^17 (log2 units) below those near."""
    b, h, hk, s, d, n = 1, 2, 1, 544, 64, 4
    x = inputs(b, h, hk, s, d, 9110)
    sl = slopes_of(h, slopes) if not isinstance(slopes, float) else steep(h, slopes)
    z = scores_of(cap, sl, prefix)
    g = {k: to_layout(ra, v.cuda(), layout, n) for k, v in x.items()}
    place = oracle.token_of_position(layout, n, s).reshape(n, -1)  # tokens of every shard
    for step in range(n):
        out, lse = ra.ring_attn_fwd_step(g["q"], g["k"], g["v"], step, layout, n, causal, scores=z)
        check_no_device_error(ra)
        want = {name: (np.zeros(shape), np.zeros(shape)) for name, shape in (("out", (b, h, s, d)), ("lse", (b, h, s)))}
        for r in range(n):
            gq, gk = place[r], place[(r - step) % n]
            for a in range(h):
                e = head_bounds(x["q"][0, a, gq], x["k"][0, 0, gk], x["v"][0, 0, gk], gq, gk, d ** -0.5, cap,
                                0.0 if sl is None else float(sl[a]), causal, prefix[0] if prefix else 0)
                for name, (val, tol) in want.items():
                    val[0, a, gq], tol[0, a, gq] = e[name], e["tol"][name]
        assert_within("out", to_original(ra, out, layout, n), want["out"])
        assert_within("lse", lse_to_original(ra, lse, layout, n), want["lse"])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap,slope,gain", [(0.0, -100.0, 1.0), (0.0, 100.0, 1.0), (90.0, -60.0, 1.0), (0.0, 0.01, 200.0),
                                            (40.0, -100.0, 1.0)])
def test_far_scores_of_whole_calls(causal, cap, slope, gain):
    """Rows whose largest score is 2^14 and more: a bias that rises with the distance, or large products next to one."""
    b, h, hk, s, d = 1, 2, 1, 600, 128
    x = inputs(b, h, hk, s, d, 9120, gain)
    x["k"] = (x["k"].float() * gain).bfloat16()
    sl = steep(h, slope)
    g = {k: v.cuda() for k, v in x.items()}
    z = scores_of(cap, sl, None)
    out, lse = ra.ring_attn_fwd(g["q"], g["k"], g["v"], "contiguous", 1, causal, scores=z)
    check_no_device_error(ra)
    want = expect(x["q"], x["k"], x["v"], None, d ** -0.5, cap, sl, causal, None)
    assert_within("lse", lse, want["lse"])
    assert_within("out", out, want["out"])
