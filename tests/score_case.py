"""Expected results of attention with changed scores, with bounds of what the kernels' roundings may add."""
import numpy as np

from oracle import scores as osc

BF = 2.0 ** -8   # half a step of bf16
EPS = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def head_bounds(q, k, v, gq, gk, scale, cap=0.0, slope=0.0, causal=False, prefix=0, do=None):
    """osc.head's results and, in "tol", a bound for each.

    Scores.  bf16 products are exact in fp32, a sum of d of them is off by d 2^-24 sum|q k|; the cap
    has slope at most 1 and is off by cap 2^-21 (exponential 2^-22, reciprocal 2^-23, three roundings,
    or the polynomial's 2^-22.4 of at most 0.54 cap); the bias is a product and a sum of fp32
    numbers up to slope * distance: 4 roundings; scaling to log2 units and taking the maximum or
    lse off: 4 roundings of numbers up to |z|.  P carries that error relatively (twice: the sum's or the lse's
    own), the exponential's 2^-21 and, as an operand, half a step of bf16; sums of n terms n 2^-24."""
    q, k, v = f64(q), f64(k), f64(v)
    r = osc.head(q, k, v, gq, gk, scale, cap, slope, causal, prefix, None if do is None else f64(do))
    n, d = len(gk), q.shape[1]
    see = np.isfinite(r["z"])
    dist = np.abs(np.asarray(gq)[:, None] - np.asarray(gk)[None, :])
    zmax = np.where(see, np.abs(r["z"]), 0.0).max(1, initial=0.0)
    s_err = d * EPS * scale * (np.abs(q) @ np.abs(k).T) + cap * 2.0 ** -21 + 4 * EPS * abs(slope) * dist + 4 * EPS * zmax[:, None]
    # what a row's weights may be off by relatively: the errors of the keys that count, as their weights have them, and the
    # largest of those with a weight that bf16 notices
    e = np.where(see & (r["P"] > 2.0 ** -30), s_err, 0.0).max(1, initial=0.0)
    rel = 2 * e + 2.0 ** -21 + n * EPS
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0.0)
    size = r["P"] @ np.abs(v)
    big = np.abs(v).max(initial=0.0)
    tol = {"out": BF * np.abs(r["out"]) + size * (BF * 1.01 + rel[:, None]) + n * 2.0 ** -29 * big + 1e-30,
           "lse": rel + 2.0 ** -21 * np.abs(lse) + 1e-6}
    if do is not None:
        ado = np.abs(f64(do))
        dD = (ado * tol["out"]).sum(1) + d * EPS * (ado * np.abs(r["out"])).sum(1)
        aw = np.abs(r["dP"] - r["D"][:, None])
        # the cap's derivative 1 - t^2: t is off by 2^-20
        dx = r["P"] * (aw * (r["g"] * (BF * 1.02 + rel[:, None]) + 2.0 ** -19 * (cap > 0))
                       + r["g"] * (dD[:, None] + d * EPS * (ado @ np.abs(v).T)))
        full = r["P"] * aw * r["g"]
        tol["dq"] = scale * ((dx + n * EPS * full) @ np.abs(k)) + BF * np.abs(r["dq"]) + 1e-30
        tol["dk"] = scale * ((dx + len(gq) * EPS * full).T @ np.abs(q))
        tol["dv"] = (r["P"] * (BF * 1.01 + rel[:, None] + len(gq) * EPS)).T @ ado
    r["tol"] = tol
    return r


def expect(q, k, v, do, scale, cap, slopes, causal, prefix, cu=None):
    """Per name (value, bound) of (b, h, s, d) tensors in original order; with cu: b = 1, packed sequences."""
    q, k, v = f64(q), f64(k), f64(v)
    do = None if do is None else f64(do)
    b, h, s, d = q.shape
    hk = k.shape[1]
    names = ["out", "lse"] + (["dq", "dk", "dv"] if do is not None else [])
    shape = {"out": q.shape, "lse": (b, h, s), "dq": q.shape, "dk": k.shape, "dv": v.shape}
    val, tol = ({n: np.zeros(shape[n]) for n in names} for _ in range(2))
    ends = [0, s] if cu is None else [int(c) for c in cu]
    for n in range(b):
        for i, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
            if lo == hi:
                continue
            t = np.arange(hi - lo)
            pre = 0 if prefix is None else int(prefix[n if cu is None else i])
            for a in range(h):
                c = a // (h // hk)
                r = head_bounds(q[n, a, lo:hi], k[n, c, lo:hi], v[n, c, lo:hi], t, t, scale, cap,
                                0.0 if slopes is None else float(slopes[a]), causal, pre,
                                None if do is None else do[n, a, lo:hi])
                for name in names:
                    at = (n, c if name in ("dk", "dv") else a, slice(lo, hi))
                    val[name][at] += r[name]
                    tol[name][at] += r["tol"][name]
    for name in ("dk", "dv"):
        if name in val:
            tol[name] += BF * np.abs(val[name]) + 1e-30
    return {n: (val[n], tol[n]) for n in names}


def assert_within(name, got, want):
    ref, tol = want
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), f"{name}: infinite values differ"
    assert np.isfinite(got[fine]).all(), f"{name}: non-finite values"
    over = np.abs(got[fine] - ref[fine]) - tol[fine]
    assert over.size == 0 or over.max() <= 0, (f"{name}: {int((over > 0).sum())} of {over.size} beyond the bound, by "
                                               f"{over.max():.3e}")
    norm = np.linalg.norm(ref[fine])
    if norm > 0 and name != "lse":  # what the plain calls keep, too
        rel = np.linalg.norm(got[fine] - ref[fine]) / norm
        assert rel <= 5e-3, f"{name}: relative L2 {rel:.2e}"
