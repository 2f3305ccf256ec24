"""A paged 4-bit cache with its sequences, for the cache tests: device tensors and
the oracle's numbers for them."""
import numpy as np
import torch

from oracle import cache as oc


class Case:
    """n_new[i] new tokens of sequence i, kv[i] tokens in its cache after them.

    order: memory order of the cache's (page, head, row) dimensions.  Pages are
    taken from the pool in random order; every byte that no token owns holds
    0xff (a NaN scale)."""

    def __init__(self, n_new, kv, h, hk, d, page, seed=0, order=(0, 1, 2), pad_rows=0, spare=2):
        self.n_new, self.kv, self.h, self.hk, self.d, self.page = list(n_new), list(kv), h, hk, d, page
        self.rng = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + pad_rows
        need = [-(-max(m, 0) // page) for m in kv]
        self.n_pages, width = sum(need) + spare, max(max(need), 1)
        ids = self.rng.permutation(self.n_pages)
        self.table = np.full((len(kv), width), -7, dtype=np.int32)  # entries past the length: not a page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.shape = (self.n_pages, hk, page)
        self.order = order
        self.page_table = torch.tensor(self.table, device="cuda")
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device="cuda")

    def _alloc(self, fill, width):
        dims = [self.shape[i] for i in self.order]
        back = [self.order.index(i) for i in range(3)]
        return torch.full((*dims, width), fill, dtype=torch.uint8, device="cuda").permute(*back, 3)

    def cache(self, ra):
        a = [self._alloc(0xff, w) for w in (self.d // 2, self.d // 16) * 2]
        self.bytes = a
        return ra.KVCache(a[0], a[1].view(torch.float8_e4m3fn), a[2], a[3].view(torch.float8_e4m3fn))

    def where(self, i, lo, hi):
        """Physical (pages, rows) of tokens [lo, hi) of sequence i."""
        t = np.arange(lo, hi)
        return self.table[i, t // self.page], t % self.page

    def fill(self, ra, k=None, v=None):
        """A cache that holds quantised random keys and values; self.k[i], self.v[i]: their values (fp64)."""
        cache = self.cache(ra)
        host = [x.cpu().numpy() for x in self.bytes]
        self.k, self.v = [], []
        for i, m in enumerate(self.kv):
            gain = np.exp(0.5 * self.rng.standard_normal((self.hk, self.d)))
            for j, (x, keep) in enumerate(((self.rng.standard_normal((max(m, 0), self.hk, self.d)) * gain, self.k),
                                           (self.rng.standard_normal((max(m, 0), self.hk, self.d)), self.v))):
                codes, scales = oc.quantise(x)
                pg, row = self.where(i, 0, max(m, 0))
                host[2 * j][pg, :, row], host[2 * j + 1][pg, :, row] = codes, scales
                keep.append(oc.dequantise(codes, scales))
        for x, y in zip(self.bytes, host):
            x.copy_(torch.from_numpy(y))
        return cache

    def queries(self, gain=1.0):
        return (torch.tensor(self.rng.standard_normal((self.rows, self.h, self.d)) * gain)).bfloat16().cuda()

    def expect(self, q, causal, scale=None):
        """(out, lse, tol_out, tol_lse) over rows [0, cu[-1]).

        Bounds.  Scores: the products of bf16 and 6-bit numbers are exact, their d-term fp32
        sums are off by at most d 2^-24 sum|q k|, and exp carries that into p relatively
        (2 d 2^-24: the maximum is off as well).  p is rounded to fp16: half a step, 2^-11,
        and below fp16's normal range by 2^-25 absolutely, with p's largest at least 2^4.  Sums of
        m terms: m 2^-24.  out is rounded to bf16: 2^-8.  The exponential is good to 2^-21."""
        scale = self.d ** -0.5 if scale is None else scale
        total = int(self.cu[-1])
        out, lse = np.zeros((total, self.h, self.d)), np.zeros((self.h, total))
        to, tl = np.zeros_like(out), np.zeros_like(lse)
        qf = q.float().cpu().numpy().astype(np.float64)
        for i, (n, m) in enumerate(zip(self.n_new, self.kv)):
            r = slice(self.cu[i], self.cu[i + 1])
            before = m - n + 1 + np.arange(n) if causal else np.full(n, m)
            o, ls, size, dots = oc.attention(qf[r], self.k[i], self.v[i], scale, np.clip(before, 0, max(m, 0)))
            out[r], lse[:, r] = o, ls
            s_err = 2 * self.d * 2.0 ** -24 * dots.T[..., None] + 2.0 ** -21 + max(m, 1) * 2.0 ** -24
            big = np.abs(self.v[i]).max(initial=0.0)
            to[r] = 2.0 ** -8 * np.abs(o) + size * (2.0 ** -11 * 1.01 + s_err) + max(m, 1) * 2.0 ** -29 * big + 1e-30
            tl[:, r] = s_err[..., 0].T + 2.0 ** -22 * np.abs(np.where(np.isfinite(ls), ls, 0.0)) + 1e-6
        return out, lse, to, tl


def assert_within(name, got, ref, tol):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), f"{name}: infinite values differ"
    assert np.isfinite(got[fine]).all(), f"{name}: non-finite values"
    over = np.abs(got[fine] - ref[fine]) - tol[fine]
    assert over.size == 0 or over.max() <= 0, f"{name}: {int((over > 0).sum())} of {over.size} beyond the bound, by {over.max():.3e}"
