"""Plain forms in 64 bits of the adapter operators, and batches to try them on."""
import numpy as np
import torch

BF = torch.bfloat16


def segments(kind: str, M: int, S: int, n: int, rng):
    """seg_start [S + 1] and seg_adapter [S] of a batch.
    one: a single request; each: a row per request; ragged: random lengths, from
    three requests on with an empty one, one without adapter and one with an
    adapter past the pool; inside: ragged, and rows before the first request
    and after the last; outside: boundaries beyond the batch, which are clamped."""
    if kind == "one":
        start, ad = np.array([0, M]), np.array([int(rng.integers(n))])
    elif kind == "each":
        start, ad = np.arange(M + 1), rng.integers(0, n, M)
    else:
        lo, hi = (0, M) if kind != "inside" else (M // 5, M - M // 7)
        start = np.sort(rng.integers(lo, hi + 1, S + 1))
        if kind != "inside":
            start[0], start[-1] = lo, hi
        if kind == "outside":
            start[0], start[-1] = -9, M + 11
        ad = rng.integers(0, n, S)
        if S >= 3:
            start[2] = start[1]
            ad[2 % S] = -1
            ad[S - 1] = n + 3
    return start.astype(np.int32), ad.astype(np.int32)


def row_ids(start, ad, M: int, n: int) -> np.ndarray:
    ids = np.full(M, -1)
    for s, a in enumerate(ad):
        ids[max(0, start[s]):max(0, min(M, start[s + 1]))] = a if 0 <= a < n else -1
    return ids


class Batch:
    """Random pool, batch and activations; everything as torch tensors on the GPU."""

    def __init__(self, M, K, N, R, kind="ragged", S=5, n=3, seed=0, ranks=None):
        rng = np.random.default_rng(seed)
        self.M, self.K, self.N, self.R, self.n = M, K, N, R, n
        self.start, self.ad = segments(kind, M, S, n, rng)
        self.S = len(self.ad)
        self.ids = row_ids(self.start, self.ad, M, n)
        r = rng.integers(0, R + 1, n) if ranks is None else np.array(ranks)
        r[0] = R if ranks is None else r[0]
        self.r = r.astype(np.int32)
        self.sc = rng.uniform(0.25, 2.0, n).astype(np.float32)
        x = rng.standard_normal((M, K)).astype(np.float32)
        x[:, :max(1, K // 50)] *= 20
        a = rng.standard_normal((n, R, K)).astype(np.float32) / np.sqrt(K)
        b = rng.standard_normal((n, N, R)).astype(np.float32) * 0.1
        for i in range(n):  # what is past the rank must not matter
            a[i, r[i]:] = np.nan
            b[i, :, r[i]:] = np.inf
        cpu = lambda v: torch.from_numpy(v)  # noqa: E731
        self.x, self.a, self.b = (cpu(v).to(BF) for v in (x, a, b))
        self.rng = rng

    def pool(self):
        """(rank, scale, seg_start, seg_adapter) on the GPU."""
        return tuple(torch.from_numpy(v).cuda() for v in (self.r, self.sc, self.start, self.ad))

    def down(self):
        """t and its bound sum |x a| in 64 bits."""
        x = self.x.double().numpy()
        t, mag = np.zeros((self.M, self.R)), np.zeros((self.M, self.R))
        for i in range(self.n):
            rows, r = self.ids == i, self.r[i]
            a = self.a[i, :r].double().numpy()
            t[rows, :r] = x[rows] @ a.T
            mag[rows, :r] = np.abs(x[rows]) @ np.abs(a).T
        return t, mag

    def up(self, t):
        """scale * t b^T and sum |scale t b| in 64 bits."""
        d, mag = np.zeros((self.M, self.N)), np.zeros((self.M, self.N))
        for i in range(self.n):
            rows, r = self.ids == i, self.r[i]
            b = self.b[i, :, :r].double().numpy()
            s = float(self.sc[i])
            d[rows] = s * (t[rows, :r] @ b.T)
            mag[rows] = s * (np.abs(t[rows, :r]) @ np.abs(b).T)
        return d, mag

    def up_bound(self, t, tmag, mag):
        """How far scale * t b^T may be off: fp32 sums of K and R + a few terms
        (2^-24 a term of the sum of magnitudes, doubled for the order), and 16
        bits kept of t by the split (2^-17 of each product)."""
        d, dm = self.up(tmag)
        return mag * (2.0 ** -17 + (self.R + 8) * 2.0 ** -23) + dm * (self.K + 8) * 2.0 ** -23
