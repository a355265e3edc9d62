"""The sampler's sums, where their rounding could be seen: totals of many equal
weights, cuts that end near the whole, rows whose bulk lies below the bins. The
same row has to give the same token and the same probability, bit for bit, in
every form that a call may be launched in (clusters that hold the rows, clusters
in several waves, a CTA per row of 512 or 1024 threads).

Tolerances are the header's: with C the sum of what a cut or the draw goes by, a
token is the definition's, or the one across a border within 2^-22 C (EPS); its
probability within 2^-21 of itself: two such sums and the fp32 result.
"""
import numpy as np
import pytest
import torch

from oracle import decode as od

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 2.0 ** -22
LAST_U = 1 - 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_qgemv_gb300 import build
    build.build()
    import skinny_gemm_qgemv_gb300 as qq
    qq.lib()
    qq.device_error(clear=True)
    yield qq
    assert qq.device_error(clear=True) == 0


class Ranked:
    """A row's order and summed weights, for many settings."""

    def __init__(self, x, temperature=1.0):
        self.order, self.C, _, _ = od.sample(x, 0.0, temperature)
        self.rank = np.empty(len(x), np.int64)
        self.rank[self.order] = np.arange(len(self.order))
        self.w = np.diff(self.C, prepend=0.0)
        self.x, self.T = np.asarray(x, np.float64), float(temperature)

    def kept(self, p):
        return len(self.C) if p >= 1 else int((self.C < p * self.C[-1]).sum()) + 1

    def check(self, u, p, token, prob):
        u, p, j, ok = float(np.float32(u)), float(np.float32(p)), self.rank[token], False
        weight = np.exp((self.x[token] - self.x[self.order[0]]) / self.T)
        for n in {self.kept(p)} | ({self.kept(p * (1 + f) + f) for f in (EPS, -EPS)} if p < 1 else set()):
            n = min(max(n, 1), len(self.C))
            lo, hi = (min(int((self.C[:n] <= (u + f) * self.C[n - 1]).sum()), n - 1) for f in (-EPS, EPS))
            want = weight / self.C[n - 1]
            ok |= lo <= j <= hi and abs(prob - want) <= 2.0 ** -21 * want + 2.0 ** -149
        assert ok, (u, p, token, prob, int(j), self.kept(p), self.order[min(self.kept(p), len(self.C)) - 1])


def test_temperatures_just_above_one(q):
    """A few tokens far above a broad bulk that has some of the mass: 22 logits below the maximum are within the bins at
    any temperature, and a temperature of 1.2 takes about as long as one of 0.99 (a row that ends below them takes twenty
    times as long)."""
    rng = np.random.default_rng(14)
    M, V = 152, 151936
    x = torch.from_numpy(rng.standard_normal((8, V)) * 2).float()
    x[:, :200] = 15 - 1.3 * torch.arange(1, 201).log()
    d, times = x[torch.arange(M) % 8].to(DEV), []
    u, p = rng.random(M), np.full(M, 0.95)
    for T in (0.99, 1.2):
        args = [torch.full((M,), v, device=DEV) for v in (T, 0.95)]
        du = torch.from_numpy(u).float().to(DEV)
        a, b = q.sample_logits(d, du, temperature=args[0], top_p=args[1])
        took = []
        for _ in range(7):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(5):
                q.sample_logits(d, du, temperature=args[0], top_p=args[1])
            end.record()
            end.synchronize()
            took.append(start.elapsed_time(end))
        times.append(sorted(took)[3])
        rows = [Ranked(y.numpy(), np.float32(T)) for y in x]
        for m in range(24):
            rows[m % 8].check(u[m], p[m], int(a[m]), float(b[m]))
    assert times[1] < 5 * times[0], times
