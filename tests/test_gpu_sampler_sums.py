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


def in_batches(q, x, row, settings, batches):
    """Case i is row `row[i]` of x with the i-th settings; the cases in calls of M rows each, for all M of `batches`:
    equal in all of them. Returns the first one's tokens and probabilities."""
    d, row, n, first = x.to(DEV), torch.tensor(row), len(row), None
    t = {k: torch.tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32) for k, v in settings.items()}
    for M in batches:
        tokens, probs = [], []
        for i in range(0, n, M):
            at = torch.arange(i, i + M) % n
            a, b = q.sample_logits(d[row[at].to(DEV)], **{k: v[at].to(DEV) for k, v in t.items()})
            keep = min(M, n - i)
            tokens.append(a[:keep].cpu().numpy()), probs.append(b[:keep].cpu().numpy())
        got = np.concatenate(tokens), np.concatenate(probs)
        first = first or got
        assert np.array_equal(got[0], first[0]), (M, np.nonzero(got[0] != first[0])[0][:5])
        assert np.array_equal(got[1].view(np.int32), first[1].view(np.int32)), \
            (M, np.nonzero(got[1] != first[1])[0][:5], got[1][got[1] != first[1]][:3], first[1][got[1] != first[1]][:3])
    return first


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_p_over_a_bulk_of_one_value(q, dtype):
    """700 tokens above a bulk that has about half of the mass; top-p ends among the first ones, next to a border."""
    rng = np.random.default_rng(11)
    V, x, rows = 151936, [], []
    for i in range(12):
        y = np.full(V, -5.2 - 0.11 * i)
        y[rng.choice(V, 700, replace=False)] = 0.5 - rng.random(700) * 2.5
        x.append(torch.from_numpy(y).to(dtype))
        rows.append(Ranked(x[-1].float().numpy()))
    row, u, p = [], [], []
    for i, r in enumerate(rows):
        for j, f in enumerate((-10, -5, -2.5, -1.25, 1.25, 2.5, 5, 10)):
            n = 60 + 9 * j + i
            while r.x[r.order[n]] == r.x[r.order[n - 1]] and n < 300:  # (bf16: to the end of equal ones)
                n += 1
            row.append(i), u.append(LAST_U), p.append(np.float32(r.C[n - 1] / r.C[-1] + f * EPS))
    tokens, probs = in_batches(q, torch.stack(x), row, dict(u=u, top_p=p), (96, 8, 32, 512))
    for i in range(len(row)):
        rows[row[i]].check(u[i], p[i], int(tokens[i]), float(probs[i]))


def test_top_p_near_one(q):
    """250 tokens have all but 3.5 to 4 * 2^-22 of the mass, some hundred more a little, a bulk of one value the rest: what
    the definition keeps of it is drawn."""
    rng = np.random.default_rng(12)
    V, x, rows = 50021, [], []
    for i in range(6):
        at = rng.permutation(V)
        y = np.empty(V)
        y[at[:250]] = -17 * rng.random(250)
        y[at[0]] = 0.0
        y[at[250:850]] = -20.5 - rng.random(600)
        y[at[850:]] = np.log(np.exp(y[at[:250]]).sum() * (3.55 + 0.06 * i) * EPS / (V - 850))
        x.append(torch.from_numpy(y).float())
        rows.append(Ranked(x[-1].numpy()))
    row, u, p = [], [], []
    for i in range(6):
        for top_p in (1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -22, 1 - 2.0 ** -21, 1 - 2.0 ** -20, 1 - 2.0 ** -18):
            for v in (LAST_U, 1 - 2.0 ** -22, 0.5):
                row.append(i), u.append(v), p.append(top_p)
    tokens, probs = in_batches(q, torch.stack(x), row, dict(u=u, top_p=p), (108, 6, 32, 512))
    for i in range(len(row)):
        rows[row[i]].check(u[i], p[i], int(tokens[i]), float(probs[i]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature,gap", [(8.0, 25.0), (64.0, 40.0), (3.9, 45.0)])
def test_a_bulk_below_the_bins(q, dtype, temperature, gap):
    """One token far above a bulk of one value, hot rows: most of the mass lies below the bins."""
    V, x, rows = 151936, [], []
    for i in range(4):
        y = torch.full((V,), -gap - 0.37 * i).to(dtype)
        y[77 + i] = 1.0
        x.append(y)
        rows.append(Ranked(y.float().numpy(), temperature))
    row, u, p = [], [], []
    for i in range(4):
        for k, v in enumerate((1e-5, 0.3, 0.71, LAST_U)):
            row.append(i), u.append(v), p.append((1.0, 0.9, 1 - 2.0 ** -22)[(i + k) % 3])
    T = [temperature] * len(row)
    tokens, probs = in_batches(q, torch.stack(x), row, dict(u=u, top_p=p, temperature=T), (16, 3, 32, 160))
    for i in range(len(row)):
        rows[row[i]].check(u[i], p[i], int(tokens[i]), float(probs[i]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [20001, 151936])
def test_a_row_gives_the_same_in_every_batch(q, V, dtype):
    """All settings; rows of few values, where cuts end among thousands of nearly equal tokens, among them."""
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((24, V)) * rng.choice([0.5, 2.0, 4.0], (24, 1)))
    for i in range(0, 24, 3):
        x[i] = (x[i] * 3).round() / 3 + 1e-4 * torch.from_numpy(rng.standard_normal(V))
    x[1::4, rng.choice(V, 150, replace=False)] += 8
    n = 192
    settings = dict(u=rng.random(n), temperature=rng.choice([0.4, 0.8, 1.0, 1.7, 20.0], n),
                    top_k=rng.choice([0, 0, 20, 300, 500, 3000], n), top_p=rng.choice([1.0, 0.5, 0.9, 0.99, 0.999], n),
                    min_p=rng.choice([0.0, 0.0, 0.05, 1e-3], n))
    row = [i % 24 for i in range(n)]
    tokens, probs = in_batches(q, x.to(dtype), row, settings, (n, 1, 32, 100, 600))
    f32 = x.to(dtype).float().numpy()
    for i in range(0, n, 5):
        own = {k: (int(v[i]) if k == "top_k" else np.float32(v[i])) for k, v in settings.items()}
        u = own.pop("u")
        order, C, kept, at = od.sample(f32[row[i]], u, **own)
        if order[at] == tokens[i]:  # (borders within EPS are the other tests')
            want = np.exp((float(f32[row[i]][order[at]]) - float(f32[row[i]][order[0]])) / float(own["temperature"])) / C[kept - 1]
            assert abs(probs[i] - want) <= 2.0 ** -21 * want or own["top_p"] < 1, (i, own, probs[i], want)


@pytest.mark.parametrize("M,V,dtype", [
    (160, 170001, torch.bfloat16), (160, 180000, torch.bfloat16), (160, 180000, torch.float32), (170, 180001, torch.bfloat16),
    (48, 151936, torch.float32), (100, 151936, torch.float32), (139, 151936, torch.bfloat16), (64, 262147, torch.float32),
    (21, 393216, torch.float32)])
def test_launch_forms(q, M, V, dtype):
    """Rows of one value; rows that all lie at one or the other end of one bin (the largest sums of deviations); masked
    rows of fewer tokens than top-k; ordinary ones. Clusters in waves and CTAs per row, at the widest rows of each."""
    rng = np.random.default_rng(M + V)
    kinds = torch.empty((8, V), dtype=torch.float64)
    kinds[0] = 1.25
    kinds[1] = -(300 + 0.4998) / (64 * 1.4426950408889634)
    kinds[2] = -(300 - 0.4998) / (64 * 1.4426950408889634)
    kinds[1:3, 5] = 0.0
    kinds[3] = float("-inf")
    kinds[3, rng.choice(V, 7, replace=False)] = torch.from_numpy(rng.standard_normal(7))
    kinds[4:] = torch.from_numpy(rng.standard_normal((4, V)) * 2)
    kinds[5, rng.choice(V, 100, replace=False)] += 9
    kinds = kinds.to(dtype)
    u, p = rng.random(M), np.where(np.arange(M) // 8 % 2, 0.9, 1.0)
    k = np.where(np.arange(M) % 8 == 3, 50, 0)
    got = []
    for top_k in (None, torch.from_numpy(k).to(DEV)):
        a, b = q.sample_logits(kinds[torch.arange(M) % 8].to(DEV), torch.from_numpy(u).float().to(DEV), top_k=top_k,
                               top_p=torch.from_numpy(p).float().to(DEV))
        got.append((a.cpu().numpy(), b.cpu().numpy()))
    assert all(np.array_equal(x, y) for x, y in zip(*got))
    rows = [Ranked(y.float().numpy()) for y in kinds]
    for m in list(range(min(M, 16))) + list(range(max(16, M - 16), M)):
        rows[m % 8].check(u[m], p[m], int(got[0][0][m]), float(got[0][1][m]))


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
