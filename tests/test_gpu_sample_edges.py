"""ssd_filter_probs and ssd_sample at edges of their settings, of the values in a row and of a cluster's life."""
import numpy as np
import pytest
import torch

from oracle import sample_oracle as Q
from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_sample import MIX, NEAR, RTOL, _check_row, _dev, _rows, _settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V", [(1, 40), (3, 1000), (7, 5003), (40, 257), (160, 3001), (2, 128256)])
def test_clusters_whose_ctas_start_at_different_times(R, V):
    """Short and long rows of clusters of one to eight CTAs, launched into a busy GPU: a CTA is handed its
    neighbours' largest values as soon as they have them, however late it started itself."""
    rng = np.random.default_rng(R + V)
    kw, _ = _settings([MIX[r % len(MIX)] for r in range(R)])
    x = _dev(_rows(rng, R, V), False)
    u = torch.from_numpy(rng.random(R).astype(np.float32)).cuda()
    want, ref = S.ssd_filter_probs(x, **kw), S.ssd_sample(x, u, **kw)
    a = torch.randn((2048, 2048), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(side):
            a = (a @ a).clamp_(-1, 1)
        got.append((S.ssd_filter_probs(x, **kw), S.ssd_sample(x, u, **kw)))
    torch.cuda.synchronize()
    for p, t in got:
        assert torch.equal(p, want) and torch.equal(t["token"], ref["token"]) and torch.equal(t["prob"], ref["prob"])


@pytest.mark.parametrize("V", [1, 7, 1000, 40000])
@pytest.mark.parametrize("k", [0, 5, 600, 3000])
def test_settings_that_are_no_number_cut_nothing(V, k):
    """NaN top-p and min-p (of either sign): as if they were not given; with top-k by the sorted list, by bins, and without it."""
    rng = np.random.default_rng(V + k)
    nan = float("nan")
    given = [(0.8, k, nan, nan), (0.8, k, 1.0, nan), (0.8, k, nan, 0.0), (0.8, k, 0.9, nan), (0.8, k, nan, 0.01), (0.8, k, 1.0, -nan), (0.0, k, nan, nan)]
    alike = [(t, k, 1.0 if p != p else p, 0.0 if m != m else m) for t, k, p, m in given]
    kw, _ = _settings(given)
    plain, ora = _settings(alike)
    x = _dev(np.repeat(_rows(rng, 1, V), len(given), 0), False)
    u = torch.full((len(given),), 0.6875, device="cuda")
    got, want = S.ssd_filter_probs(x, **kw), S.ssd_filter_probs(x, **plain)
    assert torch.equal(got, want)
    a, b = S.ssd_sample(x, u, **kw), S.ssd_sample(x, u, **plain)
    assert torch.equal(a["token"], b["token"]) and torch.equal(a["prob"], b["prob"])
    z = x.cpu().numpy()
    assert sum(_check_row(got[r].cpu().double().numpy(), z[r], ora[r]) for r in range(len(ora))) >= len(ora) - 1


def _runs_of_inf(V, n, at, rest, rng):
    """A row with n infinities side by side from `at` on, and a NaN before and behind them."""
    z = np.full(V, -np.inf, np.float32)
    if rest == "some":
        z[rng.integers(0, V, max(1, V // 50))] = 1.5
    elif rest == "all":
        z = rng.standard_normal(V).astype(np.float32)
    z[at:at + n] = np.inf
    z[max(at - 1, 0):at] = np.nan
    z[at + n:at + n + 1] = np.nan
    return z


# top-k below, at and above the number of infinities, of live tokens, of lists and of tokens; greedy; the other cuts beside it
INF_SETTINGS = [(1.0, 3, 1.0, 0.0), (1.0, 5, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (1.0, 600, 1.0, 0.5), (1.3, 2000, 0.7, 0.0), (0.0, 0, 1.0, 0.0), (0.0, 7, 0.5, 0.1),
                (1.0, 0, 0.6, 0.0), (1.0, 0, 1.0, 0.3), (1e-3, 5, 1.0, 0.0), (1e20, 9, 1.0, 0.0), (1.0, 0, 1.0, 0.0)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rest", ["none", "some", "all"])
@pytest.mark.parametrize("V,n,at", [(8, 4, 0), (8, 8, 0), (9, 4, 4), (30, 8, 8), (30, 5, 3), (1000, 4, 512), (1000, 8, 41), (5003, 16, 4096), (40000, 8, 39992), (40000, 1200, 20000),
                                    (600001, 4, 300000)])
def test_runs_of_infinities(V, n, at, rest, bf16):
    """+inf counts as the largest finite number wherever it stands: whole vectors of it, with NaN beside, too."""
    rng = np.random.default_rng(V + n)
    rows = [s for s in INF_SETTINGS if s[1] <= V]
    z = np.stack([_runs_of_inf(V, n, at, rest, rng) for _ in rows])
    kw, ora = _settings(rows)
    x = _dev(z, bf16)
    z = x.float().cpu().numpy()
    u = ((np.arange(len(rows)) * 5 % 16 + 0.37) / 16).astype(np.float32)
    full = torch.full((len(rows), V), 7.0, device="cuda")
    out = dict(token=torch.full((len(rows),), -5, dtype=torch.int32, device="cuda"), prob=torch.full((len(rows),), -5.0, device="cuda"))
    S.ssd_sample(x, torch.from_numpy(u).cuda(), **kw, out=out, probs_out=full)
    assert torch.equal(full, S.ssd_filter_probs(x, **kw))
    p, tok, prob = full.cpu().double().numpy(), out["token"].cpu().numpy(), out["prob"].cpu().numpy()
    compared = 0
    for r in range(len(rows)):
        if not _check_row(p[r], z[r], ora[r]):
            continue
        want, _, gap = Q.token(z[r], u[r], **ora[r])
        if gap >= NEAR:
            compared += 1
            assert tok[r] == want and prob[r] == p[r, want], (rows[r], tok[r], want)
    assert compared >= len(rows) - 2


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [3, 64, 5000])
def test_smallest_temperatures(V, bf16):
    """A temperature between 0 and log2(e) 2^-120 counts as that in every cut, also in what top-p looks at."""
    least = float(np.log2(np.e)) * 2.0 ** -120
    rows = [(t, k, p, m) for t in (1e-45, 1e-40, 1e-37, 1.0853631e-36) for k, p, m in ((0, 0.9, 0.0), (0, 0.3, 0.0), (2, 0.9, 0.0), (2000, 0.8, 0.0), (0, 1.0, 0.2), (0, 0.999, 0.0))]
    rng = np.random.default_rng(V)
    z = -(np.arange(V) * 1e-37 * 64 / V) + rng.integers(0, 3, V) * 1e-38
    x = _dev(np.repeat(rng.permutation(z)[None].astype(np.float32), len(rows), 0), bf16)
    kw, ora = _settings(rows)
    u = torch.full((len(rows),), 0.40625, device="cuda")
    got, tok = S.ssd_filter_probs(x, **kw), S.ssd_sample(x, u, **kw)["token"].cpu().numpy()
    z = x.float().cpu().numpy()
    compared = 0
    for r, o in enumerate(ora):
        o["temperature"] = least
        if not _check_row(got[r].cpu().double().numpy(), z[r], o):
            continue
        compared += 1
        want, _, gap = Q.token(z[r], 0.40625, **o)
        assert gap < NEAR or tok[r] == want
    assert compared >= len(rows) - 2


@pytest.mark.parametrize("V", [1 << 20, 128256, 5003])
@pytest.mark.parametrize("units", [0.3, 0.55, 1.1, 1.45, 2.6, 700.0])
def test_cuts_in_a_long_tail_of_small_weights(V, units):
    """One token and V - 1 equal ones whose weight is `units` of 2^-43, to which sums round it: what stays ends
    within the documented distance of the border, 2^-28 top_p sum + V 2^-43, and no further."""
    ps = [1 - 2.0 ** -24, 1 - 2.0 ** -22, 1 - 2.0 ** -18, 0.999, 0.5]
    z = np.full((len(ps), V), np.log(units * 2.0 ** -43), np.float32)
    z[:, V // 3] = 0.0
    kw, _ = _settings([(1.0, 0, p, 0.0) for p in ps])
    got = S.ssd_filter_probs(torch.from_numpy(z).cuda(), **kw).cpu().double().numpy()
    w = float(np.exp(np.float64(z[0, 0])))
    total = 1 + (V - 1) * w
    for r, p in enumerate(ps):
        n = int((got[r] > 0).sum())
        target, off = p * total, 2.0 ** -28 * p * total + V * 2.0 ** -43
        before = lambda j: 0.0 if j == 0 else 1 + (j - 1) * w  # noqa: B023  (of the token at place j)
        assert n >= 1 and got[r, V // 3] > 0
        assert n == 1 or before(n - 1) < target + off
        assert n == V or before(n) >= target - off
        # equal tokens by their index, and the probabilities those of what stays
        first = np.flatnonzero(got[r] > 0)
        assert (np.delete(np.arange(V), V // 3)[:n - 1] == first[first != V // 3]).all()
        sum_ = 1 + (n - 1) * w
        np.testing.assert_allclose(got[r, first], np.where(first == V // 3, 1.0, w) / sum_, rtol=RTOL + V * 2.0 ** -44)


@pytest.mark.parametrize("k", [0, 3, 5000])
def test_min_p_above_one_counts_as_one(k):
    z = torch.randn((3, 6000), device="cuda").clamp_(max=2.0)
    z[:, [7, 100, 4444, 5999]] = 2.5
    m = torch.tensor([1.0, 2.0, float("inf")], device="cuda")
    got = S.ssd_filter_probs(z, top_k=torch.full((3,), k, dtype=torch.int32, device="cuda"), min_p=m)
    for r in range(3):
        assert (got[r] > 0).nonzero()[:, 0].tolist() == [7, 100, 4444, 5999][:k or None]
