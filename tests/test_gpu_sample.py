"""ssd_filter_probs and ssd_sample against the fp64 oracle: cuts, ties, masks, types, strides and
lengths from one token to rows beyond a cluster's shared memory.

Tolerance of a probability: its weight and the sum are off by 2^-29 relative each, the fp32 number
that holds it by 2^-24 (one rounding; the products before it are carried as pairs): 2^-23.9 with
2^-126 for numbers that fp32 holds no better. Which tokens stay is compared where no border of a cut
lies within 2^-27 of the sum it compares (the inputs are drawn; a row that fails this is counted
and has to be rare)."""
import numpy as np
import pytest
import torch

from oracle import sample_oracle as Q
from speculative_decoding_copy_gb300 import _binding as S

pytestmark = pytest.mark.gpu
RTOL = 2.0 ** -23.9
NEAR = 2.0 ** -27


def _rows(rng, R, V, std=2.5, heads=20):
    z = rng.standard_normal((R, V)) * std
    for r in range(R):
        at = rng.integers(0, V, min(heads, V))
        z[r, at] += rng.uniform(2, 12) / np.arange(1, len(at) + 1) ** 0.3
    return z.astype(np.float32)


def _dev(z, bf16):
    t = torch.from_numpy(np.ascontiguousarray(z)).cuda()
    return t.to(torch.bfloat16) if bf16 else t


def _settings(rows):
    """[(temperature, top_k, top_p, min_p)] -> keyword tensors, and the oracle's keywords."""
    t, k, p, m = zip(*rows)
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")
    kw = dict(temperature=f(t), top_k=torch.tensor(k, dtype=torch.int32, device="cuda"), top_p=f(p), min_p=f(m))
    ora = [dict(temperature=float(np.float32(a)), top_k=b, top_p=float(np.float32(c)), min_p=float(np.float32(d))) for a, b, c, d in rows]
    return kw, ora


def _check_row(got, z, setting):
    """True where the row could be compared (no border too near)."""
    at, w, near = Q.kept(z, **setting)
    if near < NEAR:
        return False
    want = Q.probs(z, **setting)
    np.testing.assert_allclose(got, want, rtol=RTOL, atol=2.0 ** -126)
    # what was cut is zero exactly
    cut = np.ones(len(z), bool)
    cut[at] = False
    assert not got[cut].any()
    return True


MIX = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (0.8, 20, 0.95, 0.0), (1.0, 0, 1.0, 0.1), (0.6, 1000, 0.8, 0.02),
       (0.0, 5, 0.5, 0.5), (1.0, 1, 1.0, 0.0), (2.0, 7, 0.3, 0.9), (1e-3, 0, 0.99, 0.0), (1.0, 0, 1e-6, 0.0), (1e4, 0, 0.999, 0.0)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 257, 1000, 4097, 32000, 50257])
def test_filter_lengths_types_and_settings(V, bf16):
    rng = np.random.default_rng(V)
    kw, ora = _settings(MIX)
    x = _dev(_rows(rng, len(MIX), V), bf16)
    got = S.ssd_filter_probs(x, **kw).cpu().double().numpy()
    z = x.float().cpu().numpy()
    ok = [_check_row(got[r], z[r], ora[r]) for r in range(len(MIX))]
    assert sum(ok) >= len(ok) - 1


@pytest.mark.parametrize("V,bf16,R", [(128256, False, 5), (151936, True, 12), (128257, True, 3), (128255, False, 40), (600001, False, 2), (1 << 20, False, 2),
                                      (1 << 20, True, 2)])
def test_filter_vocabularies(V, bf16, R):
    """Whole vocabularies, odd rows, many rows (other cluster sizes), rows beyond shared memory."""
    rng = np.random.default_rng(V + R)
    kw, ora = _settings([MIX[(r * 5 + 2) % len(MIX)] for r in range(R)])
    x = _dev(_rows(rng, R, V), bf16)
    got = S.ssd_filter_probs(x, **kw).cpu().double().numpy()
    z = x.float().cpu().numpy()
    ok = [_check_row(got[r], z[r], ora[r]) for r in range(R)]
    assert sum(ok) >= len(ok) - 1


def _special(kind, V, rng):
    z = rng.standard_normal(V).astype(np.float32)
    if kind == "equal":
        z[:] = 3.25
    elif kind == "two values":
        z = np.where(rng.random(V) < 0.3, 1.0, 0.0).astype(np.float32)
    elif kind == "zeros of both signs":
        z = np.where(rng.random(V) < 0.5, 0.0, -0.0).astype(np.float32)
        z[rng.integers(0, V, V // 4)] = -1.0
    elif kind == "inf":
        z[rng.random(V) < 0.9] = -np.inf
        z[[V // 3, V // 2]] = np.inf
    elif kind == "nan":
        z[rng.random(V) < 0.5] = np.nan
    elif kind == "lowest":
        z[rng.random(V) < 0.9] = np.finfo(np.float32).min
    elif kind == "all lowest":
        z[:] = np.finfo(np.float32).min
    elif kind == "nothing":
        z[:] = np.where(rng.random(V) < 0.5, -np.inf, np.nan)
    elif kind == "one":
        z[:] = -np.inf
        z[V - 1] = -5.0
    elif kind == "huge":
        z = (z * 1e38).astype(np.float32)
    elif kind == "tiny":
        z = (z * 1e-40).astype(np.float32)
    elif kind == "last":
        z[V - 1] = 50.0
    elif kind == "ascending":
        z = (np.arange(V) * 1e-3).astype(np.float32)
    return z


KINDS = ["equal", "two values", "zeros of both signs", "inf", "nan", "lowest", "all lowest", "nothing", "one", "huge", "tiny", "last", "ascending"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [9, 1021, 40000])
def test_filter_rows_that_are_unlike_logits(kind, V):
    rng = np.random.default_rng(7)
    z = np.stack([_special(kind, V, rng) for _ in MIX])
    # fewer tokens than top-k asks for, and cuts inside a run of equal ones
    rows = [(t, min(k, V // 2 + 1) if k else 0, p, m) for t, k, p, m in MIX]
    kw, ora = _settings(rows)
    got = S.ssd_filter_probs(torch.from_numpy(z).cuda(), **kw).cpu().double().numpy()
    assert np.isfinite(got).all()
    ok = [_check_row(got[r], z[r], ora[r]) for r in range(len(rows))]
    assert sum(ok) >= (len(ok) - 2 if kind in ("equal", "two values", "zeros of both signs", "inf", "all lowest") else len(ok) - 1)


@pytest.mark.parametrize("n,p,kept", [(4, 0.5, 2), (10, 0.7, 7), (8, 0.875, 7), (1000, 0.5, 500), (4096, 0.25, 1024)])
def test_top_p_at_an_exact_border(n, p, kept):
    """n equal tokens: the sum before the j-th is j / n exactly, compared with the fp32 number top_p."""
    z = torch.full((1, n + 5), float("-inf"), device="cuda")
    z[0, 3:3 + n] = -2.5
    got = S.ssd_filter_probs(z, top_p=torch.tensor([p], device="cuda"))[0].cpu().numpy()
    want = int((np.arange(n) / n < float(np.float32(p))).sum())
    assert want == kept or abs(want - kept) == 1
    assert (got > 0).sum() == want and (got[3:3 + want] > 0).all()


def test_settings_serve_runs_of_rows_and_missing_ones_mean_all():
    rng = np.random.default_rng(3)
    z = _rows(rng, 12, 2000)
    x = torch.from_numpy(z).cuda()
    k = torch.tensor([3, 0, 11], dtype=torch.int32, device="cuda")
    got = S.ssd_filter_probs(x, top_k=k).cpu().numpy()
    assert [(got[r] > 0).sum() for r in range(12)] == [3] * 4 + [2000] * 4 + [11] * 4
    flat = S.ssd_filter_probs(x.view(3, 4, 2000), top_k=k)
    assert flat.shape == (3, 4, 2000) and np.array_equal(flat.cpu().numpy().reshape(12, 2000), got)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 3, 64])
def test_row_strides_and_neighbours(pad, bf16):
    """Rows of a wider buffer: the columns behind a row are not part of it, and an output between
    others leaves those as they were."""
    rng = np.random.default_rng(pad)
    V, R = 5003, 6
    wide = _rows(rng, R, V + pad)
    wide[:, V:] = 100.0
    x = _dev(wide, bf16)[:, :V]
    kw, ora = _settings(MIX[:R])
    buf = torch.full((R * V + 64,), -7.0, device="cuda")
    out = buf[32:32 + R * V].view(R, V)
    S.ssd_filter_probs(x, **kw, out=out)
    z = x.float().cpu().numpy()
    assert sum(_check_row(out[r].cpu().double().numpy(), z[r], ora[r]) for r in range(R)) >= R - 1
    assert (buf[:32] == -7).all() and (buf[32 + R * V:] == -7).all()


def test_rows_of_absent_tokens_stay_as_they_were():
    rng = np.random.default_rng(5)
    B, NB, Dmax, V = 3, 3, 4, 1500
    x = torch.from_numpy(_rows(rng, B * (1 + NB * Dmax), V)).cuda().view(B, 1 + NB * Dmax, V)
    blk = torch.tensor([[4, 0, 2], [0, 0, 0], [1, 3, 4]], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, -3.0)
    full = S.ssd_filter_probs(x)
    for b in range(B):
        for k in range(NB):
            x[b, 1 + k * Dmax + int(blk[b, k]):1 + (k + 1) * Dmax] = float("nan")      # never looked at
    S.ssd_filter_probs(x, blk_len=blk, Dmax=Dmax, out=out)
    for b in range(B):
        for r in range(1 + NB * Dmax):
            there = r == 0 or (r - 1) % Dmax < int(blk[b, (r - 1) // Dmax])
            assert torch.equal(out[b, r], full[b, r]) if there else (out[b, r] == -3).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("R,V", [(1, 128256), (37, 50257), (300, 1000), (5, 3), (64, 151936)])
def test_tokens(R, V, bf16):
    rng = np.random.default_rng(R + V)
    rows = [MIX[r % len(MIX)] for r in range(R)]
    kw, ora = _settings(rows)
    x = _dev(_rows(rng, R, V), bf16)
    u = (rng.integers(0, 1 << 24, R) / (1 << 24)).astype(np.float32)
    full = torch.empty((R, V), device="cuda")
    got = S.ssd_sample(x, torch.from_numpy(u).cuda(), **kw, probs_out=full)
    assert torch.equal(full, S.ssd_filter_probs(x, **kw))
    tok, prob, z = got["token"].cpu().numpy(), got["prob"].cpu().double().numpy(), x.float().cpu().numpy()
    skipped = 0
    for r in range(R):
        want, p, gap = Q.token(z[r], u[r], **ora[r])
        if Q.kept(z[r], **ora[r])[2] < NEAR or gap < NEAR:
            skipped += 1
            continue
        assert tok[r] == want, (r, tok[r], want)
        np.testing.assert_allclose(prob[r], p, rtol=RTOL)
        assert prob[r] == full[r, want].item()
    assert skipped <= max(1, R // 20)


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_of_rows_unlike_logits(kind):
    rng = np.random.default_rng(11)
    V = 3001
    us = np.array([0.0, 2.0 ** -24, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan, np.inf, 1e-30], np.float32)
    z = np.stack([_special(kind, V, rng) for _ in us])
    kw, ora = _settings([MIX[0]] * len(us))
    got = S.ssd_sample(torch.from_numpy(z).cuda(), torch.from_numpy(us).cuda(), **kw)["token"].cpu().numpy()
    for r, u in enumerate(us):
        c = Q.clean(z[r])
        if u <= 2.0 ** -24 or not u < 1:
            # the ends: the first or last token whose weight is not below 2^-44 of the largest
            top = c.max()
            live = np.nonzero(c - top > np.log(2.0 ** -44))[0] if top > -np.inf else [-1]
            sure = np.nonzero(c - top > np.log(2.0 ** -20))[0] if top > -np.inf else [-1]
            if u >= 1:
                assert sure[-1] <= got[r] <= live[-1]
            elif u <= 0 or u != u:
                assert got[r] == live[0] or live[0] <= got[r] <= sure[0]
            continue
        want, _, gap = Q.token(z[r], u)
        assert got[r] == want or gap < NEAR


def test_draws_follow_the_distribution():
    """Every uniform of a grid of n: token i gets its share of the grid, off by less than its two ends."""
    z = torch.log(torch.tensor([0.05, 0.3, 0.01, 0.24, 0.4], device="cuda"))
    n = 4096
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    tok = S.ssd_sample(z.expand(n, 5).contiguous(), u)["token"].cpu().numpy()
    share = np.bincount(tok, minlength=5)
    assert (np.diff(tok) >= 0).all()
    assert np.abs(share - np.array([0.05, 0.3, 0.01, 0.24, 0.4]) * n).max() < 1.01


def test_no_rows_and_reported_settings():
    x = torch.zeros((0, 100), device="cuda")
    assert S.ssd_filter_probs(x).shape == (0, 100)
    assert S.ssd_sample(x, torch.zeros(0, device="cuda"))["token"].shape == (0,)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.randn((3, 100), device="cuda")
    for bad in (-1.0, float("nan")):
        got = S.ssd_filter_probs(x, torch.tensor([1.0, bad, 1.0], device="cuda"), ws=ws)
        assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE
        assert got[1].argmax() == x[1].argmax() and (got[1] > 0).sum() == 1
    S.ssd_filter_probs(x, torch.tensor([0.0, float("inf"), 1e-45], device="cuda"), ws=ws)
    assert S.ssd_read_device_error(ws) == S.SSD_OK


def test_repeats_bit_for_bit_on_another_stream_and_from_a_graph():
    rng = np.random.default_rng(9)
    kw, _ = _settings([MIX[r % len(MIX)] for r in range(24)])
    x = _dev(_rows(rng, 24, 40001), True)
    u = torch.rand(24, device="cuda")
    probs = torch.empty((24, 40001), device="cuda")
    want = S.ssd_sample(x, u, **kw, probs_out=probs)
    ref = probs.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = S.ssd_filter_probs(x, **kw)
    named = S.ssd_sample(x, u, **kw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, ref) and torch.equal(named["token"], want["token"])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = dict(token=torch.empty(24, dtype=torch.int32, device="cuda"), prob=torch.empty(24, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.ssd_filter_probs(x, **kw, out=probs, ws=ws)
        S.ssd_sample(probs.log(), u, out=out, ws=ws)
    x2 = _dev(_rows(rng, 24, 40001), True)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(probs, S.ssd_filter_probs(x2, **kw))
    assert torch.equal(out["token"], S.ssd_sample(probs.log(), u)["token"])


def test_refusals():
    x = torch.zeros((4, 100), device="cuda")
    one = torch.ones(1, device="cuda")
    with pytest.raises(ValueError, match="dtype"):
        S.ssd_filter_probs(x.half())
    with pytest.raises(ValueError, match="dense"):
        S.ssd_filter_probs(x.t())
    with pytest.raises(ValueError, match="evenly"):
        S.ssd_filter_probs(torch.zeros((2, 3, 8), device="cuda")[:, :2])
    with pytest.raises(ValueError, match="divide"):
        S.ssd_filter_probs(x, torch.ones(3, device="cuda"))
    with pytest.raises(ValueError, match="top_k"):
        S.ssd_filter_probs(x, one, one)
    with pytest.raises(ValueError, match="top_p must be"):
        S.ssd_filter_probs(x, one, top_p=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="rows are not"):
        S.ssd_filter_probs(x, blk_len=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), Dmax=2)
    with pytest.raises(ValueError, match="out must be"):
        S.ssd_filter_probs(x, out=torch.zeros((4, 99), device="cuda"))
    with pytest.raises(ValueError, match="overlap"):
        S.ssd_filter_probs(x, out=x)
    with pytest.raises(ValueError, match="u must be"):
        S.ssd_sample(x, torch.zeros(3, device="cuda"))
    with pytest.raises(S.SsdError, match="unsupported"):
        S.ssd_filter_probs(torch.zeros((1, (1 << 20) + 1), device="cuda"))
    with pytest.raises(ValueError, match="rows must not overlap"):
        S.ssd_filter_probs(torch.zeros((1, 100), device="cuda").expand(4, 100))
