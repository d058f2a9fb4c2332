"""ssd_filter_probs and ssd_sample over the widest rows, with most of the weight in few bins: a CTA then
adds more than 2^16 weights to one of them, and their sum has to stay exact."""
import numpy as np
import pytest
import torch

from oracle import sample_oracle as Q
from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_sample import NEAR, RTOL, _check_row, _dev, _settings

pytestmark = pytest.mark.gpu


def _rows(V, kind):
    """Long runs of one value, then another run ("runs") or a slope ("slope") in which the cuts lie."""
    rng = np.random.default_rng(V)
    head = 5 * V // 8
    out = []
    for a in (-0.1, -0.7, -1.3, -2.9):
        z = np.full(V, a, np.float32)
        z[head:] = a - 0.25 if kind == "runs" else a - 0.25 - np.arange(V - head) * (4.0 / (V - head))
        z[rng.integers(0, V, 3)] = (0.0, -0.01, -0.02)
        out.append(z)
    return np.stack(out).astype(np.float32)


SETTINGS = [(1.0, 0, 0.9, 0.0), (1.0, 0, 0.83, 0.0), (1.0, 7, 0.97, 0.0), (0.9, 0, 0.88, 0.0)]


def _with_k(V):
    return [(t, k and int(0.8 * V) + k, p, m) for t, k, p, m in SETTINGS]


@pytest.mark.parametrize("kind", ["runs", "slope"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 5, 600001, 270000])
def test_cuts_behind_long_runs_of_equal_tokens(V, bf16, kind):
    rows = _with_k(V)
    kw, ora = _settings(rows)
    x = _dev(_rows(V, kind), bf16)
    got = S.ssd_filter_probs(x, **kw).cpu().double().numpy()
    z = x.float().cpu().numpy()
    ok = [_check_row(got[r], z[r], ora[r]) for r in range(len(rows))]
    assert sum(ok) >= len(ok) - 1


@pytest.mark.parametrize("R", [40, 160, 320])
def test_many_of_the_widest_rows(R):
    """Other cluster sizes: one row with the same answer in every place."""
    V = 1 << 20
    x = _dev(_rows(V, "runs")[3:4], True)
    want = S.ssd_filter_probs(x, top_p=torch.tensor([0.9], device="cuda"))[0]
    ora = dict(top_p=float(np.float32(0.9)))
    assert Q.kept(x[0].float().cpu().numpy(), **ora)[2] >= NEAR
    assert _check_row(want.cpu().double().numpy(), x[0].float().cpu().numpy(), ora)
    wide = x.expand(R, V).contiguous()
    u, full = torch.full((R,), 0.625, device="cuda"), torch.empty((R, V), device="cuda")
    got = S.ssd_sample(wide, u, top_p=torch.full((R,), 0.9, device="cuda"), probs_out=full)
    assert all(torch.equal(full[r], want) for r in range(R))
    tok, p, gap = Q.token(x[0].float().cpu().numpy(), 0.625, **ora)
    assert gap < NEAR or (got["token"] == tok).all()
    np.testing.assert_allclose(got["prob"].cpu().double().numpy(), p, rtol=RTOL)
