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
