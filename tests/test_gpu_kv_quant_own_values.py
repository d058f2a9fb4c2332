"""Own-block values of any size in the attention over the 8-bit cache: they set the weights' reference only as
far as they count in the output, and do not overflow."""
import numpy as np
import pytest
import torch

import kv_quant_helpers as H
from oracle import ssd_oracle as O
from speculative_decoding_copy_gb300 import workloads as WL

pytestmark = pytest.mark.gpu


class Scaled(H.AttnCase):
    """Value scales times 2^prefix_exp and own values times 2^own_exp[block], both exact; flat scores or not."""

    def __init__(self, lengths, NB, Dmax, G, dh, prefix_exp, own_exp, flat):
        B = len(lengths)
        super().__init__(101, lengths, NB, Dmax, G, 2, dh, 32, True, blk_len=np.full((B, NB), Dmax), pow2=True)
        if flat:
            self.k_scale[:] = 2.0 ** -30
        self.v_scale *= np.float32(2.0 ** prefix_exp)
        f = np.repeat(2.0 ** np.asarray(own_exp, np.float64), Dmax)
        self.vc64 = self.vc64 * f[None, :, None, None]
        self.vc = WL.f32_to_bf16_bits(self.vc64.astype(np.float32))
        assert np.array_equal(O.bf16_to_f64(self.vc), self.vc64)

    def compare(self, out):
        """Each error has its bound by arithmetic: scores 2^-11 in log2 units (kv_quant_helpers); over few rows
        fp16 weights, 2^-11, over many three e5m2 numbers behind fp16 for the prefix (2^-9 + 2^-11) and bf16 for
        the own block (2^-8), so 2^-10 or 3 x 2^-9 of sum p |v| with the scores; half of the formats' least step
        for a code while the largest p s (s the value scale, of an own key the one its values would have) has
        at least 2^7 or 2^11: 2^-32 or 2^-28 of it; the merge of many rows."""
        many = self.many(self.q.shape[2] // 2)
        got, probs, bad = out.cpu().numpy().astype(np.float64), {}, []
        for (b, t), (o, size) in self.oracle(probs=probs).items():
            P, G = int(self.prefix[b]), o.shape[0] // 2
            for h, (p, v) in enumerate(probs[b, t]):
                rows = slice(h * G, (h + 1) * G)
                sv = self.v_scales(b)[h]
                own = 2.0 ** (np.floor(np.log2(np.abs(v[P:]).max(1))) - 8)
                top = (p * np.concatenate([sv, own])).max(1)
                codes = (np.abs(v[:P]) / sv[:, None]).sum(0)
                tol = size[rows] * (3 * 2.0 ** -9 if many else 2.0 ** -10) + top[:, None] * codes * (2.0 ** -28 if many else 2.0 ** -32)
                if many:
                    d = self.dh // 2
                    for half in (slice(0, d), slice(d, None)):
                        tol[:, half] += (p @ np.abs(v[:, half]).max(1))[:, None] * 2.0 ** -14
                worst = float((np.abs(got[b, t, rows] - o[rows]) / tol).max())
                if not worst <= 1:
                    bad.append((b, t, h, worst))
        assert not bad, bad[:6]


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("exp", [-90, -60, -45, -32, 0, 12])
@pytest.mark.parametrize("dh,NB,Dmax", [(64, 1, 1), (128, 2, 2), (64, 2, 10), (128, 2, 20)])
def test_own_and_cached_values_of_one_size(dh, NB, Dmax, exp, flat):
    case = Scaled([5000, 333, 0], NB, Dmax, 4, dh, exp, [exp] * NB, flat)
    case.compare(H.run(case))


@pytest.mark.parametrize("dh,Dmax", [(64, 2), (128, 2), (64, 20), (128, 20)])
def test_blocks_of_values_far_apart(dh, Dmax):
    """Three blocks: own values far above the cache's, far below them, and alike; what one block's are like
    does not show in the rows of another."""
    case = Scaled([1000, 200], 3, Dmax, 2, dh, -30, [60, -70, -30], True)
    case.compare(H.run(case))


@pytest.mark.parametrize("exp", [100, 110, 120])
@pytest.mark.parametrize("dh,NB,Dmax", [(64, 1, 1), (128, 1, 2), (64, 1, 20), (128, 2, 20)])
def test_own_values_near_the_end_of_the_range(dh, NB, Dmax, exp):
    """Finite values give finite outputs."""
    case = Scaled([700, 0], NB, Dmax, 4, dh, 0, [exp] * NB, False)
    out = H.run(case)
    assert bool(torch.isfinite(out).all())
    case.compare(out)
