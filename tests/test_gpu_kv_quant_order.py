"""Orders that the waits of the many-rows attention over the 8-bit cache have to keep: many own-block
tiles a row tile (more than the ring holds), and references that move in every tile."""
import numpy as np
import pytest
import torch

import kv_quant_helpers as H
from speculative_decoding_copy_gb300 import _binding as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [[0], [900, 130]])
@pytest.mark.parametrize("NB,Dmax,G", [(40, 32, 2), (9, 256, 1), (5, 200, 3)])
@pytest.mark.parametrize("dh", [64, 128])
def test_many_own_block_tiles(dh, NB, Dmax, G, prefix):
    """Up to eighteen tiles of 128 own-block slots a row tile, few of their tokens present: fifty calls give
    the same bits, and the oracle's values."""
    rng = np.random.default_rng(NB)
    blk_len = rng.integers(0, 8, (len(prefix), NB)).astype(np.int32)
    blk_len[:, -1] = Dmax
    case = H.AttnCase(83, prefix, NB, Dmax, G, 2, dh, 64, True, blk_len=blk_len)
    assert case.many(G)
    case.poison()
    out = H.run(case)
    case.check(out)
    a, kw = case.args(), case.kw()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for _ in range(50):
        again = torch.full_like(out, 7.0)
        S.ssd_verify_attn_quant(*a, **kw, out=again, ws=ws)
        assert torch.equal(again, out)
    assert S.ssd_read_device_error(ws) == S.SSD_OK


@pytest.mark.parametrize("dh,Dmax", [(64, 20), (128, 20), (128, 90)])
def test_references_that_move_in_every_tile(dh, Dmax):
    """Scores grow from page to page, so every tile rescales the output right behind the product of the
    tile before: fifty calls give the same bits, and the oracle's values."""
    case = H.AttnCase(89, [1500, 700], 1, Dmax, 4, 2, dh, 16, True, q_scale=6.0, pow2=True, blk_len=np.full((2, 1), Dmax))
    for row in case.table:
        for j, pg in enumerate(row):
            case.k_scale[pg] = 2.0 ** (-9 + 0.5 * (j // 2))
    out = H.run(case)
    rng = np.random.default_rng(3)
    case.check(out, {(b, int(t)) for b in range(2) for t in rng.integers(0, Dmax, 8)}, wide=4.0)
    a, kw = case.args(), case.kw()
    for _ in range(50):
        assert torch.equal(S.ssd_verify_attn_quant(*a, **kw, out_f32=True), out)
