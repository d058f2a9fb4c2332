"""The 8-bit cache's calls through the checked build: canaries around every buffer that is written stay intact, no
index check fails, and the results are those of the normal build bit for bit."""
import numpy as np
import pytest
import torch

import kv_quant_helpers as H
from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_checked import Guarded

pytestmark = pytest.mark.gpu
dev = H.dev


def both(call, *written):
    """call(*buffers) by the normal and the checked build on equal copies of `written`; returns the checked one's."""
    normal = [x.clone() for x in written]
    call(*normal)
    G = Guarded()
    mine = [G.like(x) for x in written]
    with S.use_library(S.CHECKED_LIB_PATH) as L:
        assert L.ssd_checked_build() == 1
        S.ssd_read_check_error()
        call(*mine)
        assert G.intact(), "a canary region was written"
        assert S.ssd_read_check_error() == S.SSD_OK
    for a, b in zip(normal, mine):
        assert torch.equal(a, b)
    return mine


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("NB,Dmax,G", [(1, 1, 4), (2, 4, 2), (3, 20, 4), (40, 32, 2), (1, 1, 64)])
def test_attention(paged, dh, NB, Dmax, G):
    case = H.AttnCase(103, [0, 1, 129, 700, 128], NB, Dmax, G, 2, dh, 32, paged)
    case.poison()
    a, kw = case.args(), case.kw()
    out = torch.full(case.q.shape, 7.0, dtype=torch.float32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out, ws = both(lambda o, w: S.ssd_verify_attn_quant(*a, **kw, out=o, ws=w), out, ws)
    case.check(out)
    assert S.ssd_read_device_error(ws) == S.SSD_OK


@pytest.mark.parametrize("tokens", [128, 300])
@pytest.mark.parametrize("dh,sb,f32", [(64, 16, False), (128, 64, True), (128, 128, False)])
def test_append_and_commit(dh, sb, f32, tokens):
    rng = np.random.default_rng(dh + sb)
    B, Hkv, NB, Dmax = 5, 3, 2, 70
    c = [dev(x) for _ in range(2) for x in H.cache(rng, B, Hkv, tokens, dh, sb)]
    c = [c[0], c[2], c[1], c[3]]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rows = torch.from_numpy(rng.standard_normal((2, B, NB * Dmax, Hkv, dh)).astype(np.float32)).to("cuda")
    rows = rows if f32 else rows.bfloat16()
    slots = dev(np.concatenate([p * tokens + 128 - 58 - p + np.arange(58 + p) for p in range(B)] + [[-1, -1]]).astype(np.int32))
    k, v = (x.reshape(-1, Hkv, dh)[:len(slots)] for x in rows)
    *_, ws = both(lambda *b: S.ssd_append_kv_quant(k, v, slots, *b[:4], sb, ws=b[4]), *c, ws)
    prefix, best, n_out = (dev(np.array(x, np.int32)) for x in
                           ([0, 1, tokens - Dmax, 55, 13], [0, 1, 1, -1, 0], [Dmax + 1, 2, Dmax + 1, 1, 30]))
    new = torch.zeros_like(prefix)
    *_, new, ws = both(lambda *b: S.ssd_commit_kv_quant(*b[:4], rows[0], rows[1], prefix, best, n_out, Dmax, sb, new_len=b[4], ws=b[5]),
                       *c, new, ws)
    assert new.tolist() == [Dmax, 2, tokens, 55, 42]
    assert S.ssd_read_device_error(ws) == S.SSD_OK


@pytest.mark.parametrize("B,pps,cap", [(5, 4, 900), (1100, 3, 70000)])
def test_page_tables(B, pps, cap):
    rng = np.random.default_rng(B)
    held, table = np.zeros(B, np.int32), np.full((B, pps), -1, np.int32)
    stack, n = rng.permutation(B * pps - 1).astype(np.int32), np.array([B * pps - 1], np.int32)
    state = [dev(x) for x in (held, table, stack, n)]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    cur = i32(B)
    for add in (dev(rng.integers(0, 64 if B > 99 else 200, B).astype(np.int32)), i32(B)):      # grown, then trimmed
        more = [i32(B + 1), i32(cap), i32(B), torch.zeros(256, dtype=torch.uint8, device="cuda")]
        *state, _, _, served, ws = both(
            lambda *b: S.ssd_page_tables(cur, add, *b[:4], cap, out=dict(row_start=b[4], slot_map=b[5], served=b[6]), ws=b[7]), *state, *more)
        assert bool(served.all()) and S.ssd_read_device_error(ws) == S.SSD_OK
    assert int(state[3]) == B * pps - 1
