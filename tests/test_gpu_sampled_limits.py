"""Sampled continuations at the ends of their ranges: thousands of sequences, the longest blocks and most
slots, nothing present, and tensors whose elements pass 2^31."""
import numpy as np
import pytest
import torch

from oracle import sample_oracle as Q
from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_attn_shared import DEV, Case
from test_gpu_sample import NEAR, _check_row, _rows, _settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(B=4096, S_len=130, G=1, Hkv=1), dict(B=1500, S_len=70, G=2, Hkv=2), dict(B=1030, S_len=0, G=1, Hkv=1)],
                         ids=lambda k: "B%d" % k["B"])
@pytest.mark.parametrize("f32", [False, True])
def test_thousands_of_sequences_some_without_tokens(kw, f32):
    rng = np.random.default_rng(kw["B"])
    B = kw["B"]
    own = [int(n) for n in rng.integers(0, 4, B)]
    own[B - 1] = 131
    c = Case(21, own=own, dh=64, f32=f32, blk=rng.integers(0, 2, (B, 1)).tolist(), slack=0, **{k: v for k, v in kw.items() if k != "B"})
    c.check(c.run())


@pytest.mark.parametrize("kw", [dict(NB=1, Dmax=256, own=[40, 0]), dict(NB=70, Dmax=3, own=[9]), dict(NB=32, Dmax=256, own=[129])],
                         ids=lambda k: "NB%d" % k["NB"])
def test_long_blocks_and_many_slots(kw):
    rng = np.random.default_rng(kw["NB"])
    blk = rng.integers(0, kw["Dmax"] + 1, (len(kw["own"]), kw["NB"]))
    blk[:, 0] = kw["Dmax"]
    c = Case(22, S_len=200, G=1, Hkv=1, dh=64, blk=blk.tolist(), **kw)
    c.check(c.run())


@pytest.mark.parametrize("f32", [False, True])
def test_nothing_present(f32):
    c = Case(23, S_len=300, own=[200, 1], NB=2, Dmax=3, blk=[[0, 0], [0, 0]], f32=f32)
    out = torch.full(c.q.shape, -3.0, dtype=c.q.dtype, device=DEV)
    c.run(out=out)
    assert (out == -3).all()


@pytest.mark.parametrize("paged", [False, True])
def test_keys_beyond_32_bits(paged):
    """The small case's keys where offsets in elements and bytes pass 2^32: the same bits come out."""
    c = Case(24, S_len=300, own=[200, 129, 64], Dmax=3, dh=128, Hkv=2, paged=paged)
    args, tables = c.device()
    want = S.ssd_verify_attn_shared(*args, c.Dmax, **tables)
    far = 1 << 32                                             # elements
    if paged:
        first = far // (2 * 128 * 128)                        # pages before the small case's
        for i in (4, 5):
            big = torch.empty((first + args[i].shape[0], 2, 128, 128), dtype=torch.bfloat16, device=DEV)
            big[first:] = args[i]
            args[i] = big
        tables = {k: t + first for k, t in tables.items()}
    else:
        rows = far // 128 // 2                                # of a head of the prompt, of a sequence
        for i in (1, 2):
            big = torch.empty((2, rows * 2, 128), dtype=torch.bfloat16, device=DEV)
            big[:, :args[i].shape[1]] = args[i]
            args[i] = big
        for i in (4, 5):
            big = torch.empty((3, 2, rows, 128), dtype=torch.bfloat16, device=DEV)
            big[:, :, :args[i].shape[2]] = args[i]
            args[i] = big
    got = S.ssd_verify_attn_shared(*args, c.Dmax, **tables)
    assert torch.equal(got, want)
    c.check(got)


def test_logit_rows_beyond_32_bits():
    """Rows so far apart, and so many, that their elements pass 2^31 in the input and in the output."""
    V, R = 1 << 20, 2100
    rng = np.random.default_rng(25)
    few = _rows(rng, 3, V)
    kw, ora = _settings([(0.9, 0, 0.9, 0.0)])
    x = torch.empty((R, V + 8), dtype=torch.bfloat16, device=DEV)[:, :V]
    few = torch.from_numpy(few).to(DEV).to(torch.bfloat16)
    for r in range(3):
        x[r::3] = few[r]
    u = torch.full((R,), 0.4375, device=DEV)
    out = torch.empty((R, V), device=DEV)
    got = S.ssd_sample(x, u, **kw, probs_out=out)
    ok = 0
    for r in range(3):
        ok += _check_row(out[r].cpu().double().numpy(), few[r].float().cpu().numpy(), ora[0])
        for s in (R - 3 + r, R // 2 // 3 * 3 + r):
            assert torch.equal(out[s], out[r])
        assert (got["token"][r::3] == got["token"][r]).all() and got["token"][r] >= 0
    assert ok >= 2


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("R,V", [(1, 50257), (8, 128256), (64, 20000), (300, 5003)])
def test_top_k_of_hundreds(R, V, bf16):
    """Sorted lists of one and of several CTAs, lists too long to be sorted, and the bins beyond; drawn from the
    list and from the row."""
    rng = np.random.default_rng(R)
    rows = [(t, k, p, m) for k in (257, 512, 513, 700, 1000, 1024, 1025, 2100) for t, p, m in ((1.0, 1.0, 0.0), (1.5, 0.97, 0.0), (0.8, 0.9, 0.01))]
    rows = [rows[(7 * r) % len(rows)] for r in range(R)]
    kw, ora = _settings(rows)
    z = _rows(rng, R, V)
    z[::3] = np.round(z[::3] * 4) / 4                        # many ties, at the borders too
    x = torch.from_numpy(z).to(DEV)
    x = x.to(torch.bfloat16) if bf16 else x
    u = (rng.integers(0, 1 << 24, R) / (1 << 24)).astype(np.float32)
    full = torch.empty((R, V), device=DEV)
    got = S.ssd_sample(x, torch.from_numpy(u).to(DEV), **kw, probs_out=full)
    tok, prob, p, z = got["token"].cpu().numpy(), got["prob"].cpu().numpy(), full.cpu().double().numpy(), x.float().cpu().numpy()
    compared = 0
    for r in range(R):
        if not _check_row(p[r], z[r], ora[r]):
            continue
        want, _, gap = Q.token(z[r], u[r], **ora[r])
        if gap < NEAR:
            continue
        compared += 1
        assert tok[r] == want and prob[r] == p[r, want]
    assert compared >= R - max(1, R // 20)
