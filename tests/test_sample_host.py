"""The entry points of sampled continuations of one prompt check their arguments on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_copy_gb300 import _binding as S

A = 1 << 40            # plausible, aligned addresses that nothing dereferences
FAR = 1 << 36          # more than a buffer's size apart
P = [A + i * FAR for i in range(14)]
INV, UNS, WS = S.SSD_ERR_INVALID, S.SSD_ERR_UNSUPPORTED, S.SSD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    import os
    from speculative_decoding_copy_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    return S.lib()


def _set(args, **kw):
    for k, v in kw.items():
        setattr(args, k, v)
    return args


def _rows(**kw):
    return _set(S.RowsArgs(P[0], S.SSD_F32, 6, 1000, 1000, 2, *P[1:5]), **kw)


def _attn(**kw):
    return _set(S.AttnSharedArgs(*P[:11], None, None, S.SSD_BF16, S.SSD_BF16, 2, 2, 4, 8, 2, 128, 0, 0, 0.0, 300, 256, 2), **kw)


ROWS = [(dict(dtype=7), INV), (dict(R=-1), INV), (dict(V=0), INV), (dict(row_stride=999), INV), (dict(rows_per=0), INV), (dict(logits=None), INV),
        (dict(V=(1 << 20) + 1, row_stride=1 << 21), UNS), (dict(R=1 << 28), UNS), (dict(row_stride=1 << 60), UNS), (dict(logits=A + 2), INV),
        (dict(top_p=P[3] + 1), INV)]


@pytest.mark.parametrize("kw,want", ROWS, ids=str)
def test_rows_refused(L, kw, want):
    a = ctypes.byref(_rows(**kw))
    assert L.ssd_filter_probs(a, None, 0, 0, P[6], P[8], 256, None) == want
    assert L.ssd_sample(a, P[5], P[6], P[7], None, P[8], 256, None) == want


def test_filter_refused(L):
    call = lambda blk=None, NB=0, D=0, out=P[6], ws=P[8], n=256, **kw: L.ssd_filter_probs(ctypes.byref(_rows(**kw)), blk, NB, D, out, ws, n, None)
    assert call(out=None) == INV and call(out=P[0] + 400) == INV and call(out=P[6] + 2) == INV
    assert call(blk=P[5], NB=0, D=3) == INV and call(blk=P[5], NB=2, D=2) == INV          # 6 rows are no 1 + 2 x 2 a sequence
    assert call(blk=P[6] + 8, NB=1, D=2) == INV                                            # the output over the lengths
    assert call(ws=None) == WS and call(ws=P[8] + 8) == WS and call(n=255) == WS
    assert L.ssd_filter_probs(None, None, 0, 0, P[6], P[8], 256, None) == INV
    assert call(R=0, out=None, ws=None) == S.SSD_OK


def test_sample_refused(L):
    call = lambda u=P[5], tok=P[6], prob=P[7], full=None, ws=P[8], n=256, **kw: L.ssd_sample(ctypes.byref(_rows(**kw)), u, tok, prob, full, ws, n, None)
    assert call(u=None) == INV and call(tok=None) == INV and call(tok=P[5]) == INV and call(prob=P[6] + 4) == INV
    assert call(full=P[0] - 8) == INV and call(full=P[9] + 1) == INV
    assert call(ws=None) == WS and call(n=0) == WS
    assert L.ssd_sample(None, P[5], P[6], P[7], None, P[8], 256, None) == INV
    assert call(R=0, u=None, ws=None) == S.SSD_OK


ATTN = [(dict(B=-1), INV), (dict(Hq=7), INV), (dict(dh=96), UNS), (dict(dtype=3), INV), (dict(dtype=S.SSD_F32, out_dtype=S.SSD_BF16), INV), (dict(scale=-1.0), INV),
        (dict(scale=float("nan")), INV), (dict(Dmax=300), UNS), (dict(NB=3000), UNS), (dict(Hq=2 * 65), UNS), (dict(B=5000), UNS), (dict(q=None), INV),
        (dict(shared_len=None), INV), (dict(prefix_len=None), INV), (dict(k_shared=None), INV), (dict(v_cache=None), INV), (dict(q=P[0] + 2), UNS), (dict(out=P[0]), INV),
        (dict(out=P[6] + 16), INV), (dict(S_max=1 << 28), UNS), (dict(P_max=1 << 27, Hkv=8, Hq=8), UNS), (dict(shared_table=P[11], shared_pages=3), INV),
        (dict(block_table=P[12], pages_per_seq=0), INV), (dict(block_table=P[12], pages_per_seq=2, num_pages=0), INV),
        (dict(block_table=P[12], pages_per_seq=2, num_pages=1 << 23), UNS), (dict(block_table=P[12], pages_per_seq=2, shared_table=P[11], shared_pages=0), INV)]


@pytest.mark.parametrize("kw,want", ATTN, ids=str)
def test_attention_refused(L, kw, want):
    assert L.ssd_verify_attn_shared(ctypes.byref(_attn(**kw)), P[13], 1 << 40, None) == want
    if want == UNS or "out" not in kw:
        assert L.ssd_verify_attn_shared_workspace_size(ctypes.byref(_attn(**kw))) == 0


def test_attention_of_nothing(L):
    assert L.ssd_verify_attn_shared(ctypes.byref(_attn(B=0)), None, 0, None) == S.SSD_OK
    assert L.ssd_verify_attn_shared(None, P[13], 1 << 40, None) == INV
    assert L.ssd_verify_attn_shared_workspace_size(ctypes.byref(_attn(B=0))) == 256


def test_host_tensors_are_rejected():
    x, i, f = torch.zeros((2, 10)), torch.zeros(1, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_filter_probs(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_sample(x, f)
    q = torch.zeros((1, 1, 2, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_verify_attn_shared(q, q[0], q[0], i, q, q, q, q, i, i.view(1, 1), 1)
