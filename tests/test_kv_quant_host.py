"""The 8-bit cache's entry points check their arguments on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_copy_gb300 import _binding as S

A = 1 << 40            # plausible, aligned addresses that nothing dereferences
FAR = 1 << 36          # more than a buffer's size apart
P = [A + i * FAR for i in range(11)]


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


def _pages(**kw):
    return _set(S.PagesArgs(*P[:9], 2, 4, 10, 8), **kw)


def _append(**kw):
    return _set(S.AppendQuantArgs(*P[:7], S.SSD_BF16, 2, 64, 16, 3, 128, 128, 4, 128), **kw)


def _commit(**kw):
    return _set(S.CommitQuantArgs(*P[:10], None, S.SSD_BF16, 2, 1, 4, 2, 64, 16, 0, 256, 2), **kw)


def _attn(**kw):
    return _set(S.AttnQuantArgs(*P[:10], None, S.SSD_BF16, 2, 1, 4, 4, 2, 64, 16, 0, 0.0, 256, 2), **kw)


INV, UNS = S.SSD_ERR_INVALID, S.SSD_ERR_UNSUPPORTED


@pytest.mark.parametrize("make,fn,bad", [
    (_pages, "ssd_page_tables", [(dict(B=-1), INV), (dict(n_free=None), INV), (dict(slot_map=None), INV), (dict(slot_cap=0), INV),
                                 (dict(cur_len=None), INV), (dict(block_table=None), INV), (dict(free_pages=None), INV),
                                 (dict(num_pages=1 << 24), UNS), (dict(slot_cap=1 << 31), UNS), (dict(pages_per_seq=1 << 21), UNS), (dict(served=P[0] + 4), INV), (dict(slot_map=P[2] - 4), INV)]),
    (_append, "ssd_append_kv_quant", [(dict(dtype=5), INV), (dict(T=-1), INV), (dict(dh=96), UNS), (dict(scale_block=8), UNS),
                                      (dict(k_stride=64), INV), (dict(v_stride=132), UNS), (dict(k_new=A + 2), UNS),
                                      (dict(k_cache=A + 4), UNS), (dict(slot_map=None), INV), (dict(v_scale=None), INV),
                                      (dict(num_pages=1 << 24), UNS), (dict(page_tokens=0), INV),
                                      (dict(k_stride=1 << 60), UNS), (dict(v_cache=P[3] + 16), INV), (dict(k_new=P[4] - 16), INV)]),
    (_commit, "ssd_commit_kv_quant", [(dict(dtype=5), INV), (dict(B=-1), INV), (dict(Dmax=257), UNS), (dict(dh=32), UNS),
                                      (dict(scale_block=256), UNS), (dict(new_len=P[6]), INV), (dict(P_max=-1), INV),
                                      (dict(P_max=1 << 30), UNS), (dict(block_table=P[10]), INV), (dict(k_cand=A + 8), UNS), (dict(NB=1 << 30, B=1 << 30), UNS),
                                      (dict(n_out=None), INV)]),
    (_attn, "ssd_verify_attn_quant", [(dict(Hq=5), INV), (dict(dh=80), UNS), (dict(scale_block=24), UNS), (dict(out_dtype=7), INV),
                                      (dict(Dmax=300), UNS), (dict(NB=4000), UNS), (dict(Hq=2 * 65), UNS), (dict(scale=-1.0), INV),
                                      (dict(q=None), INV), (dict(k_cache=None), INV), (dict(q=A + 2), UNS), (dict(P_max=1 << 29), UNS),
                                      (dict(out=P[1] + 16), INV), (dict(block_table=P[10]), INV), (dict(block_table=P[10], pages_per_seq=2, num_pages=1 << 23), UNS)]),
])
def test_bad_arguments_come_back_before_any_launch(L, make, fn, bad):
    call = lambda a, ws=A, n=256: getattr(L, fn)(ctypes.byref(a), ws, n, None)
    for kw, want in bad:
        assert call(make(**kw)) == want, kw
    for ws, n in ((None, 256), (A + 8, 256), (A, 255)):
        assert call(make(), ws, n) == S.SSD_ERR_WORKSPACE
    assert getattr(L, fn)(None, A, 256, None) == INV


def test_nothing_to_do_launches_nothing(L):
    assert L.ssd_append_kv_quant(ctypes.byref(_append(T=0)), None, 0, None) == S.SSD_OK
    assert L.ssd_commit_kv_quant(ctypes.byref(_commit(B=0)), None, 0, None) == S.SSD_OK
    assert L.ssd_verify_attn_quant(ctypes.byref(_attn(B=0)), None, 0, None) == S.SSD_OK
    assert L.ssd_verify_attn_quant_workspace_size(ctypes.byref(_attn())) == 256
    assert L.ssd_verify_attn_quant_workspace_size(ctypes.byref(_attn(dh=80))) == 0


def test_host_tensors_are_rejected():
    z, i = torch.zeros((2, 2, 128, 64), dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    s, x = torch.zeros((2, 2, 1)), torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_verify_attn_quant(x, z, z, s, s, x, x, i, i.view(2, 1), 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_append_kv_quant(x[0], x[0], i, z, z, s, s)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_commit_kv_quant(z, z, s, s, x, x, i, i, i, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssd_page_tables(i, i, i, i.view(2, 1), i, i[:1], 0)
