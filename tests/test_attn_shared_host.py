"""ssd_verify_attn_shared: the documented limit of a call's work, and arguments that are not used (no GPU needed)."""
import ctypes

import pytest

from speculative_decoding_copy_gb300 import _binding as S
from test_sample_host import L, _attn, _set  # noqa: F401  (L: the library, a fixture)

UNITS = 1 << 30


def _units(a):
    """Units of work as the header counts them."""
    G, NT = a.Hq // a.Hkv, a.NB * a.Dmax
    parts = lambda n: a.Hkv * -(-n // (2 * (128 // G)))
    return 2 * parts(a.B * NT) * (-(-a.S_max // 128) + 2) + 2 * a.B * parts(NT) * (-(-a.P_max // 128) + 2)


# (out lies behind the largest of these caches)
SIZES = [dict(B=64, NB=32, Dmax=256, Hq=64, Hkv=1, S_max=2048 * 128), dict(B=128, NB=64, Dmax=128, Hq=40, Hkv=1, S_max=1000 * 128 - 5),
         dict(B=4096, NB=1, Dmax=255, Hq=56, Hkv=1, S_max=77)]


@pytest.mark.parametrize("kw", SIZES, ids=lambda k: "B%d" % k["B"])
def test_most_work_of_a_call(L, kw):  # noqa: F811
    lo, hi = 1, 1 << 20
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if _units(_attn(P_max=mid, **kw)) < UNITS:
            lo = mid
        else:
            hi = mid
    assert _units(_attn(P_max=lo, **kw)) < UNITS <= _units(_attn(P_max=hi, **kw)) and lo % 128 == 0
    call = lambda a: L.ssd_verify_attn_shared(ctypes.byref(_set(a, out=1 << 50)), None, 0, None)
    # (a call that would be taken still lacks a workspace, or a GPU)
    assert L.ssd_verify_attn_shared_workspace_size(ctypes.byref(_attn(P_max=lo, **kw))) > 0
    assert call(_attn(P_max=lo, **kw)) in (S.SSD_ERR_WORKSPACE, S.SSD_ERR_CUDA)
    assert L.ssd_verify_attn_shared_workspace_size(ctypes.byref(_attn(P_max=hi, **kw))) == 0
    assert call(_attn(P_max=hi, **kw)) == S.SSD_ERR_UNSUPPORTED


def test_most_rows_of_out(L):  # noqa: F811
    kw = dict(NB=32, Dmax=256, Hq=1024, Hkv=16, S_max=0, P_max=0)
    for B, ok in ((255, True), (256, False)):
        assert (L.ssd_verify_attn_shared_workspace_size(ctypes.byref(_attn(B=B, **kw))) > 0) == ok


@pytest.mark.parametrize("kw", [dict(k_shared=(1 << 40) + 2), dict(v_shared=1 << 48), dict(S_max=1 << 40), dict(S_max=-1), dict(k_shared=None, v_shared=None, S_max=300)],
                         ids=str)
def test_prompt_in_pages_leaves_its_own_buffers_unused(L, kw):  # noqa: F811
    """With a shared_table the shared keys come from the pool: k_shared, v_shared and S_max may hold anything."""
    a = _attn(block_table=1 << 41, pages_per_seq=2, shared_table=1 << 42, shared_pages=3, num_pages=9)
    _set(a, out=1 << 48, **kw)
    assert L.ssd_verify_attn_shared_workspace_size(ctypes.byref(a)) > 0
    assert L.ssd_verify_attn_shared(ctypes.byref(a), None, 0, None) in (S.SSD_ERR_WORKSPACE, S.SSD_ERR_CUDA)
