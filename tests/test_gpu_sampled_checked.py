"""The calls for sampled continuations of one prompt through the checked build: canaries around every buffer that is
written stay intact, no index check fails, and the results are those of the normal build bit for bit."""
import pytest
import torch

from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_attn_shared import Case
from test_gpu_kv_quant_checked import both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(S_len=700, own=[5, 0, 300], Dmax=3, G=7, Hkv=2), dict(S_len=257, own=[130, 1], NB=5, Dmax=16, blk=[[16, 0, 3, 1, 16]] * 2),
                                dict(S_len=0, own=[130] * 200, G=1, Hkv=1), dict(S_len=20000, own=[0, 0], G=64, Hkv=1, Dmax=4)])
@pytest.mark.parametrize("dh,paged,f32", [(128, False, False), (64, True, False), (128, False, True)])
def test_attention(kw, dh, paged, f32):
    c = Case(21, dh=dh, paged=paged, f32=f32, **kw)
    args, tables = c.device()
    out = torch.full_like(args[0], 7.0)
    n = S.ssd_verify_attn_shared_workspace_size(S.attn_shared_args(*args, c.Dmax, out, **tables))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def call(o, w):
        S.ssd_verify_attn_shared(*args, c.Dmax, **tables, out=o, ws=w)
        assert S.ssd_read_device_error(w) == S.SSD_OK
        w.zero_()                        # what a workspace holds behind a call is not compared

    out, _ = both(call, out, ws)
    c.check(out)


@pytest.mark.parametrize("V,bf16", [(1000, False), (32001, True), (128256, False), (600001, False)])
def test_sampling(V, bf16):
    g = torch.Generator(device="cuda").manual_seed(V)
    R = 6
    x = torch.randn((R, V), generator=g, device="cuda") * 3
    x = x.bfloat16() if bf16 else x
    t = lambda *v: torch.tensor(v, device="cuda")
    kw = dict(temperature=t(1.0, 0.7, 0.0, 1.3, 1.0, 0.9), top_k=t(0, 50, 0, 1000, 0, 5).int(), top_p=t(0.9, 1.0, 1.0, 0.95, 1.0, 0.5), min_p=t(0.0, 0.0, 0.0, 0.1, 0.05, 0.0))
    u = torch.rand(R, generator=g, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    probs, tok, prob = torch.full((R, V), 7.0, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, device="cuda")
    both(lambda p, i, q, w: S.ssd_sample(x, u, **kw, probs_out=p, out=dict(token=i, prob=q), ws=w), probs, tok, prob, ws)
    both(lambda p, w: S.ssd_filter_probs(x, **kw, out=p, ws=w), probs, ws)
