"""ssd_verify_attn_shared against the fp64 oracle.

Tolerance, bf16: the output's own rounding 2^-8 |out|; the weights of shared and own keys are rounded
(2^-8 each) and divided by the sum of the rounded ones, which moves the output by at most
2 * 2^-8 * sum w |v - out|; fp32 arithmetic (scores of |s| < 2^6 in log2 units to 2^-24 of the products'
sum, exponentials to 2^-22) adds less than 2^-12 of that sum and 2^-16 of the output. fp32: the last
ones alone."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attn_shared_oracle as A
from speculative_decoding_copy_gb300 import _binding as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, seed, S_len, own, NB=1, Dmax=1, G=4, Hkv=2, dh=128, paged=False, f32=False, blk=None, spare=3, slack=5, q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        B, NT = len(own), NB * Dmax
        kind = torch.float32 if f32 else torch.bfloat16
        new = lambda *s: torch.randn(s, generator=g).to(kind)
        self.q = (torch.randn((B, NT, Hkv * G, dh), generator=g) * q_scale).to(kind)
        self.cand = new(B, NT, Hkv, dh), new(B, NT, Hkv, dh)
        self.shared = new(Hkv, S_len, dh), new(Hkv, S_len, dh)
        self.own = [(new(Hkv, P, dh), new(Hkv, P, dh)) for P in own]
        self.blk = torch.full((B, NB), Dmax, dtype=torch.int32) if blk is None else torch.tensor(blk, dtype=torch.int32).view(B, NB)
        self.Dmax, self.S_len, self.f32 = Dmax, S_len, f32
        most = max(own)
        nan = lambda *s: torch.full(s, float("nan")).to(kind)
        # whatever is not a key is NaN: behind the lengths, in unused pages, in absent slots
        self.table = self.shared_table = self.k_shared = self.v_shared = None
        if paged:
            n, pps = -(-S_len // 128), max(1, -(-most // 128))
            order = torch.randperm(n + B * pps + spare, generator=g).to(torch.int32)
            self.shared_table, self.table = order[:max(n, 1)].clone(), order[n:n + B * pps].clone().view(B, pps)
            caches = [nan(len(order), Hkv, 128, dh) for _ in "kv"]
            for c in range(2):
                for j in range(n):
                    part = self.shared[c][:, 128 * j:128 * (j + 1)]
                    caches[c][int(order[j]), :, :part.shape[1]] = part
                for b, P in enumerate(own):
                    for j in range(-(-P // 128)):
                        part = self.own[b][c][:, 128 * j:128 * (j + 1)]
                        caches[c][int(self.table[b, j]), :, :part.shape[1]] = part
        else:
            caches = [nan(B, Hkv, most + slack, dh) for _ in "kv"]
            kv = [nan(Hkv, S_len + slack, dh) for _ in "kv"]
            for c in range(2):
                kv[c][:, :S_len] = self.shared[c]
                for b, P in enumerate(own):
                    caches[c][b, :, :P] = self.own[b][c]
            self.k_shared, self.v_shared = kv
        self.caches = caches
        t = torch.arange(NT)
        self.present = (t % Dmax)[None, :] < self.blk[:, t // Dmax]
        k, v = (x.clone() for x in self.cand)
        k[~self.present] = float("nan")
        v[~self.present] = float("nan")
        self.cand_nan = k, v
        self.lens = torch.tensor([S_len], dtype=torch.int32), torch.tensor(own, dtype=torch.int32)
        self.seen = None

    def device(self):
        d = lambda x: None if x is None else x.to(DEV)
        return [d(x) for x in (self.q, self.k_shared, self.v_shared, self.lens[0], *self.caches, *self.cand_nan, self.lens[1], self.blk)], \
            dict(block_table=d(self.table), shared_table=d(self.shared_table))

    def run(self, **kw):
        args, tables = self.device()
        return S.ssd_verify_attn_shared(*args, self.Dmax, **tables, **kw)

    def check(self, out, out_bf16=None):
        f = lambda x: x.double().numpy()
        want = A.attention(f(self.q), [f(x) for x in self.shared], [[f(x) for x in o] for o in self.own], [f(x) for x in self.cand],
                           self.blk.numpy(), self.Dmax)
        got = out.double().cpu().numpy()
        half = 2.0 ** -8 if (out.dtype == torch.bfloat16) else 0.0
        weights = 2.0 ** -12 if self.f32 else 2 * 2.0 ** -8 + 2.0 ** -12
        for (b, t), (o, spread) in want.items():
            tol = (half + 2.0 ** -16) * np.abs(o) + weights * spread + 1e-7
            err = np.abs(got[b, t] - o)
            assert (err <= tol).all(), (b, t, float((err / tol).max()))


SHAPES = [
    # one token, no keys but its own; a shared prompt alone; an own prefix alone
    dict(S_len=0, own=[0, 0]), dict(S_len=1, own=[0]), dict(S_len=0, own=[1, 3]),
    dict(S_len=128, own=[128, 0, 127]), dict(S_len=129, own=[1, 130, 257]), dict(S_len=700, own=[5, 0, 300, 128, 64]),
    # blocks, some absent; more tokens than a row tile, than a pair of them
    dict(S_len=300, own=[40, 0], NB=3, Dmax=5, blk=[[5, 0, 2], [0, 0, 1]]),
    dict(S_len=257, own=[130], NB=5, Dmax=16), dict(S_len=200, own=[20, 300, 0], NB=9, Dmax=16, G=8, Hkv=1),
    dict(S_len=300, own=[10] * 70, G=4, Hkv=1),
    # heads: one a key head, odd groups, a whole tile's
    dict(S_len=190, own=[30, 31], G=1, Hkv=3, NB=2, Dmax=3), dict(S_len=515, own=[60, 0, 7], G=7, Hkv=2, Dmax=5),
    dict(S_len=333, own=[129], G=64, Hkv=1, Dmax=3), dict(S_len=140, own=[50, 50], G=3, Hkv=5, NB=4, Dmax=20),
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "S%d own%s" % (k["S_len"], k["own"][:3]))
@pytest.mark.parametrize("dh,paged,f32", [(128, False, False), (64, False, False), (128, True, False), (64, True, False), (128, False, True), (64, False, True),
                                          (128, True, True), (64, True, True)])
def test_against_oracle(kw, dh, paged, f32):
    c = Case(1, dh=dh, paged=paged, f32=f32, **kw)
    c.check(c.run())


@pytest.mark.parametrize("dh", [64, 128])
def test_long_prompt_and_fp32_output(dh):
    c = Case(2, S_len=9001, own=[700, 33], Dmax=3, G=4, Hkv=1, dh=dh)
    c.check(c.run())
    c.check(c.run(out_f32=True))


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("kw", [dict(S_len=40000, own=[300, 0, 129], G=64, Hkv=1, Dmax=3), dict(S_len=30100, own=[1] * 6, G=4, Hkv=2),
                                dict(S_len=0, own=[130] * 400, G=1, Hkv=1), dict(S_len=5000, own=[1, 129, 257, 0, 300] * 60, G=2, Hkv=2),
                                dict(S_len=6000, own=[700] * 3, NB=3, Dmax=43, G=2, Hkv=2)], ids=["long", "narrow", "short", "mixed", "wide"])
def test_runs_of_several_tiles_and_segments(kw, dh):
    """More units than CTAs: runs of several key tiles, of several segments that end inside a tile, one
    and two row tiles in turns."""
    c = Case(13, dh=dh, **kw)
    c.check(c.run())


def test_scale_and_sharp_scores():
    """Scores that differ by hundreds: the reference maximum moves, most weights vanish."""
    c = Case(3, S_len=1500, own=[400], Dmax=4, G=4, Hkv=1, q_scale=12.0)
    c.check(c.run())
    d = Case(4, S_len=600, own=[100], Dmax=2, G=2, Hkv=2, f32=True)
    args, tables = d.device()
    got = S.ssd_verify_attn_shared(*args, d.Dmax, scale=0.02)
    f = lambda x: x.double().numpy()
    want = A.attention(f(d.q), [f(x) for x in d.shared], [[f(x) for x in o] for o in d.own], [f(x) for x in d.cand], d.blk.numpy(), d.Dmax, 0.02)
    for (b, t), (o, _) in want.items():
        np.testing.assert_allclose(got[b, t].cpu().numpy(), o, rtol=1e-4, atol=1e-5)


def test_maxima_that_grow_along_the_keys():
    c = Case(5, S_len=1024, own=[640], Dmax=2, G=4, Hkv=1)
    ramp = torch.linspace(0.1, 6.0, 1024)[None, :, None]
    c.shared = ((c.shared[0].float().abs() * ramp).to(torch.bfloat16), c.shared[1])
    c.q = c.q.float().abs().to(torch.bfloat16)
    c.k_shared[:, :1024] = c.shared[0]
    c.check(c.run())


def test_rows_of_absent_tokens_stay_and_neighbours_too():
    c = Case(6, S_len=200, own=[17, 0, 140], NB=2, Dmax=4, blk=[[4, 1], [0, 0], [0, 3]])
    buf = torch.full((c.q.numel() + 256,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[128:128 + c.q.numel()].view(c.q.shape)
    c.run(out=out)
    c.check(out)
    assert (out[~c.present.to(DEV)] == -7).all() and (buf[:128] == -7).all() and (buf[-128:] == -7).all()


def test_equals_attention_over_the_whole_prefix():
    """The same keys as one prefix of ssd_verify_attn: both within the rounding of two bf16 outputs."""
    c = Case(7, S_len=512, own=[256, 256], NB=2, Dmax=8, G=4, Hkv=2, slack=0)
    got = c.run(out_f32=True)
    both = [torch.stack([torch.cat([c.shared[i], c.own[b][i]], 1) for b in range(2)]).to(DEV) for i in range(2)]
    P = torch.tensor([768, 768], dtype=torch.int32, device=DEV)
    want = S.ssd_verify_attn(c.q.to(DEV), *both, c.cand[0].to(DEV), c.cand[1].to(DEV), P, c.blk.to(DEV), c.Dmax, out_f32=True)
    assert (got - want).abs().max() < 2.0 ** -7


def test_infinities_in_masked_places_and_in_keys():
    c = Case(8, S_len=130, own=[3, 140], NB=2, Dmax=3, Hkv=1)
    for t in (*c.caches, c.k_shared, c.v_shared):
        t[torch.isnan(t)] = float("inf")
    c.check(c.run())
    # a key at -inf along a positive query weighs nothing; a value that is no number reaches its rows only
    c = Case(9, S_len=140, own=[0, 5], Hkv=1, G=1)
    c.q = c.q.abs()
    c.k_shared[0, 77] = float("-inf")
    got = c.run(out_f32=True)
    assert torch.isfinite(got).all()
    d = Case(9, S_len=140, own=[0, 5], Hkv=1, G=1)
    d.caches[1][1, 0, 2, 4] = float("nan")
    got = d.run(out_f32=True).cpu()
    assert torch.isfinite(got[0]).all() and torch.isnan(got[1, 0, 0, 4]) and torch.isfinite(got[1, 0, 0, 5:]).all()


def test_reported_errors():
    c = Case(10, S_len=200, own=[10, 20], paged=True)
    args, tables = c.device()
    n = S.ssd_verify_attn_shared_workspace_size(S.attn_shared_args(*args, c.Dmax, torch.empty_like(args[0]), **tables))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    c.check(S.ssd_verify_attn_shared(*args, c.Dmax, **tables, ws=ws))
    assert S.ssd_read_device_error(ws) == S.SSD_OK
    for which, bad in (("shared_len", 10 ** 6), ("prefix", 200), ("prefix", -1), ("page", 99), ("shared page", -4)):
        args, tables = c.device()
        if which == "shared_len":
            args[3][0] = bad
        elif which == "prefix":
            args[8][1] = bad
        elif which == "page":
            tables["block_table"][0, 0] = bad
        else:
            tables["shared_table"][1] = bad
        S.ssd_verify_attn_shared(*args, c.Dmax, **tables, ws=ws)
        assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE, which
        assert S.ssd_read_device_error(ws) == S.SSD_OK


def test_repeats_bit_for_bit_from_a_graph_and_on_another_stream():
    c = Case(11, S_len=2000, own=[300, 0, 129, 511], NB=3, Dmax=5, paged=True)
    args, tables = c.device()
    out = torch.zeros_like(args[0])
    n = S.ssd_verify_attn_shared_workspace_size(S.attn_shared_args(*args, c.Dmax, out, **tables))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    want = c.run(out=torch.zeros_like(args[0])).clone()
    g = torch.cuda.CUDAGraph()
    S.ssd_verify_attn_shared(*args, c.Dmax, **tables, out=out, ws=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        S.ssd_verify_attn_shared(*args, c.Dmax, **tables, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # lengths and blocks are read on the device: the same graph serves the next step
    args[8].copy_(torch.tensor([299, 1, 0, 500], dtype=torch.int32))
    args[9].copy_(torch.tensor([[5, 0, 1], [0, 2, 0], [0, 0, 0], [3, 3, 3]], dtype=torch.int32))
    out.zero_()
    g.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = S.ssd_verify_attn_shared(*args, c.Dmax, **tables, out=torch.zeros_like(out), stream=side)
    torch.cuda.synchronize()
    # bit for bit: sequence 1's new key is one of the places that hold no number
    assert torch.equal(out.view(torch.int16), other.view(torch.int16))


def test_refusals():
    c = Case(12, S_len=64, own=[10])
    args, _ = c.device()
    call = lambda *a, **kw: S.ssd_verify_attn_shared(*a, c.Dmax, **kw)
    change = lambda i, x: args[:i] + [x] + args[i + 1:]
    with pytest.raises(ValueError, match="v_shared"):
        call(*change(2, args[2][:, :-1].contiguous()))
    with pytest.raises(ValueError, match="shared_len must be"):
        call(*change(3, torch.zeros(2, dtype=torch.int32, device=DEV)))
    with pytest.raises(ValueError, match="dtype"):
        call(*change(4, args[4].float()))
    with pytest.raises(ValueError, match="goes with a block_table"):
        call(*args, shared_table=torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="overlap"):
        call(*args, out=args[0])
    with pytest.raises(ValueError, match="pages of"):
        call(*args, block_table=torch.zeros((1, 1), dtype=torch.int32, device=DEV))
    with pytest.raises(S.SsdError, match="workspace"):
        call(*args, ws=torch.zeros(256, dtype=torch.uint8, device=DEV))
    wide = torch.zeros((1, 1, 8, 96), dtype=torch.bfloat16, device=DEV)
    kv, sh = torch.zeros((1, 2, 10, 96), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 64, 96), dtype=torch.bfloat16, device=DEV)
    cand = torch.zeros((1, 1, 2, 96), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(S.SsdError, match="unsupported"):
        call(wide, sh, sh, args[3], kv, kv, cand, cand, args[8], args[9])
    assert S.ssd_verify_attn_shared(*[x[:0] if i in (0, 4, 5, 6, 7, 8, 9) else x for i, x in enumerate(args)], c.Dmax).shape[0] == 0
