"""Sampled continuations of one prompt, the calls together: tokens drafted from a cut distribution, verified
by attention over the shared prompt, the target's rows cut by the same settings, accepted by rejection
sampling and committed behind each sequence's own prefix."""
import numpy as np
import pytest
import torch

from oracle import attn_shared_oracle as A
from oracle import sample_oracle as Q
from speculative_decoding_copy_gb300 import _binding as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Rollout:
    """A toy model of one attention layer: everything a token contributes comes from tables."""

    def __init__(self, seed, B=5, K=4, V=3001, Hq=8, Hkv=2, dh=64, prompt=300, room=64):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(torch.bfloat16).to(DEV)
        self.B, self.K, self.V, self.Hq, self.Hkv, self.dh = B, K, V, Hq, Hkv, dh
        self.q_of, self.k_of, self.v_of = new(V, Hq, dh), new(V, Hkv, dh), new(V, Hkv, dh)
        self.draft = new(V, V, k=1.5).float()
        self.head = new(Hq * dh, V, k=0.2).float()
        self.k_shared, self.v_shared = new(Hkv, prompt, dh), new(Hkv, prompt, dh)
        self.shared_len = torch.tensor([prompt], dtype=torch.int32, device=DEV)
        self.k_cache, self.v_cache = new(B, Hkv, room, dh) * 0, new(B, Hkv, room, dh) * 0
        self.prefix = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.blk = torch.full((B, 1), K, dtype=torch.int32, device=DEV)
        f = lambda *v: torch.tensor((v * B)[:B], dtype=torch.float32, device=DEV)
        self.setting = dict(temperature=f(0.7, 1.0, 0.0), top_k=torch.tensor(([50, 0, 0] * B)[:B], dtype=torch.int32, device=DEV), top_p=f(0.9, 0.95, 1.0), min_p=f(0.0, 0.02, 0.0))
        self.last = torch.randint(0, V, (B,), generator=g).to(DEV)
        self.u = torch.rand((8, B, 2 * K + 2), generator=g).to(DEV)
        self.ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        self.drf = torch.zeros((B, K, V), device=DEV)
        self.tgt = torch.zeros((B, 1 + K, V), device=DEV)

    def step(self, n):
        """One draft-and-verify step; everything it made."""
        u, tok, chain = self.u[n], self.last, []
        for i in range(self.K):
            row = torch.empty((self.B, self.V), device=DEV)
            got = S.ssd_sample(self.draft[tok], u[:, i].contiguous(), **self.setting, probs_out=row, ws=self.ws)
            tok = got["token"].long()
            chain.append(got["token"])
            self.drf[:, i] = row
        chain = torch.stack(chain, 1)
        # the current token's own position and those of the drafted ones are one block of K + 1
        block = torch.cat([self.last[:, None], chain.long()], 1)
        q, k, v = self.q_of[block], self.k_of[block], self.v_of[block]
        full = torch.full_like(self.blk, self.K + 1)
        attn = S.ssd_verify_attn_shared(q, self.k_shared, self.v_shared, self.shared_len, self.k_cache, self.v_cache, k, v, self.prefix, full, self.K + 1, out_f32=True)
        logits = attn.flatten(2) @ self.head
        S.ssd_filter_probs(logits, **self.setting, blk_len=self.blk, Dmax=self.K, out=self.tgt, ws=self.ws)
        acc = S.ssd_accept(self.tgt, self.drf, chain.view(self.B, 1, self.K), self.blk, u[:, self.K:2 * self.K].reshape(self.B, 1, self.K).contiguous(),
                           u[:, -1].contiguous(), mode=S.SSD_SAMPLE, kind=S.SSD_PROBS_F32, K=self.K, chain_blk=0)
        # the current token and the accepted ones enter the own cache: n_out of the block's K + 1 rows
        before = self.prefix.clone()
        S.ssd_commit_kv(self.k_cache, self.v_cache, k.contiguous(), v.contiguous(), self.prefix, acc["best_blk"], acc["n_out"] + 1, self.K + 1, ws=self.ws)
        self.last = acc["out_tok"].gather(1, (acc["n_out"] - 1)[:, None].long())[:, 0].long()
        return dict(chain=chain, q=q, k=k, v=v, attn=attn, logits=logits, acc=acc, before=before, drf=self.drf.clone(), tgt=self.tgt.clone())


def test_steps_of_a_rollout():
    r = Rollout(1)
    setting = [{k: (int if k == "top_k" else float)(v[b]) for k, v in r.setting.items()} for b in range(r.B)]
    f = lambda t: t.double().cpu().numpy()
    kept = 0
    for n in range(4):
        caches = [r.k_cache.clone(), r.v_cache.clone()]
        s = r.step(n)
        torch.cuda.synchronize()
        assert S.ssd_read_device_error(r.ws) == S.SSD_OK
        before, acc = s["before"].tolist(), {k: v.cpu().numpy() for k, v in s["acc"].items()}
        # attention over prompt, own prefix and block
        own = [[f(c[b, :, :before[b]]) for c in caches] for b in range(r.B)]
        want = A.attention(f(s["q"]), [f(r.k_shared), f(r.v_shared)], own, [f(s["k"]), f(s["v"])], np.full((r.B, 1), r.K + 1), r.K + 1)
        for (b, t), (o, spread) in want.items():
            assert (np.abs(f(s["attn"])[b, t] - o) <= 2.0 ** -16 * np.abs(o) + (2.0 ** -7 + 2.0 ** -12) * spread + 1e-7).all()
        drf, tgt, chain, u = f(s["drf"]), f(s["tgt"]), s["chain"].cpu().numpy(), r.u[n].cpu().numpy()
        for b in range(r.B):
            for i in range(1 + r.K):
                p = Q.probs(f(s["logits"])[b, i], **setting[b])
                if Q.kept(f(s["logits"])[b, i], **setting[b])[2] > 2.0 ** -27:
                    np.testing.assert_allclose(tgt[b, i], p, rtol=2.0 ** -23.9, atol=2.0 ** -126)
            # each drafted token was possible, and accepted iff u q < p in turn
            a = 0
            while a < r.K and np.float64(u[b, r.K + a]) * drf[b, a, chain[b, a]] < tgt[b, a, chain[b, a]]:
                a += 1
            assert (drf[b, np.arange(r.K), chain[b]] > 0).all()
            assert acc["n_out"][b] == a + 1 and (acc["out_tok"][b, :a] == chain[b, :a]).all()
            assert tgt[b, a, acc["out_tok"][b, a]] > 0
            kept += a
            m = before[b] + a + 1
            assert int(r.prefix[b]) == m
            rows = torch.cat([s["k"][b, :a + 1]]).transpose(0, 1)
            assert torch.equal(r.k_cache[b, :, before[b]:m], rows)
    assert kept > 0


def test_a_step_captured_and_replayed():
    """Draft, attention, cut rows and acceptance as one graph: the same results as the eager calls, and from
    other inputs copied into its buffers those of their eager calls."""
    r = Rollout(2)
    x = r.draft[r.last].clone()
    u = r.u[0].clone()
    tok = dict(token=torch.empty(r.B, dtype=torch.int32, device=DEV), prob=torch.empty(r.B, device=DEV))
    row = torch.empty((r.B, r.V), device=DEV)
    q, k, v = (t[:r.B * (r.K + 1)].clone().view(r.B, r.K + 1, *t.shape[1:]) for t in (r.q_of, r.k_of, r.v_of))
    full = torch.full_like(r.blk, r.K + 1)
    out = torch.empty(q.shape, dtype=torch.float32, device=DEV)
    a = S.attn_shared_args(q, r.k_shared, r.v_shared, r.shared_len, r.k_cache, r.v_cache, k, v, r.prefix, full, r.K + 1, out)
    aws = torch.zeros(S.ssd_verify_attn_shared_workspace_size(a), dtype=torch.uint8, device=DEV)
    logits = torch.empty((r.B, r.K + 1, r.V), device=DEV)
    us = [u[:, i].contiguous() for i in range(2)]

    def step():
        S.ssd_sample(x, us[0], **r.setting, out=tok, probs_out=row, ws=r.ws)
        S.ssd_verify_attn_shared(q, r.k_shared, r.v_shared, r.shared_len, r.k_cache, r.v_cache, k, v, r.prefix, full, r.K + 1, out=out, ws=aws)
        torch.matmul(out.flatten(2), r.head, out=logits)
        S.ssd_filter_probs(logits, **r.setting, blk_len=r.blk, Dmax=r.K, out=r.tgt, ws=r.ws)

    def results():
        step()
        torch.cuda.synchronize()
        return [t.clone() for t in (tok["token"], tok["prob"], row, out, r.tgt)]

    first = results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for t in (row, out, r.tgt):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, (tok["token"], tok["prob"], row, out, r.tgt)))
    x.copy_(r.draft[(r.last + 1) % r.V])
    r.prefix.copy_(torch.tensor([3, 0, 64, 17, 1], dtype=torch.int32))
    r.blk.copy_(torch.tensor([[4], [0], [2], [1], [3]], dtype=torch.int32))
    want = results()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (tok["token"], tok["prob"], row, out, r.tgt)))


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace and outputs."""
    r, s = Rollout(3), Rollout(4, B=7, prompt=3000)
    streams = [torch.cuda.Stream() for _ in range(2)]

    def calls(o, stream):
        full = torch.full_like(o.blk, o.K + 1)
        q, k, v = (t[:o.B * (o.K + 1)].view(o.B, o.K + 1, *t.shape[1:]) for t in (o.q_of, o.k_of, o.v_of))
        att = S.ssd_verify_attn_shared(q, o.k_shared, o.v_shared, o.shared_len, o.k_cache, o.v_cache, k, v, o.prefix, full, o.K + 1, stream=stream)
        probs = S.ssd_filter_probs(o.draft[:40], stream=stream, top_p=torch.full((1,), 0.9, device=DEV))
        return att, probs

    torch.cuda.synchronize()
    alone = [calls(o, None) for o in (r, s)]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [calls(o, st) for o, st in zip((r, s), streams)]
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
