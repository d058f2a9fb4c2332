"""A serving step over the 8-bit cache as one captured graph: pages, the last token's row, verification
attention, acceptance, commit and trim, every call reading what the one before wrote."""
import numpy as np
import pytest
import torch

import kv_quant_helpers as H
from oracle import kv_quant_oracle as K
from oracle import ssd_oracle as O
from speculative_decoding_copy_gb300 import _binding as S

pytestmark = pytest.mark.gpu
dev = H.dev


@pytest.mark.parametrize("NB,Dmax,G", [(1, 1, 4), (2, 2, 4), (3, 6, 4), (2, 20, 8)])
@pytest.mark.parametrize("dh", [64, 128])
def test_a_captured_serving_step(dh, NB, Dmax, G):
    """Five replays with new inputs in place: the tables, lengths, codes and decisions are the oracle's, the
    attention within tolerance. The appended row lies one place before the committed ones and differs
    from them, so that no call can be left out unseen."""
    rng = np.random.default_rng(dh + Dmax)
    B, Hkv, sb, pps, V = 4, 2, 32, 5, 40
    length = np.array([127, 0, 254, 383 - Dmax], np.int32)
    held = -(-length // 128)
    pool = B * pps + 3
    order = rng.permutation(pool).astype(np.int32)
    table, at = np.full((B, pps), -1, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    stack, n = np.concatenate([order[at:], np.zeros(at, np.int32)]).astype(np.int32), pool - at
    c = [x for w in range(2) for x in H.cache(rng, pool, Hkv, 128, dh, sb)]         # k codes, k scales, v codes, v scales
    t = [dev(c[i]) for i in (0, 2, 1, 3)]
    d = [dev(x) for x in (held, table, stack, np.array([n], np.int32))]
    len_d, one = dev(length), dev(np.ones(B, np.int32))
    room, zero = dev(np.full(B, 1 + Dmax, np.int32)), dev(np.zeros(B, np.int32))
    NT = NB * Dmax

    def inputs():
        case = H.AttnCase(int(rng.integers(1 << 30)), [1] * B, NB, Dmax, G, Hkv, dh, sb, True)
        tok = rng.integers(0, V, (B, NB, Dmax)).astype(np.int32)
        tgt = rng.standard_normal((B, 1 + NT, V)).astype(np.float32)
        for b in range(B):                                       # a run of each block is what the target says
            for k in range(NB):
                for i in range(int(rng.integers(0, case.blk_len[b, k] + 1))):
                    tgt[b, 0 if i == 0 else 1 + k * Dmax + i - 1, tok[b, k, i]] += 20.0
        row, row64 = H.bf16(rng, B, 2, Hkv, dh)
        return case, tok, tgt, row, row64

    def host(x):
        case, tok, tgt, row, _ = x
        return [case.q, case.kc, case.vc, case.blk_len, tok, tgt, np.ascontiguousarray(row[:, 0]), np.ascontiguousarray(row[:, 1])]

    x = inputs()
    q, kc, vc, blk_len, tok, tgt, k_row, v_row = held_in = [dev(a) for a in host(x)]
    out = torch.zeros((B, NT, Hkv * G, dh), dtype=torch.float32, device="cuda")
    acc = S.alloc_accept_outputs(B, NB, Dmax, "cuda")
    new_len = torch.zeros_like(len_d)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kind = dict(mode=S.SSD_GREEDY, kind=S.SSD_LOGITS_F32)
    need = S.ssd_accept_workspace_size(S.accept_args(S.SSD_GREEDY, S.SSD_LOGITS_F32, tgt, None, tok, blk_len, 0, -1, None, None, acc))
    acc_ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = S.ssd_page_tables(len_d, room, *d, B * (1 + Dmax), ws=ws)
        slots = got["slot_map"].view(B, 1 + Dmax)[:, 0].contiguous()
        S.ssd_append_kv_quant(k_row, v_row, slots, *t, sb, ws=ws)
        with_row = len_d + one
        S.ssd_verify_attn_quant(q, *t, kc, vc, with_row, blk_len, Dmax, sb, out=out, ws=ws, block_table=d[1])
        S.ssd_accept(tgt, None, tok, blk_len, None, None, **kind, out=acc, ws=acc_ws)
        S.ssd_commit_kv_quant(*t, kc, vc, with_row, acc["best_blk"], acc["n_out"], Dmax, sb, new_len=new_len, block_table=d[1], ws=ws)
        S.ssd_page_tables(new_len, zero, *d, 0, ws=ws)
        len_d.copy_(new_len)
    grown = 0
    for step in range(5):
        if step:
            x = inputs()
            for a, b in zip(held_in, host(x)):
                a.copy_(dev(b))
        case, tok_h, tgt_h, _, row64 = x
        graph.replay()
        n, _, want, served, err = K.page_tables(length, np.full(B, 1 + Dmax, np.int32), held, table, stack, n, B * (1 + Dmax))
        assert served.all() and not err
        for w in range(2):
            K.append(row64[:, w], want.reshape(B, -1)[:, 0], c[2 * w], c[2 * w + 1], sb)
        case.prefix, case.table = length + 1, table
        case.k_codes, case.k_scale, case.v_codes, case.v_scale = c
        case.check(out)
        ref = O.verify_step_accept("greedy", "logits_f32", tgt_h, None, tok_h, case.blk_len, NB, 0, None, None)
        for key in ("acc_len", "best_blk", "n_out", "out_tok"):
            np.testing.assert_array_equal(acc[key].cpu().numpy(), ref[key], err_msg=key)
        for w, rows in enumerate((case.kc64, case.vc64)):
            new, ok = K.commit(rows, length + 1, ref["best_blk"], ref["n_out"], Dmax, c[2 * w], c[2 * w + 1], sb, table)
            assert ok.all()
        grown += int((new - length - 1).sum())
        length = new.astype(np.int32)
        n, *_ = K.page_tables(length, np.zeros(B, np.int32), held, table, stack, n, 0)
        np.testing.assert_array_equal(len_d.cpu().numpy(), length)
        np.testing.assert_array_equal(got["slot_map"].cpu().numpy(), want)
        for a, b in zip(d, (held, table, stack, [n])):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        for a, b in zip(t, (c[0], c[2], c[1], c[3])):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
    assert grown > 0
    assert S.ssd_read_device_error(ws) == S.SSD_OK and S.ssd_read_device_error(acc_ws) == S.SSD_OK
