"""The 8-bit cache on the GPU against its oracle: page tables and slot maps and the cache's
bytes exactly, attention within a derived tolerance; its edges, errors, streams and graphs;
and a serving loop that uses all four calls."""
import numpy as np
import pytest
import torch

import kv_quant_helpers as H
from oracle import kv_quant_oracle as K
from oracle import ssd_oracle as O
from speculative_decoding_copy_gb300 import _binding as S
from speculative_decoding_copy_gb300 import workloads as WL

pytestmark = pytest.mark.gpu
dev = H.dev


# ---------------------------------------------------------------------------- page tables
def _books(rng, B, pps, spare, empty=False):
    held = np.zeros(B, np.int32) if empty else rng.integers(0, pps + 1, B).astype(np.int32)
    n = int(held.sum())
    order = rng.permutation(n + spare).astype(np.int32)
    table, at = np.full((B, pps), -1, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    stack = np.zeros(n + spare, np.int32)
    stack[:spare] = order[n:]
    return held, table, stack, spare


@pytest.mark.parametrize("B,pps,spare,cap", [(1, 3, 4, 300), (7, 5, 9, 2000), (33, 4, 0, 40000), (1024, 3, 700, 9000),
                                             (1025, 3, 500, 0), (2500, 2, 4000, 600000)])
def test_page_tables_match_the_oracle(B, pps, spare, cap):
    rng = np.random.default_rng(B)
    held, table, stack, n = _books(rng, B, pps, spare)
    d = [dev(x) for x in (held, table, stack, np.array([n], np.int32))]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    seen = set()
    for step in range(4):
        cur = rng.integers(0, pps * 128 + 1, B).astype(np.int32)
        add = np.minimum(rng.integers(0, 200, B), pps * 128 - cur).astype(np.int32)
        add[rng.random(B) < 0.3] = 0
        if cap == 0:
            add[:] = 0
        n, start, slots, served, err = K.page_tables(cur, add, held, table, stack, n, cap)
        got = S.ssd_page_tables(dev(cur), dev(add), *d, cap, ws=ws)
        for name, ref in (("row_start", start), ("slot_map", slots), ("served", served)):
            np.testing.assert_array_equal(got[name].cpu().numpy(), ref, err_msg=name)
        for t, ref in zip(d, (held, table, stack, [n])):
            np.testing.assert_array_equal(t.cpu().numpy(), ref)
        assert S.ssd_read_device_error(ws) == (S.SSD_ERR_DEVICE if err else S.SSD_OK)
        seen |= set(served.tolist())
    assert 1 in seen


def test_page_tables_report_and_leave_what_does_not_fit():
    """Negative lengths, too long a sequence and a spoiled page count: left alone, not served."""
    rng = np.random.default_rng(3)
    held, table, stack, n = _books(rng, 6, 4, 9)
    held[4] = 9                                        # more pages than the table has
    cur = np.array([10, -1, 600, 5, 10, 100], np.int32)
    add = np.array([200, 5, 0, -7, 3, 20], np.int32)
    d = [dev(x) for x in (held, table, stack, np.array([n], np.int32))]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    n, start, slots, served, err = K.page_tables(cur, add, held, table, stack, n, 400)
    got = S.ssd_page_tables(dev(cur), dev(add), *d, 400, ws=ws)
    assert err and S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE
    assert served.tolist() == [1, 0, 0, 0, 0, 1]
    for name, ref in (("row_start", start), ("slot_map", slots), ("served", served)):
        np.testing.assert_array_equal(got[name].cpu().numpy(), ref, err_msg=name)
    for t, ref in zip(d, (held, table, stack, [n])):
        np.testing.assert_array_equal(t.cpu().numpy(), ref)


def test_page_tables_keep_within_a_spoiled_stack():
    """n_free out of range, ids outside the pool, a stack without room, more rows than slots."""
    i32 = lambda *v: dev(np.array(v, np.int32))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    # 3 pages claimed free + 1 more than the pool has
    d = [i32(0), torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), i32(0, 77, 2), i32(4)]
    got = S.ssd_page_tables(i32(0), i32(300), *d, 350, ws=ws)
    assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE
    s = got["slot_map"].cpu().numpy()
    assert d[1].cpu().tolist() == [[2, 77, 0, -1]] and d[3].cpu().tolist() == [0]
    assert (s[:128] == 256 + np.arange(128)).all() and (s[128:256] == -1).all() and (s[256:300] == np.arange(44)).all()
    assert (s[300:] == -1).all()
    # trimming onto a full stack drops the page; rows past slot_cap are not written
    d = [i32(1), i32(1).view(1, 1), i32(0, 1), i32(2)]
    S.ssd_page_tables(i32(0), i32(0), *d, 0, ws=ws)
    assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE and d[3].cpu().tolist() == [2] and d[1].cpu().tolist() == [[-1]]
    d = [i32(0), i32(-1).view(1, 1), i32(1, 0), i32(2)]
    got = S.ssd_page_tables(i32(3), i32(9), *d, 4, ws=ws)
    assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE and got["slot_map"].cpu().tolist() == [3, 4, 5, 6]
    # nothing at all
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = S.ssd_page_tables(e, e, e, e.view(0, 0), e, i32(0), 3, ws=ws)
    assert got["row_start"].cpu().tolist() == [0] and got["slot_map"].cpu().tolist() == [-1] * 3
    assert S.ssd_read_device_error(ws) == S.SSD_OK


# ---------------------------------------------------------------------------- writers
def _same_cache(c, t):
    for ref, got in zip(c, t):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dh,sb,Hkv,tokens", [(128, 128, 2, 128), (64, 16, 3, 128), (128, 32, 1, 128), (64, 64, 2, 301),
                                              (128, 16, 2, 1000)])
def test_append_is_exact(f32, dh, sb, Hkv, tokens):
    """Prompts, single tokens and runs that start inside blocks, block scales that grow, padding
    rows; rows of a stride; whatever is not written keeps its bytes."""
    rng = np.random.default_rng(dh + sb + Hkv)
    pages = 9 if tokens == 128 else 3
    c = [x for w in range(2) for x in H.cache(rng, pages, Hkv, tokens, dh, sb, pow2=(w == 0))]
    t = [dev(x) for x in c]
    order = rng.permutation(pages)
    lens = rng.integers(0, tokens // 2, pages)
    for step in range(6):
        runs = []
        for pg in order:
            n = int(rng.choice([0, 1, 1, 3, tokens // 3]))
            n = min(n, tokens - lens[pg])
            runs.append(pg * tokens + lens[pg] + np.arange(n))
            lens[pg] += n
        slots = np.concatenate(runs + [np.full(2, -1)]).astype(np.int32)
        if step == 3:
            slots = np.insert(slots, 0, [-1, -5]).astype(np.int32)     # padding in front too
        T = len(slots)
        x = (rng.standard_normal((T, 2, Hkv, dh)) * 2.0 ** rng.integers(-3, 4, (T, 2, 1, 1))).astype(np.float32)
        if f32:
            full, x64 = dev(x), x.astype(np.float64)
        else:
            bits = WL.f32_to_bf16_bits(x)
            full, x64 = dev(bits).view(torch.bfloat16), O.bf16_to_f64(bits)
        K.append(x64[:, 0], slots, c[0], c[1], sb)
        K.append(x64[:, 1], slots, c[2], c[3], sb)
        ws = S.ssd_append_kv_quant(full[:, 0], full[:, 1], dev(slots), t[0], t[2], t[1], t[3], sb)
        assert S.ssd_read_device_error(ws) == S.SSD_OK
        _same_cache(c, t)


def test_append_of_many_rows():
    """Long prompts: ranges of rows a CTA walks, runs across their borders."""
    rng = np.random.default_rng(8)
    Hkv, dh, pages = 2, 64, 64
    for sb in (16, 32, 64, 128):
        c = [x for w in range(2) for x in H.cache(rng, pages, Hkv, 128, dh, sb)]
        t = [dev(x) for x in c]
        parts, at = [], 0
        for n in (1000, 129, 3, 1, 2047, 640, 17):
            first = int(rng.integers(0, 128))
            use = -(-(first + n) // 128)
            pos = first + np.arange(n)
            parts.append((at + pos // 128) * 128 + pos % 128)
            at += use
        slots = np.concatenate(parts).astype(np.int32)
        bits, x64 = H.bf16(rng, len(slots), 2, Hkv, dh)
        K.append(x64[:, 0], slots, c[0], c[1], sb)
        K.append(x64[:, 1], slots, c[2], c[3], sb)
        full = dev(bits)
        S.ssd_append_kv_quant(full[:, 0], full[:, 1], dev(slots), t[0], t[2], t[1], t[3], sb)
        _same_cache(c, t)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sb", [16, 32, 64, 128])
def test_append_of_a_large_prompt(sb, f32):
    """Enough rows that a CTA walks 128 of them, all its groups at work."""
    rng = np.random.default_rng(sb)
    T, Hkv, dh, pages = 16500, 16, 64, 135
    c = [x for w in range(2) for x in H.cache(rng, pages, Hkv, 128, dh, sb)]
    t = [dev(x) for x in c]
    order = rng.permutation(pages)
    pos = 5 + np.arange(T)
    slots = (order[pos // 128] * 128 + pos % 128).astype(np.int32)
    slots[7040 - 5:7168 - 5] = -1        # whole blocks: a hole inside one would leave it two runs, whose order is open
    if f32:
        x = rng.standard_normal((T, 2, Hkv, dh)).astype(np.float32)
        rows, x64 = dev(x), x.astype(np.float64)
    else:
        bits, x64 = H.bf16(rng, T, 2, Hkv, dh)
        rows = dev(bits)
    K.append(x64[:, 0], slots, c[0], c[1], sb)
    K.append(x64[:, 1], slots, c[2], c[3], sb)
    S.ssd_append_kv_quant(rows[:, 0], rows[:, 1], dev(slots), t[0], t[2], t[1], t[3], sb)
    _same_cache(c, t)


def test_append_edges():
    """Infinities, NaN, zero rows, borders of a scale, tiny and huge rows, slots past the pool."""
    rng = np.random.default_rng(9)
    Hkv, dh, sb = 1, 64, 16
    c = [x for w in range(2) for x in H.cache(rng, 4, Hkv, 128, dh, sb)]
    t = [dev(x) for x in c]
    x = np.zeros((9, Hkv, dh), np.float32)
    x[0] = rng.standard_normal((Hkv, dh)) * 1e-30
    x[1, 0, 3], x[1, 0, 4] = np.inf, -np.inf
    x[2] = np.nan
    x[3, 0, :5] = [448, -448, 2.0 ** -9, 2.0 ** -10, -0.0]
    x[4, 0, 0] = np.nextafter(np.float32(448 * 2.0 ** 20), np.float32(np.inf))
    x[5] = 3e38
    x[6] = 0
    x[7] = 1e-45
    x[8] = rng.standard_normal((Hkv, dh))
    slots = np.array([0, 1, 2, 16, 17, 40, 128, 129, 4 * 128], np.int32)
    for i in range(9):                                  # one row a call, then all at once into fresh places
        K.append(x[i:i + 1].astype(np.float64), slots[i:i + 1], c[0], c[1], sb)
        K.append(-x[i:i + 1].astype(np.float64), slots[i:i + 1], c[2], c[3], sb)
        ws = S.ssd_append_kv_quant(dev(x[i:i + 1]), dev(-x[i:i + 1]), dev(slots[i:i + 1]), t[0], t[2], t[1], t[3], sb)
        assert S.ssd_read_device_error(ws) == (S.SSD_ERR_DEVICE if i == 8 else S.SSD_OK)
    _same_cache(c, t)
    slots = slots + 256
    K.append(x.astype(np.float64), slots, c[0], c[1], sb)
    K.append(x.astype(np.float64), slots, c[2], c[3], sb)
    S.ssd_append_kv_quant(dev(x), dev(x), dev(slots), t[0], t[2], t[1], t[3], sb)
    _same_cache(c, t)
    e = torch.empty((0, Hkv, dh), device="cuda")
    S.ssd_append_kv_quant(e, e, torch.empty(0, dtype=torch.int32, device="cuda"), t[0], t[2], t[1], t[3], sb)
    _same_cache(c, t)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dh,sb,Dmax", [(128, 16, 20), (64, 128, 1), (128, 64, 256), (64, 32, 7)])
def test_commit_is_exact(f32, paged, dh, sb, Dmax):
    rng = np.random.default_rng(dh + sb + Dmax)
    B, NB, Hkv, P_max = 8, 2, 2, 640
    prefix = np.array([0, 1, sb - 1, sb, 127, 128, P_max - 1, 300], np.int32)
    best = np.array([0, 1, 1, 0, 1, -1, 0, 1], np.int32)
    n_out = np.array([Dmax + 1, 2, Dmax, 1, Dmax + 1, Dmax, 3, min(Dmax + 1, 100)], np.int32)
    if paged:
        table = rng.permutation(B * 5 + 2)[:B * 5].reshape(B, 5).astype(np.int32)
        table[7, 2] = -1                                # its run starts at 300: page 2
        c = [x for w in range(2) for x in H.cache(rng, B * 5 + 2, Hkv, 128, dh, sb, pow2=(w == 0))]
    else:
        table = None
        c = [x for w in range(2) for x in H.cache(rng, B, Hkv, P_max, dh, sb, pow2=(w == 0))]
    t = [dev(x) for x in c]
    x = rng.standard_normal((2, B, NB * Dmax, Hkv, dh)).astype(np.float32) * 3
    bits = WL.f32_to_bf16_bits(x)
    cand, x64 = (dev(x), x.astype(np.float64)) if f32 else (dev(bits), O.bf16_to_f64(bits))
    ref, ok = K.commit(x64[0], prefix, best, n_out, Dmax, c[0], c[1], sb, table)
    K.commit(x64[1], prefix, best, n_out, Dmax, c[2], c[3], sb, table)
    pre = dev(prefix)
    args = (t[0], t[2], t[1], t[3], cand[0], cand[1], pre, dev(best), dev(n_out), Dmax, sb)
    new, ws = S.ssd_commit_kv_quant(*args, block_table=None if table is None else dev(table))
    assert S.ssd_read_device_error(ws) == (S.SSD_OK if ok.all() else S.SSD_ERR_DEVICE)
    assert ok.any() and not ok.all()
    np.testing.assert_array_equal(new.cpu().numpy(), ref)
    np.testing.assert_array_equal(pre.cpu().numpy(), prefix)
    _same_cache(c, t)
    # the lengths are not updated in place: the same call again changes nothing
    S.ssd_commit_kv_quant(*args, new_len=new, block_table=None if table is None else dev(table))
    _same_cache(c, t)


# ---------------------------------------------------------------------------- attention
LENGTHS = [0, 1, 15, 16, 17, 127, 128, 129, 300]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("G,NB,Dmax,sb", [(1, 1, 1, 128), (4, 1, 1, 16), (3, 2, 2, 64), (8, 1, 2, 32), (5, 1, 5, 16),
                                          (2, 3, 5, 32), (16, 1, 3, 128), (64, 1, 1, 64)])
def test_attention_matches_the_oracle(paged, dh, G, NB, Dmax, sb):
    case = H.AttnCase(G + dh + sb, LENGTHS, NB, Dmax, G, 2, dh, sb, paged)
    case.check(H.run(case))
    case.check(H.run(case, f32=False))


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("G,NB,Dmax,sb", [(4, 1, 13, 128), (7, 3, 5, 16), (8, 2, 9, 64), (1, 9, 16, 32), (64, 1, 1, 128), (13, 1, 10, 64),
                                          (3, 1, 130, 16)])
def test_attention_of_many_rows_matches_the_oracle(paged, dh, G, NB, Dmax, sb):
    case = H.AttnCase(7 * G + NB + Dmax, LENGTHS, NB, Dmax, G, 2, dh, sb, paged)
    assert case.many(G)
    case.poison()
    case.check(H.run(case))


@pytest.mark.parametrize("dh,G,NB,Dmax", [(128, 4, 1, 1), (64, 4, 4, 20), (128, 4, 4, 20), (128, 8, 5, 20), (128, 1, 9, 16),
                                          (128, 2, 1, 256), (128, 7, 3, 40), (64, 2, 1, 200), (128, 32, 2, 9)])
@pytest.mark.parametrize("sb", [16, 128])
def test_attention_of_many_rows_and_long_prefixes(dh, G, NB, Dmax, sb):
    case = H.AttnCase(G * Dmax + sb, [4100, 77, 0, 1153], NB, Dmax, G, 2, dh, sb, True)
    rng = np.random.default_rng(1)
    present = [(b, t) for b in range(4) for t in range(NB * Dmax) if t % Dmax < case.blk_len[b, t // Dmax]]
    pick = {present[i] for i in rng.choice(len(present), min(24, len(present)), replace=False)} | {present[0], present[-1]}
    case.check(H.run(case), pick)


@pytest.mark.parametrize("dh,NB,Dmax", [(64, 2, 3), (128, 2, 3), (64, 4, 20), (128, 4, 20)])
@pytest.mark.parametrize("paged", [False, True])
def test_attention_never_looks_at_masked_places(dh, NB, Dmax, paged):
    """NaN in every code, scale, query and candidate that no present token may see."""
    case = H.AttnCase(7, [0, 1, 130, 200, 385], NB, Dmax, 4, 2, dh, 32, paged)
    case.poison()
    case.check(H.run(case))


@pytest.mark.parametrize("dh,NB,Dmax", [(128, 2, 3), (128, 4, 20), (64, 2, 3), (64, 4, 20)])
def test_attention_keeps_a_spoiled_candidate_to_its_block(dh, NB, Dmax):
    """An infinite key or value of one present token reaches the rows that see it, no others."""
    case = H.AttnCase(11, [70, 200], NB, Dmax, 2, 2, dh, 64, True, blk_len=np.full((2, NB), Dmax))
    clean = H.run(case)
    case.vc[0, 1, 0, 5], case.kc[1, Dmax + 1, 1, :] = 0x7f80, 0x7fc0
    out = H.run(case).cpu().numpy()
    ref = clean.cpu().numpy().copy()
    ref[0, 1:Dmax, 0:2, 5] = np.inf                     # tokens 2.. of block 0, the heads of kv head 0
    ref[1, Dmax + 1:2 * Dmax, 2:4] = np.nan
    bad = ~np.isfinite(ref)
    assert (np.isnan(out[1, Dmax + 1:2 * Dmax, 2:4])).all() and (out[0, 1:Dmax, 0:2, 5] == np.inf).all()
    np.testing.assert_allclose(out[~bad], ref[~bad], rtol=2e-3, atol=2e-3)


@pytest.mark.parametrize("dh,Dmax", [(128, 1), (128, 20), (64, 3), (64, 20)])
def test_attention_with_block_scales_far_apart(dh, Dmax):
    """Blocks of zero values (the least scale), of scale zero, and of scales 2^12 apart: the
    probabilities of their keys still count, and the small blocks lose nothing to the large."""
    case = H.AttnCase(13, [700, 333], 2, Dmax, 4, 2, dh, 16, True, pow2=True, blk_len=np.full((2, 2), Dmax))
    rng = np.random.default_rng(2)
    kind = rng.integers(0, 4, case.v_scale.shape)
    blocks = case.v_codes.reshape(*case.v_codes.shape[:2], 8, 16, dh)
    blocks[kind == 1] = 0
    case.v_scale[kind == 1] = 2.0 ** -100
    case.v_scale[kind == 2] *= 2.0 ** -12
    case.v_scale[kind == 3] = 0.0
    case.k_scale[rng.random(case.k_scale.shape) < 0.2] = 0.0
    case.check(H.run(case))


@pytest.mark.parametrize("v_scale", [2.0 ** -16, 2.0 ** -8, 2.0 ** 6])
@pytest.mark.parametrize("dh,Dmax", [(64, 1), (64, 20), (128, 1), (128, 20)])
def test_attention_of_a_flat_prefix_beside_heavy_own_keys(dh, Dmax, v_scale):
    """Thousands of keys of equal small weight, which the own-block keys, without a value scale,
    must not push to the low end of the probabilities' range."""
    case = H.AttnCase(73, [5000, 333], 1, Dmax, 4, 2, dh, 64, True, blk_len=np.full((2, 1), Dmax))
    case.k_scale[:] = 2.0 ** -30
    case.v_scale[:] = v_scale
    case.check(H.run(case))


@pytest.mark.parametrize("dh,Dmax", [(128, 1), (128, 20), (64, 20)])
def test_attention_with_sharp_and_growing_scores(dh, Dmax):
    """Scores of +-60 whose maximum keeps growing along the prefix, far past every threshold."""
    case = H.AttnCase(17, [2000], 2, Dmax, 4, 1, dh, 16, True, q_scale=6.0, pow2=True, blk_len=np.full((1, 2), Dmax))
    for j, pg in enumerate(case.table[0]):
        case.k_scale[pg] = 2.0 ** (-9 + j // 4)
    case.check(H.run(case), wide=4.0)                   # score magnitudes of 4 x 32 in log2 units


def test_attention_shares_pages_and_reports_bad_ones():
    case = H.AttnCase(19, [256, 256], 1, 2, 4, 2, 128, 64, True, blk_len=np.full((2, 1), 2))
    case.table[1] = case.table[0]
    case.check(H.run(case))
    for Dmax, bad in ((2, len(case.k_codes)), (20, -3)):
        case = H.AttnCase(20, [256, 256], 2, Dmax, 4, 2, 128, 64, True)
        case.table[1, 1] = bad
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        out = S.ssd_verify_attn_quant(*case.args(), **case.kw(), ws=ws, out_f32=True)
        assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE
        case.table[1, 1] = 0                            # read as page 0
        case.check(out)
        case.prefix[1] = 1000                           # past the table: counts as no prefix
        out = S.ssd_verify_attn_quant(*case.args(), **case.kw(), ws=ws, out_f32=True)
        assert S.ssd_read_device_error(ws) == S.SSD_ERR_DEVICE
        case.prefix[1] = 0
        case.check(out)


def test_attention_scale_argument_and_no_sequences():
    case = H.AttnCase(23, [90], 1, 2, 2, 1, 64, 32, False, blk_len=[[2]])
    out = H.run(case, scale=0.25)
    k, v = (K.values(c, s, 32, case.prefix) for c, s in ((case.k_codes, case.k_scale), (case.v_codes, case.v_scale)))
    ref = K.attention(case.q64, k, v, case.kc64, case.vc64, case.blk_len, 2, scale=0.25)
    for (b, t), (o, size) in ref.items():
        np.testing.assert_allclose(out[b, t].cpu().numpy(), o, atol=float(size.max()) * 2.0 ** -9)
    case = H.AttnCase(24, [90], 1, 1, 2, 1, 64, 32, False)
    a = [x[:0] if torch.is_tensor(x) else x for x in case.args()]
    assert S.ssd_verify_attn_quant(*a).shape == (0, 1, 2, 64)


def test_attention_repeats_bit_for_bit():
    for Dmax in (1, 20):
        case = H.AttnCase(29, [3000, 500, 64], 2, Dmax, 4, 2, 128, 128, True)
        a = H.run(case)
        for _ in range(3):
            assert torch.equal(a, H.run(case))


@pytest.mark.parametrize("prefix,Dmax", [([4096] * 8, 9), ([20000], 9), ([30000], 13), ([4096, 100], 5), ([900] * 20, 1)])
@pytest.mark.parametrize("dh", [64, 128])
def test_attention_is_stable_over_many_calls(dh, prefix, Dmax):
    """The end of a CTA's products, the merge and the ring's reuse are ordered by waits: every
    one of many calls gives the first one's bits, and those are right."""
    case = H.AttnCase(43, prefix, 1, Dmax, 4, 2, dh, 64, True, blk_len=np.full((len(prefix), 1), Dmax))
    a, kw = case.args(), case.kw()
    first = S.ssd_verify_attn_quant(*a, **kw, out_f32=True)
    out = [torch.empty_like(first) for _ in range(200)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for o in out:
        S.ssd_verify_attn_quant(*a, **kw, out=o, ws=ws)
    assert all(torch.equal(o, first) for o in out)
    assert S.ssd_read_device_error(ws) == S.SSD_OK
    case.check(first)


@pytest.mark.parametrize("dh,NB,Dmax", [(64, 2, 3), (128, 1, 1), (128, 3, 20)])
def test_attention_without_a_prefix(dh, NB, Dmax):
    """Empty prefixes, and a contiguous cache of no tokens."""
    case = H.AttnCase(47, [0, 0, 0], NB, Dmax, 4, 2, dh, 16, False)
    case.check(H.run(case))
    case.k_codes, case.v_codes, case.k_scale, case.v_scale = (
        x[:, :, :0] for x in (case.k_codes, case.v_codes, case.k_scale, case.v_scale))
    case.check(H.run(case))


@pytest.mark.parametrize("B,NB,Dmax", [(400, 1, 1), (400, 2, 4), (97, 1, 2), (257, 1, 6)])
def test_attention_of_many_sequences(B, NB, Dmax):
    """More sequences than threads of a CTA: they run in their own order; fewer: by length."""
    case = H.AttnCase(53, list(np.random.default_rng(B).integers(0, 300, B)), NB, Dmax, 4, 1, 128, 32, True)
    case.check(H.run(case))


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("NB,Dmax,G", [(300, 16, 2), (1024, 8, 1), (8192, 1, 1), (32, 256, 1)])
def test_attention_of_many_sparse_blocks(dh, NB, Dmax, G):
    """One present token in each of many blocks: rows of one tile far apart in the slots."""
    blk_len = np.zeros((1, NB), np.int32)
    blk_len[:, ::max(1, NB // 300)] = 1
    blk_len[0, NB - 1] = Dmax
    case = H.AttnCase(59, [200], NB, Dmax, G, 1, dh, 128, True, blk_len=blk_len)
    case.poison()
    case.check(H.run(case))


@pytest.mark.parametrize("Dmax", [1, 20])
def test_pages_past_four_billion_bytes(Dmax):
    """A pool of 5 GB each of keys and values, of which the last pages are used."""
    pages, Hkv, dh, sb = 40000, 8, 128, 64
    case = H.AttnCase(61, [700, 130], 1, Dmax, 4, Hkv, dh, sb, True, blk_len=np.full((2, 1), Dmax))
    t = [torch.zeros((pages, Hkv, 128, dh), dtype=torch.uint8, device="cuda") for _ in range(2)]
    t += [torch.zeros((pages, Hkv, 128 // sb), dtype=torch.float32, device="cuda") for _ in range(2)]
    assert t[0].nbytes > 1 << 32
    held = len(case.k_codes)
    for x, part in zip(t, (case.k_codes, case.v_codes, case.k_scale, case.v_scale)):
        x[pages - held:] = dev(part)
    a = case.args()
    a[1:5] = t
    table = dev(case.table + pages - held)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    case.check(S.ssd_verify_attn_quant(*a, out_f32=True, block_table=table, ws=ws))
    # rows appended and committed behind the prefixes, in pages as far out
    c = [case.k_codes, case.k_scale, case.v_codes, case.v_scale]
    place = np.array([case.table[b, P // 128] * 128 + P % 128 for b, P in enumerate(case.prefix)], np.int32)
    K.append(case.kc64[:, 0], place, c[0], c[1], sb)
    K.append(case.vc64[:, 0], place, c[2], c[3], sb)
    S.ssd_append_kv_quant(a[5][:, 0], a[6][:, 0], dev(place + (pages - held) * 128), *t, sb, ws=ws)
    best, n_out = np.zeros(2, np.int32), np.full(2, Dmax + 1, np.int32)
    new, ok = K.commit(case.kc64, case.prefix + 1, best, n_out, Dmax, c[0], c[1], sb, case.table)
    K.commit(case.vc64, case.prefix + 1, best, n_out, Dmax, c[2], c[3], sb, case.table)
    assert ok.all()
    got, _ = S.ssd_commit_kv_quant(*t, a[5], a[6], dev(case.prefix + 1), dev(best), dev(n_out), Dmax, sb, block_table=table, ws=ws)
    np.testing.assert_array_equal(got.cpu().numpy(), new)
    _same_cache(c, [t[0][pages - held:], t[2][pages - held:], t[1][pages - held:], t[3][pages - held:]])
    assert not t[0][:pages - held].any() and not t[1][:pages - held].any()
    assert S.ssd_read_device_error(ws) == S.SSD_OK


# ---------------------------------------------------------------------------- streams, graphs
@pytest.mark.parametrize("Dmax", [1, 20])
def test_on_another_stream_and_in_two_graphs(Dmax):
    """Two graphs that share a workspace, replayed in turn with changed inputs; a side stream."""
    case = H.AttnCase(31, [700, 130], 1, Dmax, 4, 2, 128, 64, True, blk_len=np.full((2, 1), Dmax))
    a, kw = case.args(), case.kw()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ref = S.ssd_verify_attn_quant(*a, **kw, out_f32=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = S.ssd_verify_attn_quant(*a, **kw, out_f32=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    short = dev(np.array([10, 10], np.int32))
    b = list(a)
    b[7] = short
    ref_short = S.ssd_verify_attn_quant(*b, **kw, out_f32=True)
    outs, graphs = [], []
    for args in (a, b):
        o = torch.zeros_like(ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.ssd_verify_attn_quant(*args, **kw, out=o, ws=ws)
        outs.append(o)
        graphs.append(g)
    for _ in range(3):
        for g, o, r in zip(graphs, outs, (ref, ref_short)):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, r)
    assert S.ssd_read_device_error(ws) == S.SSD_OK


def test_two_streams_at_once():
    """Calls that run side by side, with a workspace each."""
    cases = [H.AttnCase(67 + i, [3000, 700], 1, (1, 20)[i], 4, 2, 128, 64, True) for i in range(2)]
    args = [c.args() for c in cases]
    tables = [c.kw()["block_table"] for c in cases]
    refs = [torch.zeros(c.q.shape, dtype=torch.float32, device="cuda") for c in cases]      # absent rows are not written
    for a, t, r in zip(args, tables, refs):
        S.ssd_verify_attn_quant(*a, block_table=t, out=r)
    outs = [[torch.zeros_like(r) for _ in range(20)] for r in refs]
    ws = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for k in range(20):
        for i, s in enumerate(streams):
            S.ssd_verify_attn_quant(*args[i], block_table=tables[i], out=outs[i][k], ws=ws[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for os, r in zip(outs, refs) for o in os)


def test_a_captured_step_is_replayed():
    """Pages, rows, attention and the commit of a decoding step in one graph: three replays give
    what three steps of the oracle give."""
    rng = np.random.default_rng(71)
    B, Hkv, G, dh, sb, pps = 3, 2, 4, 128, 32, 4
    length = np.array([127, 5, 254], np.int32)
    held, table = np.array([1, 1, 2], np.int32), np.full((B, pps), -1, np.int32)
    table[0, 0], table[1, 0], table[2, :2] = 3, 0, (7, 5)
    stack, n = np.array([1, 2, 4, 6, 8, 9, 10, 11, 0, 0, 0, 0], np.int32), 8
    c = [x for w in range(2) for x in H.cache(rng, len(stack), Hkv, 128, dh, sb)]
    t = [dev(x) for x in c]
    d = [dev(x) for x in (held, table, stack, np.array([n], np.int32))]
    len_d, one, zero = dev(length), dev(np.ones(B, np.int32)), dev(np.zeros(B, np.int32))
    bits, x64 = H.bf16(rng, B, 1, 2, Hkv, dh)
    kd, vd = (dev(np.ascontiguousarray(bits[:, :, w])) for w in range(2))
    n_out, new_len = dev(np.full(B, 2, np.int32)), dev(length)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = S.ssd_page_tables(len_d, one, *d, B, ws=ws)
        S.ssd_append_kv_quant(kd[:, 0], vd[:, 0], got["slot_map"], t[0], t[2], t[1], t[3], sb, ws=ws)
        S.ssd_commit_kv_quant(t[0], t[2], t[1], t[3], kd, vd, len_d, zero, n_out, 1, sb, new_len=new_len, block_table=d[1], ws=ws)
        len_d.copy_(new_len)
    for _ in range(3):
        graph.replay()
        n, start, slots, served, err = K.page_tables(length, np.ones(B, np.int32), held, table, stack, n, B)
        assert served.all() and not err
        for w in range(2):
            K.append(x64[:, 0, w], slots, c[2 * w], c[2 * w + 1], sb)
            new, ok = K.commit(x64[:, :, w], length, np.zeros(B, np.int32), np.full(B, 2, np.int32), 1, c[2 * w], c[2 * w + 1], sb, table)
            assert ok.all()
        length = new
        np.testing.assert_array_equal(len_d.cpu().numpy(), length)
        np.testing.assert_array_equal(got["slot_map"].cpu().numpy(), slots)
        for x, ref in zip(d, (held, table, stack, [n])):
            np.testing.assert_array_equal(x.cpu().numpy(), ref)
        _same_cache(c, t)
    assert S.ssd_read_device_error(ws) == S.SSD_OK


# ---------------------------------------------------------------------------- together
def test_a_serving_loop_uses_all_calls():
    """Prompts admitted, written, decoded and verified, committed, trimmed; a sequence ends and
    its pages serve another. Tables, lengths, codes and scales stay equal to the oracle's, the
    attention within tolerance, over a loop without a host copy between the calls."""
    rng = np.random.default_rng(41)
    B, Hkv, G, dh, sb, NB, Dmax, pps, pool = 5, 2, 4, 128, 64, 2, 6, 6, 22
    held, table = np.zeros(B, np.int32), np.full((B, pps), -1, np.int32)
    stack, n = rng.permutation(pool).astype(np.int32), pool
    c = [x for w in range(2) for x in H.cache(rng, pool, Hkv, 128, dh, sb)]
    t = [dev(x) for x in c]
    d = [dev(x) for x in (held, table, stack, np.array([n], np.int32))]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    length = np.zeros(B, np.int32)
    len_d = dev(length)
    for step in range(5):
        # prompts: everybody at first, later one that takes a finished sequence's place
        add = np.zeros(B, np.int32)
        if step == 0:
            add[:] = [500, 1, 127, 128, 300]
        elif step == 3:
            length[1] = 0
            len_d = dev(length)
            add[1] = 400
        if add.any():
            cap = int(add.sum()) + 7
            n, start, slots, served, err = K.page_tables(length, add, held, table, stack, n, cap)
            assert served.all() and not err
            got = S.ssd_page_tables(len_d, dev(add), *d, cap, ws=ws)
            bits, x64 = H.bf16(rng, cap, 2, Hkv, dh)
            K.append(x64[:, 0], slots, c[0], c[1], sb)
            K.append(x64[:, 1], slots, c[2], c[3], sb)
            rows = dev(bits)
            S.ssd_append_kv_quant(rows[:, 0], rows[:, 1], got["slot_map"], t[0], t[2], t[1], t[3], sb, ws=ws)
            length = length + add
            len_d = len_d + dev(add)
        # pages for the accepted tokens of a step
        room = np.full(B, Dmax, np.int32)
        n, *_ , served, err = K.page_tables(length, room, held, table, stack, n, 0)[:4] + (False,)
        S.ssd_page_tables(len_d, dev(room), *d, B * Dmax, ws=ws)
        case = H.AttnCase(step, [1] * B, NB, Dmax, G, Hkv, dh, sb, True)
        case.prefix, case.table = length, table
        case.k_codes, case.k_scale, case.v_codes, case.v_scale = c
        kd, vd, blk = dev(case.kc), dev(case.vc), dev(case.blk_len)
        out = S.ssd_verify_attn_quant(dev(case.q), t[0], t[2], t[1], t[3], kd, vd, len_d, blk, Dmax, sb, ws=ws, out_f32=True,
                                      block_table=d[1])
        case.check(out)
        best = rng.integers(-1, NB, B).astype(np.int32)
        n_out = np.array([1 + rng.integers(0, case.blk_len[b, best[b]] + 1) if best[b] >= 0 else 1 for b in range(B)], np.int32)
        new, ok = K.commit(case.kc64, length, best, n_out, Dmax, c[0], c[1], sb, table)
        K.commit(case.vc64, length, best, n_out, Dmax, c[2], c[3], sb, table)
        assert ok.all()
        len_d, _ = S.ssd_commit_kv_quant(t[0], t[2], t[1], t[3], kd, vd, len_d, dev(best), dev(n_out), Dmax, sb, block_table=d[1],
                                         ws=ws)
        length = new
        n, *_ = K.page_tables(length, np.zeros(B, np.int32), held, table, stack, n, 0)
        S.ssd_page_tables(len_d, torch.zeros_like(len_d), *d, 0, ws=ws)
        assert S.ssd_read_device_error(ws) == S.SSD_OK
        np.testing.assert_array_equal(len_d.cpu().numpy(), length)
        for x, ref in zip(d, (held, table, stack, [n])):
            np.testing.assert_array_equal(x.cpu().numpy(), ref)
        _same_cache(c, t)


# ---------------------------------------------------------------------------- refusals
def test_refusals():
    case = H.AttnCase(37, [90, 40], 2, 3, 2, 2, 64, 32, True)
    a, kw = case.args(), case.kw()
    call = lambda i, v, **more: S.ssd_verify_attn_quant(*[v if j == i else x for j, x in enumerate(a)], **{**kw, **more})
    for i, v in ((0, a[0].float()), (0, a[0][:, :5].contiguous()), (1, a[1].int()), (1, a[1][:, :, :64].contiguous()), (2, a[2][:1]),
                 (3, a[3].double()), (3, a[3][:, :, :2].contiguous()), (5, a[5][:, :4].contiguous()), (6, a[6].cpu()),
                 (7, a[7].long()), (7, a[7][:1]), (8, a[8].view(1, 4)), (9, 4), (10, 48), (0, a[0].transpose(1, 2))):
        with pytest.raises(ValueError):
            call(i, v)
    with pytest.raises(ValueError):
        call(-1, None, out=torch.empty((2, 6, 4, 32), device="cuda"))
    with pytest.raises(ValueError, match="overlap"):
        call(-1, None, out=a[0])
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(S.SsdError):
            call(-1, None, scale=bad)
    words = torch.zeros(2 * 6 * 4 * 64, dtype=torch.float32, device="cuda")
    with pytest.raises(S.SsdError, match="invalid"):       # the result over a scale
        call(3, words[:a[3].numel()].view(a[3].shape), out=words.view(2, 6, 4, 64))
    with pytest.raises(S.SsdError):                        # a workspace off its alignment
        call(-1, None, ws=torch.zeros(512, dtype=torch.uint8, device="cuda")[16:272])
    with pytest.raises(S.SsdError):
        call(-1, None, ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    k = a[5].view(12, 2, 64)
    slots = torch.zeros(12, dtype=torch.int32, device="cuda")
    cache = (a[1], a[2], a[3], a[4], 32)
    with pytest.raises(ValueError):
        S.ssd_append_kv_quant(k, k, slots[:3], *cache)
    with pytest.raises(ValueError):
        S.ssd_append_kv_quant(k.transpose(1, 2), k, slots, *cache)
    with pytest.raises(ValueError, match="overlap"):
        S.ssd_append_kv_quant(k, k, slots, a[1], a[1], a[3], a[4], 32)
    wide = torch.zeros((12, 2 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    odd = torch.as_strided(wide, (12, 2, 64), (2 * 64 + 4, 64, 1))
    with pytest.raises(S.SsdError, match="unsupported"):   # rows that are not 16 bytes apart
        S.ssd_append_kv_quant(odd, odd, slots, *cache)
    with pytest.raises(ValueError, match="overlap"):
        S.ssd_commit_kv_quant(a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[7], a[7], 3, 32, new_len=a[7], **kw)
    with pytest.raises(ValueError):
        S.ssd_commit_kv_quant(a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[7], a[7], 4, 32, **kw)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        S.ssd_page_tables(i32(2), i32(3), i32(2), i32(2, 4), i32(9), i32(1), 4)
    with pytest.raises(ValueError):
        S.ssd_page_tables(i32(2), i32(2), i32(2), i32(2, 4), i32(9), i32(1), -1)
    both = i32(4)
    with pytest.raises(ValueError, match="overlap"):
        S.ssd_page_tables(both[:2], i32(2), both[1:3], i32(2, 4), i32(9), i32(1), 4)
