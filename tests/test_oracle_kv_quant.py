"""Pins of the 8-bit cache's oracle: the e4m3 format against torch's, the block scale's
definition, what a grown scale does to earlier rows, page bookkeeping against its
invariants, attention over exactly representable rows."""
import numpy as np
import pytest
import torch

from oracle import kv_quant_oracle as K
from oracle import ssd_oracle as O


def test_codes_are_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(K.E4M3, ref)


def test_encoding_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    grid = K.E4M3[:127]
    x = np.concatenate([rng.standard_normal(4000) * 100, rng.standard_normal(4000) * 2.0 ** -8, grid, (grid[1:] + grid[:-1]) / 2])
    x = np.concatenate([x, -x]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(K.encode(x), ref)
    assert K.encode([np.inf, -np.inf, 1e9]).tolist() == [0x7e, 0xfe, 0x7e] and K.encode(np.nan) == 0x7f


@pytest.mark.parametrize("k", [-100, -30, -1, 0, 7, 100])
def test_least_scale_at_its_borders(k):
    s = 2.0 ** k
    assert K.least_scale(448 * s) == s
    assert K.least_scale(np.nextafter(448 * s, np.inf)) == 2 * s
    assert K.least_scale(0.0) == 2.0 ** -100


def test_a_grown_scale_moves_only_earlier_rows():
    rng = np.random.default_rng(2)
    codes, scale = np.full((1, 1, 32, 8), 0x55, np.uint8), np.full((1, 1, 2), np.nan)
    x = rng.standard_normal((5, 1, 8))
    K.append(x, np.arange(5), codes, scale, 16)
    before, s0 = codes.copy(), scale[0, 0, 0]
    K.append(x[:2] * 64, np.arange(5, 7), codes, scale, 16)
    assert scale[0, 0, 0] == 64 * s0 and np.isnan(scale[0, 0, 1])
    # a factor 64 is exact but for the codes that fall under the smallest normal one
    np.testing.assert_allclose(K.E4M3[codes[0, 0, :5]] * 64, K.E4M3[before[0, 0, :5]], atol=2.0 ** -10 * 64)
    np.testing.assert_array_equal(codes[0, 0, 7:], before[0, 0, 7:])
    # a block's first row starts it afresh
    K.append(x[:1] * 2.0 ** -9, np.array([0]), codes, scale, 16)
    assert scale[0, 0, 0] <= s0


def _books(rng, B, pps, spare):
    held = rng.integers(0, pps + 1, B).astype(np.int32)
    n = int(held.sum())
    order = rng.permutation(n + spare).astype(np.int32)
    table, at = np.full((B, pps), -1, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    stack = np.zeros(n + spare, np.int32)
    stack[:spare] = order[n:]
    return held, table, stack, spare


@pytest.mark.parametrize("seed", range(6))
def test_no_page_is_lost_or_held_twice(seed):
    rng = np.random.default_rng(seed)
    B, pps = 7, 5
    held, table, stack, n = _books(rng, B, pps, int(rng.integers(0, 12)))
    for _ in range(5):
        cur = rng.integers(0, 400, B).astype(np.int32)
        add = np.minimum(rng.integers(0, 300, B), pps * 128 - cur).astype(np.int32)
        n, start, slots, served, err = K.page_tables(cur, add, held, table, stack, n, int(add.sum()) + 3)
        assert not err
        pages = sorted(table[table >= 0].tolist() + stack[:n].tolist())
        assert pages == list(range(len(stack)))
        assert ((table >= 0).sum(1) == held).all()
        for b in range(B):
            if served[b]:
                assert held[b] == -(-(cur[b] + add[b]) // 128)
            got = slots[start[b]:start[b + 1]]
            assert (got >= 0).all() if served[b] else (got == -1).all()
        assert (slots[start[-1]:] == -1).all()


def test_attention_agrees_with_the_plain_cache():
    """Rows that e4m3 holds exactly: the cache's attention is ssd_oracle's over those rows."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, dh, P, NB, Dmax = 2, 4, 2, 8, 40, 2, 3
    codes = rng.integers(0, 0x7e, (B, Hkv, P, dh)).astype(np.uint8)
    scale = 2.0 ** rng.integers(-9, -5, (B, Hkv, 3)).astype(np.float64)
    prefix = np.array([40, 17], np.int32)
    rows = K.values(codes, scale, 16, prefix)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    q, kd, vd = f(B, NB * Dmax, Hq, dh), f(B, NB * Dmax, Hkv, dh), f(B, NB * Dmax, Hkv, dh)
    blk = np.array([[3, 1], [0, 2]], np.int32)
    full = (K.E4M3[codes] * np.repeat(scale, 16, 2)[:, :, :P, None]).astype(np.float32)
    ref = O.verify_attention(q, full, full, kd, vd, prefix, blk, Dmax, "f32")
    got = K.attention(q.astype(np.float64), rows, rows, kd.astype(np.float64), vd.astype(np.float64), blk, Dmax)
    assert got.keys() == ref.keys()
    for key in ref:
        np.testing.assert_allclose(got[key][0], ref[key], rtol=1e-12)
