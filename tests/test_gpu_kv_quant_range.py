"""The range of the probabilities in the attention over the 8-bit cache: a long tail of keys that are each
small beside one, and together hold most of the mass."""
import numpy as np
import pytest

import kv_quant_helpers as H
from oracle import kv_quant_oracle as K
from oracle import ssd_oracle as O
from speculative_decoding_copy_gb300 import workloads as WL

pytestmark = pytest.mark.gpu


class Tail(H.AttnCase):
    """Prefix keys of scores spread by `spread` nats, of which key 5 of sequence b lies above[b] log2 units
    over their mean and has small values; own-block keys of negligible score. All values are positive,
    so that errors of one sign show in the output."""

    def __init__(self, P, Dmax, G, dh, sb, above, spread, Hkv=1):
        B = len(above)
        super().__init__(97, [P] * B, 1, Dmax, G, Hkv, dh, sb, True, blk_len=np.full((B, 1), Dmax), spare=0)
        rng = self.rng
        u = rng.standard_normal(dh)
        u *= np.sqrt(dh) / np.linalg.norm(u)                    # scores are u . k / sqrt(dh)
        self.u, ln2 = u, np.log(2.0)
        q = np.broadcast_to(u, self.q.shape) * (1 + 0.02 * rng.standard_normal(self.q.shape))
        self.q = WL.f32_to_bf16_bits(q.astype(np.float32))
        self.q64 = O.bf16_to_f64(self.q)
        kc = np.broadcast_to(u * (-30 * ln2 / np.sqrt(dh)), self.kc.shape)
        self.kc = WL.f32_to_bf16_bits(kc.astype(np.float32))
        self.kc64 = O.bf16_to_f64(self.kc)
        self.table[1:, 1:] = self.table[0, 1:]                  # the first page is each sequence's own
        k = rng.standard_normal((P, Hkv, dh)) * spread
        v = 0.5 + rng.random((P, Hkv, dh))
        v[5] = 2.0 ** -4
        for b in range(B):
            k[5] = u * (above[b] * ln2 / np.sqrt(dh))
            self.write(b, *((k, v) if b == 0 else (k[:128], v[:128])))

    def write(self, b, k, v):
        pos = np.arange(len(k))
        slots = self.table[b, pos // 128] * 128 + pos % 128
        K.append(k, slots, self.k_codes, self.k_scale, self.sb)
        K.append(v, slots, self.v_codes, self.v_scale, self.sb)

    def bound(self, b, o, heads, many):
        """The most that a row [Hq][dh] may be off, by arithmetic alone (errors of one sign all along).

        A probability: scores 2^-11 in log2 units (kv_quant_helpers), so 2^-11; over many rows fp16
        (half a step, 2^-11) and then three e5m2 numbers, each half a step (2^-3) of what the one before
        left: 2^-9; together under 2^-8. Over few rows fp16: with the scores 2^-10.
        Below the formats' normal numbers half their least step, while the key of the largest weight p_j s_j
        (s_j the value scale) has at least 2^11 (many: 2^-17) or 2^7 (few: 2^-25), for a code.
        The merge of many rows rounds to 2^-14 of the largest of dh / 2 elements of a share."""
        P, G, dh = int(self.prefix[b]), o.shape[0] // len(heads), self.dh
        sv = self.v_scales(b)
        tol = np.zeros_like(o)
        for h, (p, v) in enumerate(heads):
            rows = slice(h * G, (h + 1) * G)
            top = (p[:, :P] * sv[h]).max(1)
            codes = (np.abs(v[:P]) / sv[h][:, None]).sum(0)
            tol[rows] = (p @ np.abs(v)) * (2.0 ** -8 if many else 2.0 ** -10)
            tol[rows] += top[:, None] * codes * (2.0 ** -28 if many else 2.0 ** -32)
            if many:
                for half in (slice(0, dh // 2), slice(dh // 2, dh)):
                    tol[rows, half] += (p @ np.abs(v[:, half]).max(1))[:, None] * 2.0 ** -14
        return tol

    def compare(self, out, slots):
        many = self.many(self.q.shape[2] // self.kc.shape[2])
        got = out.cpu().numpy().astype(np.float64)
        probs, bad = {}, []
        for (b, t), (o, _) in self.oracle(slots, probs).items():
            worst = float((np.abs(got[b, t] - o) / self.bound(b, o, probs[b, t], many)).max())
            if not worst <= 1:
                bad.append((b, t, worst, float(np.abs(got[b, t] / o - 1).max())))
        assert not bad, bad


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("dh,P,B", [(128, 32768, 2), (128, 32768, 24), (64, 16384, 24)])
def test_a_long_tail_beside_one_large_key_of_many_rows(dh, P, B, spread):
    case = Tail(P, 20, 4, dh, 128, np.log2(P) - 3 + 5 * np.arange(B) / B, spread, Hkv=4)
    assert case.many(4)
    case.compare(H.run(case), {(b, (7 * b) % 20) for b in range(B)})


@pytest.mark.parametrize("dh", [64, 128])
def test_a_value_block_of_a_large_scale_of_many_rows(dh):
    """One block whose values need a scale 2^11 to 2^16 above the others', in one element alone and at scores
    a little above theirs: the other elements keep their bits."""
    P, B = 16384, 24
    case = Tail(P, 20, 4, dh, 64, [0.0] * B, 0.0)
    for b in range(B):
        k = np.broadcast_to(case.u * ((0.3 + 0.7 * b / B) * np.log(2) / np.sqrt(dh)), (128, 1, dh))
        v = 0.5 + case.rng.random((128, 1, dh))
        v[64:] = 0
        v[64:, :, 0] = 2.0 ** (11 + b % 6)
        case.write(b, k, v)
    case.compare(H.run(case), {(b, (7 * b) % 20) for b in range(B)})


def test_a_long_tail_beside_one_large_key_of_few_rows():
    """So many sequences, most of them empty, that one CTA of three warps takes a whole prefix."""
    P, B, more = 65536, 12, 60000
    case = Tail(P, 1, 1, 64, 128, 15 + 3.5 * np.arange(B) / B, 0.0)
    empty = lambda x: np.concatenate([x, np.zeros((more,) + x.shape[1:], x.dtype)])
    case.q, case.kc, case.vc, case.table, case.prefix = map(empty, (case.q, case.kc, case.vc, case.table, case.prefix))
    case.q64, case.kc64, case.vc64 = map(empty, (case.q64, case.kc64, case.vc64))
    case.blk_len = np.ones((B + more, 1), np.int32)
    assert not case.many(1)
    case.compare(H.run(case), {(b, 0) for b in range(B)})
