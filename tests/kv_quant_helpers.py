"""Inputs and comparisons of the 8-bit cache's GPU tests."""
import numpy as np
import torch

from oracle import kv_quant_oracle as K
from oracle import ssd_oracle as O
from speculative_decoding_copy_gb300 import _binding as S
from speculative_decoding_copy_gb300 import workloads as WL

DEV = "cuda"


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


def bf16(rng, *shape, scale=1.0):
    """Random bf16 rows: (bit patterns, their fp64 values)."""
    bits = WL.f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))
    return bits, O.bf16_to_f64(bits)


def cache(rng, pages, Hkv, tokens, dh, sb, pow2=True):
    """A filled cache: codes and scales (powers of two, or any)."""
    table = K.encode(rng.standard_normal(1 << 16) * 100)
    codes = table[rng.integers(0, len(table), (pages, Hkv, tokens, dh))]
    scale = 2.0 ** rng.integers(-8, -5, (pages, Hkv, -(-tokens // sb)))
    if not pow2:
        scale = scale * (1 + rng.random(scale.shape))
    return codes, scale.astype(np.float32)


class AttnCase:
    """One attention call over a random cache, and its oracle."""

    def __init__(self, seed, prefix, NB, Dmax, G, Hkv, dh, sb, paged, q_scale=1.5, blk_len=None, spare=2, pow2=False,
                 order=None):
        rng = self.rng = np.random.default_rng(seed)
        B = len(prefix)
        self.prefix, self.Dmax, self.sb, self.dh = np.asarray(prefix, np.int32), Dmax, sb, dh
        NT, most = NB * Dmax, max(1, max(prefix))
        if paged:
            pps = -(-most // 128)
            pages, tokens = B * pps + spare, 128
            ids = rng.permutation(pages) if order is None else order(pages)
            self.table = ids[:B * pps].reshape(B, pps).astype(np.int32)
        else:
            pages, tokens, self.table = B, most, None
        self.k_codes, self.k_scale = cache(rng, pages, Hkv, tokens, dh, sb, pow2)
        self.v_codes, self.v_scale = cache(rng, pages, Hkv, tokens, dh, sb, pow2)
        self.q, self.q64 = bf16(rng, B, NT, Hkv * G, dh, scale=q_scale)
        self.kc, self.kc64 = bf16(rng, B, NT, Hkv, dh)
        self.vc, self.vc64 = bf16(rng, B, NT, Hkv, dh)
        self.blk_len = np.asarray(blk_len if blk_len is not None else rng.integers(0, Dmax + 1, (B, NB)), np.int32)
        if blk_len is None:
            self.blk_len[0, 0] = Dmax

    def poison(self):
        """NaN codes and scales wherever the call must not look."""
        for b, P in enumerate(self.prefix):
            for codes, scale in ((self.k_codes, self.k_scale), (self.v_codes, self.v_scale)):
                if self.table is None:
                    codes[b, :, P:] = 0x7f
                    scale[b, :, -(-P // self.sb):] = np.nan
                else:
                    for j, pg in enumerate(self.table[b]):
                        left = max(0, P - 128 * j)
                        codes[pg, :, left:] = 0x7f
                        scale[pg, :, -(-left // self.sb):] = np.nan
        NB = self.blk_len.shape[1]
        absent = np.arange(self.Dmax)[None, None, :] >= self.blk_len[:, :, None]
        absent = absent.reshape(len(self.prefix), NB * self.Dmax)
        for x in (self.q, self.kc, self.vc):
            x[absent] = 0x7fc0

    def args(self):
        t = [dev(x) for x in (self.q, self.k_codes, self.v_codes, self.k_scale, self.v_scale, self.kc, self.vc,
                              self.prefix, self.blk_len)]
        return t + [self.Dmax, self.sb]

    def kw(self):
        return dict(block_table=None if self.table is None else dev(self.table))

    def oracle(self, slots=None, probs=None):
        k = K.values(self.k_codes, self.k_scale, self.sb, self.prefix, self.table)
        v = K.values(self.v_codes, self.v_scale, self.sb, self.prefix, self.table)
        return K.attention(self.q64, k, v, self.kc64, self.vc64, self.blk_len, self.Dmax, slots, probs=probs)

    def v_scales(self, b):
        """The value scale of every prefix key of sequence b: [Hkv][prefix]."""
        pages = [b] if self.table is None else self.table[b, :-(-int(self.prefix[b]) // 128)]
        s = [np.repeat(self.v_scale[p].astype(np.float64), self.sb, 1)[:, :self.v_codes.shape[2]] for p in pages]
        s = np.concatenate(s, 1) if s else np.zeros((self.kc.shape[2], 0))
        return np.maximum(s[:, :self.prefix[b]], 2.0 ** -100)

    def many(self, G):
        """Whether the call takes the kernel for many rows."""
        rows, (pages, Hkv) = self.q.shape[1] * G, self.k_codes.shape[:2]
        capacity = self.k_codes.shape[2] if self.table is None else self.table.shape[1] * 128
        groups = len(self.prefix) * Hkv * -(-rows // 16)
        return not (rows <= 16 or (rows <= 48 and groups <= 152 and groups * capacity <= 1 << 17))

    def tolerance(self, b, o, size, heads, f32, wide):
        """Per element [Hq][dh]; heads = [(p, v)] of the kv heads, size = sum_j p_j |v_j|.

        Both paths: scores are off by less than 2^-11 in log2 units (fp32 sums over at most 128
        products of total magnitude <= 32, 2^-23 each; q as two e4m3 numbers is off by 2^-18 of
        its largest per element) and exponentials by 2^-21, which acts on size; a bf16 output
        adds half a step of its own, 2^-8 |out|.

        Few rows: probabilities are rounded to 11 bits, 2^-11 size, and below the fp16 range by
        2^-25 each while the largest weight is at least 1: N 2^-25 448 max v_scale.

        Many rows: a probability is rounded to an e4m3 number and what is left (at most 2^-4 of
        it) to an e5m2 number (half a step 2^-3), or by half of 2^-16, e5m2's least step, where that is more, while the key with the largest
        weight p_j s_j (s the value scale) has at least 2^4. Over a binade of the first and of
        the second number the product of the two uniform errors has a standard deviation under
        (2^-4 / sqrt 3)(2^-3 / sqrt 3) = 2^-7 / 3 < 2^-8 / sqrt 3; with sum_j p_j = 1 the least
        step is (max_i p_i s_i / 2^4) 2^-17 for a code, over sqrt 3 (the maximum runs over the
        own-block keys too, which enter it with s = 2^-16). Both are independent from key to key:
        six standard deviations of their sums are allowed (for a single key 2^-5.4, over the 2^-7
        it can be off by). The merge rounds a share's row to 2^-14 of its largest element:
        2^-14 sum_j p_j max_d |v_jd|."""
        tol = np.zeros_like(o)
        G = o.shape[0] // len(heads)
        many = self.many(G)
        P = int(self.prefix[b])
        sv = self.v_scales(b)
        for h, (p, v) in enumerate(heads):
            rows = slice(h * G, (h + 1) * G)
            if not many:
                tol[rows] = size[rows] * 2.0 ** -10 * wide + P * 2.0 ** -25 * 448 * float(sv.max(initial=0))
                continue
            rel = (p ** 2) @ (v ** 2) * (2.0 ** -8) ** 2 / 3
            top = np.maximum((p[:, :P] * sv[h]).max(1, initial=0.0), p[:, P:].max(1, initial=0.0) * 2.0 ** -16)
            codes2 = ((v[:P] / sv[h][:, None]) ** 2).sum(0)
            floor = (top[:, None] * 2.0 ** -4 * 2.0 ** -17) ** 2 / 3 * codes2[None, :]
            most = p @ np.abs(v).max(1)
            tol[rows] = 6 * np.sqrt(rel + floor) + size[rows] * 2.0 ** -11 * wide + most[:, None] * 2.0 ** -14
        return tol + (0 if f32 else np.abs(o) * 2.0 ** -8) + 1e-30

    def check(self, out, slots=None, wide=1.0):
        """Every present row within tolerance of the oracle."""
        f32 = out.dtype == torch.float32
        got = out.cpu().numpy().astype(np.float64) if f32 else O.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
        probs = {}
        ref = self.oracle(slots, probs)
        assert ref
        for (b, t), (o, size) in ref.items():
            tol = self.tolerance(b, o, size, probs[b, t], f32, wide)
            err = np.abs(got[b, t] - o)
            assert (err <= tol).all(), (b, t, float((err / tol).max()))
        return ref


def run(case, fill=7.0, f32=True, **kw):
    """Call the attention into a buffer of `fill`; absent rows must keep it."""
    B, NT, Hq, dh = case.q.shape
    out = torch.full((B, NT, Hq, dh), fill, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    S.ssd_verify_attn_quant(*case.args(), out=out, ws=ws, **case.kw(), **kw)
    torch.cuda.synchronize()
    assert S.ssd_read_device_error(ws) == S.SSD_OK
    keep = np.arange(case.Dmax)[None, None, :] >= case.blk_len[:, :, None]
    keep = torch.from_numpy(keep.reshape(B, NT)).to(DEV)
    assert bool((out[keep] == fill).all()), "a row of an absent token was written"
    return out
