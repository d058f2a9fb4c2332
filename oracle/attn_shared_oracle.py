"""Plain fp64 restatement of the attention over a shared prompt, an own prefix and the own block."""
import numpy as np


def attention(q, shared, own, cand, blk_len, Dmax, scale=None):
    """q [B][NT][Hq][dh]; shared = (k, v) [Hkv][S][dh]; own = list over b of (k, v) [Hkv][P_b][dh];
    cand = (k, v) [B][NT][Hkv][dh]; blk_len [B][NB]. Returns {(b, t): (out [Hq][dh], spread [Hq][dh])}
    for the present tokens; spread is sum_j w_j |v_j - out|, what a rounding of the weights can move."""
    B, NT, Hq, dh = q.shape
    Hkv = cand[0].shape[2]
    G, scale = Hq // Hkv, scale or dh ** -0.5
    got = {}
    for b in range(B):
        for t in range(NT):
            k, pos = divmod(t, Dmax)
            if pos >= blk_len[b][k]:
                continue
            out, spread = np.zeros((Hq, dh)), np.zeros((Hq, dh))
            for h in range(Hkv):
                keys = np.concatenate([shared[0][h], own[b][0][h], cand[0][b, k * Dmax:t + 1, h]])
                vals = np.concatenate([shared[1][h], own[b][1][h], cand[1][b, k * Dmax:t + 1, h]])
                for g in range(h * G, (h + 1) * G):
                    z = keys @ q[b, t, g] * scale
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    out[g] = w @ vals
                    spread[g] = w @ np.abs(vals - out[g])
            got[b, t] = (out, spread)
    return got
