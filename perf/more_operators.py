"""Sampled continuations of one prompt: what is measured.

Three operators that a serving loop calls when many sequences go on from one long prompt and are
sampled instead of decoded greedily:

  shared  ssd_verify_attn_shared  block-triangular verification (one token: decode) of a batch whose
                                  sequences share a prompt's keys: those once for all, then each
                                  sequence's own keys and its own candidate block
  filter  ssd_filter_probs        the distributions that temperature, top-k, top-p and min-p leave of
                                  logit rows (what the acceptance verifies against)
  sample  ssd_sample              a token from such a distribution, by a given uniform number (the
                                  drafter's tokens with their rows, or plain sampled decoding)

With `own` false, run() computes them with elementary torch operations; with `own` true it calls the
framework.
"""
import torch

own = False

PAGE = 128


# ---------------------------------------------------------------------------- cases
def _shared(name, B, NB, Dmax, Hq, Hkv, prompt, lo, hi, dh=128, paged=False, absent=False, f32=False):
    return dict(name=name, op="shared", B=B, NB=NB, Dmax=Dmax, Hq=Hq, Hkv=Hkv, prompt=prompt, lo=lo, hi=hi, dh=dh, paged=paged, absent=absent, f32=f32)


def _filter(name, B, NB, Dmax, V, mix, std=2.5, bf16=True, absent=False, masked=0.0):
    return dict(name=name, op="filter", B=B, NB=NB, Dmax=Dmax, V=V, mix=mix, std=std, bf16=bf16, absent=absent, masked=masked)


def _sample(name, B, V, mix, std=2.5, bf16=True, probs=False, pad=0, masked=0.0):
    return dict(name=name, op="sample", B=B, V=V, mix=mix, std=std, bf16=bf16, probs=probs, pad=pad, masked=masked)


def listed():
    return [
        # two samples of a short prompt, their second tokens: the smallest attention call, where latency counts
        _shared("shared_two", 2, 1, 1, 32, 8, 512, 1, 1),
        # 64 samples of a prompt of 8192 tokens, a token each, after up to 500 of their own, in pages
        _shared("shared_decode", 64, 1, 1, 32, 8, 8192, 20, 500, paged=True),
        # a chain draft of five tokens behind an odd prompt, head dim 64, seven query heads a key head
        _shared("shared_chain_dh64", 12, 1, 5, 14, 2, 1999, 0, 300, dh=64),
        # eight samples verify four copied continuations of twenty tokens each: the benchmark's blocks, a prompt of 4096
        _shared("shared_verify", 8, 4, 20, 32, 8, 4096, 1, 1500),
        # batched serving, eight continuations and a chain block, some absent, one prompt of 16384, pages: the largest
        _shared("shared_batch", 32, 9, 16, 32, 8, 16384, 0, 2048, paged=True, absent=True),
        # one user's chain draft of seven tokens: eight rows to verify
        _filter("filter_chain", 1, 1, 7, 128256, "served", bf16=False),
        # the benchmark's verification rows, every token present, fp32 logits
        _filter("filter_verify", 1, 4, 20, 128256, "nucleus", bf16=False),
        # batched serving rows, a setting for each sequence, some blocks absent
        _filter("filter_batch", 8, 9, 16, 151936, "served", absent=True),
        # wide distributions (high temperature, top-p alone), where the nucleus holds thousands of tokens
        _filter("filter_wide", 8, 4, 20, 32000, "nucleus", std=1.0),
        # one drafted token with its row, from the drafter's fp32 logits
        _sample("sample_draft", 1, 128256, "served", bf16=False, probs=True),
        # 64 users' next tokens, logits in a padded buffer
        _sample("sample_64", 64, 151936, "served", pad=128),
        # 256 users, a grammar that leaves one token in a hundred
        _sample("sample_grammar", 256, 128256, "topk", masked=0.99),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["shared", "shared", "filter", "sample"])
    if op == "shared":
        while True:
            B, NB, Dmax = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4, 5, 9]), _log(rng, 1, 24)
            G, Hkv = rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.choice([1, 2, 4, 8])
            prompt, hi = _log(rng, 16, 32768), _log(rng, 1, 4096)
            if B * NB * Dmax * G * Hkv * (prompt + hi) <= 32 * 144 * 32 * 16384 // 4:
                break
        f32 = rng.random() < 0.1 and B * NB * Dmax * G * Hkv * (prompt + hi) <= 1 << 26
        c = _shared("", B, NB, Dmax, G * Hkv, Hkv, prompt - rng.choice([0, 0, 1, 5]), rng.randint(0, hi), hi, rng.choice([64, 128, 128]),
                    rng.random() < 0.4 and not f32, rng.random() < 0.4, f32)
    else:
        V, bf16 = rng.choice([_log(rng, 500, 160000), _log(rng, 500, 160000), 32000, 128256, 151936]), rng.random() < 0.6
        mix, std = rng.choice(["served", "served", "nucleus", "topk", "plain"]), rng.choice([1.0, 2.5, 2.5, 4.0])
        masked = rng.choice([0.0, 0.0, 0.5, 0.99])
        if op == "filter":
            while True:
                B, NB, Dmax = _log(rng, 1, 16), rng.choice([1, 1, 2, 4, 5, 9]), _log(rng, 1, 24)
                if B * (1 + NB * Dmax) * V <= 8 * 145 * 151936 // 2:
                    break
            c = _filter("", B, NB, Dmax, V, mix, std, bf16, rng.random() < 0.5, masked)
        else:
            c = _sample("", min(_log(rng, 1, 300), 40000000 // V), V, mix, std, bf16, rng.random() < 0.4, rng.choice([0, 0, 1, 128]), masked)
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi]: the same ones for every seed."""
    return [hi] if n == 1 else [round(lo + (hi - lo) * i / (n - 1)) for i in range(n)]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _blocks(c, h):
    """Lengths of the candidate blocks: all full, or some absent and some short."""
    blk = torch.full((c["B"], c["NB"]), c["Dmax"], dtype=torch.int32)
    if c["absent"]:
        blk = torch.where(torch.rand(blk.shape, generator=h) < 0.4, 0, torch.randint(0, c["Dmax"] + 1, blk.shape, generator=h)).to(torch.int32)
        blk[0, 0] = c["Dmax"]
    return blk.cuda()


def _settings(c, n, h):
    """Sampling settings of n sequences: temperature, top-k, top-p, min-p (0, 0, 1, 0: not used)."""
    pick = lambda *v: torch.tensor(v)[torch.randint(0, len(v), (n,), generator=h)]
    t, k, p, m = torch.ones(n), torch.zeros(n, dtype=torch.int32), torch.ones(n), torch.zeros(n)
    if c["mix"] == "served":        # each user's own choice, a greedy one among them now and then
        t, k, p, m = pick(0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2), pick(0, 20, 50, 0, 1000), pick(1.0, 0.8, 0.9, 0.95), pick(0.0, 0.0, 0.05, 0.1)
    elif c["mix"] == "nucleus":
        t, p = pick(0.8, 1.0, 1.3), pick(0.9, 0.95, 0.99)
    elif c["mix"] == "topk":
        t, k = pick(0.7, 1.0), pick(1, 40, 64)
    return [v.cuda() for v in (t.float(), k.to(torch.int32), p.float(), m.float())]


def _logits(c, g, rows, width):
    """Rows as a language model gives them: a bulk, and some tens of tokens that fit the context."""
    z = _randn(g, rows, width) * c["std"]
    n = min(40, c["V"])
    at = torch.randint(0, c["V"], (rows, n), generator=g, device="cuda")
    lift = torch.rand((rows, 1), generator=g, device="cuda") * 8 + 4
    z.scatter_add_(1, at, lift / torch.arange(1, n + 1, device="cuda") ** 0.3)
    if c["masked"]:
        ban = torch.rand((rows, width), generator=g, device="cuda") < c["masked"]
        ban[:, 0] = False
        z.masked_fill_(ban, float("-inf"))
        del ban
    return z.to(torch.bfloat16) if c["bf16"] else z


def prepare(case, seed):
    c = dict(case)
    h, g = torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c=c)
    B, op = c["B"], c["op"]
    if op == "sample":
        s["logits"] = _logits(c, g, B, c["V"] + c["pad"])[:, :c["V"]]
        s["settings"] = _settings(c, B, h)
        s["u"] = (torch.randint(0, 1 << 24, (B,), generator=h).float() / (1 << 24)).cuda()
        s["probs"] = torch.zeros((B, c["V"]), device="cuda") if c["probs"] else None
        return s
    NT = c["NB"] * c["Dmax"]
    s["blk_len"] = _blocks(c, h)
    if op == "filter":
        s["logits"] = _logits(c, g, B * (1 + NT), c["V"]).view(B, 1 + NT, c["V"])
        s["settings"] = _settings(c, B, h)
        s["probs"] = torch.zeros((B, 1 + NT, c["V"]), device="cuda")
        return s
    Hkv, dh, S = c["Hkv"], c["dh"], c["prompt"]
    kind = torch.float32 if c["f32"] else torch.bfloat16
    own_len = torch.tensor(_spread(c["lo"], c["hi"], B), dtype=torch.int32)[torch.randperm(B, generator=h)]
    new = lambda *shape: _randn(g, *shape).to(kind)
    s["shared_table"] = s["table"] = s["k_shared"] = s["v_shared"] = None
    if c["paged"]:
        n, pps = -(-S // PAGE), max(1, -(-c["hi"] // PAGE))
        order = torch.randperm(n + B * pps + 3, generator=h).to(torch.int32).cuda()
        s["shared_table"], s["table"] = order[:n].clone(), order[n:n + B * pps].clone().view(B, pps)
        s["k_cache"], s["v_cache"] = (new(len(order), Hkv, PAGE, dh) for _ in "kv")
    else:
        s["k_shared"], s["v_shared"] = (new(Hkv, S, dh) for _ in "kv")
        s["k_cache"], s["v_cache"] = (new(B, Hkv, max(1, c["hi"]), dh) for _ in "kv")
    s["k_cand"], s["v_cand"] = (new(B, NT, Hkv, dh) for _ in "kv")
    s["q"] = (_randn(g, B, NT, c["Hq"], dh) * 1.5).to(kind)
    s["shared_len"], s["prefix"] = torch.tensor([S], dtype=torch.int32, device="cuda"), own_len.cuda()
    s["out"] = torch.zeros_like(s["q"])
    return s


# ---------------------------------------------------------------------------- plain forms
def _keys(s, which):
    """The prompt's keys (or values) [Hkv][S][dh] and the sequences' own [B][Hkv][n][dh], in fp32."""
    cache, S = s[which + "_cache"], s["c"]["prompt"]
    if s["table"] is None:
        return s[which + "_shared"].float(), cache.float()
    take = lambda t: cache[t.long()].float()
    return take(s["shared_table"]).transpose(0, 1).flatten(1, 2)[:, :S], take(s["table"]).transpose(1, 2).flatten(2, 3)


def _plain_shared(s):
    c = s["c"]
    B, NB, Dmax, Hq, Hkv, dh = (c[k] for k in ("B", "NB", "Dmax", "Hq", "Hkv", "dh"))
    NT, G = NB * Dmax, Hq // Hkv
    q = s["q"].float().view(B, NT, Hkv, G, dh).permute(2, 0, 1, 3, 4).reshape(Hkv, B * NT * G, dh) * dh ** -0.5
    mine = q.view(Hkv, B, NT * G, dh).transpose(0, 1)
    k_all, k_own = _keys(s, "k")
    z = torch.matmul(q, k_all.transpose(1, 2)).masked_fill_(torch.arange(c["prompt"], device="cuda") >= s["shared_len"], float("-inf"))
    z_own = torch.matmul(mine, k_own.transpose(2, 3))
    beyond = torch.arange(k_own.shape[2], device="cuda")[None, :] >= s["prefix"][:, None]
    z_own.masked_fill_(beyond[:, None, None, :], float("-inf"))
    z_blk = torch.matmul(mine, s["k_cand"].float().permute(0, 2, 3, 1))
    t = torch.arange(NT, device="cuda")
    see = (t[:, None] // Dmax == t[None, :] // Dmax) & (t[None, :] <= t[:, None])
    z_blk.masked_fill_(~see.repeat_interleave(G, 0), float("-inf"))
    del k_all, k_own
    own_top = torch.maximum(z_own.amax(-1, keepdim=True), z_blk.amax(-1, keepdim=True)).transpose(0, 1).reshape(Hkv, -1, 1)
    top = torch.maximum(z.amax(-1, keepdim=True), own_top)
    mine_top = top.view(Hkv, B, NT * G, 1).transpose(0, 1)
    z, z_own, z_blk = z.sub_(top).exp_(), z_own.sub_(mine_top).exp_(), z_blk.sub_(mine_top).exp_()
    v_all, v_own = _keys(s, "v")
    o = torch.matmul(z_own, v_own) + torch.matmul(z_blk, s["v_cand"].float().transpose(1, 2))
    o += torch.matmul(z, v_all).view(Hkv, B, NT * G, dh).transpose(0, 1)
    total = z_own.sum(-1, keepdim=True) + z_blk.sum(-1, keepdim=True) + z.sum(-1, keepdim=True).view(Hkv, B, NT * G, 1).transpose(0, 1)
    o = (o / total).view(B, Hkv, NT, G, dh).permute(0, 2, 1, 3, 4).reshape(B, NT, Hq, dh)
    present = t[None, :] % Dmax < s["blk_len"][:, t // Dmax]
    return torch.where(present[:, :, None, None], o, 0).to(s["q"].dtype)


def _plain_weights(z, temperature, top_k, top_p, min_p):
    """z [R][V]; settings [R]. exp((z - max) / temperature) of the tokens that stay, 0 for the others, in 64 bits: the
    sums run over the vocabulary and the cuts depend on values next to a border."""
    z = z.float().nan_to_num(nan=float("-inf"), posinf=torch.finfo(torch.float32).max, neginf=float("-inf"))
    V = z.shape[1]
    order = torch.sort(z, dim=1, descending=True, stable=True)
    some = order.values[:, :1] > float("-inf")
    d = order.values.double() - torch.where(some, order.values[:, :1], 0).double()
    t = temperature[:, None].double()
    w = torch.where(t > 0, torch.exp(d / torch.where(t > 0, t, 1)), (torch.arange(V, device=z.device) == 0)[None, :].double())
    w.masked_fill_(order.values == float("-inf"), 0)
    del d
    place = torch.arange(V, device=z.device)[None, :]
    n = torch.where((top_k <= 0) | (top_k > V), V, top_k)[:, None]
    w.masked_fill_(place >= n, 0)
    run_ = torch.cumsum(w, 1)
    cut = ((run_ - w) >= top_p[:, None].double() * run_[:, -1:]) & (top_p < 1)[:, None]
    del run_
    cut |= w < min_p[:, None].double().clamp(max=1)
    w.masked_fill_(cut & (place > 0), 0)
    return torch.zeros_like(w).scatter_(1, order.indices, w)


def _plain_filter(s):
    c = s["c"]
    B, NB, Dmax, V = c["B"], c["NB"], c["Dmax"], c["V"]
    NT = NB * Dmax
    t = torch.arange(NT, device="cuda")
    need = torch.cat([torch.ones((B, 1), dtype=torch.bool, device="cuda"), t[None, :] % Dmax < s["blk_len"][:, t // Dmax]], 1)
    b, r = need.nonzero(as_tuple=True)
    w = _plain_weights(s["logits"][b, r], *(v[b] for v in s["settings"]))
    w /= w.sum(1, keepdim=True).clamp(min=1e-300)
    s["probs"][b, r] = w.float()
    return s["probs"]


def _plain_sample(s):
    w = _plain_weights(s["logits"], *s["settings"])
    total = w.sum(1, keepdim=True)
    token = (torch.cumsum(w, 1) > s["u"][:, None].double() * total).to(torch.uint8).argmax(1)
    token = torch.where(total[:, 0] > 0, token, -1)
    w /= total.clamp(min=1e-300)
    out = [token.to(torch.int32), torch.where(token >= 0, w.gather(1, token.clamp(min=0)[:, None])[:, 0], 0).float()]
    return out + [w.float()] if s["c"]["probs"] else out


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if own:
        import speculative_decoding_copy_gb300 as ssd
        if op == "shared":
            if "ws" not in s:
                n = ssd.ssd_verify_attn_shared_workspace_size(ssd.attn_shared_args(
                    s["q"], s["k_shared"], s["v_shared"], s["shared_len"], s["k_cache"], s["v_cache"], s["k_cand"], s["v_cand"], s["prefix"],
                    s["blk_len"], s["c"]["Dmax"], s["out"], block_table=s["table"], shared_table=s["shared_table"]))
                s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            return ssd.ssd_verify_attn_shared(s["q"], s["k_shared"], s["v_shared"], s["shared_len"], s["k_cache"], s["v_cache"], s["k_cand"],
                                              s["v_cand"], s["prefix"], s["blk_len"], s["c"]["Dmax"], out=s["out"], ws=s["ws"],
                                              block_table=s["table"], shared_table=s["shared_table"])
        if "ws" not in s:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        t, k, p, m = s["settings"]
        if op == "filter":
            return ssd.ssd_filter_probs(s["logits"], t, k, p, m, blk_len=s["blk_len"], Dmax=s["c"]["Dmax"], out=s["probs"], ws=s["ws"])
        got = ssd.ssd_sample(s["logits"], s["u"], t, k, p, m, probs_out=s["probs"], ws=s["ws"])
        return [got["token"], got["prob"]] + ([s["probs"]] if s["c"]["probs"] else [])
    return {"shared": _plain_shared, "filter": _plain_filter, "sample": _plain_sample}[op](s)


def work(case):
    c = case
    B = c["B"]
    es = 4 if c.get("f32") or c.get("bf16") is False else 2
    if c["op"] == "sample":
        n = float(B) * c["V"]
        return dict(bytes=n * (es + (4 if c["probs"] else 0)) + 24.0 * B, flops=5 * n)
    NT = c["NB"] * c["Dmax"]
    part = 0.3 if c["absent"] else 1.0          # the present tokens
    if c["op"] == "filter":
        n = B * (1 + NT * part) * c["V"]
        return dict(bytes=n * (es + 4), flops=6 * n)
    n, rows, Hkv, dh = float(sum(_spread(c["lo"], c["hi"], B))), NT * c["Hq"] * part, c["Hkv"], c["dh"]
    byt = es * dh * (2 * Hkv * (c["prompt"] + n + B * NT * part) + 2 * B * rows)
    return dict(bytes=byt, flops=4 * rows * dh * (n + B * (c["prompt"] + c["Dmax"] / 2)))


# ---------------------------------------------------------------------------- in 64 bits, from the definition
def _exact_row(z, t, k, p, m):
    """Probabilities [V] of one row z (64 bits): the tokens in their order, best first, as long as the rules let them in."""
    z = torch.where(torch.isnan(z), -torch.inf, z).clamp(max=float(torch.finfo(torch.float32).max))
    out = torch.zeros_like(z)
    live = (z > -torch.inf).nonzero()[:, 0]
    if len(live) == 0:
        return out
    at = live[torch.argsort(-z[live], stable=True)]
    if t <= 0:
        out[at[0]] = 1
        return out
    if k > 0:
        at = at[:k]
    e = torch.exp((z[at] - z[at[0]]) / t)
    keep = len(at)
    if p < 1:
        before = torch.cumsum(e, 0) - e
        keep = min(keep, int((before < p * e.sum()).sum()))
    if m > 0:
        keep = min(keep, int((e >= min(m, 1.0)).sum()))
    keep = max(keep, 1)
    out[at[:keep]] = e[:keep] / e[:keep].sum()
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "sample":
        rows, settings = s["logits"], [v.double().tolist() for v in s["settings"]]
        tokens, probs, full = [], [], []
        for r in range(c["B"]):
            q = _exact_row(rows[r].double(), settings[0][r], int(settings[1][r]), settings[2][r], settings[3][r])
            i = int(torch.searchsorted(torch.cumsum(q, 0), float(s["u"][r]) * float(q.sum()), right=True)) if float(q.sum()) > 0 else -1
            tokens.append(i)
            probs.append(float(q[i]) if i >= 0 else 0.0)
            if c["probs"]:
                full.append(q)
        out = [torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.tensor(probs, dtype=torch.float64, device="cuda")]
        return out + [torch.stack(full)] if c["probs"] else out
    B, NB, Dmax = c["B"], c["NB"], c["Dmax"]
    NT = NB * Dmax
    blk = s["blk_len"].tolist()
    if c["op"] == "filter":
        if B * (1 + NT) * c["V"] > 2e8:
            return None
        out = torch.zeros((B, 1 + NT, c["V"]), dtype=torch.float64, device="cuda")
        settings = [v.double().tolist() for v in s["settings"]]
        for b in range(B):
            for r in range(1 + NT):
                if r == 0 or (r - 1) % Dmax < blk[b][(r - 1) // Dmax]:
                    out[b, r] = _exact_row(s["logits"][b, r].double(), settings[0][b], int(settings[1][b]), settings[2][b], settings[3][b])
        return out
    Hq, Hkv, dh, S = c["Hq"], c["Hkv"], c["dh"], c["prompt"]
    if B * NT * Hq * (S + c["hi"]) * dh > 2 ** 40:
        return None
    G = Hq // Hkv
    out = torch.zeros((B, NT, Hq, dh), dtype=torch.float64, device="cuda")
    for b in range(B):
        tt = torch.tensor([t for t in range(NT) if t % Dmax < blk[b][t // Dmax]], device="cuda", dtype=torch.long)
        if len(tt) == 0:
            continue
        P = int(s["prefix"][b])
        ban = ((tt[:, None] // Dmax != tt[None, :] // Dmax) | (tt[None, :] > tt[:, None])).repeat_interleave(G, 0)
        for head in range(Hkv):
            kv = []
            for w in "kv":
                if c["paged"]:
                    first = torch.cat([s[w + "_cache"][i, head] for i in s["shared_table"].tolist()])[:S]
                    mine = torch.cat([s[w + "_cache"][i, head] for i in s["table"][b].tolist()])[:P]
                else:
                    first, mine = s[w + "_shared"][head][:S], s[w + "_cache"][b, head][:P]
                kv.append(torch.cat([first.double(), mine.double(), s[w + "_cand"][b, tt, head].double()]))
            z = (s["q"][b, tt, head * G:(head + 1) * G].double().reshape(-1, dh) / dh ** 0.5) @ kv[0].T
            z[:, S + P:].masked_fill_(ban, float("-inf"))
            out[b, tt, head * G:(head + 1) * G] = (torch.softmax(z, 1) @ kv[1]).view(len(tt), G, dh)
    return out
