"""The 8-bit key/value cache of the speculate-and-verify step: what is measured.

Four operators, as a serving loop calls them one after another:

  pages    ssd_page_tables        block tables and slot maps from request lengths
  append   ssd_append_kv_quant    prompt (or decode) rows quantised into the cache at their slots
  commit   ssd_commit_kv_quant    the accepted candidates' rows quantised into the cache
  attn     ssd_verify_attn_quant  block-triangular verification (one token: decode) over that cache

The cache holds e4m3 codes and one fp32 scale for each block of `sb` tokens and kv head; pages are
128 tokens. With `own` false, run() computes them with elementary torch operations; with `own` true
it calls the framework.
"""
import numpy as np
import torch

own = False

PAGE = 128
LOG_MIN = -100          # least exponent of a block scale


# ---------------------------------------------------------------------------- cases
def _attn(name, B, NB, Dmax, Hq, Hkv, lo, hi, dh=128, sb=128, paged=True, absent=False):
    return dict(name=name, op="attn", B=B, NB=NB, Dmax=Dmax, Hq=Hq, Hkv=Hkv, dh=dh, lo=lo, hi=hi, sb=sb, paged=paged, absent=absent)


def _append(name, B, lo, hi, Hkv, cur_lo=0, cur_hi=0, dh=128, sb=128, f32=False):
    return dict(name=name, op="append", B=B, lo=lo, hi=hi, cur_lo=cur_lo, cur_hi=cur_hi, Hkv=Hkv, dh=dh, sb=sb, f32=f32)


def _commit(name, B, NB, Dmax, Hkv, cur_lo, cur_hi, dh=128, sb=128, paged=True):
    return dict(name=name, op="commit", B=B, NB=NB, Dmax=Dmax, Hkv=Hkv, cur_lo=cur_lo, cur_hi=cur_hi, dh=dh, sb=sb, paged=paged)


def _pages(name, B, cur_lo, cur_hi, add_lo, add_hi, pps):
    return dict(name=name, op="pages", B=B, cur_lo=cur_lo, cur_hi=cur_hi, add_lo=add_lo, add_hi=add_hi, pps=pps)


def listed():
    return [
        # one user decoding a token after a prompt of 4096: the smallest attention call, where latency counts
        _attn("decode_one", 1, 1, 1, 32, 8, 4096, 4096),
        # 64 users decoding a token each, prefixes of 2k to 8k: the cache's bytes count
        _attn("decode_64", 64, 1, 1, 32, 8, 2048, 8192),
        # a chain draft of five tokens behind odd short prefixes, head dim 64, contiguous cache, scales of 32 tokens
        _attn("chain_dh64", 7, 1, 5, 14, 2, 1, 1500, dh=64, sb=32, paged=False),
        # four copied continuations of twenty tokens, prefix 4096: the benchmark's verification
        _attn("verify_4096", 1, 4, 20, 32, 8, 4096, 4096),
        # batched serving, eight continuations and a chain block, some of them absent, prefixes of 1k to 16k: the largest
        _attn("verify_batch", 32, 9, 16, 32, 8, 1024, 16384, sb=16, absent=True),
        # 64 query heads, prefixes of 32768: long context
        _attn("verify_long", 4, 5, 20, 64, 8, 32768, 32768),
        # four prompts of up to 8192 tokens written at once
        _append("append_prompt", 4, 2500, 8192, 8),
        # one new token for each of 64 sequences, somewhere inside their blocks
        _append("append_decode", 64, 1, 1, 8, 100, 8000),
        # the accepted tokens of one user
        _commit("commit_one", 1, 4, 20, 8, 4096, 4096),
        # the accepted tokens of a serving batch, contiguous cache, scales of 16 tokens
        _commit("commit_32", 32, 9, 16, 8, 1024, 2000, sb=16, paged=False),
        # pages for a step's candidates of 64 sequences, taken before it and trimmed behind it
        _pages("pages_step", 64, 2048, 8192, 17, 21, 72),
        # 512 prompts admitted and their requests ended
        _pages("pages_admit", 512, 0, 0, 100, 4000, 32),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "commit", "pages"])
    dh, sb, paged = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), rng.random() < 0.6
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "attn":
        while True:
            B, NB, Dmax = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4, 5, 9]), _log(rng, 1, 24)
            G, hi = rng.choice([1, 2, 3, 4, 5, 7, 8]), _log(rng, 1, 32768)
            lo = rng.randint(0, hi)
            if B * NB * Dmax * G * Hkv * hi <= 32 * 144 * 32 * 16384 // 4 and B * hi * Hkv <= 64 * 8192 * 8:
                c = _attn("", B, NB, Dmax, G * Hkv, Hkv, lo, hi, dh, sb, paged, rng.random() < 0.5)
                break
    elif op == "append":
        B, hi = _log(rng, 1, 64), _log(rng, 1, 8192)
        hi = max(1, min(hi, 32768 // B))
        cur = _log(rng, 1, 2000)
        c = _append("", B, rng.randint(0, hi), hi, Hkv, rng.randint(0, cur), cur, dh, sb, rng.random() < 0.3)
    elif op == "commit":
        cur = _log(rng, 1, 4000)
        c = _commit("", _log(rng, 1, 64), rng.randint(1, 9), _log(rng, 1, 24), Hkv, rng.randint(0, cur), cur, dh, sb, paged)
    else:
        cur, add = _log(rng, 1, 6000), _log(rng, 1, 3000)
        c = _pages("", _log(rng, 1, 700), rng.randint(0, cur), cur, rng.randint(0, add), add, -(-(cur + add) // PAGE) + rng.randint(0, 5))
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi]: the same ones for every seed."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi], np.int64)


def _lens(c, lo, hi, g, off=0):
    v = _spread(c[lo], c[hi], c["B"])
    return torch.from_numpy(v)[torch.randperm(c["B"], generator=g)].to(torch.int32)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(c, g, pages, tokens):
    """Codes and scales of a cache that earlier tokens filled: values of a few units, scales that vary by block."""
    nb = -(-tokens // c["sb"])
    codes = (_randn(g, pages, c["Hkv"], tokens, c["dh"]) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.exp2(torch.randint(-8, -5, (pages, c["Hkv"], nb), generator=g, device="cuda").float())
    return codes, scale


def prepare(case, seed):
    c = dict(case)
    h, g = torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c=c)
    B = c["B"]
    if c["op"] == "pages":
        cur, add = _lens(c, "cur_lo", "cur_hi", h), _lens(c, "add_lo", "add_hi", h)
        held = (cur + PAGE - 1) // PAGE
        most = B * (-(-(c["cur_hi"] + c["add_hi"]) // PAGE) + 2) + 16
        order = torch.randperm(most, generator=h).to(torch.int32)
        used = torch.arange(c["pps"])[None, :] < held[:, None]
        table = torch.full((B, c["pps"]), -1, dtype=torch.int32)
        n = int(held.sum())
        table[used] = order[:n]
        free = torch.zeros(most, dtype=torch.int32)
        free[:most - n] = order[n:]
        s |= dict(cur=cur, add=add, held=held, table=table, free=free, n_free=torch.tensor([most - n], dtype=torch.int32), none=torch.zeros(B, dtype=torch.int32))
        s = {k: v.cuda() if torch.is_tensor(v) else v for k, v in s.items()}
        s["cap"] = B * c["add_hi"]
        return s
    Hkv, dh = c["Hkv"], c["dh"]
    if c["op"] == "attn":
        prefix, most = _lens(c, "lo", "hi", h), c["hi"]
    elif c["op"] == "append":
        prefix, most = _lens(c, "cur_lo", "cur_hi", h), c["cur_hi"] + c["hi"]
    else:
        prefix, most = _lens(c, "cur_lo", "cur_hi", h), c["cur_hi"] + c["Dmax"]
    pps = max(1, -(-most // PAGE))
    if c.get("paged", True):
        pages, tokens = B * pps + 3, PAGE
        s["table"] = torch.randperm(pages, generator=h)[:B * pps].view(B, pps).to(torch.int32).cuda()
    else:
        pages, tokens = B, max(1, most)
        s["table"] = None
    s["k_cache"], s["k_scale"] = _cache(c, g, pages, tokens)
    s["v_cache"], s["v_scale"] = _cache(c, g, pages, tokens)
    s["prefix"] = prefix.cuda()
    if c["op"] == "append":
        add = _lens(c, "lo", "hi", h)
        T = int(add.sum())
        b = torch.repeat_interleave(torch.arange(B), add.long())
        pos = torch.arange(T) - (torch.cumsum(add, 0) - add)[b] + prefix[b]
        s["slots"] = (s["table"].cpu()[b, pos // PAGE].long() * PAGE + pos % PAGE).to(torch.int32).cuda()
        # the rows sit in a projection's output of keys and values together
        kv = _randn(g, T, 2, Hkv, dh) * torch.exp2(torch.randint(-2, 3, (T, 2, Hkv, 1), generator=g, device="cuda").float())
        kv = kv if c["f32"] else kv.to(torch.bfloat16)
        s["k_new"], s["v_new"] = kv[:, 0], kv[:, 1]
        return s
    NB, Dmax = c["NB"], c["Dmax"]
    NT = NB * Dmax
    s["k_cand"] = _randn(g, B, NT, Hkv, dh).to(torch.bfloat16)
    s["v_cand"] = _randn(g, B, NT, Hkv, dh).to(torch.bfloat16)
    if c["op"] == "commit":
        s["best"] = torch.randint(-1 if B > 4 else 0, NB, (B,), generator=h, dtype=torch.int32).cuda()
        s["n_out"] = torch.randint(1 if B > 4 else Dmax, Dmax + 2, (B,), generator=h, dtype=torch.int32).cuda()
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    s["q"] = (_randn(g, B, NT, c["Hq"], dh) * 1.5).to(torch.bfloat16)
    blk = torch.full((B, NB), Dmax, dtype=torch.int32)
    if c["absent"]:
        blk = torch.where(torch.rand((B, NB), generator=h) < 0.4, 0, torch.randint(0, Dmax + 1, (B, NB), generator=h)).to(torch.int32)
        blk[0, 0] = Dmax
    s["blk_len"] = blk.cuda()
    s["out"] = torch.zeros_like(s["q"])
    return s


# ---------------------------------------------------------------------------- plain forms
def _plain_pages(s, cur, add, cap):
    """Grows or trims every sequence's table to ceil((cur + add) / 128) pages; updates the state in place."""
    table, held, free = s["table"], s["held"], s["free"]
    pps, N = table.shape[1], free.shape[0]
    want = (cur + add + PAGE - 1) // PAGE
    grow, trim = (want - held).clamp(min=0), (held - want).clamp(min=0)
    avail = s["n_free"] + trim.sum()
    run_ = torch.cumsum(grow, 0)
    served = ((grow == 0) | (run_ <= avail)) & (want <= pps)
    col = torch.arange(pps, device=table.device)[None, :]
    gone = (col >= want[:, None]) & (col < held[:, None])
    at = s["n_free"] + (torch.cumsum(trim, 0) - trim)[:, None] + col - want[:, None]
    more = torch.cat([free, free.new_zeros(1)])
    more.scatter_(0, torch.where(gone, at, N).flatten().long(), table.flatten())
    new = served[:, None] & (col >= held[:, None]) & (col < want[:, None])
    src = avail - 1 - ((run_ - grow)[:, None] + col - held[:, None])
    table.copy_(torch.where(gone, -1, torch.where(new, more[src.clamp(0, N).long()], table)))
    free.copy_(more[:N])
    s["n_free"].copy_(avail - (grow * served).sum())
    held.copy_(torch.where(served, want, held))
    start = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)]).to(torch.int32)
    t = torch.arange(cap, device=table.device, dtype=torch.int32)
    b = torch.searchsorted(start[1:], t, right=True)
    inside = b < cur.shape[0]
    b = b.clamp(max=cur.shape[0] - 1)
    p = cur[b] + t - start[b]
    slot = table[b, (p // PAGE).clamp(0, pps - 1)] * PAGE + p % PAGE
    return start, torch.where(inside & served[b], slot, -1), served.to(torch.int32)


def _pow2_scale(a):
    """The least power of two s with a <= 448 s (448 = 0.875 2^9), exponent at least -100."""
    m, e = torch.frexp(a)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(a > 0, k, LOG_MIN).clamp(min=LOG_MIN).float())


def _plain_write(x, slots, codes, scale, sb):
    """Quantises rows x [T][Hkv][dh] into the slots of a cache of pages [pages][Hkv][tokens][dh], in place."""
    pages, H, tokens, dh = codes.shape
    nb = scale.shape[2]
    x = x.float()
    page, off = slots // tokens, slots % tokens
    blk, row = off // sb, off % sb
    ids, at = torch.unique(page * nb + blk, return_inverse=True)
    U = ids.shape[0]
    pg, bk = ids // nb, ids % nb
    top = torch.zeros((U, H), device=x.device).scatter_reduce_(0, at[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    first = torch.full((U,), sb, device=x.device, dtype=row.dtype).scatter_reduce_(0, at, row, "amin")
    old = scale[pg, :, bk]
    need = _pow2_scale(top)
    now = torch.where((first == 0)[:, None], need, torch.maximum(old, need))
    # rows that the block already holds, under the new scale
    r = torch.arange(sb, device=x.device)
    where = (bk[:, None] * sb + r).clamp(max=tokens - 1)
    have = codes[pg[:, None], :, where]                                    # [U][sb][H][dh]
    again = (have.view(torch.float8_e4m3fn).float() * (old / now)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = ((r[None, :] < first[:, None])[:, :, None] & (now > old)[:, None, :])[..., None]
    u, j = (r[None, :] < torch.minimum(first, tokens - bk * sb)[:, None]).nonzero(as_tuple=True)
    codes[pg[u], :, where[u, j]] = torch.where(keep, again, have)[u, j]
    scale[pg, :, bk] = now
    codes[page, :, off] = (x / now[at][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(s):
    return [s["k_cache"].view(torch.float8_e4m3fn), s["k_scale"], s["v_cache"].view(torch.float8_e4m3fn), s["v_scale"]]


def _plain_commit(s):
    c = s["c"]
    B, NB, Dmax = c["B"], c["NB"], c["Dmax"]
    n = torch.where(s["best"] >= 0, s["n_out"] - 1, 0)
    b, i = (torch.arange(Dmax, device="cuda")[None, :] < n[:, None]).nonzero(as_tuple=True)
    pos = s["prefix"][b].long() + i
    tokens = s["k_cache"].shape[2]
    page = b if s["table"] is None else s["table"][b, pos // tokens].long()
    slots = page * tokens + pos % tokens
    src = s["best"][b] * Dmax + i
    _plain_write(s["k_cand"][b, src], slots, s["k_cache"], s["k_scale"], c["sb"])
    _plain_write(s["v_cand"][b, src], slots, s["v_cache"], s["v_scale"], c["sb"])
    return _values(s) + [torch.add(s["prefix"], n, out=s["new_len"])]


def _gather(codes, scale, table, sb):
    """The cache as fp32 values [B][Hkv][tokens][dh], through the block table if there is one."""
    if table is not None:
        codes, scale = codes[table.long()].transpose(1, 2).flatten(2, 3), scale[table.long()].transpose(1, 2).flatten(2, 3)
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(sb, -1)[..., :codes.shape[2], None]


def _plain_attn(s):
    c = s["c"]
    B, NB, Dmax, Hq, Hkv, dh = (c[k] for k in ("B", "NB", "Dmax", "Hq", "Hkv", "dh"))
    NT, G = NB * Dmax, Hq // Hkv
    q = s["q"].float().view(B, NT, Hkv, G, dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, NT * G, dh)
    k = _gather(s["k_cache"], s["k_scale"], s["table"], c["sb"])
    own_ = torch.matmul(q, s["k_cand"].float().permute(0, 2, 3, 1)) * dh ** -0.5
    pre = torch.matmul(q, k.transpose(2, 3)) * dh ** -0.5
    del k
    t = torch.arange(NT, device="cuda")
    see = (t[:, None] // Dmax == t[None, :] // Dmax) & (t[None, :] <= t[:, None])
    own_.masked_fill_(~see.repeat_interleave(G, 0), float("-inf"))
    beyond = torch.arange(pre.shape[3], device="cuda")[None, :] >= s["prefix"][:, None]
    pre.masked_fill_(beyond[:, None, None, :], float("-inf"))
    top = torch.maximum(own_.amax(-1, keepdim=True), pre.amax(-1, keepdim=True))
    own_, pre = own_.sub_(top).exp_(), pre.sub_(top).exp_()
    total = own_.sum(-1, keepdim=True) + pre.sum(-1, keepdim=True)
    o = torch.matmul(own_, s["v_cand"].float().transpose(1, 2))
    o += torch.matmul(pre, _gather(s["v_cache"], s["v_scale"], s["table"], c["sb"]))
    o = (o / total).view(B, Hkv, NT, G, dh).permute(0, 2, 1, 3, 4).reshape(B, NT, Hq, dh)
    present = t[None, :] % Dmax < s["blk_len"][:, t // Dmax]
    return torch.where(present[:, :, None, None], o, 0).to(torch.bfloat16)


# ---------------------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    if own:
        import speculative_decoding_copy_gb300 as ssd
        if "ws" not in s:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        if c["op"] == "pages":
            a = ssd.ssd_page_tables(s["cur"], s["add"], s["held"], s["table"], s["free"], s["n_free"], s["cap"], ws=s["ws"])
            ssd.ssd_page_tables(s["cur"], s["none"], s["held"], s["table"], s["free"], s["n_free"], 0, ws=s["ws"])
            return [a["row_start"], a["slot_map"], a["served"], s["table"], s["held"], s["free"], s["n_free"]]
        if c["op"] == "append":
            ssd.ssd_append_kv_quant(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], c["sb"], ws=s["ws"])
            return _values(s)
        if c["op"] == "commit":
            ssd.ssd_commit_kv_quant(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["k_cand"], s["v_cand"], s["prefix"], s["best"], s["n_out"],
                                    c["Dmax"], c["sb"], new_len=s["new_len"], block_table=s["table"], ws=s["ws"])
            return _values(s) + [s["new_len"]]
        return ssd.ssd_verify_attn_quant(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["k_cand"], s["v_cand"], s["prefix"],
                                         s["blk_len"], c["Dmax"], c["sb"], out=s["out"], ws=s["ws"], block_table=s["table"])
    if c["op"] == "pages":
        # a step takes pages for its new tokens; behind it what was not kept goes back
        start, slots, served = _plain_pages(s, s["cur"], s["add"], s["cap"])
        _plain_pages(s, s["cur"], s["none"], 0)
        return [start, slots, served, s["table"], s["held"], s["free"], s["n_free"]]
    if c["op"] == "append":
        _plain_write(s["k_new"], s["slots"], s["k_cache"], s["k_scale"], c["sb"])
        _plain_write(s["v_new"], s["slots"], s["v_cache"], s["v_scale"], c["sb"])
        return _values(s)
    if c["op"] == "commit":
        return _plain_commit(s)
    return _plain_attn(s)


def work(case):
    c = case
    B = c["B"]
    if c["op"] == "pages":
        cur, add = _spread(c["cur_lo"], c["cur_hi"], B), _spread(c["add_lo"], c["add_hi"], B)
        moved = float(add.sum()) / PAGE
        return dict(bytes=4.0 * (2 * 4 * B + 4 * moved + B * c["add_hi"] + 2 * B), flops=0.0)
    Hkv, dh = c["Hkv"], c["dh"]
    if c["op"] == "append":
        n = float(_spread(c["lo"], c["hi"], B).sum())
        return dict(bytes=2 * n * Hkv * dh * ((4 if c["f32"] else 2) + 1) + 4 * n + 64.0 * B, flops=4 * n * Hkv * dh)
    if c["op"] == "commit":
        n = B * c["Dmax"] * (0.5 if B > 4 else 1.0)
        return dict(bytes=2 * n * Hkv * dh * 3 + 64.0 * B, flops=4 * n * Hkv * dh)
    n, NT = float(_spread(c["lo"], c["hi"], B).sum()), c["NB"] * c["Dmax"]
    part = 0.3 if c["absent"] else 1.0          # the present tokens
    rows = NT * c["Hq"] * part
    byt = 2 * n * Hkv * (dh + 4 / c["sb"]) + 4 * B * rows * dh + 4 * B * NT * part * Hkv * dh
    return dict(bytes=byt, flops=4 * rows * dh * (n + B * c["Dmax"] / 2))


# ---------------------------------------------------------------------------- in 64 bits, from the definition
_E4M3 = np.array([((-1.0) ** (i >> 7)) * ((i & 7) / 8 * 2.0 ** -6 if (i >> 3) & 15 == 0 else (1 + (i & 7) / 8) * 2.0 ** (((i >> 3) & 15) - 7)) for i in range(256)])


def _nearest(v):
    """Nearest e4m3 value, ties to the even code; |v| <= 448."""
    grid = _E4M3[:127]
    a = np.abs(v)
    hi = np.searchsorted(grid, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(grid[pick], v)


def _exact_write(x, slots, vals, scale, sb):
    """x [T][H][dh]; vals [pages][H][tokens][dh]: code values; slots in order, each block's rows side by side."""
    tokens = vals.shape[2]
    t, T = 0, len(slots)
    while t < T:
        page, off = divmod(int(slots[t]), tokens)
        blk, row = divmod(off, sb)
        n = 1
        while t + n < T and slots[t + n] == slots[t] + n and row + n < sb and off + n < tokens:
            n += 1
        part = x[t:t + n]
        top = np.abs(part).max((0, 2))
        need = 2.0 ** np.maximum(np.where(top > 0, np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), LOG_MIN), LOG_MIN)
        old = scale[page, :, blk].copy()
        now = need if row == 0 else np.maximum(old, need)
        if row:
            held = vals[page, :, blk * sb:off]
            vals[page, :, blk * sb:off] = np.where((now > old)[:, None, None], _nearest(held * (old / now)[:, None, None]), held)
        vals[page, :, off:off + n] = _nearest(part / now[None, :, None]).transpose(1, 0, 2)
        scale[page, :, blk] = now
        t += n


def exact(case, seed):
    c = dict(case)
    if c["op"] == "pages":
        return None
    s = prepare(case, seed)
    if c["op"] in ("append", "commit"):
        f = lambda t: t.double().cpu().numpy()
        slots, rows = None, None
        if c["op"] == "append":
            slots, rows = s["slots"].cpu().numpy().astype(np.int64), (f(s["k_new"]), f(s["v_new"]))
            if len(slots) > 40000:
                return None
        else:
            best, n_out, pre = (s[k].cpu().numpy().astype(np.int64) for k in ("best", "n_out", "prefix"))
            tokens = s["k_cache"].shape[2]
            sl, kr, vr = [], [], []
            kc, vc = f(s["k_cand"]), f(s["v_cand"])
            for b in range(c["B"]):
                for i in range(int(n_out[b]) - 1 if best[b] >= 0 else 0):
                    p = int(pre[b]) + i
                    page = b if s["table"] is None else int(s["table"][b, p // tokens])
                    sl.append(page * tokens + p % tokens)
                    kr.append(kc[b, best[b] * c["Dmax"] + i])
                    vr.append(vc[b, best[b] * c["Dmax"] + i])
            slots, rows = np.array(sl, np.int64), (np.array(kr), np.array(vr))
        got = []
        for x, w in zip(rows, ("k", "v")):
            vals, scale = _E4M3[s[w + "_cache"].cpu().numpy()], f(s[w + "_scale"])
            if len(slots):
                _exact_write(x, slots, vals, scale, c["sb"])
            got += [vals, scale]
        if c["op"] == "commit":
            got.append(None)
        return got
    B, NB, Dmax, Hq, Hkv, dh = (c[k] for k in ("B", "NB", "Dmax", "Hq", "Hkv", "dh"))
    if B * NB * Dmax * Hq * c["hi"] * dh > 2 ** 42:
        return None
    G, NT = Hq // Hkv, NB * Dmax
    value = torch.from_numpy(_E4M3).cuda()
    out = torch.zeros((B, NT, Hq, dh), dtype=torch.float64, device="cuda")
    for b in range(B):
        P = int(s["prefix"][b])
        pages = [b] if s["table"] is None else s["table"][b].long()
        sc, codes = {}, {}
        for w in ("k", "v"):
            codes[w] = torch.cat(list(s[w + "_cache"][pages]), 1)[:, :P]
            sc[w] = torch.cat(list(s[w + "_scale"][pages]), 1).double().repeat_interleave(c["sb"], 1)[:, :P]
        ok = [t for t in range(NT) if t % Dmax < int(s["blk_len"][b, t // Dmax])]
        if not ok:
            continue
        tt = torch.tensor(ok, device="cuda")
        ban = ((tt[:, None] // Dmax != tt[None, :] // Dmax) | (tt[None, :] > tt[:, None])).repeat_interleave(G, 0)
        for h in range(Hkv):
            qq = s["q"][b, tt, h * G:(h + 1) * G].double().reshape(-1, dh) / dh ** 0.5
            kk = torch.cat([value[codes["k"][h].long()] * sc["k"][h][:, None], s["k_cand"][b, tt, h].double()])
            vv = torch.cat([value[codes["v"][h].long()] * sc["v"][h][:, None], s["v_cand"][b, tt, h].double()])
            z = qq @ kk.T
            z[:, P:].masked_fill_(ban, float("-inf"))
            z = torch.softmax(z, 1)
            out[b, tt, h * G:(h + 1) * G] = (z @ vv).view(len(ok), G, dh)
    return out
