"""The cache and attention operators around the indexer, as measured cases.

Three operators: rotated FP8 rows for the indexer (``rotate_quantise``), the append of rotated keys and values to a
paged 8-bit cache (``cache_append``), and attention over that cache (``cache_attend``): over whole sequences, or over
the positions that the indexer selected.  ``run`` computes them in plain torch, or through the library where ``own``
is set."""

import math

import torch

own = False

E4M3_MAX = 448.0
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode step's indexer queries: 16 sequences, one token each
        dict(name="rows_decode_16", op="rows", S=16, H=64, D=128, act="bf16", rot=64, inter=False, pos0=1048560),
        # the indexer queries of a whole prefill of 16,384 tokens
        dict(name="rows_prefill_16k", op="rows", S=16384, H=64, D=128, act="bf16", rot=64, inter=False, pos0=0),
        # one new token for each of 16 sequences, in the middle of their blocks
        dict(name="append_decode_16", op="append", B=16, q_lo=1, q_hi=1, past_lo=100, past_hi=60000, Hq=64, Hkv=8, D=128,
             page=64, block=16, act="bf16", rot=128, inter=False),
        # a prefill chunk of one sequence behind 8,192 cached tokens
        dict(name="append_chunk_8k", op="append", B=1, q_lo=8192, q_hi=8192, past_lo=8192, past_hi=8192, Hq=64, Hkv=8,
             D=128, page=64, block=64, act="bf16", rot=128, inter=False),
        # several prompts of odd lengths, smaller heads, part of each head rotated, pages of 96 tokens
        dict(name="append_ragged_odd", op="append", B=7, q_lo=1, q_hi=701, past_lo=0, past_hi=333, Hq=16, Hkv=4, D=64,
             page=96, block=32, act="fp16", rot=32, inter=True),
        # a chat's first answers: one sequence, a few hundred cached tokens; latency counts
        dict(name="attend_one_short", op="attend", B=1, q_lo=1, q_hi=1, len_lo=333, len_hi=333, Hq=64, Hkv=8, D=128,
             page=64, block=16, act="bf16", sel=0, causal=True),
        # a decode batch over long contexts of different lengths
        dict(name="attend_decode_16", op="attend", B=16, q_lo=1, q_hi=1, len_lo=16384, len_hi=65536, Hq=64, Hkv=8, D=128,
             page=64, block=16, act="bf16", sel=0, causal=True),
        # one query over 1,048,576 tokens with one shared key and value head
        dict(name="attend_decode_1m", op="attend", B=1, q_lo=1, q_hi=1, len_lo=1048576, len_hi=1048576, Hq=64, Hkv=1,
             D=128, page=64, block=64, act="bf16", sel=0, causal=True),
        # a few drafted tokens a sequence, checked together; odd lengths, smaller heads
        dict(name="attend_verify_odd", op="attend", B=9, q_lo=1, q_hi=5, len_lo=777, len_hi=12001, Hq=32, Hkv=4, D=64,
             page=96, block=32, act="fp16", sel=0, causal=True),
        # a prefill chunk of 2,048 tokens at the end of 16,384
        dict(name="attend_chunk_2k", op="attend", B=1, q_lo=2048, q_hi=2048, len_lo=16384, len_hi=16384, Hq=64, Hkv=8,
             D=128, page=64, block=64, act="bf16", sel=0, causal=True),
        # a decode batch over the 2,048 positions that the indexer selected in each context
        dict(name="attend_selected_16", op="attend", B=16, q_lo=1, q_hi=1, len_lo=16384, len_hi=65536, Hq=64, Hkv=8,
             D=128, page=64, block=16, act="bf16", sel=2048, causal=True),
        # a prefill chunk of 1,024 tokens, each over its own 2,048 selected positions
        dict(name="attend_selected_1k", op="attend", B=1, q_lo=1024, q_hi=1024, len_lo=16384, len_hi=16384, Hq=64, Hkv=8,
             D=128, page=64, block=16, act="bf16", sel=2048, causal=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "append", "append", "attend", "attend", "attend"])
    act, D, inter = rng.choice(["bf16", "fp16"]), rng.choice([64, 128, 128]), rng.random() < 0.4
    rot = rng.choice([0, 16, 32, 48, 64] + ([96, 128, 128] if D == 128 else [64]))
    if op == "rows":
        return dict(op=op, S=_log_int(rng, 1, 16384), H=rng.choice([1, 4, 8, 16, 32, 64]), D=D, act=act, rot=rot, inter=inter,
                    pos0=rng.choice([0, rng.randrange(1000000)]))
    block = rng.choice([1, 8, 16, 16, 32, 64, 128])
    page = block * rng.choice([1, 2, 3, 4] if block > 8 else [3, 4, 8, 16])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 6, 8, 16] if Hkv > 2 else [4, 8, 12, 16, 32, 64])
    while Hkv * group > 64:
        group //= 2
    case = dict(op=op, B=1, q_lo=1, q_hi=1, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, block=block, act=act)
    if op == "append":
        case["B"] = _log_int(rng, 1, 64)
        case["q_hi"] = _log_int(rng, 1, 8192 // case["B"])
        case["q_lo"] = rng.choice([1, case["q_hi"]])
        case["past_lo"], case["past_hi"] = 0, _log_int(rng, 1, 65536 // case["B"])
        return dict(case, rot=rot, inter=inter)
    kind = rng.choice(["decode", "verify", "chunk", "selected", "selected"])
    case.update(sel=0, causal=True)
    if kind in ("decode", "verify"):
        case["B"] = _log_int(rng, 1, 32)
        case["q_hi"] = 1 if kind == "decode" else rng.randint(2, 16)
        case["len_hi"] = _log_int(rng, 64, min(1 << 20, (1 << 22) // (case["B"] * Hkv)))
        if kind == "verify":  # the plain form holds every score
            case["len_hi"] = min(case["len_hi"], (1 << 28) // (case["B"] * case["q_hi"] * case["Hq"]))
        case["len_lo"] = max(case["q_hi"], case["len_hi"] // rng.choice([1, 4, 50]))
        case["len_hi"] = max(case["len_hi"], case["len_lo"])
        case["causal"] = rng.random() < 0.8
    elif kind == "chunk":
        case["B"] = _log_int(rng, 1, 6)
        case["q_hi"] = _log_int(rng, 17, 2048 // case["B"])
        case["q_lo"] = max(1, case["q_hi"] // rng.choice([1, 3]))
        case["len_lo"] = case["q_hi"]
        case["len_hi"] = max(case["q_hi"], _log_int(rng, 64, 16384))
        case["causal"] = rng.random() < 0.8
    else:
        case["B"] = _log_int(rng, 1, 16)
        case["q_hi"] = rng.choice([1, _log_int(rng, 1, 1024 // case["B"])])
        case["sel"] = rng.choice([64, 512, 2048, 2048, 2051])
        case["len_lo"] = case["q_hi"] + rng.randrange(200)
        case["len_hi"] = case["len_lo"] + _log_int(rng, 64, 65536 // case["B"])
    return case


def _lengths(case, key, n):
    """n whole numbers spread evenly from case[key + "_lo"] to case[key + "_hi"], both among them where n > 1."""
    lo, hi = case[key + "_lo"], case[key + "_hi"]
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _layout(case):
    """Rows and cached tokens of each sequence, the latter with the rows."""
    B = case["B"]
    q = _lengths(case, "q", B)
    if case["op"] == "append":
        return q, [a + b for a, b in zip(reversed(_lengths(case, "past", B)), q)]
    n = _lengths(case, "len", B)
    n = n[::2] + n[1::2][::-1]
    return q, [max(a, b) for a, b in zip(n, q)]


# --------------------------------------------------------------------------------------------------------- inputs --

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _rope_table(n, rot):
    """[n, rot] fp32: cosines, then sines, of position * 10000^(-2i/rot); the angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s, no less than 2^-100."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e + 127) << 23).view(torch.float32)  # 2^e by its bits


def _filled_cache(gen, n_pages, case):
    """Codes and scales of a cache whose blocks hold normal values of different sizes."""
    page, block, Hkv, D = case["page"], case["block"], case["Hkv"], case["D"]
    codes = torch.empty((n_pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_pages, page // block, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (page * Hkv * D))
    for p0 in range(0, n_pages, step):
        p1 = min(n_pages, p0 + step)
        x = _randn(gen, p1 - p0, page // block, block, Hkv, D)
        x *= torch.exp(0.4 * _randn(gen, p1 - p0, page // block, block, Hkv, 1))  # tokens of different norms
        s = _pow2_scale(x.abs().amax(dim=(2, 4)))
        codes[p0:p1] = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(p1 - p0, page, Hkv, D)
        scale[p0:p1] = s
    return codes, scale


def _page_table(gen, lens, page):
    """Pages of each sequence in shuffled order, -1 behind them, and the number of pages of the cache."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 2


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    act, D = ACT[case["act"]], case["D"]
    if case["op"] == "rows":
        x = _randn(gen, case["S"], case["H"], D) * torch.exp(0.5 * _randn(gen, case["S"], case["H"], 1))
        pos = torch.arange(case["S"], dtype=torch.int32, device="cuda") + case["pos0"]
        return dict(case=case, x=x.to(act), positions=pos,
                    table=_rope_table(case["pos0"] + case["S"], case["rot"]) if case["rot"] else None)
    q_lens, lens = _layout(case)
    S = sum(q_lens)
    table, n_pages = _page_table(gen, lens, case["page"])
    st = dict(case=case, max_q=max(q_lens), page_table=table,
              cu_q=torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32, device="cuda"),
              kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    st["k_cache"], st["k_scale"] = _filled_cache(gen, n_pages, case)
    st["v_cache"], st["v_scale"] = _filled_cache(gen, n_pages, case)
    if case["op"] == "append":
        gain = torch.exp(0.4 * _randn(gen, S, 1, 1))
        st["k"] = (_randn(gen, S, case["Hkv"], D) * gain).to(act)
        st["v"] = _randn(gen, S, case["Hkv"], D).to(act)
        st["q"] = _randn(gen, S, case["Hq"], D).to(act)
        st["table"] = _rope_table(max(lens), case["rot"]) if case["rot"] else None
        return st
    st["q"] = (_randn(gen, S, case["Hq"], D) * 1.5).to(act)
    if case["sel"]:
        # distinct ascending positions up to each row's own, -1 behind them, as the indexer writes them
        W = case["sel"]
        idx = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
        count = torch.empty((S,), dtype=torch.int32, device="cuda")
        r = 0
        for nq, n in zip(q_lens, lens):
            for i in range(nq):
                see = n - nq + i + 1
                take = min(see, W)
                idx[r, :take] = torch.randperm(see, generator=gen, device="cuda", dtype=torch.int32)[:take].sort().values
                r += 1
            count[r - nq:r] = (torch.arange(nq, device="cuda", dtype=torch.int32) + (n - nq + 1)).clamp(max=W)
        st["sel_idx"], st["sel_len"] = idx, count
    return st


# ------------------------------------------------------------------------------------------------------ the calls --

def run(st):
    op = st["case"]["op"]
    if own:
        return {"rows": _own_rows, "append": _own_append, "attend": _own_attend}[op](st)
    return {"rows": _plain_rows, "append": _plain_append, "attend": _plain_attend}[op](st)


def _own_rows(st):
    from head_weighted_relu_b200 import indexer as I
    codes, scale = I.rotate_quantise(st["x"], st["positions"], st["table"], interleaved=st["case"]["inter"])
    return dict(codes=codes.view(torch.float8_e4m3fn), scale=scale)


def _own_append(st):
    from head_weighted_relu_b200 import indexer as I
    cache = I.KVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    q_rot = I.cache_append(cache, st["k"], st["v"], st["cu_q"], st["kv_len"], st["page_table"], table=st["table"],
                           interleaved=st["case"]["inter"], q=st["q"])
    return _cache_outputs(st, q_rot)


def _own_attend(st):
    from head_weighted_relu_b200 import indexer as I
    cache = I.KVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    selected = (st["sel_idx"], st["sel_len"]) if "sel_idx" in st else None
    out, lse = I.cache_attend(cache, st["q"], st["cu_q"], st["kv_len"], st["page_table"], max_q=st["max_q"],
                              causal=st["case"]["causal"], selected=selected, with_lse=True)
    return dict(out=out, lse=lse)


def _cache_outputs(st, q_rot):
    return dict(k=st["k_cache"].view(torch.float8_e4m3fn), v=st["v_cache"].view(torch.float8_e4m3fn),
                k_scale=st["k_scale"], v_scale=st["v_scale"], q=q_rot)


# ----------------------------------------------------------------------------------------------------- plain forms --

def _rotate(x, table, positions, inter):
    """fp32 rows [S, H, D] with their first rot dimensions rotated by their position."""
    if table is None:
        return x
    half = table.shape[1] // 2
    c, s = table[positions.long()].unsqueeze(1).split(half, dim=-1)
    y = x.clone()
    if inter:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def _plain_rows(st):
    y = _rotate(st["x"].float(), st["table"], st["positions"], st["case"]["inter"])
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return dict(codes=(y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale=scale)


def _rows_of(st):
    """Sequence, index within its sequence and position of every query row."""
    r = torch.arange(st["q"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["cu_q"], r, right=True) - 1
    i = r - st["cu_q"][b]
    return b, i, st["kv_len"][b] - (st["cu_q"][b + 1] - st["cu_q"][b]) + i


def _plain_append(st):
    case = st["case"]
    page, block = case["page"], case["block"]
    b, i, pos = _rows_of(st)
    old = (st["kv_len"] - st["cu_q"].diff()) % block          # old tokens of each sequence's first block
    first = (st["kv_len"] - st["cu_q"].diff()) - old          # position of that block's first token
    slot = st["page_table"][b, pos // page].long() * page + pos % page
    j = torch.arange(block, device="cuda")
    at = first[:, None] // page
    old_slot = st["page_table"][torch.arange(case["B"], device="cuda")[:, None], at].long() * page + first[:, None] % page + j
    keep = j < old[:, None]                                   # [B, block]: rows of old tokens in a block that grows
    for name, x in (("k", _rotate(st["k"].float(), st["table"], pos, case["inter"])), ("v", st["v"].float())):
        codes = st[name + "_cache"].view(-1, case["Hkv"], case["D"])
        scale = st[name + "_scale"].view(-1, case["Hkv"])
        blk = (slot // block)[:, None].expand(-1, case["Hkv"])
        amax = torch.zeros_like(scale).scatter_reduce_(0, blk, x.abs().amax(-1), "amax")
        fresh = torch.zeros_like(scale).scatter_reduce_(0, blk, (pos % block == 0).float()[:, None].expand_as(blk), "amax")
        need = _pow2_scale(amax)
        new = torch.where(amax > 0, need, scale.clamp(min=2.0 ** -100))
        new = torch.where(fresh > 0, need, torch.maximum(new, scale))
        rows = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").scatter_(0, slot // block, True)
        new = torch.where(rows[:, None], new, scale)
        ob, was = old_slot // block, codes[old_slot]
        again = was.view(torch.float8_e4m3fn).float() * (scale[ob] / new[ob])[..., None]
        codes[old_slot] = torch.where(keep[..., None, None], again.to(torch.float8_e4m3fn).view(torch.uint8), was)
        codes[slot] = (x / new[slot // block][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(new)
    return _cache_outputs(st, _rotate(st["q"].float(), st["table"], pos, case["inter"]).to(st["q"].dtype))


def _values(codes, scale, slot, block):
    """fp32 values of the cache's tokens `slot` (any shape): [..., Hkv, D]."""
    x = codes.view(-1, *codes.shape[2:])[slot].view(torch.float8_e4m3fn).float()
    return x.mul_(scale.view(-1, scale.shape[-1])[slot // block][..., None])


def _softmax_product(s, v):
    """Scores [..., rows, keys] (-inf where masked) and values [..., keys, D]: outputs, and the log of the sums."""
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total)), (top + total.log()).squeeze(-1)


def _plain_attend(st):
    case = st["case"]
    page, block, Hkv, D = case["page"], case["block"], case["Hkv"], case["D"]
    G, S, c = case["Hq"] // Hkv, st["q"].shape[0], 1.0 / math.sqrt(case["D"])
    b, i, pos = _rows_of(st)
    last = pos if case["causal"] else st["kv_len"][b] - 1
    if case["sel"]:
        at = st["sel_idx"]
        seen = (torch.arange(at.shape[1], device="cuda") < st["sel_len"][:, None]) & (at >= 0) & (at <= last[:, None])
        at = torch.where(seen, at, torch.zeros_like(at))
        slot = st["page_table"][b[:, None], at // page].long() * page + at % page               # [S, W]
        k = _values(st["k_cache"], st["k_scale"], slot, block).transpose(1, 2)                  # [S, Hkv, W, D]
        s = (st["q"].float().view(S, Hkv, G, D) @ k.transpose(2, 3)).mul_(c)
        del k
        s.masked_fill_(~seen[:, None, None], -math.inf)
        o, lse = _softmax_product(s, _values(st["v_cache"], st["v_scale"], slot, block).transpose(1, 2))
        return dict(out=o.reshape(S, -1, D).to(st["q"].dtype), lse=lse.reshape(S, -1))
    B, Q, L = case["B"], st["max_q"], st["page_table"].shape[1] * page
    t = torch.arange(L, device="cuda")
    slot = st["page_table"][:, t // page].clamp(min=0).long() * page + t % page                 # [B, L]
    q = torch.zeros((B, Q, Hkv, G, D), device="cuda")
    q[b, i] = st["q"].float().view(S, Hkv, G, D)
    end = torch.full((B, Q), -1, dtype=torch.int32, device="cuda")
    end[b, i] = last
    k = _values(st["k_cache"], st["k_scale"], slot, block).permute(0, 2, 3, 1)                   # [B, Hkv, D, L]
    s = (q.transpose(1, 2).reshape(B, Hkv, Q * G, D) @ k).mul_(c).view(B, Hkv, Q, G, L)
    del k
    s.masked_fill_((t > end[..., None])[:, None, :, None], -math.inf)
    o, lse = _softmax_product(s.view(B, Hkv, Q * G, L), _values(st["v_cache"], st["v_scale"], slot, block).transpose(1, 2))
    o, lse = o.view(B, Hkv, Q, G, D).transpose(1, 2)[b, i], lse.view(B, Hkv, Q, G).transpose(1, 2)[b, i]
    return dict(out=o.reshape(S, -1, D).to(st["q"].dtype), lse=lse.reshape(S, -1))


# ------------------------------------------------------------------------------------------------------------ work --

def work(case):
    act, D = 2, case["D"]
    if case["op"] == "rows":
        n = case["S"] * case["H"]
        return dict(bytes=n * D * (act + 1) + 4 * n + 4 * case["S"] * (case["rot"] + 1), flops=4 * n * D)
    q_lens, lens = _layout(case)
    S, Hq, Hkv = sum(q_lens), case["Hq"], case["Hkv"]
    if case["op"] == "append":
        blocks = sum(-(-n // case["block"]) - (n - q) // case["block"] for q, n in zip(q_lens, lens))
        moved = 2 * S * Hkv * D * (act + 1) + 2 * S * Hq * D * act + 2 * blocks * Hkv * 4 + 4 * S * case["rot"]
        return dict(bytes=moved, flops=3 * S * (Hq + Hkv) * case["rot"] + 4 * S * Hkv * D)
    if case["sel"]:
        seen = [min(n - q + i + 1, case["sel"]) for q, n in zip(q_lens, lens) for i in range(q)]
        pairs = sum(seen)
        # tokens that at least one row names: all of those named where there are few, at most the sequence
        tokens, r = 0, 0
        for q, n in zip(q_lens, lens):
            tokens += min(n, sum(seen[r:r + q]))
            r += q
        extra = 4 * pairs
    else:
        pairs = sum(q * (n - q) + q * (q + 1) // 2 if case["causal"] else q * n for q, n in zip(q_lens, lens))
        tokens, extra = sum(lens), 0
    moved = tokens * Hkv * (2 * D + 8 / case["block"]) + 2 * S * Hq * D * act + 4 * S * Hq + extra
    return dict(bytes=moved, flops=4 * pairs * Hq * D)


# ----------------------------------------------------------------------------------------------------------- exact --

def _e4m3_values():
    """The value of each of the 256 codes, from the format: sign, 4 exponent bits of bias 7, 3 of mantissa."""
    out = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.nan if c & 127 == 127 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _to_codes(y):
    """fp64 values of at most 448 in size to the nearest e4m3 value's code, ties to the even code."""
    grid = _e4m3_values()[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs()
    lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)  # differ at a tie alone
    code = torch.where(lo % 2 == 0, lo, hi)
    return torch.where(y < 0, code + 128, code).to(torch.uint8)


def _exact_rotation(x, rot, positions, inter):
    y = x.clone()
    for d in range(rot // 2):
        angle = positions.double() * 10000.0 ** (-2.0 * d / rot)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        m, n = (2 * d, 2 * d + 1) if inter else (d, d + rot // 2)
        y[:, :, m] = x[:, :, m] * c - x[:, :, n] * s
        y[:, :, n] = x[:, :, n] * c + x[:, :, m] * s
    return y


def exact(case, seed):
    st = prepare(case, seed)
    values = _e4m3_values()
    if case["op"] == "rows":
        y = _exact_rotation(st["x"].double(), case["rot"], st["positions"], case["inter"])
        top = y.abs().max(-1).values
        scale = torch.where(top > 0, top / 448, 1.0)
        return dict(codes=values[_to_codes(y / scale[..., None]).int()], scale=scale)
    q_lens, lens = _layout(case)
    page, block, D, G = case["page"], case["block"], case["D"], case["Hq"] // case["Hkv"]
    if case["op"] == "append":
        where = torch.cat([torch.arange(n - q, n, device="cuda") for q, n in zip(q_lens, lens)])
        got = {}
        for name in ("k", "v"):
            x = st[name].double()
            if name == "k":
                x = _exact_rotation(x, case["rot"], where, case["inter"])
            codes, scale = st[name + "_cache"].clone(), st[name + "_scale"].double()
            r = 0
            for s, (q, n) in enumerate(zip(q_lens, lens)):
                pos = n - q
                while pos < n:
                    end = min(n, (pos // block + 1) * block)
                    p, b, o = int(st["page_table"][s, pos // page]), pos % page // block, pos % block
                    rows, at = x[r:r + end - pos], pos % page
                    # log2 of the size, decided by comparison
                    e = torch.ceil(torch.log2(rows.abs().amax((0, 2)).clamp(min=2.0 ** -91) / 448)).clamp(min=-100)
                    new = 2.0 ** e
                    if o:
                        new = torch.maximum(new, scale[p, b])
                        was = values[codes[p, at - o:at].int()] * scale[p, b][:, None]
                        codes[p, at - o:at] = _to_codes(was / new[:, None])
                    codes[p, at:at + end - pos] = _to_codes(rows / new[:, None])
                    scale[p, b] = new
                    r, pos = r + end - pos, end
            got[name], got[name + "_scale"] = values[codes.int()], scale
        got["q"] = _exact_rotation(st["q"].double(), case["rot"], where, case["inter"])
        return got
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    r = 0
    for s, (q, n) in enumerate(zip(q_lens, lens)):
        t = torch.arange(n, device="cuda")
        p, o = st["page_table"][s, t // page].long(), t % page
        for h in range(case["Hkv"]):
            k = values[st["k_cache"][p, o, h].int()] * st["k_scale"][p, o // block, h].double()[:, None]
            v = values[st["v_cache"][p, o, h].int()] * st["v_scale"][p, o // block, h].double()[:, None]
            heads = slice(h * G, h * G + G)
            step = max(1, (1 << 28) // (G * n))
            for i in range(0, q, step):
                rows = slice(r + i, r + min(q, i + step))
                m = rows.stop - rows.start
                z = torch.einsum("rgd,td->rgt", st["q"][rows, heads].double(), k) / math.sqrt(D)
                see = t <= (n - q + torch.arange(i, i + m, device="cuda"))[:, None] if case["causal"] else t[None] < n
                if case["sel"]:
                    named = torch.zeros((m, n + 1), dtype=torch.bool, device="cuda")
                    idx = st["sel_idx"][rows].long()
                    named.scatter_(1, torch.where(idx < 0, n, idx), True)
                    see = see & named[:, :n]
                z = z.masked_fill(~see[:, None].expand_as(z), -math.inf)
                lse[rows, heads] = torch.logsumexp(z, -1)
                out[rows, heads] = torch.einsum("rgt,td->rgd", torch.softmax(z, -1), v)
        r += q
    return dict(out=out, lse=lse)
