"""Binary64 reference of the cache operators (rotated FP8 rows, append, attention),
written from their definitions in include/hwr_indexer.h, on the CPU.  Shares no
code with the CUDA path."""

import math

import numpy as np
import torch


def e4m3_values():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[c] = -v if c & 128 else v
    return out


VALUES = e4m3_values()
GRID = VALUES[:127]


def to_code(y):
    """Nearest e4m3 code of |y| <= 448, ties to even; NaN (and infinities) to 0x7F."""
    a = np.abs(y)
    bad = ~np.isfinite(y)
    a = np.where(bad, 0, a)
    mid = (GRID[1:] + GRID[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")
    hi = np.searchsorted(mid, a, side="right")
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    code = np.where(np.signbit(y), code + 128, code)
    return np.where(bad, 0x7F, code).astype(np.uint8)


def rotate(x, positions, rot, interleaved, base=10000.0):
    """x [S, H, D] float64 rotated at positions [S]; the angles from fp32 table
    entries, as a caller's table holds them."""
    y = x.copy()
    if rot == 0:
        return y
    half = rot // 2
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * inv
    c = np.cos(ang).astype(np.float32).astype(np.float64)[:, None]
    s = np.sin(ang).astype(np.float32).astype(np.float64)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def block_scale(amax):
    """Least power of two s with amax <= 448 s, at least 2^-100."""
    e = -100
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rows_of(cu_q, kv_len):
    """(sequence, position) of each row that belongs to a sequence."""
    out = []
    for b, n in enumerate(kv_len):
        for r in range(cu_q[b], cu_q[b + 1]):
            out.append((r, b, n - (cu_q[b + 1] - r)))
    return out


def append(k_codes, v_codes, k_scale, v_scale, k, v, cu_q, kv_len, table, rot, interleaved, rot_rows=None):
    """The cache after an append, as new arrays, and the rotated float64 values
    that each written code rounds: {(name, page, offset, head): row}."""
    pages, page, heads, D = k_codes.shape
    nb = k_scale.shape[1]
    block = page // nb
    rows = rows_of(cu_q, kv_len)
    pos = np.zeros(k.shape[0])
    for r, _, p in rows:
        pos[r] = max(p, 0)
    kr = rotate(k, pos, rot, interleaved)
    out = {"k": k_codes.copy(), "v": v_codes.copy()}
    scales = {"k": k_scale.astype(np.float64).copy(), "v": v_scale.astype(np.float64).copy()}
    written = {}
    groups = {}
    for r, b, p in rows:
        if p < 0 or p // page >= table.shape[1] or not 0 <= table[b, p // page] < pages:
            continue
        if rot and rot_rows is not None and p >= rot_rows:
            continue
        groups.setdefault((int(table[b, p // page]), (p % page) // block), []).append((p, r))
    for (pg, bl), members in groups.items():
        first = min(p for p, _ in members)
        o0 = first % page
        kept = range(bl * block, o0)      # earlier tokens of the block
        for name, x in (("k", kr), ("v", v)):
            for h in range(heads):
                vals = np.stack([x[r, h] for _, r in members])
                fin = np.abs(vals[np.isfinite(vals)])
                s = block_scale(fin.max() if fin.size else 0.0)
                if len(kept):
                    old = scales[name][pg, bl, h]
                    s = max(s, old, 2.0 ** -100)
                    for o in kept:
                        out[name][pg, o, h] = to_code(VALUES[out[name][pg, o, h]] * (old / s))
                scales[name][pg, bl, h] = s
                for p, r in members:
                    out[name][pg, p % page, h] = to_code(x[r, h] / s)
                    written[(name, pg, p % page, h)] = (x[r, h], s)
    return out["k"], out["v"], scales["k"], scales["v"], kr, written


def attend(k_codes, v_codes, k_scale, v_scale, q, cu_q, kv_len, table, scale, causal=True, selected=None):
    """out, lse and, for tolerances, per (row, head): the weighted size of the
    values sum_j p_j |v_j| [S, Hq, D] and the largest scale * sum_d |q_d k_d|."""
    pages, page, heads, D = k_codes.shape
    block = page // k_scale.shape[1]
    S, Hq, _ = q.shape
    G = Hq // heads
    out = np.zeros((S, Hq, D))
    size = np.zeros((S, Hq, D))
    lse = np.full((S, Hq), -np.inf)
    reach = np.zeros((S, Hq))
    owned = np.zeros(S, dtype=bool)
    for r, b, p in rows_of(cu_q, kv_len):
        owned[r] = True
        end = min(p + 1, kv_len[b]) if causal else kv_len[b]
        if selected is None:
            seen = np.arange(max(end, 0))
        else:
            e = selected[0][r, :max(0, min(int(selected[1][r]), selected[0].shape[1]))].astype(np.int64)
            seen = e[(e >= 0) & (e < end)]
        seen = seen[seen // page < table.shape[1]]
        pg = table[b, seen // page].astype(np.int64)
        ok = (pg >= 0) & (pg < pages)
        seen, pg = seen[ok], pg[ok]
        if seen.size == 0:
            continue
        o = seen % page
        for h in range(heads):
            kk = VALUES[k_codes[pg, o, h]] * k_scale[pg, o // block, h].astype(np.float64)[:, None]
            vv = VALUES[v_codes[pg, o, h]] * v_scale[pg, o // block, h].astype(np.float64)[:, None]
            qq = q[r, h * G:(h + 1) * G]
            s = scale * (qq @ kk.T)
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            l = w.sum(-1, keepdims=True)
            w = w / l
            out[r, h * G:(h + 1) * G] = w @ vv
            size[r, h * G:(h + 1) * G] = w @ np.abs(vv)
            lse[r, h * G:(h + 1) * G] = (m + np.log(l))[:, 0]
            reach[r, h * G:(h + 1) * G] = abs(scale) * (np.abs(qq) @ np.abs(kk).T).max(-1)
    return out, lse, size, reach, owned


def to_np(t):
    return t.detach().cpu().double().numpy() if t.dtype != torch.uint8 else t.detach().cpu().numpy()
