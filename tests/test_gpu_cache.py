"""The operators around the indexer on the GPU against their binary64 reference:
rotated FP8 rows, the append to the paged 8-bit cache, and attention over it,
at the sizes, layouts and masks where they can go wrong; then the whole serving
step, from projections to the attention's output."""

import numpy as np
import pytest
import torch

from tests import cache_reference as R

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _I():
    from head_weighted_relu_b200 import indexer as I
    return I


def _dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


# --------------------------------------------------------------- FP8 rows --

def _half_step(y, s):
    """Largest distance of y from the nearest e4m3 value times s, for |y| <= 448 s:
    half a step, 2^-4 of the value or, below the normal range, 2^-10 s."""
    return np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10)


@pytest.mark.parametrize("S,H,D,act,rot,inter", [
    (1, 1, 64, "bf16", 64, False), (1, 64, 128, "bf16", 64, False), (3, 5, 128, "fp16", 128, True),
    (37, 64, 128, "bf16", 48, False), (65, 4, 64, "fp16", 16, True), (130, 3, 64, "bf16", 48, False),
    (700, 7, 128, "fp16", 112, False), (257, 32, 128, "bf16", 0, False), (19, 64, 64, "bf16", 32, True),
])
def test_rotate_quantise(cuda_ok, S, H, D, act, rot, inter):
    I = _I()
    g = torch.Generator().manual_seed(S * 1000 + H)
    wide = torch.randn(S, H * D + 24, generator=g).to(ACT[act])
    wide[0, : D] = 0                                   # a zero row
    wide = wide.cuda()
    x = wide[:, 8: 8 + H * D].view(S, H, D) if S > 0 else wide
    x = wide.as_strided((S, H, D), (H * D + 24, D, 1), 8)   # a slice of a wider projection
    pos = torch.randint(0, 5000, (S,), generator=g, dtype=torch.int32)
    table = I.rope_table(5000, rot) if rot else None
    codes, scale = I.rotate_quantise(x, pos.cuda(), table, interleaved=inter)
    y = R.rotate(R.to_np(x), pos.numpy(), rot, inter)
    amax = np.abs(y).max(-1)
    want = np.where(amax > 0, amax / 448, 1.0)
    sc = R.to_np(scale)
    # a rotated value: two products and a sum in FP32, each within 2^-24 of at
    # most |a| + |b| <= 2 amax(x); and the division
    size = np.abs(R.to_np(x)).max(-1)
    slip = 6 * 2.0 ** -24 * size
    assert (np.abs(sc - want) <= slip / 448 + 2.0 ** -23 * want).all()
    got = R.VALUES[codes.cpu().numpy()] * sc[..., None]
    assert (np.abs(got - y) <= _half_step(y, sc[..., None]) * (1 + 2.0 ** -20) + 2 * slip[..., None]).all()
    # without a rotation, the plain formula in FP32 bit for bit (on the CPU: the
    # GPU's division of a tensor by a number multiplies by its reciprocal instead)
    if rot == 0:
        xf = x.float().cpu()
        s2 = xf.abs().amax(-1)
        s2 = torch.where(s2 > 0, s2 / 448, torch.ones_like(s2))
        assert torch.equal(scale.cpu(), s2)
        assert torch.equal(codes.cpu(), (xf / s2[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("act,D,rot,inter", [("bf16", 128, 128, False), ("bf16", 128, 64, False), ("fp16", 64, 64, True),
                                             ("fp16", 128, 48, False), ("bf16", 64, 16, True)])
def test_rotation_rounds_each_product_on_its_own(cuda_ok, act, D, rot, inter):
    """Rotated q and FP8 rows bit for bit as the formula in FP32, no product fused
    with the sum (which the CPU's separate operations do not do either)."""
    I = _I()
    S, H = 300, 5
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(S, H, D, generator=g).to(ACT[act])
    rt = I.rope_table(S, rot)
    c, s = rt.cpu()[:, None].split(rot // 2, dim=-1)
    xf = x.float()
    y = xf.clone()
    a, b = (xf[..., 0:rot:2], xf[..., 1:rot:2]) if inter else (xf[..., :rot // 2], xf[..., rot // 2:rot])
    ra, rb = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    cache = I.allocate_cache(1, 512, 1, D, 16)
    k = torch.zeros(S, 1, D, dtype=ACT[act], device="cuda")
    cu, kv = _dev(np.array([0, S], dtype=np.int32)), _dev(np.array([S], dtype=np.int32))
    q = I.cache_append(cache, k, k, cu, kv, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), table=rt,
                       interleaved=inter, q=x.cuda())
    assert torch.equal(q.cpu(), y.to(ACT[act]))
    codes, scale = I.rotate_quantise(x.cuda(), None, rt, interleaved=inter)
    want = y.abs().amax(-1) / 448
    assert torch.equal(scale.cpu(), want)
    assert torch.equal(codes.cpu(), (y / want[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("act", ["bf16", "fp16"])
def test_rotate_quantise_over_the_whole_range(cuda_ok, act):
    """Rows of every magnitude that the type holds, subnormal scales among them, and
    values from the row's largest down to nothing: scale and codes as IEEE division
    gives them."""
    I = _I()
    g = torch.Generator().manual_seed(8)
    lo, hi = (-133, 127) if act == "bf16" else (-24, 15)
    mag = 2.0 ** torch.arange(lo, hi, dtype=torch.float64)
    rows = torch.rand(len(mag), 3, 128, generator=g, dtype=torch.float64) * 2 - 1
    rows *= 2.0 ** -(torch.arange(128) % 24)                      # down to below the least code
    rows[:, 1, 5] = 1.9921875                                     # the largest fraction of 8 bits
    x = (rows * mag[:, None, None]).to(ACT[act])
    codes, scale = I.rotate_quantise(x.cuda())
    xf = x.float()
    amax = xf.abs().amax(-1)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert torch.equal(scale.cpu(), want)
    z = (xf / want[..., None]).clamp(-448, 448)                   # (a subnormal scale is coarse: past 448 by its rounding)
    assert torch.equal(codes.cpu(), z.to(torch.float8_e4m3fn).view(torch.uint8))


def test_append_of_many_rows(cuda_ok):
    """Large enough for q to go through a kernel of its own: the same rows as in
    pieces, and the cache with them."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(5)
    S, Hq, heads, D = 2200, 64, 2, 128
    q, k, v = (torch.randn(S, n, D, generator=g, device="cuda").bfloat16() for n in (Hq, heads, heads))
    rt = I.rope_table(S, 128)
    table = torch.arange(18, dtype=torch.int32, device="cuda").flip(0).view(1, 18)
    one, two = (I.allocate_cache(18, 128, heads, D, 128) for _ in range(2))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    whole = I.cache_append(one, k, v, ints(0, S), ints(S), table, table=rt, q=q)
    parts = [I.cache_append(two, k[a:b], v[a:b], ints(0, b - a), ints(b), table, table=rt, q=q[a:b])
             for a, b in ((0, 128), (128, 1024), (1024, 2048), (2048, S))]
    assert torch.equal(whole, torch.cat(parts))
    used = [i for i in range(18)][::-1]
    for pg, n in ((p, min(128, S - 128 * i)) for i, p in enumerate(used)):
        assert torch.equal(one.k[pg, :n], two.k[pg, :n]) and torch.equal(one.v[pg, :n], two.v[pg, :n])
    assert torch.equal(one.k_scale, two.k_scale) and torch.equal(one.v_scale, two.v_scale)


def test_rotate_quantise_bad_rows(cuda_ok):
    I = _I()
    x = torch.randn(6, 2, 64, device="cuda").bfloat16()
    x[4, 1, 3] = float("nan")
    x[5, 0, 9] = float("inf")
    table = I.rope_table(100, 64)
    pos = torch.tensor([0, 99, 100, -1, 5, 5], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scale = I.rotate_quantise(x, pos, table, status=status)
    c = codes.cpu().numpy() & 0x7F
    assert status.item() == I.STATUS_TOKEN
    assert (c[2:4] == 0x7F).all() and (scale[2:4] == 1).all()
    assert (c[4, 1] == 0x7F).all() and (c[5, 0] == 0x7F).all()
    assert (c[:2] != 0x7F).all() and (c[4, 0] != 0x7F).all() and (c[5, 1] != 0x7F).all()
    assert I.indexer_read_status(status) == I.STATUS_TOKEN and status.item() == 0
    # written into the rows of a larger key array
    keys = torch.zeros(10, 64, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(10, device="cuda")
    I.rotate_quantise(x[:2, :1], pos[:2], table, out=(keys[3:5], ks[3:5]))
    assert torch.equal(keys[3:5], codes[:2, 0]) and torch.equal(ks[3:5], scale[:2, 0])
    assert keys[:3].eq(0).all() and keys[5:].eq(0).all()


# ------------------------------------------------------------------ cache --

def _random_cache(rng, pages, page, heads, D, block, hnd=False, garbage=True):
    """Cache tensors (pages uninitialised in spirit: NaN codes and NaN scales)."""
    I = _I()
    shape = (pages, heads, page, D) if hnd else (pages, page, heads, D)
    k = torch.full(shape, 0x7F if garbage else 0, dtype=torch.uint8, device="cuda")
    v = torch.full(shape, 0xFF if garbage else 0, dtype=torch.uint8, device="cuda")
    if hnd:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks = torch.full((pages, page // block, heads), float("nan"), device="cuda")
    return I.KVCache(k, v, ks, ks.clone())


def _tables(rng, kv_len, page, extra_pages=2, width=None):
    need = [-(-max(n, 0) // page) for n in kv_len]
    order = rng.permutation(sum(need) + extra_pages)
    w = width or max(max(need), 1)
    table = np.full((len(kv_len), w), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + extra_pages


def _snapshot(cache):
    return [x.detach().cpu().numpy().copy() for x in cache]


APPENDS = [
    # q_lens, kv_len (with them), Hq, heads, D, page, block, act, rot, inter, hnd
    ([1], [1], 4, 1, 128, 16, 16, "bf16", 128, False, False),
    ([1, 1, 1], [17, 64, 100], 8, 2, 128, 64, 16, "bf16", 64, False, False),
    ([5, 0, 33, 1], [5, 9, 130, 48], 6, 3, 64, 48, 16, "fp16", 32, True, True),
    ([70, 3], [200, 3], 4, 4, 64, 96, 32, "fp16", 64, False, False),
    ([129, 1], [129, 65], 2, 2, 128, 128, 64, "bf16", 112, False, True),
    ([300], [333], 8, 8, 128, 128, 128, "bf16", 128, True, False),
    ([7, 2, 9], [40, 2, 9], 5, 5, 64, 3, 1, "bf16", 48, False, False),
    ([20, 30], [31, 77], 4, 1, 128, 24, 8, "fp16", 0, False, False),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"q{c[0]}-b{c[6]}-{c[7]}")
def test_cache_append(cuda_ok, case):
    I = _I()
    q_lens, kv_len, Hq, heads, D, page, block, act, rot, inter, hnd = case
    rng = np.random.default_rng(sum(kv_len))
    S = sum(q_lens) + 3                                    # three rows behind the last sequence
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    table, pages = _tables(rng, kv_len, page)
    cache = _random_cache(rng, pages, page, heads, D, block, hnd)
    rt = I.rope_table(max(kv_len), rot) if rot else None
    # earlier tokens, appended first: their block scales are what the new ones meet
    past = [n - q for n, q in zip(kv_len, q_lens)]
    for step, (ql, kl) in enumerate([(past, past), (q_lens, kv_len)]):
        n = sum(ql) + 3
        gain = np.exp(rng.normal(size=(n, 1, 1)) + 2 * step)
        k = _dev(rng.normal(size=(n, heads, D)) * gain, ACT[act])
        v = _dev(rng.normal(size=(n, heads, D)), ACT[act])
        q = _dev(rng.normal(size=(n, Hq, D)), ACT[act])
        q_out = torch.full_like(q, 7.0)
        c = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        before = _snapshot(cache)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (k, v, _dev(c), _dev(np.array(kl, dtype=np.int32)), _dev(table))
        got_q = I.cache_append(cache, *args, table=rt, interleaved=inter, q=q, q_out=q_out, status=status)
        after = _snapshot(cache)
        assert status.item() == 0 and got_q is q_out
        wk, wv, wks, wvs, kr, written = R.append(*before, R.to_np(k), R.to_np(v), c, kl, table, rot, inter)
        for name, got, want, gs, ws in (("k", after[0], wk, after[2], wks), ("v", after[1], wv, after[3], wvs)):
            np.testing.assert_array_equal(gs, ws.astype(np.float32))        # powers of two, exactly
            mask = np.zeros(got.shape[:3], dtype=bool)
            for (nm, pg, o, h), (y, s) in written.items():
                if nm != name:
                    continue
                mask[pg, o, h] = True
                slip = 6 * 2.0 ** -24 * np.abs(R.to_np(k)).max() if name == "k" and rot else 0.0
                err = np.abs(R.VALUES[got[pg, o, h]] * s - y)
                assert (err <= _half_step(y, s) * (1 + 2.0 ** -20) + slip).all()
            np.testing.assert_array_equal(got[~mask], want[~mask])          # all else bit for bit
        # q: rotated rows, one rounding to their type; rows of no sequence untouched
        own = sum(ql)
        pos = np.array([p for _, _, p in R.rows_of(c, kl)] + [0] * 3)
        want_q = R.rotate(R.to_np(q), pos, rot, inter)
        tol = torch.finfo(ACT[act]).eps / 2 * np.abs(want_q) + 6 * 2.0 ** -24 * np.abs(R.to_np(q)).max() + 2.0 ** -25
        assert (np.abs(R.to_np(q_out) - want_q)[:own] <= tol[:own]).all()
        assert (q_out[own:] == 7.0).all()
        # the same append again changes nothing
        I.cache_append(cache, *args, table=rt, interleaved=inter)
        for a, b in zip(after, _snapshot(cache)):
            np.testing.assert_array_equal(a, b)


def test_append_split_gives_the_same_scales(cuda_ok):
    """One append of 50 tokens, and the same tokens one by one: equal scales, and
    values within the roundings of a growing block."""
    I = _I()
    rng = np.random.default_rng(3)
    k = _dev(rng.normal(size=(50, 2, 64)) * np.exp(rng.normal(size=(50, 1, 1))), torch.bfloat16)
    v = _dev(rng.normal(size=(50, 2, 64)) * np.exp(rng.normal(size=(50, 1, 1))), torch.bfloat16)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    rt = I.rope_table(64, 64)
    one, many = (_random_cache(rng, 3, 32, 2, 64, 16) for _ in range(2))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    I.cache_append(one, k, v, ints(0, 50), ints(50), table, table=rt)
    for i in range(50):
        I.cache_append(many, k[i:i + 1], v[i:i + 1], ints(0, 1), ints(i + 1), table, table=rt)
    # 50 tokens fill pages 2 and half of page 0 (blocks 0, 1 of each, the last one in part)
    for a, b in ((one.k_scale, many.k_scale), (one.v_scale, many.v_scale)):
        a, b = a.cpu().numpy(), b.cpu().numpy()
        np.testing.assert_array_equal(a[[2, 0]][:, :2].ravel()[:8], b[[2, 0]][:, :2].ravel()[:8])
    for p in range(50):
        pg, o = [(2, p), (0, p - 32)][p >= 32]
        s = one.k_scale[pg, o // 16].cpu().numpy()[:, None]
        a = R.VALUES[one.k[pg, o].cpu().numpy()] * s
        b = R.VALUES[many.k[pg, o].cpu().numpy()] * s
        # each was rounded once to its own scale and, in `many`, at most 15 more
        # times where a code fell below the normal range (2^-10 s each)
        assert (np.abs(a - b) <= 2 * np.maximum(np.abs(a) * 2.0 ** -4, 2.0 ** -10 * s) + 15 * 2.0 ** -10 * s).all()


def test_append_scale_edges(cuda_ok):
    """Block maxima at the border of a power of two, zero and tiny blocks, NaN and
    infinite values."""
    I = _I()
    tops = [448.0, 449.0, 450.0, 447.0, 896.0, 898.0, 1.75, 1.7578125, 0.0, 2.0 ** -95, 2.0 ** -126, 3.0e38]
    n = len(tops)
    k = torch.zeros(n, 1, 64, device="cuda")
    for i, t in enumerate(tops):
        k[i, 0, i % 64] = t
    k = k.bfloat16()
    v = -k
    v[0, 0, 5] = float("nan")
    v[1, 0, 6] = float("-inf")
    cache = _random_cache(None, 1, n, 1, 64, 1)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    I.cache_append(cache, k, v, ints(0, n), ints(n), ints(0).view(1, 1))
    want = np.array([R.block_scale(float(x)) for x in k.float().amax((1, 2)).cpu()])
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy()[0, :, 0], want.astype(np.float32))
    np.testing.assert_array_equal(cache.v_scale.cpu().numpy()[0, :, 0], want.astype(np.float32))
    kv = cache.v.cpu().numpy()[0, :, 0]
    assert kv[0, 5] & 0x7F == 0x7F and kv[1, 6] & 0x7F == 0x7F
    assert (kv & 0x7F == 0x7F).sum() == 2
    np.testing.assert_array_equal(cache.k.cpu().numpy()[0, :, 0], R.to_code(R.to_np(k)[:, 0] / want[:, None]))


def test_append_skips_bad_pages_and_positions(cuda_ok):
    I = _I()
    rng = np.random.default_rng(9)
    cache = _random_cache(rng, 3, 16, 1, 64, 8)
    before = _snapshot(cache)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # sequence 0: pages -1 and 3 (outside); 1: a length below its rows (positions -2, -1, 0);
    # 2: positions beyond the rotation table (60 rows) and beyond the page table
    table = ints([[-1, 3, 0, -1], [1, -1, -1, -1], [-1, -1, -1, 2]])
    cu, kv = ints([0, 40, 43, 53]), ints([40, 1, 66])
    k = _dev(rng.normal(size=(53, 1, 64)), torch.bfloat16)
    q = _dev(rng.normal(size=(53, 2, 64)), torch.bfloat16)
    q_out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    I.cache_append(cache, k, k, cu, kv, table, table=I.rope_table(60, 64), q=q, q_out=q_out, status=status)
    after = _snapshot(cache)
    assert status.item() == I.STATUS_TOKEN
    wk, wv, wks, wvs, _, written = R.append(*before, R.to_np(k), R.to_np(k), cu.tolist(), kv.tolist(),
                                            table.cpu().numpy(), 64, False, rot_rows=60)
    changed = {(0, o) for o in range(8)} | {(1, 0)} | {(2, o) for o in range(8, 12)}
    assert {(pg, o) for _, pg, o, _ in written} == changed
    for pg in range(3):
        for o in range(16):
            if (pg, o) not in changed:
                assert (after[0][pg, o] == before[0][pg, o]).all()
    np.testing.assert_array_equal(after[2], wks.astype(np.float32))
    assert (q_out[40:42] == 7.0).all() and (q_out[42] != 7.0).any() and (q_out[47:] == 7.0).all()


# -------------------------------------------------------------- attention --

def _filled(rng, kv_len, heads, D, page, block, hnd=False, spread=1.0, width=None):
    """A cache with the sequences' tokens in it and NaN everywhere else."""
    table, pages = _tables(rng, kv_len, page, width=width)
    cache = _random_cache(rng, pages, page, heads, D, block, hnd)
    for b, n in enumerate(kv_len):
        for p0 in range(0, n, block):
            pg, o = table[b, p0 // page], p0 % page
            m = min(block, n - p0)
            for codes, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                codes[pg, o:o + m] = _dev(R.to_code(np.clip(rng.normal(size=(m, heads, D)) * 60, -448, 448)))
                sc[pg, o // block] = _dev((2.0 ** np.round(rng.normal(size=heads) * spread - 6)).astype(np.float32))
    return cache, table


def _check_attend(cache, q, cu, kv_len, table, scale, causal, selected, out, lse, act):
    """Tolerances, by arithmetic: a score is off by the FP32 accumulation of its D
    products, at most 2^-19 of their sizes' sum in all (each addition within 2^-22),
    and by 2^-23 of itself from the two factors; a weight by that, by the exponential
    (2^-21) and by FP16 (2^-12, or 2^-31 of the largest); the output's type rounds once."""
    want, wl, size, reach, owned = R.attend(*_snapshot(cache), R.to_np(q), cu, kv_len, table, scale, causal,
                                            None if selected is None else [x.cpu().numpy() for x in selected])
    got, gl = R.to_np(out), R.to_np(lse)
    ds = 2.0 ** -18 * reach
    rel = np.expm1(2 * ds) + 2.0 ** -20 + 2.0 ** -12
    tiny = 2.0 ** -30 * np.nanmax(np.abs(size)) * max(kv_len)
    tol = torch.finfo(ACT[act]).eps / 2 * (np.abs(want) + rel[..., None] * size) + rel[..., None] * size + tiny + 2.0 ** -25
    bad = owned[:, None, None] & ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5], bad.sum())
    empty = owned[:, None] & np.isneginf(wl)
    assert (got[empty] == 0).all() and np.isneginf(gl[empty]).all()
    fin = owned[:, None] & np.isfinite(wl)
    assert (np.abs(gl - wl)[fin] <= (ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(fin, wl, 0)))[fin]).all()
    return owned


ATTENDS = [
    # q_lens, kv_len, Hq, heads, D, page, block, act, causal, hnd
    ([1], [1], 8, 1, 128, 16, 16, "bf16", True, False),
    ([1], [333], 64, 8, 128, 64, 16, "bf16", True, False),
    ([1, 1, 1], [63, 64, 65], 16, 8, 64, 16, 16, "fp16", True, True),
    ([1], [20000], 8, 1, 128, 64, 64, "bf16", True, False),
    ([3, 0, 1, 5], [700, 4, 0, 129], 12, 4, 128, 96, 32, "bf16", True, False),
    ([2, 7], [1, 900], 20, 4, 64, 24, 8, "fp16", True, False),      # more rows than tokens: some see nothing
    ([40], [300], 16, 2, 128, 128, 128, "bf16", True, False),
    ([131, 17], [131, 500], 8, 8, 64, 3, 1, "bf16", True, True),
    ([5, 9], [257, 40], 128, 1, 128, 64, 16, "fp16", True, False),
    ([4, 3], [130, 77], 24, 2, 64, 32, 16, "bf16", False, False),
    ([90], [100], 33, 1, 128, 64, 64, "bf16", False, True),
    ([260], [700], 16, 4, 128, 64, 64, "fp16", True, False),
    ([1] * 40, list(range(1, 401, 10)), 64, 8, 128, 16, 16, "bf16", True, False),
    ([1, 3], [5000, 3001], 64, 1, 128, 64, 32, "bf16", True, False),
    ([40, 1], [2500, 1700], 16, 2, 64, 24, 8, "fp16", True, False),     # a scale every 8 tokens, many tiles
    ([150], [2900], 6, 2, 128, 48, 4, "bf16", True, False),
    ([70], [3100], 8, 2, 128, 128, 64, "fp16", True, True),
    ([1], [1], 64, 1, 64, 16, 16, "bf16", True, False),
    ([5] * 20, list(range(5, 605, 30)), 64, 64, 64, 16, 16, "bf16", True, False),     # a CTA for each (tile, head)
]


STREAM, TILE = 1, 2   # the kernels, as the binding numbers them


@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: f"q{str(c[0])[:12]}-H{c[2]}.{c[3]}-D{c[4]}-{c[7]}-{'c' if c[8] else 'n'}")
def test_cache_attend(cuda_ok, case, kernel):
    I = _I()
    q_lens, kv_len, Hq, heads, D, page, block, act, causal, hnd = case
    rng = np.random.default_rng(len(q_lens) * 1000 + Hq + D)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    S = int(cu[-1]) + 2
    cache, table = _filled(rng, kv_len, heads, D, page, block, hnd)
    wide = _dev(rng.normal(size=(S, Hq * D + 16)) * np.exp(rng.normal(size=(S, 1))), ACT[act])
    q = wide.as_strided((S, Hq, D), (Hq * D + 16, D, 1), 16)
    out = torch.full((S, Hq, D), 7.0, dtype=ACT[act], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (cache, q, _dev(cu), _dev(np.array(kv_len, dtype=np.int32)), _dev(table))
    kw = dict(causal=causal, with_lse=True, max_q=max(q_lens), kernel=kernel)
    got, lse = I.cache_attend(*args, out=out, status=status, **kw)
    assert status.item() == 0
    owned = _check_attend(cache, q, cu, kv_len, table, D ** -0.5, causal, None, got, lse, act)
    assert (out[int(cu[-1]):] == 7.0).all() and owned.sum() == cu[-1]
    again, lse2 = I.cache_attend(*args, **kw)
    n = int(cu[-1])
    assert torch.equal(got[:n], again[:n]) and torch.equal(lse[:n], lse2[:n])      # the same sums in the same order


SELECTED = [
    # q_lens, kv_len, Hq, heads, D, page, block, act, width
    ([1], [50], 8, 1, 128, 16, 16, "bf16", 64),
    ([1, 1, 1], [3000, 64, 5], 64, 8, 128, 64, 16, "bf16", 2048),
    ([30, 5], [700, 60], 16, 2, 64, 96, 32, "fp16", 130),
    ([7], [400], 64, 1, 128, 64, 64, "bf16", 300),
    ([3, 4], [200, 100], 24, 1, 64, 3, 1, "fp16", 65),
    ([200], [900], 128, 1, 128, 64, 16, "bf16", 257),
]


@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("case", SELECTED, ids=lambda c: f"q{c[0]}-H{c[2]}.{c[3]}-D{c[4]}-W{c[8]}")
def test_cache_attend_selected(cuda_ok, case, kernel):
    I = _I()
    q_lens, kv_len, Hq, heads, D, page, block, act, W = case
    rng = np.random.default_rng(W)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    S = int(cu[-1])
    cache, table = _filled(rng, kv_len, heads, D, page, block)
    q = _dev(rng.normal(size=(S, Hq, D)) * 2, ACT[act])
    idx = np.full((S, W), -1, dtype=np.int32)
    ln = np.zeros(S, dtype=np.int32)
    for r, b, p in R.rows_of(cu, kv_len):
        n = min(W, p + 1)
        n = [n, 0, n, max(n - 3, 0)][r % 4] if S > 3 else n         # also rows with nothing selected
        row = np.sort(rng.choice(p + 1, size=n, replace=False))
        if r % 4 == 2 and n > 4:                                    # out of order, twice, unseen, negative
            row = row[::-1].copy()
            row[1], row[2], row[3] = row[0], p + 1, -5
        idx[r, :n] = row
        ln[r] = n
    sel = (_dev(idx), _dev(ln))
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv_len, dtype=np.int32)), _dev(table),
                              scale=0.11, selected=sel, with_lse=True, kernel=kernel)
    _check_attend(cache, q, cu, kv_len, table, 0.11, True, sel, out, lse, act)


@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_attend_extreme_scores_and_scales(cuda_ok, kernel):
    """Scores of hundreds, value scales that differ by 2^60 within a sequence, and
    queries near the ends of their type's range."""
    I = _I()
    rng = np.random.default_rng(4)
    cache, table = _filled(rng, [500], 2, 128, 64, 16, spread=3.0)
    cache.v_scale[torch.from_numpy(table[0, :3].astype(np.int64)).cuda()] *= 2.0 ** -60
    q = _dev(rng.normal(size=(4, 8, 128)) * np.array([1e-30, 1e-3, 30.0, 300.0])[:, None, None], torch.bfloat16)
    cu, kv = np.array([0, 4], dtype=np.int32), [500]
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), with_lse=True, kernel=kernel)
    _check_attend(cache, q, cu, kv, table, 128 ** -0.5, True, None, out, lse, "bf16")


@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_attend_references_that_keep_rising(cuda_ok, kernel):
    """Keys sorted so that later ones score higher by hundreds, in steps of every
    size: the running references rise again and again, within a tile too."""
    I = _I()
    rng = np.random.default_rng(14)
    kv, D = [900], 128
    cache, table = _filled(rng, kv, 1, D, 64, 16)
    q = _dev(np.ones((3, 40, D)) * np.linspace(-1, 1, 40)[None, :, None], torch.bfloat16)
    for p in range(900):   # every dimension alike: the score is their value
        pg, o = table[0, p // 64], p % 64
        v = 448.0 * (p / 900) ** 2
        cache.k[pg, o, 0] = int(R.to_code(np.array(v)))
        cache.k_scale[pg, o // 16, 0] = 2.0 ** -5
    cu = np.array([0, 3], dtype=np.int32)
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), with_lse=True, scale=0.1,
                              kernel=kernel)
    _check_attend(cache, q, cu, kv, table, 0.1, True, None, out, lse, "bf16")
    # the other sign of the scale turns the scores round
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), with_lse=True, scale=-0.1,
                              kernel=kernel)
    _check_attend(cache, q, cu, kv, table, -0.1, True, None, out, lse, "bf16")
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), with_lse=True, scale=0.0,
                              kernel=kernel)
    _check_attend(cache, q, cu, kv, table, 0.0, True, None, out, lse, "bf16")


@pytest.mark.parametrize("G,kernel", [(4, STREAM), (40, STREAM), (4, TILE), (40, TILE)])
def test_attend_nan_reaches_only_rows_that_see_it(cuda_ok, G, kernel):
    """A NaN among the newest token's keys or values, or in one query: the rows
    before it stay as they are without it."""
    I = _I()
    rng = np.random.default_rng(5)
    cache, table = _filled(rng, [70], 2, 64, 32, 16)
    cu, kv = np.array([0, 4], dtype=np.int32), [70]
    q = _dev(rng.normal(size=(4, 2 * G, 64)), torch.float16)
    args = (_dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table))
    clean = I.cache_attend(cache, q, *args, kernel=kernel)
    pg, o = table[0, 69 // 32], 69 % 32
    cache.v[pg, o, 1, 7] = 0x7F
    got = I.cache_attend(cache, q, *args, kernel=kernel)
    assert torch.equal(got[:3], clean[:3]) and torch.equal(got[3, :G], clean[3, :G])
    assert got[3, G:, 7].isnan().all() and torch.equal(got[3, G:, :7], clean[3, G:, :7])
    cache.v[pg, o, 1, 7] = 0
    cache.k[pg, o, 0, 3] = 0xFF
    got = I.cache_attend(cache, q, *args, kernel=kernel)
    assert torch.equal(got[:3], I.cache_attend(cache, q[:3].contiguous(), _dev(np.array([0, 3], dtype=np.int32)),
                                               _dev(np.array([69], dtype=np.int32)), args[2],
                                               kernel=kernel))
    assert got[3, :G].isnan().all() and not got[3, G:].isnan().any()
    cache.k[pg, o, 0, 3] = 0
    q2 = q.clone()
    q2[1, 0, 0] = float("nan")
    got = I.cache_attend(cache, q2, *args, kernel=kernel)
    assert got[1, 0].isnan().all() and not got[1, 1:].isnan().any() and not got[[0, 2, 3]].isnan().any()


@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_attend_passes_over_bad_pages(cuda_ok, kernel):
    I = _I()
    rng = np.random.default_rng(6)
    cache, table = _filled(rng, [100, 50, 64], 2, 64, 16, 16)
    table[0, 2], table[0, 4] = -1, cache.k.shape[0]         # holes
    table[1, :4] = 1 << 30                                  # nothing left
    kv = [100, 50, 64 + 40]                                 # longer than its page table
    kv_dev = _dev(np.array(kv, dtype=np.int32))
    t2 = np.ascontiguousarray(table[:, :7])
    cu = np.array([0, 2, 3, 4], dtype=np.int32)
    q = _dev(rng.normal(size=(4, 4, 64)), torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = I.cache_attend(cache, q, _dev(cu), kv_dev, _dev(t2), with_lse=True, status=status, kernel=kernel)
    assert status.item() == I.STATUS_TOKEN
    _check_attend(cache, q, cu, kv, t2, 64 ** -0.5, True, None, out, lse, "bf16")
    assert (out[2] == 0).all()


@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_attend_calls_at_once_and_rows_on_their_own(cuda_ok, kernel):
    """Two calls side by side on two streams, with a workspace each; and a row's
    result in a batch is that of the row alone where its keys are divided alike."""
    I = _I()
    rng = np.random.default_rng(21)
    kv = [4000, 250, 3500, 1]
    cache, table = _filled(rng, kv, 1, 128, 64, 16)
    cu, n, tb = _dev(np.arange(5, dtype=np.int32)), _dev(np.array(kv, dtype=np.int32)), _dev(table)
    qs = [_dev(rng.normal(size=(4, 24, 128)), torch.bfloat16) for _ in range(2)]
    want = [I.cache_attend(cache, q, cu, n, tb, kernel=kernel) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in qs]
    for _ in range(20):
        for i, (q, s) in enumerate(zip(qs, streams)):
            got[i].append(I.cache_attend(cache, q, cu, n, tb, kernel=kernel, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    # other queries in the batch change nothing of a row
    mixed = qs[0].clone()
    mixed[[0, 2]] = qs[1][[0, 2]] * 50
    out = I.cache_attend(cache, mixed, cu, n, tb, kernel=kernel)
    assert torch.equal(out[[1, 3]], want[0][[1, 3]])


def test_pages_beyond_32_bits(cuda_ok):
    """Pages 128 MB apart, most of them past 4 GB: the same cache, append and
    attention as with the pages side by side."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(3)
    pages, page, heads, D, n, gap = 48, 64, 2, 128, 48 * 64 - 5, 1 << 27
    far = [torch.empty(pages * gap, dtype=torch.uint8, device="cuda").as_strided((pages, page, heads, D),
                                                                                 (gap, heads * D, D, 1)) for _ in range(2)]
    near = I.allocate_cache(pages, page, heads, D, 16)
    wide = I.KVCache(*far, torch.empty_like(near.k_scale), torch.empty_like(near.v_scale))
    table = torch.randperm(pages, generator=g, device="cuda").int().view(1, pages)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randn(n, heads, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    rt = I.rope_table(n, 128)
    for c in (near, wide):
        I.cache_append(c, k[:-1], v[:-1], ints(0, n - 1), ints(n - 1), table, table=rt)
        I.cache_append(c, k[-1:], v[-1:], ints(0, 1), ints(n), table, table=rt)
    used = (torch.arange(pages * page, device="cuda") < n).view(pages, page)
    order = table[0].long()
    for a, b in ((near.k, wide.k), (near.v, wide.v)):
        assert torch.equal(a[order][used], b[order][used])
    q = torch.randn(3, 24 * heads, D, generator=g, device="cuda").bfloat16()
    sel = (torch.arange(0, n - 3, 7, device="cuda").int().repeat(3, 1), ints(300, 100, 437))
    for kw in (dict(kernel=STREAM), dict(kernel=TILE), dict(selected=sel, kernel=STREAM), dict(selected=sel, kernel=TILE)):
        one, two = (I.cache_attend(c, q, ints(0, 3), ints(n), table, **kw) for c in (near, wide))
        assert torch.equal(one, two) and one.isfinite().all()


def test_attend_in_large_prefill(cuda_ok):
    """More tiles than CTAs share: against the same rows in pieces."""
    I = _I()
    rng = np.random.default_rng(22)
    n, Hq, heads, D = 1500, 32, 32, 64
    cache, table = _filled(rng, [n], heads, D, 64, 64)
    q = _dev(rng.normal(size=(n, Hq, D)), torch.bfloat16)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    whole = I.cache_attend(cache, q, ints(0, n), ints(n), _dev(table), kernel=TILE)
    for a in (0, 700, 1400):
        part = I.cache_attend(cache, q[a:a + 100].contiguous(), ints(0, 100), ints(a + 100), _dev(table), kernel=STREAM)
        x, y = whole[a:a + 100].float(), part.float()
        # both within the tolerance of their own: a rounding of the output's type, of
        # FP16 weights, and of FP32 scores, each of values no larger than the row's largest
        assert (x - y).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -10) * y.abs().max()


def test_attend_shares_pages_between_sequences(cuda_ok):
    """Two sequences with a common prefix in the same pages."""
    I = _I()
    rng = np.random.default_rng(7)
    cache, table = _filled(rng, [64, 48], 1, 128, 16, 16)
    table[1, :2] = table[0, :2]
    cu, kv = np.array([0, 1, 2], dtype=np.int32), [64, 48]
    q = _dev(rng.normal(size=(2, 16, 128)), torch.bfloat16)
    out, lse = I.cache_attend(cache, q, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), with_lse=True)
    _check_attend(cache, q, cu, kv, table, 128 ** -0.5, True, None, out, lse, "bf16")


# ---------------------------------------------------------- streams, graphs --

@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_attend_on_another_stream_and_in_graphs(cuda_ok, kernel):
    """A side stream, and two captured graphs that share one workspace, replayed
    with new lengths and pages in the same buffers."""
    I = _I()
    rng = np.random.default_rng(8)
    cache, table = _filled(rng, [900, 300], 2, 128, 64, 16, width=20)
    cu = _dev(np.array([0, 1, 2], dtype=np.int32))
    kv = _dev(np.array([900, 300], dtype=np.int32))
    tb = _dev(table)
    q = _dev(rng.normal(size=(2, 16, 128)), torch.bfloat16)
    want = I.cache_attend(cache, q, cu, kv, tb, kernel=kernel)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = I.cache_attend(cache, q, cu, kv, tb, stream=side, kernel=kernel)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(I.cache_attend_workspace_bytes(cache, q, cu, kv, tb, kernel=kernel), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for _ in range(2):
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            I.cache_attend(cache, q, cu, kv, tb, out=out, workspace=ws, kernel=kernel)
        outs.append(out)
        graphs.append(g)
    for lens in ([900, 300], [850, 299], [1, 64]):
        kv.copy_(_dev(np.array(lens, dtype=np.int32)))
        want = I.cache_attend(cache, q, cu, kv, tb, kernel=kernel)
        ws.fill_(0xFF)
        for g, out in zip(graphs, outs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_append_in_a_graph(cuda_ok):
    """A captured decode step appends at the lengths that its buffers hold when it
    is replayed."""
    I = _I()
    rng = np.random.default_rng(11)
    table = _dev(np.array([[0, 2], [1, 3]], dtype=np.int32))
    rt = I.rope_table(64, 64)
    one, two = (_random_cache(rng, 4, 32, 2, 64, 16) for _ in range(2))
    k, v = (torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu, kv = _dev(np.array([0, 1, 2], dtype=np.int32)), _dev(np.array([1, 1], dtype=np.int32))
    for t in (k, v):
        t.normal_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        I.cache_append(one, k, v, cu, kv, table, table=rt)
    for step in range(40):
        k.normal_()
        v.normal_()
        kv.fill_(step + 1)
        g.replay()
        I.cache_append(two, k, v, cu, kv, table, table=rt)
    torch.cuda.synchronize()
    for a, b in zip(_snapshot(one), _snapshot(two)):
        np.testing.assert_array_equal(a, b)


# ------------------------------------------------------------ a whole step --

@pytest.mark.parametrize("steps", [[97, 1, 3]])
def test_serving_step_from_projections_to_output(cuda_ok, steps):
    """A prefill chunk, a decode step and a draft of three tokens of one sequence:
    index rows and queries made, keys and values appended, the indexer's selection
    attended over.  Every stage against the reference on the stage's own inputs."""
    I = _I()
    rng = np.random.default_rng(12)
    H, D, Hq, heads, page, block, K, base = 32, 128, 16, 2, 32, 16, 48, 160
    rt = I.rope_table(512, 64)
    total = base + sum(steps)
    keys = torch.zeros(total, D, dtype=torch.uint8, device="cuda")
    key_scale = torch.zeros(total, device="cuda")
    cache = I.allocate_cache(16, page, heads, D, block)
    for t in (cache.k, cache.v):
        t.fill_(0x7F)
    table = _dev(rng.permutation(16).astype(np.int32)[None])
    T = 0
    for n in [base] + steps:
        rnd = lambda *s: _dev(rng.normal(size=s), torch.bfloat16)  # noqa: E731
        xi, qi, w = rnd(n, 1, D), rnd(n, H, D), _dev(rng.normal(size=(n, H)).astype(np.float32))
        q, k, v = rnd(n, Hq, D), rnd(n, heads, D), rnd(n, heads, D)
        pos = torch.arange(T, T + n, dtype=torch.int32, device="cuda")
        cu = _dev(np.array([0, n], dtype=np.int32))
        kv = _dev(np.array([T + n], dtype=np.int32))
        I.rotate_quantise(xi, pos, rt, out=(keys[T:T + n], key_scale[T:T + n]))
        qc, qs = I.rotate_quantise(qi, pos, rt)
        q_rot = I.cache_append(cache, k, v, cu, kv, table, table=rt, q=q)
        idx, ln = I.topk(qc, keys[:T + n], w, K, q_pos0=T, q_scale=qs, k_scale=key_scale[:T + n])
        out, lse = I.cache_attend(cache, q_rot, cu, kv, table, selected=(idx, ln), with_lse=True)
        assert ln.tolist() == [min(K, T + i + 1) for i in range(n)]
        _check_attend(cache, q_rot, [0, n], [T + n], table.cpu().numpy(), D ** -0.5, True, (idx, ln), out, lse, "bf16")
        # rows that see at most K positions select all of them: dense attention
        few = [i for i in range(n) if T + i < K]
        if few:
            dense = I.cache_attend(cache, q_rot, cu, kv, table)
            a, b = out[few].float(), dense[few].float()
            assert (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()
        T += n
