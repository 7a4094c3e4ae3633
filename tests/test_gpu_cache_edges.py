"""Edges of the cache operators on the GPU: scales that are no power of two, NaN
codes in tiles that only some rows see whole, beside large scores and of vanishing
weight, runs of zero values, rows beside very different ones,
rows that see nothing; large ragged batches, pages interleaved by token, results in
the place of their inputs, large appends in a graph."""

import numpy as np
import pytest
import torch

from tests import cache_reference as R
from tests.test_gpu_cache import ACT, STREAM, TILE, _check_attend, _dev, _filled, _half_step, _I, _random_cache, _snapshot

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------- append --

@pytest.mark.parametrize("D,block,act,rot", [(128, 16, "bf16", 64), (64, 32, "fp16", 0), (128, 128, "bf16", 128),
                                             (64, 128, "bf16", 0)])
@pytest.mark.parametrize("old", ["1.5*2^-7", "0.3", "1.25", "amax/448", "2^127"])
def test_append_behind_any_scale(cuda_ok, D, block, act, rot, old):
    """A block begun by another writer, whose scale is no power of two (or too large
    for its reciprocal to be a normal number): kept where the new tokens fit
    under it, raised to a power of two where they do not."""
    I = _I()
    rng = np.random.default_rng(D + block)
    heads, past, n = 3, 5, 9
    cache = _random_cache(rng, 2, block, heads, D, block)
    cache.k[1, :past] = _dev(R.to_code(np.clip(rng.normal(size=(past, heads, D)) * 100, -448, 448)))
    cache.v[1, :past] = _dev(R.to_code(np.clip(rng.normal(size=(past, heads, D)) * 100, -448, 448)))
    scale = {"1.5*2^-7": np.full(heads, 1.5 * 2.0 ** -7), "0.3": np.full(heads, 0.3), "1.25": np.full(heads, 1.25),
             "amax/448": rng.uniform(1, 4, size=heads) / 448, "2^127": np.full(heads, 2.0 ** 127)}[old].astype(np.float32)
    cache.k_scale[1, 0] = _dev(scale)
    cache.v_scale[1, 0] = _dev(scale)
    # the first head fits under the old scale, the last one may not
    x = rng.normal(size=(n, heads, D)) * np.array([0.5, 3.0, 40.0])[:, None] * float(scale[0]) * 60
    x = np.clip(x, -3e38, 3e38) if act == "bf16" else np.clip(x, -60000, 60000)
    k, v = _dev(x, ACT[act]), _dev(-x[::-1], ACT[act])
    before = _snapshot(cache)
    rt = I.rope_table(64, rot) if rot else None
    cu, kv = np.array([0, n], dtype=np.int32), [past + n]
    table = np.array([[1]], dtype=np.int32)
    I.cache_append(cache, k, v, _dev(cu), _dev(np.array(kv, dtype=np.int32)), _dev(table), table=rt)
    after = _snapshot(cache)
    wk, wv, wks, wvs, _, written = R.append(*before, R.to_np(k), R.to_np(v), cu, kv, table, rot, False)
    for name, got, want, gs, ws, was, sc0 in (("k", after[0], wk, after[2], wks, before[0], before[2]),
                                              ("v", after[1], wv, after[3], wvs, before[1], before[3])):
        np.testing.assert_array_equal(gs[1], ws[1].astype(np.float32))
        for (nm, pg, o, h), (y, s) in written.items():
            if nm == name:
                slip = 6 * 2.0 ** -24 * np.abs(R.to_np(k)[o - past, h]).max() if name == "k" and rot else 0.0
                # (a rotation beyond FP32's range is infinite, and becomes NaN codes)
                over = np.abs(y) >= 2.0 ** 128 * (1 - 2.0 ** -25)
                assert ((got[pg, o, h] & 0x7F == 0x7F) == over).all()
                y = np.where(over, 0.0, y)
                err = np.where(over, 0.0, np.abs(R.VALUES[got[pg, o, h]] * s - y))
                # rounded twice: the quotient, half a step of FP32, and the code
                assert (err <= _half_step(y, s) * (1 + 2.0 ** -20) + slip).all(), (name, o, h)
        for h in range(heads):
            if ws[1, 0, h] == sc0[1, 0, h]:
                np.testing.assert_array_equal(got[1, :past, h], was[1, :past, h])
            else:
                y, s = R.VALUES[was[1, :past, h]] * float(sc0[1, 0, h]), ws[1, 0, h]
                assert (np.abs(R.VALUES[got[1, :past, h]] * s - y) <= _half_step(y, s) * (1 + 2.0 ** -20)).all()
        np.testing.assert_array_equal(got[0], was[0])
        np.testing.assert_array_equal(got[1, past + n:], was[1, past + n:])


# -------------------------------------------------------------- attention --

@pytest.mark.parametrize("block", [16, 8])
@pytest.mark.parametrize("G,n_q,kv,max_q,causal", [(8, 40, 140, 40, True), (1, 300, 420, 300, True), (8, 16, 134, 16, True),
                                                   (3, 200, 700, 200, True), (8, 40, 140, 40, False)])
def test_nan_value_in_a_tile_that_later_rows_see_whole(cuda_ok, G, n_q, kv, max_q, causal, block):
    """Tiles of keys that a tile's first row sees in part and its last rows whole: a
    NaN value code there reaches every row that sees it."""
    I = _I()
    rng = np.random.default_rng(G * 100 + n_q)
    cache, table = _filled(rng, [kv], 2, 128, 32, block)
    first = kv - n_q + 1                                   # positions that the first row sees
    for p, d in ((50, 3), (first // 128 * 128, 77), (kv - 2, 100)):
        cache.v[table[0, p // 32], p % 32, 1, d] = 0x7F
    cu = np.array([0, n_q], dtype=np.int32)
    q = _dev(rng.normal(size=(n_q, 2 * G, 128)), torch.bfloat16)
    out = {}
    for kernel in (TILE, STREAM):
        out[kernel], lse = I.cache_attend(cache, q, _dev(cu), _ints([kv]), _dev(table), causal=causal, with_lse=True,
                                          max_q=max_q, kernel=kernel)
        _check_attend(cache, q, cu, [kv], table, 128 ** -0.5, causal, None, out[kernel], lse, "bf16")
    nan = out[TILE].isnan()
    assert torch.equal(nan, out[STREAM].isnan()) and nan[:, G:, 3].all() and not nan[:, :G].any()


def _ramp(rng, kv, heads, D, low):
    """A cache whose keys score `low`[p] in every head against a query of ones."""
    I = _I()
    page = 64
    pages = -(-kv // page)
    table = rng.permutation(pages).astype(np.int32)[None]
    cache = I.allocate_cache(pages, page, heads, D, 16)
    code = R.to_code(low).astype(np.uint8)
    flat = np.zeros((pages * page,), dtype=np.uint8)
    flat[:kv] = code
    by_page = np.empty((pages, page), dtype=np.uint8)
    by_page[table[0]] = flat.reshape(pages, page)
    cache.k.copy_(_dev(by_page)[:, :, None, None].expand(pages, page, heads, D))
    values = R.to_code(np.clip(rng.normal(size=(64, page, heads, D)) * 60, -448, 448))
    cache.v.copy_(_dev(np.resize(values, (pages, page, heads, D))))
    cache.k_scale.fill_(2.0 ** -4)
    cache.v_scale.fill_(2.0 ** -6)
    return cache, table


@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("where", [5000, 5128])
def test_nan_key_beside_large_scores(cuda_ok, kernel, where):
    """Scores of some 200 (natural) everywhere, and a NaN code in one key, in an even
    and in an odd tile: all rows that see it are NaN, whatever shares its sums."""
    I = _I()
    rng = np.random.default_rng(31)
    kv, heads, D = 20000, 4, 128
    cache, table = _ramp(rng, kv, heads, D, np.full(kv, 256.0))
    cache.k[table[0, where // 64], where % 64, 1, 9] = 0x7F
    q = torch.ones(1, heads * 8, D, dtype=torch.bfloat16, device="cuda")
    out, lse = I.cache_attend(cache, q, _ints([0, 1]), _ints([kv]), _dev(table), scale=0.1, with_lse=True, max_q=1,
                              kernel=kernel)
    assert out[0, 8:16].isnan().all() and lse[0, 8:16].isnan().all()
    assert out[0, :8].isfinite().all() and out[0, 16:].isfinite().all()


@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("kv,every,part", [(20000, 20000, 10000), (20000, 64, 16), (20000, 256, 128), (600, 600, 300)])
def test_nan_value_of_vanishing_weight(cuda_ok, kernel, kv, every, part):
    """A NaN code among the values of keys that score hundreds less than the others,
    by themselves in a warp's, a stream's or a CTA's share: 0 * NaN is NaN in
    that dimension, and there alone."""
    I = _I()
    rng = np.random.default_rng(32)
    heads, D = 2, 64
    pos = np.arange(kv)
    cache, table = _ramp(rng, kv, heads, D, np.where(pos % every < part, -256.0, 256.0))
    for p in (min(3, part - 1), (kv - 1) // every * every):
        cache.v[table[0, p // 64], p % 64, 1, 21] = 0xFF
    q = torch.ones(1, heads * 8, D, dtype=torch.bfloat16, device="cuda")
    out = I.cache_attend(cache, q, _ints([0, 1]), _ints([kv]), _dev(table), scale=0.2, max_q=1, kernel=kernel)
    nan = out.isnan()
    assert nan[0, 8:, 21].all() and nan.sum() == 8


@pytest.mark.parametrize("kernel,B,n,ones", [(STREAM, 300, 14, 0), (TILE, 1200, 14, 0), (STREAM, 300, 19, 64), (TILE, 1200, 16, 64),
                                             (STREAM, 1, 14, 64), (TILE, 1, 14, 64), (STREAM, 1, 21, 0), (TILE, 1, 21, 0)])
def test_run_of_zero_values_at_the_slack(cuda_ok, kernel, B, n, ones):
    """Blocks of zero values have the scale 2^-100.  2^n of their tokens, which score
    just under what would raise the reference that the first 256 set, then some
    values that are not zero: sums stay finite.  B sequences over the same
    pages: with many, one CTA goes over all of the keys."""
    I = _I()
    rng = np.random.default_rng(34)
    kv, D, G = 2 ** n + 256 + 64, 64, 8
    low = np.where(np.arange(kv) < 256, 0.0, 15.0)         # 15/16 * 64 dimensions * scale below: 7.5 in base 2
    cache, table = _ramp(rng, kv, 1, D, low)
    cache.v.zero_()
    cache.v_scale.fill_(2.0 ** -100)
    scale = 7.5 * np.log(2) / 60
    for p in range(kv - ones, kv):
        cache.v[table[0, p // 64], p % 64] = 0x38 + (p & 1)
        cache.v_scale[table[0, p // 64], p % 64 // 16] = 1.0
    q = torch.ones(B, G, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out, lse = I.cache_attend(cache, q, cu, _ints([kv] * B), _dev(table).expand(B, -1).contiguous(), scale=scale,
                              with_lse=True, max_q=1, kernel=kernel)
    # all dimensions are alike: scores 0 and 7.5 ln 2, values 1 and 1.125 in turn
    total = 256 + (kv - 256) * 2.0 ** 7.5
    want = 2.0 ** 7.5 * ones * 1.0625 / total
    # a row's sum is of kv/16 additions one after another or fewer, each within 2^-24;
    # scores as in the other tests (5.2 at most); weights to FP16, the output to bf16
    off = kv / 16 * 2.0 ** -24 + 2.0 ** -17
    assert (np.abs(R.to_np(lse) - np.log(total)) <= off + 2.0 ** -20).all()
    assert (np.abs(R.to_np(out) - want) <= want * (2.0 ** -8 + 2 * (off + 2.0 ** -12))).all()
    assert (out == out[:1]).all() and (lse == lse[:1]).all()


@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("first", [True, False])
def test_zero_values_count_beside_a_far_larger_scale(cuda_ok, kernel, first):
    """2^18 tokens of zero values, each 2^-27 as likely as one token whose values'
    scale is 2^100 times theirs: 1/512 of the row's sum together."""
    I = _I()
    rng = np.random.default_rng(36)
    kv, D, G = 2 ** 18 + 1, 64, 8
    at = kv - 1 if first else 0
    low = np.zeros(kv)
    low[at] = 15.0
    cache, table = _ramp(rng, kv, 1, D, low)
    cache.v.zero_()
    cache.v_scale.fill_(2.0 ** -100)
    cache.v[table[0, at // 64], at % 64] = 0x38
    cache.v_scale[table[0, at // 64], at % 64 // 16] = 1.0
    scale = 27 * np.log(2) / 60
    q = torch.ones(1, G, D, dtype=torch.bfloat16, device="cuda")
    out, lse = I.cache_attend(cache, q, _ints([0, 1]), _ints([kv]), _dev(table), scale=scale, with_lse=True, max_q=1,
                              kernel=kernel)
    # the score of 18.7 is within 2^-16; the sum's additions, at most kv/16 of them for
    # 1/512 of it, within a quarter of that
    rest = np.log1p((kv - 1) * 2.0 ** -27)
    assert (np.abs(R.to_np(lse) - 27 * np.log(2) - rest) <= rest * 2.0 ** -2).all()
    assert (np.abs(R.to_np(out) - np.exp(-rest)) <= 2.0 ** -8 + 2.0 ** -11).all()


@pytest.mark.parametrize("G,kernel", [(3, STREAM), (8, STREAM), (3, TILE), (8, TILE)])
def test_rows_do_not_depend_on_their_neighbours(cuda_ok, G, kernel):
    """Queries of one sequence share a tile, and their CTAs go over many keys each:
    another query's values, large or not, change no bit of a row."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(33)
    pages, D = 3000, 128
    cache = I.allocate_cache(pages, 64, 1, D, 16)
    for x in (cache.k, cache.v):
        x.copy_((60 * torch.randn(x.shape, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
                .view(torch.uint8))
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(2.0 ** -6)
    table = torch.randperm(pages, generator=g, device="cuda").int().view(1, pages)
    for n_q in (2, 5):
        args = (_ints([0, n_q]), _ints([pages * 64]), table)
        q = torch.randn(n_q, G, D, generator=g, device="cuda").bfloat16()
        want, wl = I.cache_attend(cache, q, *args, kernel=kernel, with_lse=True)
        for i in range(n_q):
            other = q.clone()
            other[i] *= 50
            got, gl = I.cache_attend(cache, other, *args, kernel=kernel, with_lse=True)
            keep = [j for j in range(n_q) if j != i]
            assert torch.equal(got[keep], want[keep]) and torch.equal(gl[keep], wl[keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kernel", [STREAM, TILE])
@pytest.mark.parametrize("G,block", [(8, 16), (64, 8)])
def test_rows_that_see_nothing_whatever_their_query(cuda_ok, kernel, G, block, bad):
    """Padding rows whose queries hold anything: nothing selected, nothing but unseen
    or missing tokens selected, no page, a length of zero."""
    I = _I()
    rng = np.random.default_rng(35)
    cache, table = _filled(rng, [200, 200, 64], 1, 128, 32, block)
    table[1, :] = -1
    q = _dev(rng.normal(size=(5, G, 128)), torch.bfloat16)
    clean = q.clone()
    q[[0, 1, 3, 4]] = bad
    cu, kv = _ints([0, 3, 4, 5]), _ints([200, 200, 0])
    idx = np.full((5, 300), -1, dtype=np.int32)
    idx[1, :3] = [199, 200, -7]                            # row 1 sees up to 198
    idx[2, :150] = np.arange(150)
    idx[3, :100] = np.arange(100)
    idx[4, :2] = [0, 1]
    ln = _ints([0, 3, 150, 100, 2])
    tb = _dev(table)
    for kw in (dict(selected=(_dev(idx), ln)), dict()):
        out, lse = I.cache_attend(cache, q, cu, kv, tb, with_lse=True, kernel=kernel, **kw)
        want, wl = I.cache_attend(cache, clean, cu, kv, tb, with_lse=True, kernel=kernel, **kw)
        empty = [0, 1, 3, 4] if kw else [3, 4]
        assert (out[empty] == 0).all() and lse[empty].isneginf().all()
        assert torch.equal(out[2], want[2]) and torch.equal(lse[2], wl[2]) and out[2].isfinite().all()
        if not kw:
            assert out[:2].isnan().all()


# ----------------------------------------- calls that other tests do not make --

@pytest.mark.parametrize("kernel", [STREAM, TILE])
def test_ragged_decode_batch_of_many_sequences(cuda_ok, kernel):
    """More sequences than CTAs of the streaming kernel share: one long context among
    short ones, some of them empty."""
    I = _I()
    rng = np.random.default_rng(41)
    B, D = 300, 128
    kv = rng.integers(0, 60, size=B).tolist()
    kv[17] = 3000
    cache, table = _filled(rng, kv, 2, D, 64, 16)
    cu = np.arange(B + 1, dtype=np.int32)
    q = _dev(rng.normal(size=(B, 16, D)), torch.bfloat16)
    out, lse = I.cache_attend(cache, q, _dev(cu), _ints(kv), _dev(table), with_lse=True, max_q=1, kernel=kernel)
    _check_attend(cache, q, cu, kv, table, D ** -0.5, True, None, out, lse, "bf16")


def test_pages_interleaved_by_token(cuda_ok):
    """Memory [tokens of a page, pages, heads, D], and [heads, pages, tokens, D]: the
    same cache and the same attention as page by page."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(42)
    pages, page, heads, D, n = 7, 32, 3, 64, 200
    k, v = (torch.randn(n, heads, D, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(n, 2 * heads, D, generator=g, device="cuda").half()
    table = torch.randperm(pages, generator=g, device="cuda").int().view(1, pages)
    rt = I.rope_table(n, 64)
    results = []
    for order in ((0, 1, 2), (1, 0, 2), (2, 0, 1)):
        sizes = [(pages, page, heads)[i] for i in order]
        codes = [torch.zeros(*sizes, D, dtype=torch.uint8, device="cuda").permute(*[order.index(i) for i in range(3)], 3)
                 for _ in range(2)]
        scales = [torch.zeros(pages, page // 16, heads, device="cuda") for _ in range(2)]
        cache = I.KVCache(*codes, *scales)
        for a, b in ((0, 77), (77, n)):
            I.cache_append(cache, k[a:b], v[a:b], _ints([0, b - a]), _ints([b]), table, table=rt)
        results.append([x.contiguous() for x in cache] + [I.cache_attend(cache, q, _ints([0, n]), _ints([n]), table, kernel=x)
                                                          for x in (STREAM, TILE)])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("inter", [False, True])
def test_results_in_the_place_of_their_inputs(cuda_ok, inter):
    """q rotated, and attended with, in its own memory; q large enough for a kernel
    of its own in one case."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(43)
    for n, Hq, rot in ((50, 16, 48), (1100, 128, 128)):
        cache = I.allocate_cache(-(-n // 64), 64, 4, 128, 16)
        table = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda").view(1, -1)
        k = torch.randn(n, 4, 128, generator=g, device="cuda").bfloat16()
        q = torch.randn(n, Hq, 128, generator=g, device="cuda").bfloat16()
        args = (_ints([0, n]), _ints([n]), table)
        want = I.cache_append(cache, k, k, *args, table=I.rope_table(n, rot), interleaved=inter, q=q)
        same = q.clone()
        assert I.cache_append(cache, k, k, *args, table=I.rope_table(n, rot), interleaved=inter, q=same, q_out=same) is same
        assert torch.equal(same, want)
        for kernel in (STREAM, TILE):
            x = want.clone()
            out = I.cache_attend(cache, want, *args, kernel=kernel)
            assert torch.equal(I.cache_attend(cache, x, *args, kernel=kernel, out=x), out)


def test_large_append_in_a_graph(cuda_ok):
    """q in a kernel of its own, captured and replayed with other rows and lengths,
    and what follows it in the graph."""
    I = _I()
    g = torch.Generator(device="cuda").manual_seed(44)
    n, Hq, heads, D = 1100, 128, 2, 128
    one, two = (I.allocate_cache(40, 64, heads, D, 64) for _ in range(2))
    table = torch.randperm(40, generator=g, device="cuda").int().view(1, 40)
    rt = I.rope_table(40 * 64, 128)
    q, k, v = (torch.empty(n, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, heads, heads))
    cu, kv = _ints([0, n]), _ints([n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_rot = I.cache_append(one, k, v, cu, kv, table, table=rt, q=q)
        out = I.cache_attend(one, q_rot, cu, kv, table)
    for length in (n, 2 * n):
        for x in (q, k, v):
            x.normal_(generator=g)
        kv.fill_(length)
        graph.replay()
        want = I.cache_append(two, k, v, cu, kv, table, table=rt, q=q)
        assert torch.equal(q_rot, want)
        assert torch.equal(out, I.cache_attend(two, want, cu, kv, table))
