"""Host-side argument checks of the cache calls (no GPU needed: a refused call
launches nothing), and the binding's checks of tensors."""

import ctypes

import pytest
import torch

EINVAL, EWORKSPACE, EUNSUPPORTED, ECUDA = 1, 2, 3, 4
PTR = 1 << 20   # an aligned address that a refused call never follows


@pytest.fixture(scope="module")
def I():
    from head_weighted_relu_b200 import build
    build.build()
    from head_weighted_relu_b200 import indexer
    return indexer


def _cache(I, **kw):
    d = dict(k=PTR, v=PTR, k_scale=PTR, v_scale=PTR, n_pages=10, page_stride=64 * 8 * 128, token_stride=8 * 128,
             head_stride=128, page_size=64, block=16, heads=8, D=128)
    d.update(kw)
    return I.CacheDesc(*[d[f] for f, _ in I.CacheDesc._fields_])


def _seqs(I, **kw):
    d = dict(S=4, cu_q=PTR, kv_len=PTR, page_table=PTR, table_stride=5, table_pages=5, B=2)
    d.update(kw)
    return I.Sequences(*[d[f] for f, _ in I.Sequences._fields_])


def _append(I, cache=None, seqs=None, k=PTR, v=PTR, stride=1024, act=0, rot=None, q=PTR, Hq=64, q_stride=8192, q_out=PTR):
    return I._lib.indexer_cache_append(cache or _cache(I), seqs or _seqs(I), k, v, stride, act,
                                       rot or I.Rotation(PTR, 100, 128, 0), q, Hq, q_stride, q_out, None, None)


def _attend(I, cache=None, seqs=None, att=None, q=PTR, stride=8192, si=None, sl=None, out=PTR, ws=PTR, n=1 << 40):
    a = dict(Hq=64, act=0, causal=1, sel_width=0, max_q=0, scale=0.1, kernel=0)
    a.update(att or {})
    return I._lib.indexer_cache_attend(cache or _cache(I), seqs or _seqs(I),
                                       I.Attention(*[a[f] for f, _ in I.Attention._fields_]), q, stride, si, sl, out,
                                       None, None, ws, n, None)


def test_valid_calls_get_as_far_as_the_device(I):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no GPU can follow them")
    assert _append(I) == ECUDA and _attend(I) == ECUDA
    assert I._lib.indexer_rotate_quantise(PTR, 4, 8, 128, 0, 1024, None, None, PTR, PTR, None, None) == ECUDA


@pytest.mark.parametrize("change,status", [
    (dict(k=None), EINVAL), (dict(v_scale=None), EINVAL), (dict(k=PTR + 8), EINVAL), (dict(D=96), EUNSUPPORTED),
    (dict(n_pages=0), EINVAL), (dict(block=24, page_size=48), EUNSUPPORTED), (dict(block=256, page_size=256), EUNSUPPORTED),
    (dict(page_size=40), EINVAL), (dict(page_size=0), EINVAL), (dict(heads=0), EINVAL), (dict(heads=2000), EUNSUPPORTED),
    (dict(head_stride=64), EINVAL), (dict(token_stride=1000), EINVAL), (dict(token_stride=512), EINVAL),
    (dict(page_stride=8), EINVAL), (dict(n_pages=1 << 24), EUNSUPPORTED), (dict(n_pages=1 << 40, page_stride=16), EINVAL),
])
def test_cache_descriptor(I, change, status):
    assert _append(I, cache=_cache(I, **change)) == status
    assert _attend(I, cache=_cache(I, **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(S=-1), EINVAL), (dict(B=-1), EINVAL), (dict(cu_q=None), EINVAL), (dict(kv_len=None), EINVAL),
    (dict(page_table=None), EINVAL), (dict(table_stride=4), EINVAL), (dict(S=1 << 31), EUNSUPPORTED),
    (dict(B=(1 << 20) + 1), EUNSUPPORTED),
])
def test_sequences(I, change, status):
    assert _append(I, seqs=_seqs(I, **change)) == status
    assert _attend(I, seqs=_seqs(I, **change)) == status


def test_nothing_to_do_is_no_error(I):
    assert _append(I, seqs=_seqs(I, S=0)) == 0 and _append(I, seqs=_seqs(I, B=0)) == 0
    r = I._lib.indexer_rotate_quantise
    assert r(None, 0, 8, 128, 0, 1024, None, None, None, None, None, None) == 0


def test_append_arguments(I):
    assert _append(I, k=None) == EINVAL
    assert _append(I, k=PTR + 2) == EINVAL
    assert _append(I, stride=1020) == EINVAL and _append(I, stride=512) == EINVAL
    assert _append(I, act=2) == EINVAL
    assert _append(I, q_out=None) == EINVAL and _append(I, q=None) == EINVAL
    assert _append(I, Hq=0) == EINVAL and _append(I, q_stride=128) == EINVAL
    assert _append(I, rot=I.Rotation(None, 100, 128, 0)) == EINVAL
    assert _append(I, rot=I.Rotation(PTR, 0, 128, 0)) == EINVAL
    assert _append(I, rot=I.Rotation(PTR, 100, 136, 0)) == EINVAL
    assert _append(I, rot=I.Rotation(PTR, 100, 144, 0)) == EINVAL
    assert _append(I, rot=I.Rotation(PTR, 100, 64, 2)) == EINVAL


def test_attend_arguments(I):
    for att, status in ((dict(Hq=60), EINVAL), (dict(Hq=0), EINVAL), (dict(Hq=8 * 129), EUNSUPPORTED), (dict(act=7), EINVAL),
                        (dict(causal=2), EINVAL), (dict(sel_width=-1), EINVAL), (dict(scale=float("nan")), EINVAL),
                        (dict(scale=float("inf")), EINVAL), (dict(max_q=-1), EINVAL), (dict(kernel=3), EINVAL),
                        (dict(kernel=-1), EINVAL)):
        assert _attend(I, att=att) == status, att
    assert _attend(I, seqs=_seqs(I, table_pages=1 << 28, table_stride=1 << 28)) == EUNSUPPORTED


def test_rotate_quantise_arguments(I):
    r = I._lib.indexer_rotate_quantise
    ok = dict(x=PTR, S=4, H=8, D=128, act=0, stride=1024, pos=None, rot=None, codes=PTR, scale=PTR)
    for change, status in ((dict(x=None), EINVAL), (dict(x=PTR + 4), EINVAL), (dict(S=-1), EINVAL), (dict(D=80), EUNSUPPORTED),
                           (dict(act=-1), EINVAL), (dict(stride=1000), EINVAL), (dict(stride=1028), EINVAL),
                           (dict(codes=PTR + 4), EINVAL), (dict(scale=None), EINVAL),
                           (dict(rot=I.Rotation(PTR + 4, 10, 64, 0)), EINVAL), (dict(rot=I.Rotation(PTR, 10, 24, 0)), EINVAL)):
        a = dict(ok, **change)
        assert r(a["x"], a["S"], a["H"], a["D"], a["act"], a["stride"], a["pos"], a["rot"], a["codes"], a["scale"], None,
                 None) == status, change


def test_binding_checks_tensors(I):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    good = I.KVCache(z(4, 32, 2, 64), z(4, 32, 2, 64), f(4, 2, 2), f(4, 2, 2))
    d = good.descriptor()
    assert (d.n_pages, d.page_size, d.block, d.heads, d.D, d.token_stride) == (4, 32, 16, 2, 64, 128)
    hnd = I.KVCache(z(4, 2, 32, 64).transpose(1, 2), z(4, 2, 32, 64).transpose(1, 2), f(4, 2, 2), f(4, 2, 2)).descriptor()
    assert (hnd.token_stride, hnd.head_stride, hnd.page_stride) == (64, 2048, 4096)
    for bad in (good._replace(v=z(4, 32, 2, 128)), good._replace(k_scale=f(4, 3, 2)), good._replace(k=f(4, 32, 2, 64)),
                good._replace(v_scale=f(4, 2, 3)), good._replace(v=z(4, 2, 32, 64).transpose(1, 2))):
        with pytest.raises(ValueError):
            bad.descriptor()
    cu, kv, table = z(3, dt=torch.int32), z(2, dt=torch.int32), z(2, 3, dt=torch.int32)
    bf = torch.bfloat16
    with pytest.raises(ValueError):   # a CPU cache
        I.cache_attend(good, z(2, 4, 64, dt=bf), cu, kv, table)
    with pytest.raises(ValueError):   # float32 queries
        I.cache_attend(good, f(2, 4, 64), cu, kv, table)
    with pytest.raises(ValueError):   # int64 lengths
        I.cache_attend(good, z(2, 4, 64, dt=bf), cu, kv.long(), table)
    with pytest.raises(ValueError):   # keys of another head size
        I.cache_append(good, z(2, 2, 128, dt=bf), z(2, 2, 128, dt=bf), cu, kv, table)
    with pytest.raises(ValueError):   # heads not packed
        I.rotate_quantise(z(2, 64, 4, dt=bf).transpose(1, 2))
    with pytest.raises(ValueError):
        I.allocate_cache(4, 24, 2, 64, block=16, device="cpu")


def test_rope_table(I):
    t = I.rope_table(7, 32, device="cpu")
    assert t.shape == (7, 32) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.cat([torch.ones(16), torch.zeros(16)]))
    assert abs(t[5, 3].item() - torch.cos(torch.tensor(5 * 10000 ** (-6 / 32), dtype=torch.float64)).item()) < 1e-7
