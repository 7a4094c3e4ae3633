"""Which cache layouts the calls take (no GPU needed: a refused call launches
nothing, and without a device an accepted one stops before its launch)."""

import pytest
import torch

from tests.test_cache_arguments import ECUDA, EINVAL, EUNSUPPORTED, I, _append, _attend, _cache  # noqa: F401

GB = 1 << 30


def _token_major(tokens, pages, heads=8, D=128):
    """Pages interleaved by token: [tokens of a page, pages, heads, D]."""
    return dict(n_pages=pages, page_size=tokens, page_stride=heads * D, token_stride=pages * heads * D,
                head_stride=D, heads=heads, D=D)


def _both(I, layout):  # noqa: F811
    return _append(I, cache=_cache(I, **layout)), _attend(I, cache=_cache(I, **layout))


@pytest.mark.parametrize("layout", [
    _token_major(64, 1 << 21),                                     # 128 GiB: tokens beyond 32 bits of 16 bytes
    _token_major(64, 1 << 20) | dict(page_stride=2048, token_stride=1 << 31),
    dict(n_pages=1000, page_stride=1 << 22, page_size=16, token_stride=(1 << 32) + (1 << 27)),   # over by the last pages alone
], ids=["128GiB", "gaps", "last-page"])
def test_offsets_beyond_32_bits_are_refused(I, layout):  # noqa: F811
    d = _cache(I, **layout)
    last = (d.n_pages - 1) * d.page_stride + (d.page_size - 1) * d.token_stride
    assert last >> 4 >= 1 << 32                                    # (what the kernels hold in 32 bits)
    assert _both(I, layout) == (EUNSUPPORTED, EUNSUPPORTED)


@pytest.mark.parametrize("layout", [
    _token_major(64, 1 << 20),                                     # 64 GiB and no more
    dict(n_pages=1 << 20, page_stride=1 << 16),                    # the same, page by page
    dict(n_pages=1 << 20, page_stride=1 << 16, token_stride=128, head_stride=64 * 128),
])
def test_layouts_up_to_64_gib_are_taken(I, layout):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no GPU can follow them")
    assert _both(I, layout) == (ECUDA, ECUDA)


@pytest.mark.parametrize("layout", [dict(token_stride=1 << 60), dict(head_stride=1 << 61), dict(token_stride=(1 << 62) + 1024),
                                    dict(head_stride=1 << 60, heads=1024, token_stride=128), dict(page_stride=1 << 60)])
def test_strides_whose_extent_overflows_are_refused(I, layout):  # noqa: F811
    assert _both(I, layout) == (EUNSUPPORTED, EUNSUPPORTED)


def test_strides_of_single_tokens_and_heads_do_not_count(I):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no GPU can follow them")
    assert _both(I, dict(page_size=1, block=1, token_stride=1 << 60)) == (ECUDA, ECUDA)


@pytest.mark.parametrize("layout", [
    dict(page_stride=8 * 1024, page_size=16),                      # half of each page is the next one's
    dict(page_stride=64 * 1024 - 128),
    _token_major(64, 100) | dict(token_stride=99 * 1024),          # token o + 1 of page 0 is token o of page 99
    dict(page_stride=128, token_stride=10 * 128, head_stride=64 * 128),    # heads and tokens that meet
    dict(heads=3, D=64, head_stride=64, token_stride=128, page_stride=1 << 14),
])
def test_pages_tokens_or_heads_that_share_bytes_are_refused(I, layout):  # noqa: F811
    assert _both(I, layout) == (EINVAL, EINVAL)


@pytest.mark.parametrize("layout", [
    _token_major(64, 100),
    dict(n_pages=1, page_stride=16),                               # a single page's stride counts for nothing
    dict(heads=1, head_stride=1 << 20, token_stride=128),
    dict(page_stride=2 * 64 * 1024),                               # keys and values of a page side by side
    dict(head_stride=256, token_stride=2048, page_stride=64 * 2048),       # of a head
    dict(n_pages=10, page_stride=64 * 128, token_stride=128, head_stride=10 * 64 * 128),    # heads outermost
    dict(head_stride=10 * 128, page_stride=128, token_stride=8 * 10 * 128),                 # pages innermost
])
def test_layouts_in_any_order_are_taken(I, layout):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no GPU can follow them")
    assert _both(I, layout) == (ECUDA, ECUDA)
