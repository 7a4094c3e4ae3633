"""The tile attention kernel's wait-timeout path, exercised without a device
fault: with the test hook the look-ups of the keys' places do not come, the waits
for them run out after about a millisecond each CTA, and the call must load
nothing, make its rows NaN and report bit 0 of the status word.  The next
ordinary call on the same workspace is checked against the reference."""

import numpy as np
import pytest
import torch

from tests.test_gpu_cache import ACT, _check_attend, _dev, _filled, _I

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,kv_len,Hq,heads,D,block,act", [
    ([1], [3000], 64, 1, 128, 16, "bf16"),           # one stream's rows, shares and the join
    ([40, 3], [700, 130], 16, 2, 128, 8, "bf16"),    # two streams, a place for each token
    ([70], [300], 8, 2, 64, 32, "fp16"),
    ([5] * 20, list(range(5, 605, 30)), 64, 64, 64, 16, "bf16"),   # a CTA for each (tile, head)
])
def test_wait_timeout_reports_and_device_recovers(cuda_ok, q_lens, kv_len, Hq, heads, D, block, act):
    I = _I()
    rng = np.random.default_rng(Hq)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    cache, table = _filled(rng, kv_len, heads, D, 64, block)
    q = _dev(rng.normal(size=(int(cu[-1]), Hq, D)), ACT[act])
    args = (cache, q, _dev(cu), _dev(np.array(kv_len, dtype=np.int32)), _dev(table))
    size = I.cache_attend_workspace_bytes(*args, max_q=max(q_lens), kernel=I.ATTEND_TILE)
    hook = I.ATTEND_TILE | I.ATTEND_TEST_WAIT_TIMEOUT
    assert I.cache_attend_workspace_bytes(*args, max_q=max(q_lens), kernel=hook) == size
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(with_lse=True, max_q=max(q_lens), workspace=ws, status=status)
    for _ in range(2):   # twice: the path leaves nothing behind
        out, lse = I.cache_attend(*args, kernel=hook, **kw)
        assert I.indexer_read_status(status) == 1
        assert out.isnan().all() and lse.isnan().all()
    out, lse = I.cache_attend(*args, kernel=I.ATTEND_TILE, **kw)
    assert I.indexer_read_status(status) == 0
    _check_attend(cache, q, cu, kv_len, table, D ** -0.5, True, None, out, lse, act)


def test_hook_is_of_the_tile_kernel_alone(cuda_ok):
    I = _I()
    cache = I.allocate_cache(1, 16, 1, 64, 16)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for kernel in (I.ATTEND_AUTO, I.ATTEND_STREAM):
        with pytest.raises(I.IndexerError):
            I.cache_attend(cache, q, one, one[1:], one[:1].view(1, 1), kernel=kernel | I.ATTEND_TEST_WAIT_TIMEOUT)
