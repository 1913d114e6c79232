"""Block selection and attention at the ends of what they take: hundreds of picks among
thousands of blocks, prefix sums that fall between good sequences."""
import pytest
import torch

import test_gpu_blocks_edges as edges
from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_blocks import DEV, filled_cache, gen, ints, randn, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ds41.load()
    ds41.device_status()


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert ds41.device_status() == 0


@pytest.mark.parametrize("lens,news,nh,kvh,hd,page,topk,first,local", [
    ([16000], [2], 4, 1, 64, 16, 300, 1, 2), ([30000, 9000], [5, 1], 2, 1, 64, 16, 1024, 0, 1),
    ([17000], [1], 8, 2, 128, 16, 1024, 500, 20), ([9000], [9], 3, 1, 80, 16, 257, 1, 1),
    ([16400], [1], 4, 1, 64, 16, 1024, 1, 2), ([200000], [1], 2, 1, 16, 16, 300, 1, 2)])
def test_select_hundreds_of_many_blocks(lens, news, nh, kvh, hd, page, topk, first, local):
    """More picks than the list of candidates holds, more than 512 blocks."""
    edges.test_select_over_many_blocks(lens, news, nh, kvh, hd, page, topk, first, local)


@pytest.mark.parametrize("c", [[0, 4, -3, 8], [0, 3, 100, 4, 8], [4, 6, 1, 3], [5, 9, 12, 2, 5]])
def test_prefix_sums_that_fall_between_good_sequences(c):
    """Sequences whose prefix sums fall, start below 0 or pass the tokens are skipped and reported; the others' tokens are
    worked out, wherever those stand."""
    g = gen(41)
    page, kvh, hd, nh, T = 16, 2, 64, 4, 9
    B = len(c) - 1
    lens = [60 + 7 * b for b in range(B)]
    n_pages, rows = tables(g, lens, page)
    cache = filled_cache(g, n_pages, kvh, page, hd, True)
    q = randn(g, T, nh, hd)
    idx = ints([[[0, 2]] * kvh] * T)
    o = torch.full_like(q, 7.0)
    ds41.block_attn_fwd(q, cache, ints(rows), ints(lens), ints(c), T, idx, 0.1, o=o)
    assert ds41.device_status() == 4
    # each good sequence by itself
    want = torch.full_like(q, 7.0)
    for b in range(B):
        if 0 <= c[b] <= c[b + 1] <= T:
            for t in range(c[b], c[b + 1]):
                n = lens[b] - (c[b + 1] - 1 - t)
                want[t:t + 1] = ds41.block_attn_fwd(q[t:t + 1], cache, ints(rows[b:b + 1]), ints([n]), ints([0, 1]), 1,
                                                    idx[t:t + 1], 0.1)
    assert ds41.device_status() == 0
    assert torch.equal((o == 7.0).all(-1), (want == 7.0).all(-1))
    assert (o.float() - want.float()).abs().max() <= 2e-2
