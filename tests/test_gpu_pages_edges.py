"""Pages where they could go wrong beside the plain cases: pages taken ahead of the lengths
when a pool is compacted."""
import pytest
import torch

from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_blocks import DEV, filled_cache, gen, ints
from test_gpu_pages import everything, filled_keys

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


# ---------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [True, False])
def test_compact_between_taking_pages_and_counting_them(e4m3):
    """A page taken for rows that the lengths do not count yet is somebody's: where it moves
    its entry follows, and what is written through that entry lands in a page of its own."""
    g = gen(31)
    P, kvh, hd, page = 40, 2, 32, 16
    refs = torch.ones(P, dtype=torch.int32, device=DEV)
    refs[24:] = 0
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    lens, new = ints([30, 16, 0]), ints([70, 17, 40])
    ds41.kv_pages_take(refs, table, torch.zeros_like(lens), lens, page)
    ds41.kv_pages_take(refs, table, lens, new, page)  # all of them at the end of the pool
    refs[:24] = 0                                      # whose other sequences end
    table[1, 7], table[2, 6] = P, -(1 << 31)           # no pages: behind what is looked at
    before = table.clone()
    cache, keys = filled_cache(g, P, kvh, page, hd, e4m3), filled_keys(g, P, kvh, hd)
    want = [[t[before[b, :-(-int(n) // page)].long()].clone() for t in everything(cache, keys)]
            for b, n in enumerate(new.tolist())]
    live = ds41.kv_pages_compact(cache, refs, table, lens, keys=keys)
    assert ds41.device_status() == 0
    need = [-(-n // page) for n in new.tolist()]
    assert live.item() == sum(need) and refs.tolist() == [1] * sum(need) + [0] * (P - sum(need))
    named = [p for b, n in enumerate(need) for p in table[b, :n].tolist()]
    assert sorted(named) == list(range(sum(need)))
    for b, n in enumerate(need):
        for t, w in zip(everything(cache, keys), want[b]):
            assert torch.equal(t[table[b, :n].long()], w)
        assert torch.equal(table[b, n:], before[b, n:])
    # an entry that names no page within the lengths is reported as before
    table[0, 1] = P + 3
    ds41.kv_pages_compact(cache, refs, table, lens, keys=keys)
    assert ds41.device_status() == 4
    assert table[0, 1] == P + 3
