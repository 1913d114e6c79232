"""Pages and beams where they could go wrong beside the plain cases: pages taken ahead of
the lengths when a pool is compacted, tables of more than 128 pages, whole prompts under a
beam search, many beams and the longest rows, offers of different beams next to each other."""
import math

import pytest
import torch

import test_gpu_pages as pages
from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_blocks import DEV, filled_cache, gen, ints
from test_gpu_pages import check_beam, everything, filled_keys, u8

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


@pytest.mark.parametrize("replace", [False, True])
@pytest.mark.parametrize("lens,n", [([128 * 16 + 5, 127 * 16 + 3, 129 * 16, 257 * 16 + 9], 200), ([2049] * 8, 256),
                                    ([300 * 16 + 1, 0, 5], 40)])
def test_fork_of_long_tables(lens, n, replace):
    """More pages a row than the threads of a CTA, in two launches."""
    pages.test_fork(lens, n, 1, 16, 16, n + 3, replace, True)


def test_beams_keep_their_prompts():
    """Every beam has its prompt's rows, K, V and the scales, through forks that share whole pages and copy
    the last one, and through steps that replace the beams by their children."""
    g = gen(32)
    B, W, V, page, kvh, hd = 3, 4, 300, 16, 2, 32
    n0 = [20, 33, 16]
    P = 3 * W * 6 + 4
    cache, refs = filled_cache(g, P, kvh, page, hd, True), torch.zeros(P, dtype=torch.int32, device=DEV)
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    lens = ints(n0)

    def rows(row, n):  # [tensor][n, kvh, ..]
        at = row[:-(-n // page)].long()
        return [u8(t)[at].transpose(1, 2).flatten(0, 1)[:n].clone() for t in cache]
    ds41.kv_pages_take(refs, table, torch.zeros_like(lens), lens, page)
    prompts = [rows(table[b], n) for b, n in enumerate(n0)]
    start = table.clone()
    table, lens = ds41.kv_pages_fork(cache, refs, table, lens, ints([b for b in range(B) for _ in range(W)]))
    ds41.kv_pages_free(refs, start, ints(n0), page)
    scores = torch.full((B, W), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    for step in range(20):
        scores, parents, _ = ds41.beam_select(torch.randn(B, W, V, generator=g, device=DEV) * 2, scores, W)
        table, lens = ds41.kv_pages_fork(cache, refs, table, lens, parents.view(-1), replace=True)
        new = lens + 1
        ds41.kv_pages_take(refs, table, lens, new, page)
        pos = lens.long()
        slots = torch.gather(table.long(), 1, (pos // page)[:, None])[:, 0] * page + pos % page
        k = torch.randn(B * W, kvh, hd, generator=g, device=DEV).bfloat16()
        ds41.kv_cache_write(cache, k, k, slots)
        lens = new
        for i in range(B * W):
            assert int(lens[i]) == n0[i // W] + step + 1
            for got, want in zip(rows(table[i], n0[i // W]), prompts[i // W]):
                assert torch.equal(got, want), (step, i)


# ---------------------------------------------------------------------------
# Beams
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,W,V,k", [(1, 1024, 5000, 64), (2, 700, 9000, 128), (1, 4, 1 << 22, 16)])
def test_beam_of_many_beams_and_of_long_rows(B, W, V, k):
    g = gen(33)
    x = torch.randn(B, W, V, generator=g, device=DEV).bfloat16()
    check_beam(x, torch.zeros(B, W, device=DEV), k)


def test_beam_order_of_offers_next_to_each_other():
    """Rows of n zeros, -inf besides: the sum n is exact in f32, so that a beam's offers are at s - log n but for
    the logarithm.  Scores that are log n rounded to f32 set two beams' offers 2.4e-7 .. 1e-6 apart
    (the rounding of a logarithm of 8 .. 10 in f32 alone is 4.8e-7); the logarithm is worked out
    as e ln 2 in 64 bits and that of a factor of 3/4 .. 3/2 in f32, off by 2^-25 for each of the two."""
    r = torch.Generator().manual_seed(34)
    V = 20000
    pairs = []
    while len(pairs) < 300:
        n = torch.randint(3000, V, (2,), generator=r)
        exact = n.double().log()
        s = exact.float()
        gap = (s[0].double() - exact[0]) - (s[1].double() - exact[1])
        if abs(gap) >= 2.0 ** -22:
            pairs.append((n.tolist(), s, 0 if gap > 0 else 1))
    x = torch.full((len(pairs), 2, V), -math.inf)
    want, first = [], []
    for b, (n, s, best) in enumerate(pairs):
        for w in range(2):
            at = torch.randperm(V, generator=r)[:n[w]]
            x[b, w, at] = 0.0
            if w == best:
                want.append([2 * b + w])
                first.append([int(at.min())])
    scores = torch.stack([s for _, s, _ in pairs]).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        _, parents, tokens = ds41.beam_select(x.to(DEV, dtype), scores, 1)
        wrong = [b for b, (p, w) in enumerate(zip(parents.tolist(), want)) if p != w]
        assert not wrong, f"{len(wrong)} of {len(pairs)} searches keep the lower offer"
        assert tokens.tolist() == first


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_order_of_rows_in_other_orders(dtype):
    """Beams with the same logits in other orders: their sums differ by their roundings, which check_beam bounds by
    tol for each.  Scores 2 tol apart decide; equal scores leave the order of equal logits to the sums."""
    g = gen(35)
    V, W, k = 3001, 6, 24
    tol = (V / 256 + 16) * 2.0 ** -24 + 2.0 ** -20
    row = torch.randn(V, generator=g, device=DEV).to(dtype)
    row[:8] = torch.arange(8, device=DEV).to(dtype) * 0.5 + 5  # (the best ones far apart)
    order = [torch.randperm(V, generator=g, device=DEV) for _ in range(W)]
    x = torch.stack([row[o] for o in order])[None]
    scores = (torch.arange(W, device=DEV) * 2.5 * tol)[None].float()
    _, parents, tokens = ds41.beam_select(x, scores, k)
    assert parents[0].tolist() == [W - 1 - i % W for i in range(k)]
    assert x[0, parents[0].long(), tokens[0].long()].tolist() == [row[7 - i // W].item() for i in range(k)]
    _, parents, tokens = ds41.beam_select(x, torch.zeros(1, W, device=DEV), k)
    for i in range(0, k, W):
        assert sorted(parents[0, i:i + W].tolist()) == list(range(W))
    assert x[0, parents[0].long(), tokens[0].long()].tolist() == [row[7 - i // W].item() for i in range(k)]
