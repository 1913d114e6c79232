"""The paged cache's pages on the GPU - taken, forked, freed, copied, compacted - against plain
lists (blocks_ref.py), and beam selection against 64 bits."""
import math

import pytest
import torch

import blocks_ref as br
from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_blocks import DEV, filled_cache, gen, ints

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


def u8(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def everything(cache, keys):
    return [u8(t) for t in list(cache) + list(keys) if t is not None]


def filled_keys(g, n_pages, kvh, hd):
    return ds41.BlockKeys(torch.randint(-127, 128, (n_pages, kvh, hd), generator=g, device=DEV).to(torch.int8),
                          torch.rand(n_pages, kvh, generator=g, device=DEV))


def copied(cache, keys, copies):
    """The tensors after the copies (src, dst, rows)."""
    out = [t.clone() for t in everything(cache, keys)]
    n_cache = len(out) - 2
    for s, d, rows in copies:
        for i, t in enumerate(out):
            if i < n_cache:
                t[d, :, :rows] = t[s, :, :rows]
            else:
                t[d] = t[s]
    return out


def pool(g, lens, page, spare, shared=True):
    """Sequences whose first whole pages are partly shared: refs, rows of the table."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).tolist()
    width = max(max(need, default=0), 1) + 1
    rows, at, refs = [], 0, [0] * (sum(need) + spare)
    for b, n in enumerate(need):
        row = order[at:at + n]
        at += n
        if shared and b % 2 and rows:  # as the sequence before, as far as both are full
            m = min(lens[b] // page, lens[b - 1] // page, 3)
            row[:m] = rows[-1][:m]
        rows.append(row + [-9] * (width - n))
        for p in row:
            refs[p] += 1
    return refs, rows


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("replace", [False, True])
@pytest.mark.parametrize("lens,n,kvh,hd,page,spare", [
    ([1], 1, 1, 16, 16, 2), ([40, 41, 16, 0, 33], 9, 3, 80, 16, 12), ([300, 130], 40, 2, 128, 64, 45),
    ([64, 128, 64], 5, 8, 64, 64, 0), ([255, 257], 3, 1, 96, 256, 4), ([17] * 50, 1500, 1, 32, 16, 1600)])
def test_fork(lens, n, kvh, hd, page, spare, replace, e4m3):
    g = gen(sum(lens) + n)
    refs, rows = pool(g, lens, page, spare)
    parents = torch.randint(0, len(lens), (n,), generator=g, device=DEV).tolist()
    if n > 4:
        parents[2] = -1
    cache, keys = filled_cache(g, len(refs), kvh, page, hd, e4m3), filled_keys(g, len(refs), kvh, hd)
    w_refs, w_table, w_lens, copies = br.fork(refs, rows, lens, parents, page, replace)
    want = copied(cache, keys, copies)
    r, t = ints(refs), ints(rows)
    table, out_lens = ds41.kv_pages_fork(cache, r, t, ints(lens), ints(parents), replace=replace, keys=keys)
    assert table.tolist() == w_table and out_lens.tolist() == w_lens and r.tolist() == w_refs
    assert t.tolist() == rows
    for a, b in zip(everything(cache, keys), want):
        assert torch.equal(a, b)
    ds41.kv_pages_free(r, table, out_lens, page)
    if not replace:
        assert r.tolist() == refs
    else:
        assert r.tolist() == [0] * len(refs)


def test_fork_without_pages_left():
    g = gen(1)
    refs, rows = pool(g, [20, 35], 16, 1, shared=False)
    cache = filled_cache(g, len(refs), 1, 16, 32, True)
    r = ints(refs)
    table, lens = ds41.kv_pages_fork(cache, r, ints(rows), ints([20, 35]), ints([1, 0, 1]))
    assert ds41.device_status() == 7
    free = refs.index(0)
    assert table.tolist() == [rows[1][:2] + [free, -1], [rows[0][0], -1, -1, -1], rows[1][:2] + [-1, -1]]
    assert lens.tolist() == [35, 20, 35]
    assert r.tolist() == [2 if p == rows[0][0] else 3 if p in rows[1][:2] else 1 for p in range(len(refs))]


def test_fork_reports_what_is_wrong():
    g = gen(2)
    refs, rows = pool(g, [20, 35], 16, 6, shared=False)
    cache = filled_cache(g, len(refs), 1, 16, 32, True)
    r = ints(refs)
    table, lens = ds41.kv_pages_fork(cache, r, ints(rows), ints([20, 10 ** 6]), ints([2, 1, -5, -1]))
    assert ds41.device_status() == 4
    assert table.tolist() == [[-1] * 4] * 4 and lens.tolist() == [0] * 4 and r.tolist() == refs
    rows[0][0] = len(refs)
    table, lens = ds41.kv_pages_fork(cache, r, ints(rows), ints([20, 35]), ints([0]))
    assert ds41.device_status() == 4
    assert table.tolist() == [[-1, refs.index(0), -1, -1]]


@pytest.mark.parametrize("lens,new,page", [
    ([0], [1], 16), ([16, 15, 0, 40], [17, 16, 0, 40], 16), ([5, 100], [300, 90], 64), ([1] * 1500, [40] * 1500, 16)])
def test_take_and_free(lens, new, page):
    g = gen(len(lens))
    width = max(-(-max(n, m) // page) for n, m in zip(lens, new)) + 1
    refs, rows = pool(g, lens, page, 3 + sum(max(0, -(-m // page) - -(-n // page)) for n, m in zip(lens, new)), False)
    rows = [(r + [-9] * width)[:width] for r in rows]
    r, t = ints(refs), ints(rows)
    p = br.Pool(refs)
    if len(lens) > 1000:  # (the plain list looks from the start each time)
        free = iter([i for i, x in enumerate(refs) if x == 0])
        p.take = lambda: next(free)
    want = [list(x) for x in rows]
    for b, (n, m) in enumerate(zip(lens, new)):
        for x in range(-(-n // page), -(-m // page)):
            want[b][x] = p.take()
            p.refs[want[b][x]] = 1
    ds41.kv_pages_take(r, t, ints(lens), ints(new), page)
    assert t.tolist() == want and r.tolist() == p.refs
    most = [max(n, m) for n, m in zip(lens, new)]
    ds41.kv_pages_free(r, t, ints(most), page)
    assert r.tolist() == [0] * len(refs)
    if max(most):
        ds41.kv_pages_free(r, t, ints(most), page)
        assert ds41.device_status() == 4
        assert r.tolist() == [0] * len(refs)


def test_take_from_a_large_pool_that_runs_out():
    g = gen(5)
    n = 30011
    refs = torch.randint(0, 3, (n,), generator=g, device=DEV, dtype=torch.int32)
    free = torch.nonzero(refs == 0)[:, 0].tolist()
    B, width = 700, 64
    table = torch.full((B, width), -9, dtype=torch.int32, device=DEV)
    need = torch.randint(0, width + 1, (B,), generator=g, device=DEV)
    ds41.kv_pages_take(refs, table, torch.zeros(B, dtype=torch.int32, device=DEV), (need * 16).int(), 16)
    assert ds41.device_status() == 7
    it = iter(free)
    want = [[next(it, -1) if x < m else -9 for x in range(width)] for m in need.tolist()]
    assert table.tolist() == want
    assert bool((refs > 0).all())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("P,kvh,hd,page,live", [
    (1, 1, 16, 16, 1.0), (2, 1, 16, 16, 0.5), (40, 3, 80, 16, 0.0), (300, 2, 128, 64, 0.3), (9000, 1, 16, 16, 0.6),
    (70, 8, 96, 32, 0.9)])
def test_compact(P, kvh, hd, page, live, e4m3):
    g = gen(P)
    used = torch.randperm(P, generator=g, device=DEV).tolist()[:int(P * live)]
    refs, rows, lens, at = [0] * P, [], [], 0
    width = 8
    while at < len(used):
        n = min(len(used) - at, len(rows) % 7 + 1)
        rows.append(used[at:at + n] + [-9] * (width - n))
        lens.append(n * page - len(rows) % page)
        for p in used[at:at + n]:
            refs[p] += 1
        at += n
    if len(rows) > 2:  # a page of two sequences
        rows[1][0] = rows[0][0]
        refs[rows[0][0]] += 1
    cache, keys = filled_cache(g, P, kvh, page, hd, e4m3), filled_keys(g, P, kvh, hd)
    w_refs, w_rows, w_live, moves = br.compact(refs, rows, lens, page)
    want = copied(cache, keys, [(s, d, page) for s, d in moves])
    r = ints(refs)
    t = ints(rows) if rows else torch.zeros(0, width, dtype=torch.int32, device=DEV)
    L = ints(lens) if lens else torch.zeros(0, dtype=torch.int32, device=DEV)
    got = ds41.kv_pages_compact(cache, r, t, L, keys=keys)
    assert got.tolist() == [w_live] and r.tolist() == w_refs and t.tolist() == w_rows
    for a, b in zip(everything(cache, keys), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("n,kvh,hd,page", [(1, 1, 16, 16), (7, 3, 80, 32), (300, 2, 128, 256)])
def test_copy(n, kvh, hd, page, e4m3):
    g = gen(n)
    P = 2 * n + 3
    order = torch.randperm(P, generator=g, device=DEV).tolist()
    src, dst = order[:n], order[n:2 * n]
    rows = torch.randint(0, page + 1, (n,), generator=g, device=DEV).tolist()
    cache, keys = filled_cache(g, P, kvh, page, hd, e4m3), filled_keys(g, P, kvh, hd)
    if n > 3:
        src[1], dst[2] = -1, -1
    for r in (rows, None):
        want = copied(cache, keys, [(s, d, page if r is None else r[i]) for i, (s, d) in enumerate(zip(src, dst))
                                    if s >= 0 and d >= 0])
        ds41.kv_pages_copy(cache, ints(src), ints(dst), rows=None if r is None else ints(r), keys=keys)
        for a, b in zip(everything(cache, keys), want):
            assert torch.equal(a, b)
    want = [t.clone() for t in everything(cache, keys)]
    for s, d, r in ((P, 0, 1), (0, P, 1), (-2, 1, 1), (0, 1, page + 1), (0, 1, -1)):
        ds41.kv_pages_copy(cache, ints([s]), ints([d]), rows=ints([r]), keys=keys)
        assert ds41.device_status() == 4
    for a, b in zip(everything(cache, keys), want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Beam search
# ---------------------------------------------------------------------------
def check_beam(x, scores, k, ended=None, end_token=0):
    """Parents and tokens equal, scores to the roundings: the sum of V terms in f32 (each thread at
    most V / 256 in a row and a tree above: V / 256 + 16 roundings of 2^-24, plus the exponential's 2^-21)
    shifts every offer of a beam alike, and the result is rounded to f32."""
    got = [t.tolist() for t in ds41.beam_select(x, scores, k, ended=ended, end_token=end_token)]
    want = br.beam(x, scores, k, ended, end_token)
    tol = (x.shape[2] / 256 + 16) * 2.0 ** -24 + 2.0 ** -20
    for b, w in enumerate(want):
        m = len(w)
        assert got[1][b] == [o[1] for o in w] + [-1] * (k - m), b
        assert got[2][b] == [o[2] for o in w] + [-1] * (k - m), b
        for a, o in zip(got[0][b], w):
            assert abs(a - o[0]) <= tol + 2.0 ** -23 * abs(o[0])
        assert got[0][b][m:] == [-math.inf] * (k - m)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,k", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 37, 6), (1, 4, 32000, 8), (3, 5, 4097, 10), (2, 16, 8192, 32),
    (1, 2, 70001, 128), (40, 8, 1000, 16), (1, 1, 160000, 1)])
def test_beam(B, W, V, k, dtype):
    g = gen(V + k)
    x = (torch.randn(B, W, V, generator=g, device=DEV) * 3).to(dtype)
    scores = -(torch.rand(B, W, generator=g, device=DEV) * 2).cumsum(1)
    check_beam(x, scores, k)
    ended = torch.rand(B, W, generator=g, device=DEV) < 0.4
    check_beam(x, scores, k, ended, V - 1)
    # a slice of wider rows, one that does not begin on 16 bytes
    wide = torch.randn(B, W, V + 9, generator=g, device=DEV).to(dtype)
    check_beam(wide[:, :, 3:3 + V], scores, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_equal_and_missing(dtype):
    g = gen(4)
    B, W, V, k = 2, 3, 9001, 20
    scores = torch.zeros(B, W, device=DEV)
    x = torch.zeros(B, W, V, device=DEV, dtype=dtype)
    check_beam(x, scores, k)                       # all alike: the lowest
    x[:, :, 5000:] = 1.0
    check_beam(x, scores, k)
    x[:] = -math.inf
    x[0, 1, 77], x[0, 1, 8000], x[1, 2, 9000] = 1.0, 1.0, -2.0
    check_beam(x, scores, k)                       # three offers in all
    x = (torch.randn(B, W, V, generator=g, device=DEV) * 100).to(dtype)
    x[0, 0, 3], x[0, 1, 8999], x[1, 1, 4] = math.nan, math.inf, -0.0
    x[1, 0] = 0.0
    x[1, 0, ::2] = -0.0
    scores[1, 2] = -math.inf
    check_beam(x, scores, k)
    scores[0, 2], scores[1, 0] = math.nan, math.inf
    check_beam(x, scores, k)
    x = torch.arange(V, device=DEV).to(dtype).expand(B, W, V).contiguous() / 64  # rising
    check_beam(x, torch.zeros(B, W, device=DEV), k)
    check_beam(-x, torch.zeros(B, W, device=DEV), k)


def test_beam_search_over_pages():
    """Beams go on over forked pages: a step's selection drives the fork, and every beam's
    rows are what a search on whole copies of its rows has."""
    g = gen(6)
    B, W, V, page, kvh, hd = 3, 4, 300, 16, 2, 32
    n0 = [20, 33, 16]
    P = 3 * W * 6 + 4
    cache, refs = filled_cache(g, P, kvh, page, hd, True), torch.zeros(P, dtype=torch.int32, device=DEV)
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    lens = ints(n0)
    ds41.kv_pages_take(refs, table, torch.zeros_like(lens), lens, page)
    start = table.clone()
    table, lens = ds41.kv_pages_fork(cache, refs, table, lens, ints([b for b in range(B) for _ in range(W)]))
    ds41.kv_pages_free(refs, start, ints(n0), page)
    scores = torch.full((B, W), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    store = {}
    history = [[] for _ in range(B * W)]
    for step in range(9):
        x = torch.randn(B, W, V, generator=g, device=DEV) * 2
        scores, parents, tokens = ds41.beam_select(x, scores, W)
        flat = parents.view(-1)
        table, lens = ds41.kv_pages_fork(cache, refs, table, lens, flat, replace=True)
        new = lens + 1
        ds41.kv_pages_take(refs, table, lens, new, page)
        pos = lens.long()
        slots = torch.gather(table.long(), 1, (pos // page)[:, None])[:, 0] * page + pos % page
        k = torch.randn(B * W, kvh, hd, generator=g, device=DEV).bfloat16()
        ds41.kv_cache_write(cache, k, k, slots)
        lens = new
        history = [history[p] + [(step, i)] for i, p in enumerate(flat.tolist())]
        one = ds41.make_kv_cache(B * W, kvh, page, hd)
        ds41.kv_cache_write(one, k, k, torch.arange(B * W, device=DEV) * page)
        for i in range(B * W):
            store[step, i] = u8(one.k)[i, :, 0]
        ends = [0] + lens.cumsum(0).tolist()
        got = u8(cache.k)
        for i in range(B * W):
            n = int(lens[i])
            rows = got[table[i, :-(-n // page)].long()].transpose(1, 2).flatten(0, 1)[:n]
            base = got[start[i // W, :-(-n0[i // W] // page)].long()]
            assert n == n0[i // W] + step + 1 and ends[-1] > 0 and base.numel()
            for s, at in history[i]:
                assert torch.equal(rows[n0[i // W] + s], store[s, at])
        held = [p for i in range(B * W) for p in table[i, :-(-int(lens[i]) // page)].tolist()]
        assert refs.tolist() == [held.count(p) for p in range(P)]
    ds41.kv_pages_free(refs, table, lens, page)
    assert int(refs.sum()) == 0
