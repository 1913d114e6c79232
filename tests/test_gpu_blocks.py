"""Attention over selected blocks of the paged cache on the GPU: block keys and picks equal to
the definition's, attention against 64 bits (blocks_ref.py)."""
import math

import pytest
import torch

import blocks_ref as br
import dense_ref as ref
from compressed_sparse_attention_window_gb300 import ds41

pytestmark = pytest.mark.gpu

DEV = "cuda"


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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cu(lens):
    return ints([0] + torch.tensor(lens).cumsum(0).tolist())


def filled_cache(g, n_pages, kvh, page, hd, e4m3):
    k, v = randn(g, n_pages, kvh, page, hd), randn(g, n_pages, kvh, page, hd)
    if not e4m3:
        return ds41.KvCache(k, v)
    (kc, ks), (vc, vs) = ref.quantise(k), ref.quantise(v)
    return ds41.KvCache(kc, vc, ks, vs)


def tables(g, lens, page, spare=3):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).tolist()
    width = max(max(need), 1) + 1
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-7] * (width - n))  # never looked at
        at += n
    return sum(need) + spare, rows


def sequence(cache, row, n, page):
    """k, v [n, kvh, hd] and v's scales [n, kvh] of a sequence, in 64 bits."""
    if n == 0:
        kvh, hd = cache.k.shape[1], cache.k.shape[3]
        z = torch.zeros(0, kvh, hd, dtype=torch.float64, device=DEV)
        return z, z, None
    at = torch.tensor(row[:-(-n // page)], device=DEV)
    k = ref.values(cache.k[at], None if cache.k_scales is None else cache.k_scales[at])
    v = ref.values(cache.v[at], None if cache.v_scales is None else cache.v_scales[at])
    vs = None if cache.v_scales is None else cache.v_scales[at].transpose(1, 2).flatten(0, 1)[:n]
    return k.transpose(1, 2).flatten(0, 1)[:n], v.transpose(1, 2).flatten(0, 1)[:n], vs


# ---------------------------------------------------------------------------
# Block keys
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("lens,starts,kvh,hd,page", [
    ([1], None, 1, 16, 16), ([16, 0, 33], None, 3, 80, 16), ([130, 64, 257], [129, 0, 200], 2, 128, 64),
    ([300, 17, 256], [300, 3, 255], 8, 64, 256), ([100, 31], [40, 30], 5, 96, 32)])
def test_block_keys(lens, starts, kvh, hd, page, e4m3):
    """Codes and scales bit for bit; other pages' as they were."""
    g = gen(sum(lens) + hd)
    n_pages, rows = tables(g, lens, page)
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    if lens[0] > 20:  # rows that a key could go wrong on
        cache.k.view(torch.uint8 if e4m3 else torch.bfloat16)[rows[0][0], 0] = 0
        if e4m3:
            cache.k_scales[rows[0][1], 0, 1] = math.nan
        else:
            cache.k[rows[0][1], 0, 1, 3] = math.inf
    keys = ds41.BlockKeys(torch.randint(-127, 128, (n_pages, kvh, hd), generator=g, device=DEV).to(torch.int8),
                          torch.rand(n_pages, kvh, generator=g, device=DEV))
    want = [t.clone() for t in keys]
    st = starts or [0] * len(lens)
    for b, n in enumerate(lens):
        for i in range(st[b] // page, -(-n // page)) if st[b] < n else ():
            for h in range(kvh):
                m = min(page, n - i * page)
                c, s = br.block_key(br.key_rows(cache, rows[b][i], h)[:m])
                want[0][rows[b][i], h], want[1][rows[b][i], h] = c.to(torch.int8), s
    ds41.kv_block_keys(cache, keys, ints(rows), ints(lens), max(n - s for n, s in zip(lens, st)),
                       starts=None if starts is None else ints(starts))
    assert torch.equal(keys.codes, want[0])
    assert torch.equal(keys.scales.nan_to_num(nan=-1.0), want[1].nan_to_num(nan=-1.0))


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------
SELECT = [
    # lens, new tokens, nh, kvh, hd, page, topk, first, local
    ([1], [1], 1, 1, 16, 16, 1, 0, 1),
    ([700, 33, 5000], [1, 1, 1], 8, 2, 128, 16, 12, 1, 2),
    ([300, 0, 90, 17], [40, 0, 3, 17], 12, 4, 64, 16, 5, 1, 2),
    ([513], [513], 10, 2, 80, 32, 6, 0, 1),
    ([2000], [37], 64, 1, 96, 16, 33, 2, 3),
    ([400], [5], 7, 7, 32, 64, 1024, 1, 2),
    ([260, 255], [200, 255], 4, 4, 128, 256, 1, 0, 1),
    ([9000], [33], 16, 4, 128, 16, 64, 1, 2),
]


@pytest.mark.parametrize("lens,news,nh,kvh,hd,page,topk,first,local", SELECT)
def test_select(lens, news, nh, kvh, hd, page, topk, first, local):
    g = gen(sum(lens))
    n_pages, rows = tables(g, lens, page)
    keys = ds41.BlockKeys(torch.randint(-127, 128, (n_pages, kvh, hd), generator=g, device=DEV).to(torch.int8),
                          torch.rand(n_pages, kvh, generator=g, device=DEV) + 0.01)
    keys.scales[:, 0] = keys.scales[0, 0]
    if n_pages > 8:  # equal scores, a block that does not count
        keys.codes[rows[0][3], 0] = keys.codes[rows[0][2], 0]
        keys.scales[rows[0][1], 0] = math.nan
    q = randn(g, sum(news) + 2, nh, hd)
    if sum(news) > 4:
        q[1], q[2, 0, 0], q[3] = 0.0, math.inf, math.nan
    c = cu(news)
    got = torch.full((sum(news) + 2, kvh, topk), -5, dtype=torch.int32, device=DEV)
    ds41.block_select(q, keys, page, ints(rows), ints(lens), c, max(news), max(lens), topk, first, local, idx=got)
    assert bool((got[sum(news):] == -5).all())  # behind the last sequence
    got = got.tolist()
    codes, scales = keys.codes.double(), keys.scales.double()
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        mine = torch.tensor(rows[b][:-(-n // page)], device=DEV, dtype=torch.long)
        for i in range(m):
            for h in range(kvh):
                w = br.picks(q[at + i, h * nh // kvh:(h + 1) * nh // kvh], codes[mine, h], scales[mine, h],
                             n - m + i, page, topk, first, local)
                assert got[at + i][h] == w + [-1] * (topk - len(w)), (b, i, h)
        at += m


def test_select_equal_scores():
    """All blocks alike: the lowest ones; strided queries; few scores of many values."""
    g = gen(3)
    n, page, kvh, hd, topk = 1024, 16, 2, 64, 9
    _, rows = tables(g, [n], page, 0)
    keys = ds41.make_block_keys(64, kvh, hd)
    keys.codes.fill_(1)
    keys.scales.fill_(1.0)
    qkv = randn(g, 3, 12, hd)
    got = ds41.block_select(qkv[:, :4], keys, page, ints(rows), ints([n]), cu([3]), 3, n, topk, 1, 2)
    assert got[0, 0].tolist() == list(range(7)) + [62, 63]
    assert bool((got == got[0, 0]).all())


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def random_lists(g, lens, news, kvh, page, topk):
    """idx [T, kvh, topk] and lists[t][h]: some full, some short, some empty, own block or
    not."""
    T = sum(news)
    r = torch.rand(T, kvh, generator=g, device=DEV).tolist()
    out, lists, t = [], [], 0
    for n, m in zip(lens, news):
        for i in range(m):
            cur = (n - m + i) // page
            rows = []
            for h in range(kvh):
                take = min(topk, cur + 1)
                if r[t][h] < 0.1:
                    take = 0
                elif r[t][h] < 0.3:
                    take = (take + 1) // 2
                x = torch.randperm(cur + 1, generator=g, device=DEV)[:take].tolist()
                if take and r[t][h] > 0.4 and cur not in x:
                    x[0] = cur
                rows.append(sorted(x))
            lists.append(rows)
            t += 1
    idx = [[x + [-1] * (topk - len(x)) for x in rows] for rows in lists]
    # behind the first -1 anything may stand
    idx = [[x if len(x) < 3 or x[-2] != -1 else x[:-1] + [5] for x in rows] for rows in idx]
    return ints(idx) if T else torch.zeros(0, kvh, topk, dtype=torch.int32, device=DEV), lists


TOKENS = [
    # lens, new tokens, nh, kvh, hd, page, topk, sink
    ([1], [1], 1, 1, 16, 16, 1, False),
    ([700, 33, 5000], [1, 1, 1], 8, 2, 128, 16, 12, True),
    ([300, 0, 90, 17], [4, 0, 3, 17], 12, 4, 64, 16, 5, False),
    ([513], [3], 40, 2, 80, 32, 6, True),
    ([2000, 1999], [2, 1], 64, 1, 96, 64, 33, False),
    ([3000], [1], 16, 8, 128, 64, 40, True),
    ([260, 255], [2, 5], 4, 4, 128, 256, 2, False),
    ([900] * 40, [1] * 40, 32, 8, 128, 64, 14, True),
]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("lens,news,nh,kvh,hd,page,topk,with_sink", TOKENS)
def test_tokens(lens, news, nh, kvh, hd, page, topk, with_sink, e4m3):
    g = gen(sum(lens) + topk)
    n_pages, rows = tables(g, lens, page)
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    idx, lists = random_lists(g, lens, news, kvh, page, topk)
    for b, n in enumerate(lens):  # rows behind the end may hold anything
        if n % page:
            at = rows[b][n // page]
            if e4m3:
                cache.k_scales[at, :, n % page:] = math.nan
                cache.v_scales[at, :, n % page:] = math.inf
            else:
                cache.k[at, :, n % page:] = math.nan
                cache.v[at, :, n % page:] = math.inf
    q = randn(g, sum(news) + 1, nh, hd)
    sink = torch.randn(nh, generator=g, device=DEV) if with_sink else None
    o = torch.full_like(q, 7.0)
    lse = torch.full((sum(news) + 1, nh), 7.0, device=DEV)
    full = torch.cat([idx, idx.new_full((1, kvh, topk), -1)])
    scale = hd ** -0.5
    ds41.block_attn_fwd(q, cache, ints(rows), ints(lens), cu(news), max(news), full, scale, sink=sink, o=o, lse=lse)
    assert bool((o[-1] == 7).all()) and bool((lse[-1] == 7).all())
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v, vs = sequence(cache, rows[b], n, page)
        w = br.attend(q[at:at + m], k, v, lists[at:at + m], n - m, page, scale, sink, vs)
        if m:
            ref.close(o[at:at + m], lse[at:at + m], *w)
        at += m


PROMPTS = [
    # queries, earlier rows, nh, kvh, hd, block, topk, sink
    ([1], 0, 1, 1, 16, 16, 1, False),
    ([5, 0, 130, 1], 0, 8, 2, 128, 16, 4, True),
    ([300, 77], 0, 12, 4, 64, 32, 5, False),
    ([257], 100, 10, 2, 80, 64, 3, True),
    ([40], 1000, 64, 1, 96, 64, 9, False),
    ([130], 700, 4, 4, 128, 128, 3, True),
    ([90], 1000, 5, 1, 128, 256, 2, False),
    ([33], 300, 256, 1, 64, 16, 8, True),
    ([600], 0, 2, 2, 128, 16, 6, False),
]


@pytest.mark.parametrize("lens,prior,nh,kvh,hd,block,topk,with_sink", PROMPTS)
def test_prompt(lens, prior, nh, kvh, hd, block, topk, with_sink):
    g = gen(sum(lens) + topk)
    lens_k = [n + prior if n else 0 for n in lens]
    Tq, Tk = sum(lens), sum(lens_k)
    idx, lists = random_lists(g, lens_k, lens, kvh, block, topk)
    q = randn(g, Tq + 1, nh, hd)
    kv = randn(g, Tk + 3, 2 * kvh, hd)  # (strided)
    k, v = kv[:, :kvh], kv[:, kvh:]
    kv[Tk:] = math.nan  # nobody's
    sink = torch.randn(nh, generator=g, device=DEV) if with_sink else None
    o = torch.full_like(q, 7.0)
    lse = torch.full((Tq + 1, nh), 7.0, device=DEV)
    full = torch.cat([idx, idx.new_full((1, kvh, topk), -1)])
    scale = hd ** -0.5
    ds41.block_prompt_attn_fwd(q, k, v, cu(lens), cu(lens_k), max(lens), max(lens_k), full, block, scale, sink=sink,
                               o=o, lse=lse)
    assert bool((o[-1] == 7).all()) and bool((lse[-1] == 7).all())
    at = at_k = 0
    for n, m in zip(lens, lens_k):
        w = br.attend(q[at:at + n], k[at_k:at_k + m].double(), v[at_k:at_k + m].double(), lists[at:at + n], m - n,
                      block, scale, sink)
        if n:
            ref.close(o[at:at + n], lse[at:at + n], *w)
        at, at_k = at + n, at_k + m


def test_lists_that_break_the_rules_end():
    """An entry that does not rise, or lies past the token, ends its list and is reported; a
    page outside the cache is not seen."""
    g = gen(9)
    n, page, kvh, hd = 100, 16, 1, 64
    n_pages, rows = tables(g, [n], page)
    cache = filled_cache(g, n_pages, kvh, page, hd, False)
    q = randn(g, 1, 4, hd)
    k, v, _ = sequence(cache, rows[0], n, page)
    for idx, seen in (([1, 1, 3], [1]), ([2, 1, 3], [2]), ([0, 7, 3], [0]), ([0, -2, 3], [0]), ([9, 1, 2], [])):
        w = br.attend(q, k, v, [[seen]], n - 1, page, 0.1, None)
        o, lse = torch.empty_like(q), torch.empty(1, 4, device=DEV)
        i = ints([[idx]])
        ds41.block_attn_fwd(q, cache, ints(rows), ints([n]), cu([1]), 1, i, 0.1, o=o, lse=lse)
        assert ds41.device_status() == 4
        ref.close(o, lse, *w)
        ds41.block_prompt_attn_fwd(q, k.bfloat16(), v.bfloat16(), cu([1]), cu([n]), 1, n, i, page, 0.1, o=o, lse=lse)
        assert ds41.device_status() == 4
        ref.close(o, lse, *w)
    bad = [list(rows[0])]
    bad[0][2] = n_pages
    w = br.attend(q, k, v, [[[1, 6]]], n - 1, page, 0.1, None)
    ds41.block_attn_fwd(q, cache, ints(bad), ints([n]), cu([1]), 1, ints([[[1, 2, 6]]]), 0.1, o=o, lse=lse)
    assert ds41.device_status() == 4
    ref.close(o, lse, *w)


def test_sequences_that_break_their_limits_are_skipped():
    g = gen(10)
    page, kvh, hd = 16, 2, 64
    lens, news = [40, 50], [2, 3]
    n_pages, rows = tables(g, lens, page)
    cache = filled_cache(g, n_pages, kvh, page, hd, True)
    keys = ds41.make_block_keys(n_pages, kvh, hd)
    q = randn(g, 5, 4, hd)
    idx = ints([[[0, 1]] * kvh] * 5)
    for bad_lens, c in (([1, 50], [0, 2, 5]), ([10 ** 6, 50], [0, 2, 5]), ([40, 50], [-3, 2, 5]), ([40, 50], [4, 2, 5])):
        o = torch.full_like(q, 7.0)
        ds41.block_attn_fwd(q, cache, ints(rows), ints(bad_lens), ints(c), 3, idx, 0.1, o=o)
        assert ds41.device_status() == 4
        assert bool((o[:2] == 7).all()) and not bool((o[2:] == 7).any())
        got = torch.full((5, kvh, 4), -5, dtype=torch.int32, device=DEV)
        ds41.block_select(q, keys, page, ints(rows), ints(bad_lens), ints(c), 3, 64, 4, idx=got)
        assert ds41.device_status() == 4
        assert bool((got[:2] == -5).all()) and not bool((got[2:] == -5).any())
    ds41.kv_block_keys(cache, keys, ints(rows), ints([40, 10 ** 6]), 64)
    assert ds41.device_status() == 4
    ds41.kv_block_keys(cache, keys, ints(rows), ints(lens), 8, starts=ints([32, 41]))
    assert ds41.device_status() == 4
    k = randn(g, 90, kvh, hd)
    for cq, ck in (([0, 2, 5], [0, 1, 51]), ([0, 2, 5], [0, 60, 110]), ([0, 2, 5], [-1, 40, 90])):
        o = torch.full_like(q, 7.0)
        ds41.block_prompt_attn_fwd(q, k, k, ints(cq), ints(ck), 3, 50, idx, page, 0.1, o=o)
        assert ds41.device_status() == 4
        assert bool((o[:2] == 7).all())


def test_the_run_of_a_step():
    """Rows written, keys brought up to date, blocks picked and attended to, as a captured
    graph: the same bits as eagerly, and close to attention over all rows when all are
    picked."""
    g = gen(11)
    page, kvh, hd, nh, B = 16, 2, 64, 8, 5
    lens = [int(x) for x in torch.randint(30, 200, (B,), generator=g, device=DEV)]
    n_pages, rows = tables(g, [n + 4 for n in lens], page)
    cache = filled_cache(g, n_pages, kvh, page, hd, True)
    keys = ds41.make_block_keys(n_pages, kvh, hd)
    table, L = ints(rows), ints(lens)
    ds41.kv_block_keys(cache, keys, table, L, 200)
    q, k, v = (torch.zeros(B, h, hd, dtype=torch.bfloat16, device=DEV) for h in (nh, kvh, kvh))
    c = cu([1] * B)
    one = torch.ones_like(L)

    def step(lse):
        L.add_(1)
        p = L.long() - 1
        slots = torch.gather(table.long(), 1, (p // page)[:, None])[:, 0] * page + p % page
        ds41.kv_cache_write(cache, k, v, slots)
        ds41.kv_block_keys(cache, keys, table, L, 1, starts=L - one)
        idx = ds41.block_select(q, keys, page, table, L, c, 1, 256, 6)
        return idx, ds41.block_attn_fwd(q, cache, table, L, c, 1, idx, 0.125, lse=lse)

    lse = torch.empty(B, nh, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(lse)
    torch.cuda.current_stream().wait_stream(side)
    L.copy_(ints(lens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, o = step(lse)
    L.copy_(ints(lens))
    saved = [t.clone() for t in cache if t is not None] + [t.clone() for t in keys]
    for s in range(3):
        x = randn(g, B, nh + 2 * kvh, hd)
        q.copy_(x[:, :nh]), k.copy_(x[:, nh:nh + kvh]), v.copy_(x[:, nh + kvh:])
        graph.replay()
        torch.cuda.synchronize()
        got = [idx.clone(), o.clone(), lse.clone()] + [t.clone() for t in cache] + [t.clone() for t in keys]
        for t, w in zip([t for t in cache] + list(keys), saved):
            t.copy_(w)
        L.sub_(1)
        idx2, o2 = step(lse)
        for a, b in zip(got, [idx2, o2, lse] + [t for t in cache] + list(keys)):
            assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                               b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
        saved = [t.clone() for t in cache if t is not None] + [t.clone() for t in keys]
    every = ds41.block_select(q, keys, page, table, L, c, 1, 256, 20)
    o3 = ds41.block_attn_fwd(q, cache, table, L, c, 1, every, 0.125)
    o4 = ds41.tree_attn_fwd(q, cache, table, L, c, 1, 256, 0.125)
    assert (o3.float() - o4.float()).abs().max() < 2e-2
