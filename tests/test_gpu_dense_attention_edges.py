"""The dense attention and its cache where inputs are unusual but allowed, on the
GPU: what earlier users left in a page, value rows of very different sizes, pages
that have left the window, prefix sums that do not start at 0, the largest window.

Against the definitions in 64 bits (dense_ref.py, where the tolerances are derived).
"""
import math

import pytest
import torch

import dense_ref as ref
from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_dense_attention import (DEV, _clean_status, _cuda, cu, filled_cache, gen, randn,
                                      words_of)

pytestmark = pytest.mark.gpu

# drafted tokens, query heads, key/value heads: 1 to 16 rows per key/value head,
# 17 to 128, more
FEW, MIDDLING, MANY = (2, 8, 2), (9, 16, 2), (20, 16, 1)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def packed_cache(k, v, page, e4m3, spare=2, seed=0):
    """k, v [n, kvh, hd] of one sequence in a cache of pages in no order: the cache,
    its table [1, pages]; rows and pages that are not the sequence's are zero."""
    n, kvh, hd = k.shape
    need = -(-n // page)
    order = torch.randperm(need + spare, generator=torch.Generator().manual_seed(seed))[:need]
    cache = ds41.make_kv_cache(need + spare, kvh, page, hd, e4m3)
    pos = torch.arange(n)
    ds41.kv_cache_write(cache, k, v, (order[pos // page] * page + pos % page).to(DEV))
    return cache, order.int().to(DEV).view(1, need)


def rows_of(cache, table, n):
    """The sequence's rows as 64-bit values and the scales of v."""
    pages = table[0, :-(-n // cache.k.shape[2])].long()
    k, v = (ref.values(c, s)[pages].transpose(1, 2).flatten(0, 1)[:n]
            for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)))
    vs = cache.v_scales
    return k, v, None if vs is None else vs[pages].transpose(1, 2).flatten(0, 1)[:n]


def attend(q, cache, table, n, bits=None, window=0, sink=None):
    d, nh = q.shape[:2]
    mask = None
    if bits is not None:
        mask = torch.tensor(words_of(bits, -(-d // 64)), dtype=torch.int64, device=DEV)
    lse = torch.empty(d, nh, device=DEV)
    o = ds41.tree_attn_fwd(q, cache, table, i32([n]), cu([d]), d, n, q.shape[2] ** -0.5, mask=mask,
                           sink=sink, window=window, lse=lse)
    return o, lse


# ---------------------------------------------------------------------------
# Rows behind a sequence's end
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("left", [2.0 ** 12, 2.0 ** 20, 1e30, torch.finfo(torch.float32).max,
                                  math.inf, math.nan])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
@pytest.mark.parametrize("n", [21, 700, 1001])
def test_rows_behind_the_end_are_not_used(n, shape, left):
    """Whatever scales, codes (NaN among them) and values an earlier user left there:
    the outputs are those of a cache with zeros there."""
    d, nh, kvh = shape
    page, hd = 64, 128
    g = gen(n + d)
    k, v, q = randn(g, n, kvh, hd), randn(g, n, kvh, hd), randn(g, d, nh, hd)
    for e4m3 in (True, False):
        cache, table = packed_cache(k, v, page, e4m3)
        kx, vx, vs = rows_of(cache, table, n)
        want = ref.attend(q, kx, vx, ref.tree_visible(d, n, None, 0, DEV), hd ** -0.5, None, vs)
        last = int(table[0, -1])
        for t in cache:
            if t is None:
                continue
            rows = t[last, :, n % page:]
            if t.dtype == torch.float8_e4m3fn:
                rows.view(torch.uint8).random_(0, 256, generator=g)
            else:
                rows.fill_(min(left, torch.finfo(t.dtype).max) if left < math.inf else left)
        ref.close(*attend(q, cache, table, n), *want)


# ---------------------------------------------------------------------------
# Value rows of very different sizes (e4m3)
# ---------------------------------------------------------------------------
# Here a row's weights are charged with their own sizes.  The weights p_j vs_j of an
# e4m3 cache are rounded to f16 in a unit that brings the largest of the keys that the
# row sees to 2^8 at least, so what f16's smallest step of 2^-24 adds is half of it,
# 2^-25, times 2^-8 of that largest weight, for every code: 2^-33 max_j(p_j vs_j)
# sum_j |code_j|; and no unit is below 2^-96 of the largest p_j: 2^-121 p_max sum_j
# |code_j|.  (Keys are dealt to warps and CTAs, each with a unit of its own from its
# keys, which is not larger.)
def close_by_weight(q, cache, table, n, visible, got, sink=None):
    k, v, vs = rows_of(cache, table, n)
    hd = q.shape[2]
    o, lse, tol, ltol = ref.attend(q, k, v, visible, hd ** -0.5, sink)
    per = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        s = torch.where(visible, q[:, h].double() @ k[:, h // per].T * hd ** -0.5, -math.inf)
        p = torch.exp(s - torch.where(lse[:, h] == -math.inf, 0.0, lse[:, h])[:, None])
        x = torch.where(visible.any(0), vs[:, h // per].double(), 0.0)
        codes = torch.where(visible.any(0)[:, None],
                            v[:, h // per].abs() / vs[:, h // per].double()[:, None], 0.0)
        unit = 2.0 ** -33 * (p * x).amax(1) + 2.0 ** -121 * p.amax(1)
        tol[:, h] += unit[:, None] * (visible.double() @ codes)
    ref.close(*got, o, lse, tol, ltol)


def aligned(g, d, nh, n, kvh, hd):
    """Queries and keys, with a channel that all queries have alike (a key's entry
    there moves its scores of all rows)."""
    q, k, v = randn(g, d, nh, hd), randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    return q, k, v


@pytest.mark.parametrize("gain", [2.0 ** 8, 2.0 ** 16, 2.0 ** 20, 2.0 ** 40])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
@pytest.mark.parametrize("hd", [64, 128])
def test_large_value_row_of_little_weight(hd, shape, gain):
    """Key 300 has a weight of e^-(hd^-0.5 1200) and values `gain` times the rest's."""
    d, nh, kvh = shape
    n = 800
    q, k, v = aligned(gen(d + hd), d, nh, n, kvh, hd)
    k[300, :, 0] = -300.0
    v[300] *= gain
    cache, table = packed_cache(k, v, 32, True)
    got = attend(q, cache, table, n)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, 0, DEV), got)


@pytest.mark.parametrize("gain", [2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_large_value_row_that_is_not_seen(shape, gain):
    """A sibling branch, and rows just before the window, with values `gain` times
    the rest's."""
    d, nh, kvh = shape
    n, hd = 613, 128
    q, k, v = aligned(gen(d), d, nh, n, kvh, hd)
    pre = n - d
    v[pre + 1] *= gain              # seen by drafted token 1 only
    cache, table = packed_cache(k, v, 16, True)
    bits = [1 << t | (1 if t > 1 else 0) for t in range(d)]
    got = attend(q, cache, table, n, bits)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, bits, 0, DEV), got)
    window = 200
    v[pre + 1] /= gain
    v[:pre - window + 1] *= gain    # before what the first token sees
    cache, table = packed_cache(k, v, 64, True)
    got = attend(q, cache, table, n, None, window)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, window, DEV), got)


@pytest.mark.parametrize("spread", [6, 20, 50])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
@pytest.mark.parametrize("n", [64, 3000])
def test_value_scales_far_apart(n, shape, spread):
    """Any key may hold the row's largest p_j vs_j."""
    d, nh, kvh = shape
    hd = 128
    g = gen(n + spread)
    q, k, v = randn(g, d, nh, hd), randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    k = k * 3.0
    cache, table = packed_cache(k, v, 64, True)
    e = torch.randint(-spread, spread + 1, cache.v_scales.shape, generator=g, device=DEV)
    cache.v_scales.mul_(torch.exp2(e.float()))
    sink = torch.randn(nh, generator=g, device=DEV)
    for snk in (None, sink):
        got = attend(q, cache, table, n, sink=snk)
        close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, 0, DEV), got, snk)


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -60, 2.0 ** 60, 2.0 ** 96])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_values_all_small_or_all_large(shape, size):
    d, nh, kvh = shape
    n, hd = 900, 64
    g = gen(d)
    q, k, v = randn(g, d, nh, hd), randn(g, n, kvh, hd), randn(g, n, kvh, hd) * size
    v[5] = 0.0
    cache, table = packed_cache(k, v, 128, True)
    got = attend(q, cache, table, n)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, 0, DEV), got)


# ---------------------------------------------------------------------------
# The largest windows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 31, (1 << 63) - 1])
def test_window_larger_than_any_sequence(window):
    """The results of no window, bit for bit; more queries than keys among them."""
    g = gen(90)
    for hd in (64, 128):
        for lens_q, lens_k in (([40, 9, 70], [12, 9, 3]), ([33, 200], [533, 200])):
            q, k, v = (randn(g, n, h, hd) for n, h in
                       ((sum(lens_q), 8), (sum(lens_k), 2), (sum(lens_k), 2)))
            both = [ds41.prompt_attn_fwd(q, k, v, cu(lens_q), cu(lens_k), max(lens_q), 0.1, window=w)
                    for w in (0, window)]
            assert torch.equal(*both)
    for d, nh, kvh in (FEW, MIDDLING, MANY):
        q, k, v = randn(g, d, nh, 64), randn(g, 500, kvh, 64), randn(g, 500, kvh, 64)
        cache, table = packed_cache(k, v, 32, True)
        for n in (500, d):
            both = [attend(q, cache, table, n, None, w) for w in (0, window)]
            assert all(torch.equal(a, b) for a, b in zip(*both))


# ---------------------------------------------------------------------------
# Pages that have left the window
# ---------------------------------------------------------------------------
def evict(cache, table, first):
    """The pages whose rows are all before row `first` go to someone else: out of the
    table (half of them), or kept in it with another sequence's rows, NaN among them."""
    page = cache.k.shape[2]
    for i in range(first // page):
        p = int(table[0, i])
        for t in cache:
            if t is not None and t.dtype != torch.float8_e4m3fn:
                t[p] = math.nan
            elif t is not None:
                t[p].view(torch.uint8).fill_(0x7f)  # NaN
        if i % 2 == 0 or i == first // page - 1 and i % 4 == 1:
            table[0, i] = -1


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_pages_before_the_window_may_be_gone(shape, page, e4m3):
    """No error and no trace of them, for windows that end anywhere in a page and a
    128-key block."""
    d, nh, kvh = shape
    n, hd = 1100, 64
    g = gen(page + d)
    q, k, v = randn(g, d, nh, hd), randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    pre = n - d
    up = [0]
    for t in range(1, d):
        up.append(int(torch.randint(0, t, (1,), generator=torch.Generator().manual_seed(t))))
    tree = []
    for t in range(d):
        tree.append((tree[up[t]] if t else 0) | 1 << t)
    lost = list(tree)
    lost[d // 2] = 0                # a token that sees no drafted row: it stands at pre - 1
    kept, _ = packed_cache(k, v, page, e4m3)
    _, vs = None, None
    for first in (512, 513, 527, 528, 640, 700):  # the first row that token 0 sees
        for bits in (None, tree, lost):
            window = pre - first + 1
            cache, table = packed_cache(k, v, page, e4m3)
            kx, vx, vs = rows_of(cache, table, n)
            visible = ref.tree_visible(d, n, bits, window, DEV)
            want = ref.attend(q, kx, vx, visible, hd ** -0.5, None, vs)
            evict(cache, table, first - (1 if bits is lost else 0))
            ref.close(*attend(q, cache, table, n, bits, window), *want)
            assert ds41.device_status() == 0


@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_pages_inside_the_window_are_missed(shape):
    """A page with a row that some token sees has to be there."""
    d, nh, kvh = shape
    g = gen(91)
    q, k, v = randn(g, d, nh, 64), randn(g, 600, kvh, 64), randn(g, 600, kvh, 64)
    cache, table = packed_cache(k, v, 16, True)
    pre = 600 - d
    table[0, 20] = -1               # rows 320 .. 335
    empty = [0] * d
    for window, bits, code in ((pre - 335 + 1, None, 4), (pre - 336 + 1, None, 0),
                               (pre - 335, empty, 4), (pre - 335, None, 0),
                               (pre - 336, empty, 0)):
        attend(q, cache, table, 600, bits, window)
        assert ds41.device_status() == code, (window, bits, code)


# ---------------------------------------------------------------------------
# Prefix sums of a read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [True, False])
def test_read_leaves_rows_before_the_first_sequence(e4m3):
    g = gen(92)
    cache = filled_cache(g, 6, 2, 16, 64, e4m3)
    table = i32([[0, 1, 2], [3, 4, 5]])
    for starts in (None, i32([17, 3])):
        k, v = (torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ds41.kv_cache_read(cache, table, i32([5, 30, 50]), 60, starts=starts, k=k, v=v)
        assert ds41.device_status() == 0
        want = ds41.kv_cache_read(cache, table, i32([0, 25, 45]), 45, starts=starts)
        for x, w in zip((k, v), want):
            assert bool((x[:5] == 7.0).all() and (x[50:] == 7.0).all())
            assert torch.equal(x[5:50], w)


def test_read_skips_sequences_outside_its_rows():
    """Prefix sums that fall, start below 0 or pass the outputs' rows: those sequences
    are skipped with an error."""
    g = gen(93)
    cache = filled_cache(g, 8, 2, 16, 64, True)
    table = i32([[0, 1], [2, 3], [4, 5]])
    whole = ds41.kv_cache_read(cache, table, i32([0, 20, 30, 40]), 40)
    for prefix, rows, good in (([0, 20, 30, 41], 40, (0, 30)),    # past the rows
                               ([0, 20, 50, 60], 40, (0, 20)),
                               ([0, 20, 20, 10], 40, (0, 20)),    # falls
                               ([-3, 20, 30, 40], 40, (20, 40)),  # before the rows
                               ([0, 20, 1 << 30, -(1 << 31)], 40, (0, 20))):
        k, v = (torch.full((rows, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ds41.kv_cache_read(cache, table, i32(prefix), rows, k=k, v=v)
        assert ds41.device_status() == 4, prefix
        a, b = good
        for x, w in zip((k, v), whole):
            assert torch.equal(x[a:b], w[a:b]), prefix
            assert bool((x[:a] == 7.0).all() and (x[b:] == 7.0).all()), prefix


# ---------------------------------------------------------------------------
# The smallest scales
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-35])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_scales_and_queries_next_to_nothing(shape, scale):
    """Scores that are 0 but for their last bits: the average of what a token sees."""
    d, nh, kvh = shape
    n, hd = 150, 64
    g = gen(94)
    q = randn(g, d, nh, hd) * 2.0 ** -115
    k, v = randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    for e4m3 in (True, False):
        cache, table = packed_cache(k, v, 32, e4m3)
        kx, vx, vs = rows_of(cache, table, n)
        lse = torch.empty(d, nh, device=DEV)
        o = ds41.tree_attn_fwd(q, cache, table, i32([n]), cu([d]), d, n, scale, lse=lse)
        ref.close(o, lse, *ref.attend(q, kx, vx, ref.tree_visible(d, n, None, 0, DEV), scale, None,
                                      vs))
    lse = torch.empty(d, nh, device=DEV)
    o = ds41.prompt_attn_fwd(q, k, v, cu([d]), cu([n]), d, scale, lse=lse)
    ref.close(o, lse, *ref.attend(q, k, v, ref.prompt_visible(d, n, 0, DEV), scale, None))


# ---------------------------------------------------------------------------
# A key that takes nearly all the weight and has next to no values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("size", [0.0, 2.0 ** -60, 2.0 ** -8])
@pytest.mark.parametrize("nats", [8, 30, 60, 200])
@pytest.mark.parametrize("shape", [FEW, MIDDLING, MANY])
def test_heavy_key_of_small_values(shape, nats, size):
    """As the first token of a text often is: what the others add is kept, down to
    2^-96 of the heavy key's weight."""
    d, nh, kvh = shape
    n, hd = 500, 128
    q, k, v = aligned(gen(d), d, nh, n, kvh, hd)
    at = 0 if nats == 30 else 260
    k[at, :, 0] = nats * hd ** 0.5 / 4.0
    v[at] *= size
    cache, table = packed_cache(k, v, 64, True)
    got = attend(q, cache, table, n)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, 0, DEV), got)
    sink = torch.full((nh,), float(nats), device=DEV)
    got = attend(q, cache, table, n, sink=sink)
    close_by_weight(q, cache, table, n, ref.tree_visible(d, n, None, 0, DEV), got, sink)
