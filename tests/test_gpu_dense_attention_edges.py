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
