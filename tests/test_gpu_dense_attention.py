"""Dense attention with grouped heads and its paged cache on the GPU, against
the definitions in 64 bits (dense_ref.py, where the tolerances are derived)."""
import math
import sys
import threading

import pytest
import torch

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


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0).tolist()), dtype=torch.int32,
                        device=DEV)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------
def filled_cache(g, n_pages, kvh, page, hd, e4m3):
    k, v = randn(g, n_pages, kvh, page, hd), randn(g, n_pages, kvh, page, hd)
    if not e4m3:
        return ds41.KvCache(k, v)
    (kc, ks), (vc, vs) = ref.quantise(k), ref.quantise(v)
    return ds41.KvCache(kc, vc, ks, vs)


def u8(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def bits(t):
    """Bit patterns; every NaN as one."""
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    t = torch.where(t.isnan(), torch.full_like(t, math.nan), t)
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("n,kvh,hd,page,fused", [
    (1, 1, 16, 16, False), (1, 8, 128, 64, True), (37, 3, 80, 32, False), (130, 2, 64, 256, True),
    (515, 4, 96, 16, True), (4099, 8, 128, 64, True)])
def test_write(n, kvh, hd, page, fused, e4m3):
    """Codes and scales bit for bit, other slots as they were, -1 not written."""
    g = gen(n + hd)
    n_pages = -(-n // page) + 2
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    want = [None if t is None else t.clone() for t in cache]
    if fused:
        qkv = randn(g, n, 3 * kvh, hd)
        k, v = qkv[:, kvh:2 * kvh], qkv[:, 2 * kvh:]
    else:
        k, v = randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    k = k.contiguous() if n == 1 else k
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:n]
    if n > 2:
        slots[[0, n // 2]] = -1
    if n > 100:  # rows that a scale could go wrong on
        k[1], k[2, :, 0], v[3], v[4, 0, 1] = 0.0, 1e30, 1e-38, math.inf
        k[5, 0, 2], k[6] = math.nan, -1e-40
    ds41.kv_cache_write(cache, k, v, slots)
    keep = slots >= 0
    at, off = slots[keep] // page, slots[keep] % page
    for i, x in ((0, k), (1, v)):
        if e4m3:
            codes, s = ref.quantise(x[keep])
            u8(want[i])[at, :, off] = u8(codes)
            want[2 + i][at, :, off] = s
        else:
            want[i][at, :, off] = x[keep]
    for got, w in zip(cache, want):
        if w is not None:
            assert torch.equal(bits(got), bits(w))


@pytest.mark.parametrize("hd", [16, 128])
def test_write_every_magnitude(hd):
    """Rows whose largest element is each of the bf16 numbers, zero and infinity
    among them: the scales and the codes bit for bit."""
    g = gen(5)
    tops = torch.arange(0x7f81, device=DEV)
    n = tops.numel()

    def rows(top):
        b = (torch.rand(n, 1, hd, generator=g, device=DEV, dtype=torch.float64)
             * (top[:, None, None] + 1)).long()
        near = torch.rand(n, 1, hd, generator=g, device=DEV) < 0.5  # most within 2^-10
        b = torch.where(near, (top[:, None, None] - b % (10 * 128)).clamp_min(0), b)
        at = torch.randint(hd, (n,), generator=g, device=DEV)
        b[torch.arange(n, device=DEV), 0, at] = top
        sign = torch.randint(2, b.shape, generator=g, device=DEV) << 15
        return (b | sign).to(torch.int16).view(torch.bfloat16)
    k, v = rows(tops), rows(tops.flip(0))
    cache = ds41.make_kv_cache((n + 63) // 64, 1, 64, hd)
    ds41.kv_cache_write(cache, k, v, torch.arange(n, device=DEV))
    for x, codes, scales in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        want, ws = ref.quantise(x)
        assert torch.equal(bits(scales.view(-1)[:n]), bits(ws.view(-1)))
        assert torch.equal(u8(codes).view(-1, hd)[:n], u8(want)[:, 0])


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("lens,kvh,hd,page,starts", [
    ([1], 1, 16, 16, None), ([5, 0, 33, 1], 3, 80, 16, [3, 0, 7, 15]),
    ([300, 17], 8, 128, 64, None), ([129, 64, 200], 2, 96, 32, [0, 100, 31])])
def test_read(lens, kvh, hd, page, starts, e4m3):
    g = gen(sum(lens))
    st = starts or [0] * len(lens)
    need = max(-(-(n + s) // page) for n, s in zip(lens, st))
    n_pages = need * len(lens) + 1
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    table = torch.randperm(n_pages, generator=g, device=DEV)[:need * len(lens)].view(
        len(lens), need).int()
    rows = sum(lens)
    k = torch.full((rows + 3, kvh, hd), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    sd = torch.tensor(starts, dtype=torch.int32, device=DEV) if starts else None
    ds41.kv_cache_read(cache, table, cu(lens), rows + 3, starts=sd, k=k, v=v)
    for got, c, s in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        x = ref.values(c, s).transpose(1, 2)
        at = 0
        for b, n in enumerate(lens):
            w = x[table[b].long()].flatten(0, 1)[st[b]:st[b] + n]
            e = (got[at:at + n].double() - w).abs()
            # code * scale is rounded to f32, then to bf16
            assert bool((e <= w.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
            at += n
        assert bool((got[at:] == 7.0).all()), "rows behind the last sequence"


def test_write_then_read_halves_a_step():
    """What is read back is within half an e4m3 step of what was written."""
    g = gen(3)
    n, kvh, hd, page = 200, 4, 128, 32
    cache = ds41.make_kv_cache(9, kvh, page, hd)
    k, v = randn(g, n, kvh, hd), randn(g, n, kvh, hd) * 1e-6
    slots = torch.randperm(9 * page, generator=g, device=DEV)[:n]
    ds41.kv_cache_write(cache, k, v, slots)
    table = torch.arange(9, dtype=torch.int32, device=DEV).view(1, 9)
    kr, vr = ds41.kv_cache_read(cache, table, cu([9 * page]), 9 * page)
    for x, y in ((k, kr[slots]), (v, vr[slots])):
        x, y = x.double(), y.double()
        amax = x.abs().amax(-1, keepdim=True)
        # e4m3: half a step is 2^-4 relative, 2^-10 of the smallest normal below
        # it (amax / 448 * 2^-10 absolute); s, x / s and bf16 roundings beside it
        tol = torch.maximum(x.abs() * 2.0 ** -4, amax / 448 * 2.0 ** -10) * (1 + 2.0 ** -20)
        assert bool(((x - y).abs() <= tol + (x.abs() + tol) * (2.0 ** -8 + 2.0 ** -20)).all())


def test_cache_beyond_32_bit_offsets():
    """A cache of over 2^31 elements: the last page written, read and attended."""
    g = gen(5)
    kvh, page, hd = 8, 64, 128
    n_pages = (1 << 31) // (kvh * page * hd) + 40
    cache = ds41.make_kv_cache(n_pages, kvh, page, hd)
    n = 100
    k, v = randn(g, n, kvh, hd), randn(g, n, kvh, hd)
    slots = torch.arange(n, device=DEV) + (n_pages - 2) * page
    ds41.kv_cache_write(cache, k, v, slots)
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device=DEV)
    kr, vr = ds41.kv_cache_read(cache, table, cu([n]), n)
    kq, vq = (ref.values(*ref.quantise(x)) for x in (k, v))
    assert bool(((kr.double() - kq).abs() <= kq.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    assert bool(((vr.double() - vq).abs() <= vq.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    q = randn(g, 1, 16, hd)
    lse = torch.empty(1, 16, device=DEV)
    o = ds41.tree_attn_fwd(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                           cu([1]), 1, n, hd ** -0.5, lse=lse)
    ref.close(o, lse, *ref.attend(q, kq, vq, ref.tree_visible(1, n, None, 0, DEV), hd ** -0.5, None))


# ---------------------------------------------------------------------------
# Prompts
# ---------------------------------------------------------------------------
PROMPTS = [
    # lens_q, lens_k, nh, kvh, hd, window, sink
    ([1], [1], 1, 1, 16, 0, False),
    ([1], [1], 4, 2, 64, 0, True),
    ([64], [64], 4, 2, 64, 0, True),
    ([127], [127], 8, 2, 128, 0, False),
    ([128], [128], 8, 8, 128, 0, True),
    ([129], [129], 4, 1, 128, 0, False),
    ([257], [257], 5, 1, 80, 0, True),
    ([300], [300], 6, 2, 96, 0, False),
    ([511], [511], 16, 2, 64, 0, False),
    ([700], [700], 3, 3, 128, 0, False),
    ([5, 0, 130, 1, 64], [5, 0, 130, 1, 64], 8, 2, 128, 0, True),
    ([33, 200, 7], [533, 200, 1031], 8, 4, 128, 0, False),
    ([1, 1, 1], [600, 129, 1], 32, 8, 128, 0, True),
    ([40, 9], [12, 0], 4, 2, 64, 0, False),          # queries that see nothing
    ([40, 9], [12, 0], 4, 2, 128, 0, True),
    ([300, 77], [300, 577], 8, 2, 64, 128, True),
    ([300, 77], [300, 577], 8, 2, 128, 1, False),
    ([513], [513], 4, 4, 48, 200, False),
    ([260], [1500], 2, 1, 112, 1000, True),
    ([2, 3], [4096, 4097], 64, 8, 128, 0, False),
    ([1100], [1100], 24, 1, 128, 0, False),
]


def run_prompt(g, lens_q, lens_k, nh, kvh, hd, window, sink, layout="dense", q_gain=1.0):
    Tq, Tk = sum(lens_q), sum(lens_k)
    q, k, v = randn(g, Tq, nh, hd) * q_gain, randn(g, Tk, kvh, hd), randn(g, Tk, kvh, hd)
    if layout == "fused" and lens_q == lens_k:  # slices of one projection
        qkv = torch.cat([q, k, v], 1)
        q, k, v = qkv[:, :nh], qkv[:, nh:nh + kvh], qkv[:, nh + kvh:]
    elif layout == "heads":  # heads outermost
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    snk = torch.randn(nh, generator=g, device=DEV) if sink else None
    o = torch.full((Tq + 2, nh, hd), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Tq + 2, nh), 7.0, device=DEV)
    qx = torch.cat([q, q[:1].expand(2, -1, -1)]) if layout == "dense" else q
    n = qx.shape[0]
    ds41.prompt_attn_fwd(qx, k, v, cu(lens_q), cu(lens_k), max(lens_q), hd ** -0.5, sink=snk,
                         window=window, o=o[:n], lse=lse[:n])
    assert bool((o[Tq:] == 7.0).all() and (lse[Tq:] == 7.0).all()), "rows behind the last sequence"
    at_q = at_k = 0
    for n, m in zip(lens_q, lens_k):
        want = ref.attend(q[at_q:at_q + n], k[at_k:at_k + m], v[at_k:at_k + m],
                          ref.prompt_visible(n, m, window, DEV), hd ** -0.5, snk)
        ref.close(o[at_q:at_q + n], lse[at_q:at_q + n], *want)
        at_q, at_k = at_q + n, at_k + m


@pytest.mark.parametrize("case", range(len(PROMPTS)))
@pytest.mark.parametrize("layout", ["dense", "fused", "heads"])
def test_prompt(case, layout):
    run_prompt(gen(100 + case), *PROMPTS[case], layout=layout)


def test_prompt_large_scores():
    """Scores far apart: the maximum moves a lot from tile to tile."""
    run_prompt(gen(7), [600], [900], 8, 2, 128, 0, False, q_gain=40.0)
    run_prompt(gen(8), [600], [900], 8, 2, 64, 0, True, q_gain=40.0)


def test_prompt_other_sequences_do_not_leak():
    """NaN in the neighbours' keys and values, before and behind, changes nothing."""
    g = gen(9)
    lens = [70, 45, 90]
    for hd in (64, 128):
        q, k, v = (randn(g, 205, h, hd) for h in (4, 2, 2))
        for b in (0, 2):
            at = sum(lens[:b])
            k[at:at + lens[b]] = math.nan
            v[at:at + lens[b]] = math.inf
        lse = torch.empty(205, 4, device=DEV)
        o = ds41.prompt_attn_fwd(q, k, v, cu(lens), cu(lens), 90, hd ** -0.5, lse=lse)
        s = slice(70, 115)
        ref.close(o[s], lse[s], *ref.attend(q[s], k[s], v[s], ref.prompt_visible(45, 45, 0, DEV),
                                            hd ** -0.5, None))


def test_prompt_nan_key_reaches_those_that_see_it():
    g = gen(10)
    q, k, v = randn(g, 200, 4, 64), randn(g, 200, 2, 64), randn(g, 200, 2, 64)
    k[150, 0, 3] = math.nan
    o = ds41.prompt_attn_fwd(q, k, v, cu([200]), cu([200]), 200, 0.125)
    assert bool(o[150:, :2].isnan().all()) and not bool(o[:150].isnan().any())
    assert not bool(o[:, 2:].isnan().any())


def test_prompt_no_keys_at_all():
    q = randn(gen(1), 5, 4, 64)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(5, 4, device=DEV)
    o = ds41.prompt_attn_fwd(q, e, e, cu([5]), cu([0]), 5, 0.125, lse=lse)
    assert bool((o == 0).all() and (lse == -math.inf).all())
    z = q[:0]
    assert ds41.prompt_attn_fwd(z, e, e, cu([0]), cu([0]), 0, 0.125).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# Trees
# ---------------------------------------------------------------------------
def tree_bits(rng, n):
    """Each token's bits: its own and its parent's; parents come earlier."""
    rows = []
    for t in range(n):
        up = rows[int(torch.randint(max(0, t - 5), t, (1,), generator=rng))] if t else 0
        rows.append(up | 1 << t)
    return rows


def signed(w):
    return w - (1 << 64) if w >> 63 else w


def words_of(bits, words):
    return [[signed(b >> (64 * i) & ((1 << 64) - 1)) for i in range(words)] for b in bits]


TREES = [
    # lens, drafts, nh, kvh, hd, page, e4m3, window, sink, masked
    ([1], [1], 1, 1, 16, 16, True, 0, False, False),
    ([1], [1], 4, 2, 64, 16, False, 0, True, False),
    ([64], [1], 8, 1, 128, 64, True, 0, False, False),
    ([700], [1], 32, 8, 128, 64, True, 0, True, False),
    ([700], [1], 32, 8, 128, 64, False, 0, False, False),
    ([5000, 17, 1, 2049], [1, 1, 1, 1], 64, 8, 128, 64, True, 0, True, False),
    ([9000, 63], [1, 1], 16, 1, 64, 128, False, 0, False, False),
    ([333, 100], [1, 1], 5, 1, 80, 32, True, 0, False, False),
    ([333, 100], [4, 7], 6, 2, 96, 256, True, 0, True, False),
    ([130, 40], [8, 0], 8, 2, 112, 16, False, 0, False, True),
    ([1000, 16, 400], [16, 16, 9], 32, 8, 128, 64, True, 0, False, True),
    ([1000, 16, 400], [16, 16, 9], 8, 8, 128, 16, False, 0, True, True),
    ([3000, 64], [64, 64], 64, 8, 128, 64, True, 0, False, True),
    ([3000, 64], [64, 64], 64, 8, 64, 32, False, 0, True, True),
    ([500], [200], 4, 2, 128, 64, True, 0, False, True),
    ([260, 256], [130, 256], 16, 4, 64, 32, True, 0, True, True),
    ([1000, 90], [1, 1], 8, 2, 128, 64, True, 128, True, False),
    ([1000, 90], [12, 5], 8, 2, 128, 64, True, 100, False, True),
    ([600, 610], [30, 33], 24, 1, 64, 16, False, 64, True, True),
    ([700], [12], 8, 2, 128, 64, True, 12, False, False),
]


def run_tree(g, lens, drafts, nh, kvh, hd, page, e4m3, window, sink, masked, q_heads_out=False,
             spread=0, q_gain=None):
    need = max(max(-(-n // page) for n in lens), 1)
    n_pages = need * len(lens) + 2
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    if spread:  # rows of very different sizes
        for s in cache[2:]:
            s.mul_(torch.exp2(torch.randint(-spread, spread + 1, s.shape, generator=g,
                                            device=DEV).float()))
    table = torch.randperm(n_pages, generator=g, device=DEV)[:need * len(lens)].view(
        len(lens), need).int()
    # behind each sequence's end: whatever an earlier user left there
    for b, n in enumerate(lens):
        if n % page:
            pg = int(table[b, n // page])
            for t in cache:
                if t is not None and t.dtype != torch.float8_e4m3fn:
                    t[pg, :, n % page:] = math.nan
        table[b, -(-n // page):] = -5  # never read
    Tq = sum(drafts)
    q = randn(g, Tq, nh, hd)
    if q_gain is not None:
        q = q * q_gain
    if q_heads_out:
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    snk = torch.randn(nh, generator=g, device=DEV) if sink else None
    rng = torch.Generator().manual_seed(Tq)
    bits = [tree_bits(rng, n) if masked else None for n in drafts]
    mask = None
    if masked:
        if drafts[0] > 2:
            bits[0][1] = 0  # sees no drafted token, not even itself
        words = -(-max(drafts) // 64)
        rows = [w for b in bits for w in words_of(b, words)]
        # bits past a sequence's own tokens are ignored
        at = 0
        for n in drafts:
            for t in range(at, at + n):
                if n % 64 and n < 64:
                    rows[t][0] = signed((rows[t][0] | (~0 << n)) & ((1 << 64) - 1))
            at += n
        mask = torch.tensor(rows, dtype=torch.int64, device=DEV).view(Tq, words)
    o = torch.full((Tq, nh, hd), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Tq, nh), 7.0, device=DEV)
    ds41.tree_attn_fwd(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                       cu(drafts), max(drafts), max(lens), hd ** -0.5, mask=mask, sink=snk,
                       window=window, o=o, lse=lse)
    kx, vx = ref.values(cache.k, cache.k_scales), ref.values(cache.v, cache.v_scales)
    at = 0
    for b, (n, d) in enumerate(zip(lens, drafts)):
        pages = table[b, :-(-n // page)].long()
        k, v = (x[pages].transpose(1, 2).flatten(0, 1)[:n] for x in (kx, vx))
        vs = cache.v_scales[pages].transpose(1, 2).flatten(0, 1)[:n] if e4m3 else None
        want = ref.attend(q[at:at + d], k, v, ref.tree_visible(d, n, bits[b], window, DEV),
                          hd ** -0.5, snk, vs)
        ref.close(o[at:at + d], lse[at:at + d], *want)
        at += d


@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(case):
    run_tree(gen(200 + case), *TREES[case])


def test_tree_strided_queries():
    run_tree(gen(41), *TREES[10], q_heads_out=True)
    run_tree(gen(42), *TREES[5], q_heads_out=True)


@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_of_middling_rows_over_long_caches(e4m3):
    """17 to 128 rows per key/value head: one tile of rows, odd and even numbers of
    blocks a piece, streams that end one after the other."""
    run_tree(gen(61), [4000, 2417, 900, 129], [16, 9, 16, 5], 32, 8, 128, 64, e4m3, 0, False, True)
    run_tree(gen(62), [6001], [30], 16, 4, 64, 128, e4m3, 0, True, True)
    run_tree(gen(63), [3333] * 9, [5] * 9, 16, 2, 128, 32, e4m3, 1000, False, False)


@pytest.mark.parametrize("spread", [3, 12, 40])
@pytest.mark.parametrize("case", [3, 10, 12, 15])
def test_tree_scales_far_apart(case, spread):
    """Rows whose scales differ by up to 2^(2 spread), so that the common exponent
    of the value scales moves along the way."""
    run_tree(gen(300 + case), *TREES[case], spread=spread)


@pytest.mark.parametrize("q_gain", [1e-30, 1e-4, 30.0])
@pytest.mark.parametrize("case", [3, 10, 12])
def test_tree_small_and_large_queries(case, q_gain):
    run_tree(gen(320 + case), *TREES[case], q_gain=q_gain)


def test_tree_query_with_outliers():
    """A query channel 1000 times larger than the rest, and a zero query."""
    for case in (3, 10, 12):
        c = list(TREES[case])
        q_gain = torch.ones(sum(c[1]), c[2], c[4], device=DEV, dtype=torch.bfloat16)
        q_gain[:, :, 5] = 1000.0
        q_gain[0, 1] = 0.0
        run_tree(gen(340 + case), *c, q_gain=q_gain)


def test_tree_token_that_sees_nothing():
    """No earlier rows and an empty mask row: o = 0, lse = sink or -inf."""
    g = gen(11)
    for e4m3 in (True, False):
        cache = filled_cache(g, 2, 2, 16, 64, e4m3)
        table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
        q = randn(g, 3, 4, 64)
        mask = torch.tensor([[1], [0], [5]], dtype=torch.int64, device=DEV)
        snk = torch.randn(4, generator=g, device=DEV)
        n = torch.tensor([3], dtype=torch.int32, device=DEV)
        lse = torch.empty(3, 4, device=DEV)
        o = ds41.tree_attn_fwd(q, cache, table, n, cu([3]), 3, 3, 0.125, mask=mask, lse=lse)
        assert bool((o[1] == 0).all() and (lse[1] == -math.inf).all())
        o = ds41.tree_attn_fwd(q, cache, table, n, cu([3]), 3, 3, 0.125, mask=mask, sink=snk,
                               lse=lse)
        assert bool((o[1] == 0).all())
        assert bool(((lse[1] - snk).abs() <= 2.0 ** -21 * (1 + snk.abs())).all())


def test_tree_nan_scale_of_an_unseen_row():
    """An e4m3 row that held NaN, seen by one token of the tree only."""
    g = gen(12)
    cache = filled_cache(g, 3, 2, 64, 128, True)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    n, d = 100, 4
    bad = n - d + 2  # drafted row 2
    for s in (cache.k_scales, cache.v_scales):
        s[0, :, bad - 64] = math.nan
    mask = torch.tensor([[1], [3], [4], [9]], dtype=torch.int64, device=DEV)
    q = randn(g, d, 8, 128)
    o = ds41.tree_attn_fwd(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                           cu([d]), d, n, 0.1, mask=mask)
    assert bool(o[2].isnan().all()) and not bool(o[[0, 1, 3]].isnan().any())


# ---------------------------------------------------------------------------
# Refusals on the device, streams, graphs
# ---------------------------------------------------------------------------
def test_bad_slots_and_pages_are_skipped():
    g = gen(13)
    cache = filled_cache(g, 4, 2, 16, 64, True)
    before = [t.clone() for t in cache]
    k, v = randn(g, 3, 2, 64), randn(g, 3, 2, 64)
    ds41.kv_cache_write(cache, k, v, torch.tensor([64, -2, 1 << 40], device=DEV))
    assert ds41.device_status() == 4  # DS41_E_INDEX
    assert all(torch.equal(u8(a), u8(b)) for a, b in zip(cache, before))
    table = torch.tensor([[0, 9], [-1, 1]], dtype=torch.int32, device=DEV)
    kr, vr = ds41.kv_cache_read(cache, table, cu([20, 20]), 40)
    assert ds41.device_status() == 4
    assert bool((kr[16:36] == 0).all() and (vr[16:36] == 0).all())
    assert bool((kr[:16] != 0).any() and (kr[36:] != 0).any())
    # attention: a bad page's rows are not seen
    q = randn(g, 2, 4, 64)
    lens = torch.tensor([20, 20], dtype=torch.int32, device=DEV)
    lse = torch.empty(2, 4, device=DEV)
    o = ds41.tree_attn_fwd(q, cache, table, lens, cu([1, 1]), 1, 20, 0.125, lse=lse)
    assert ds41.device_status() == 4
    kx, vx = ref.values(cache.k, cache.k_scales), ref.values(cache.v, cache.v_scales)
    for b, (pg, n) in enumerate(((0, 16), (1, 4))):
        kk, vv = kx[pg].transpose(0, 1)[:n], vx[pg].transpose(0, 1)[:n]
        ref.close(o[b:b + 1], lse[b:b + 1],
                  *ref.attend(q[b:b + 1], kk, vv, torch.ones(1, n, dtype=torch.bool, device=DEV),
                              0.125, None))


def test_bad_lengths_are_skipped():
    """A sequence that breaks its limits keeps its output rows; the others are
    computed."""
    g = gen(14)
    cache = filled_cache(g, 8, 2, 16, 64, False)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    q = randn(g, 6, 4, 64)
    for lens, cuq in (([33, 20, 20, 20], [0, 1, 2, 3, 4]),   # past the table
                      ([0, 20, 20, 20], [0, 1, 2, 3, 4]),    # fewer rows than drafted tokens
                      ([-7, 20, 20, 20], [0, 1, 2, 3, 4]),
                      ([20, 20, 20, 20], [0, 4, 5, 6, 6])):  # more than max_q
        o = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        ds41.tree_attn_fwd(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                           torch.tensor(cuq, dtype=torch.int32, device=DEV), 2, 64, 0.125, o=o)
        assert ds41.device_status() == 4
        assert bool((o[cuq[0]:cuq[1]] == 7.0).all()) and bool((o[cuq[1]:cuq[3]] != 7.0).any())
    k = randn(g, 10, 2, 64)
    for cuq, cuk in (([0, 3, 6], [0, 20, 10]), ([0, -3, 6], [0, 5, 10]), ([0, 3, 9], [0, 5, 10]),
                     ([-2, 3, 6], [0, 5, 10]), ([0, 5, 6], [0, 5, 10])):
        o = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        ds41.prompt_attn_fwd(q, k, k, torch.tensor(cuq, dtype=torch.int32, device=DEV),
                             torch.tensor(cuk, dtype=torch.int32, device=DEV), 4, 0.125, o=o)
        assert ds41.device_status() == 4


def test_other_stream_and_graph_replay():
    """The whole sequence of calls on a side stream, eager and as a graph that
    is replayed on new inputs, gives the same bits."""
    g = gen(15)
    kvh, hd, page, nh = 2, 128, 32, 8
    cache = ds41.make_kv_cache(8, kvh, page, hd)
    table = torch.tensor([[3, 1, 7], [0, 2, 5]], dtype=torch.int32, device=DEV)
    q, k, v = randn(g, 130, nh, hd), randn(g, 130, kvh, hd), randn(g, 130, kvh, hd)
    lens_t = torch.tensor([70, 60], dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(70), torch.arange(60)]).to(DEV)
    seq = torch.tensor([0] * 70 + [1] * 60, device=DEV)
    slots = table.long()[seq, pos // page] * page + pos % page
    c = cu([70, 60])
    cq = cu([9, 4])
    qt = randn(g, 13, nh, hd)
    out = {}

    def step():
        out["p"] = ds41.prompt_attn_fwd(q, k, v, c, c, 70, 0.1)
        ds41.kv_cache_write(cache, k, v, slots)
        out["k"], out["v"] = ds41.kv_cache_read(cache, table, c, 130)
        out["t"] = ds41.tree_attn_fwd(qt, cache, table, lens_t, cq, 9, 70, 0.1)

    step()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in out.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for t in cache:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
    q2, k2 = q.clone(), k.clone()
    q.copy_(randn(g, 130, nh, hd))
    k.copy_(randn(g, 130, kvh, hd))
    graph.replay()
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in out.items()}
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], got[n]) for n in got)
    assert not torch.equal(q2, q) and not torch.equal(k2, k)


def test_serving_run():
    """As they are used: a prompt, its rows cached in 8 bits, a second chunk
    over the rows read back, a tree of drafted tokens checked, the accepted ones
    written to their places, and a decode step over all of it."""
    g = gen(16)
    nh, kvh, hd, page, scale = 8, 2, 128, 32, 128 ** -0.5
    cache = ds41.make_kv_cache(12, kvh, page, hd)
    table = torch.tensor([[7, 2, 9, 4, 0, 11]], dtype=torch.int32, device=DEV)

    def slot(p):
        p = torch.as_tensor(p, device=DEV)
        return table[0].long()[p // page] * page + p % page

    def chunk(n):
        return randn(g, n, nh, hd), randn(g, n, kvh, hd), randn(g, n, kvh, hd)

    def quant(x):
        return ref.values(*ref.quantise(x))

    q1, k1, v1 = chunk(75)
    lse = torch.empty(75, nh, device=DEV)
    o = ds41.prompt_attn_fwd(q1, k1, v1, cu([75]), cu([75]), 75, scale, lse=lse)
    ref.close(o, lse, *ref.attend(q1, k1, v1, ref.prompt_visible(75, 75, 0, DEV), scale, None))
    ds41.kv_cache_write(cache, k1, v1, slot(torch.arange(75)))
    # the second chunk: its rows written, all rows read back, attended
    q2, k2, v2 = chunk(40)
    ds41.kv_cache_write(cache, k2, v2, slot(torch.arange(75, 115)))
    kr, vr = ds41.kv_cache_read(cache, table, cu([115]), 115)
    lse = torch.empty(40, nh, device=DEV)
    o = ds41.prompt_attn_fwd(q2, kr, vr, cu([40]), cu([115]), 40, scale, lse=lse)
    K, V = (torch.cat([quant(a), quant(b)]) for a, b in ((k1, k2), (v1, v2)))
    assert bool(((kr.double() - K).abs() <= K.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    ref.close(o, lse, *ref.attend(q2, kr, vr, ref.prompt_visible(40, 115, 0, DEV), scale, None))
    # five drafted tokens: 0 -> 1 -> 3, 0 -> 2 -> 4
    q3, k3, v3 = chunk(5)
    ds41.kv_cache_write(cache, k3, v3, slot(torch.arange(115, 120)))
    bits = [0b1, 0b11, 0b101, 0b1011, 0b10101]
    lse = torch.empty(5, nh, device=DEV)
    o = ds41.tree_attn_fwd(q3, cache, table, torch.tensor([120], dtype=torch.int32, device=DEV),
                           cu([5]), 5, 120, scale,
                           mask=torch.tensor(bits, dtype=torch.int64, device=DEV).view(5, 1),
                           lse=lse)
    K3, V3 = torch.cat([K, quant(k3)]), torch.cat([V, quant(v3)])
    ref.close(o, lse, *ref.attend(q3, K3, V3, ref.tree_visible(5, 120, bits, 0, DEV), scale, None))
    # 0, 2 and 4 are accepted: 2 and 4 move up, the rest is not written
    ds41.kv_cache_write(cache, k3, v3, torch.stack([torch.tensor(-1, device=DEV),
                                                    torch.tensor(-1, device=DEV), slot(116),
                                                    torch.tensor(-1, device=DEV), slot(117)]))
    q4, k4, v4 = chunk(1)
    ds41.kv_cache_write(cache, k4, v4, slot([118]))
    lse = torch.empty(1, nh, device=DEV)
    o = ds41.tree_attn_fwd(q4, cache, table, torch.tensor([119], dtype=torch.int32, device=DEV),
                           cu([1]), 1, 119, scale, lse=lse)
    K4, V4 = (torch.cat([a, quant(b)[[0, 2, 4]], quant(c)]) for a, b, c in ((K, k3, k4), (V, v3, v4)))
    ref.close(o, lse, *ref.attend(q4, K4, V4, ref.tree_visible(1, 119, None, 0, DEV), scale, None))


# ---------------------------------------------------------------------------
# Batches, groups, calls at once
# ---------------------------------------------------------------------------
def test_prompt_many_sequences():
    """More sequences than one lookup takes, empty ones among them."""
    rng = torch.Generator().manual_seed(70)
    lens = torch.randint(0, 41, (75,), generator=rng).tolist()
    lens[30:36] = [0] * 6
    run_prompt(gen(70), lens, lens, 4, 2, 128, 0, True)
    run_prompt(gen(71), lens, [n + 130 for n in lens], 8, 1, 64, 100, False)


@pytest.mark.parametrize("nh,kvh", [(300, 2), (131, 1), (256, 1), (128, 1)])
def test_prompt_groups_beyond_a_tile(nh, kvh):
    run_prompt(gen(72), [70, 5], [90, 5], nh, kvh, 64, 0, True)


def test_tree_many_sequences():
    rng = torch.Generator().manual_seed(73)
    drafts = torch.randint(0, 6, (90,), generator=rng).tolist()
    lens = [n + int(torch.randint(0, 400, (1,), generator=rng)) for n in drafts]
    lens[3], drafts[3] = 0, 0
    for nh, e4m3 in ((6, True), (6, False), (16, True), (16, False)):
        run_tree(gen(73), lens, drafts, nh, 2, 128, 32, e4m3, 0, False, True)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("nh,kvh,drafts", [(150, 1, [1]), (17, 1, [1, 1]), (300, 1, [3]),
                                           (128, 1, [1]), (129, 1, [2, 1])])
def test_tree_wide_groups(nh, kvh, drafts, e4m3):
    run_tree(gen(74), [700, 64][:len(drafts)], drafts, nh, kvh, 64, 64, e4m3, 0, True, False)


def tree_inputs(g, lens, drafts, nh, kvh, hd, page, e4m3):
    need = max(-(-n // page) for n in lens)
    cache = filled_cache(g, need * len(lens), kvh, page, hd, e4m3)
    table = torch.randperm(need * len(lens), generator=g, device=DEV).view(len(lens), need).int()
    q = randn(g, sum(drafts), nh, hd)
    return (q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), cu(drafts),
            max(drafts), max(lens), hd ** -0.5)


def test_same_bits_every_time_and_on_two_streams():
    """No result depends on the order in which CTAs finish, nor on a call that runs
    beside it on another stream with a workspace of its own."""
    g = gen(75)
    cases = [tree_inputs(g, [5000, 900], [1, 1], 32, 8, 128, 64, True),
             tree_inputs(g, [5000, 900], [16, 9], 32, 8, 128, 64, True),
             tree_inputs(g, [3000, 900], [64, 40], 64, 8, 128, 64, False)]
    q, k, v = (randn(g, 1500, h, 128) for h in (8, 2, 2))
    c = cu([1000, 500])

    def run():
        return [ds41.tree_attn_fwd(*a) for a in cases] + [
            ds41.prompt_attn_fwd(q, k, v, c, c, 1000, 0.09)]

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(6):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for outs in got:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_from_two_threads_and_no_leak():
    """Two threads, each on a stream of its own, while neither holds the other's
    outputs; what a call allocates is given back, the outputs given are returned."""
    g = gen(78)
    a = tree_inputs(g, [700, 33], [3, 1], 8, 2, 64, 32, True)
    q, k, v = (randn(g, 150, h, 64) for h in (8, 2, 2))
    c = cu([100, 50])
    cache = filled_cache(g, 5, 2, 32, 64, True)
    slots = torch.arange(150, device=DEV)
    rows = torch.arange(5, device=DEV, dtype=torch.int32)[None]

    def run():
        ds41.kv_cache_write(cache, k, v, slots)  # (both threads the same rows)
        return (ds41.tree_attn_fwd(*a), ds41.prompt_attn_fwd(q, k, v, c, c, 100, 0.1),
                *ds41.kv_cache_read(cache, rows, cu([150]), 150))
    want = run()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(100):
                if not all(torch.equal(x, y) for x, y in zip(run(), want)):
                    wrong.append(1)
        s.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and torch.cuda.memory_allocated() == before
    o, lse = torch.empty_like(want[1]), torch.empty(150, 8, device=DEV)
    refs = sys.getrefcount(o)
    for _ in range(10):
        assert ds41.prompt_attn_fwd(q, k, v, c, c, 100, 0.1, o=o, lse=lse) is o
    assert sys.getrefcount(o) == refs and torch.equal(o, want[1])
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    got = ds41.kv_cache_read(cache, rows, cu([150]), 150, k=k2, v=v2)
    assert got[0] is k2 and got[1] is v2 and torch.equal(k2, want[2])


def test_workspace_given():
    g = gen(76)
    a = tree_inputs(g, [700], [1], 8, 2, 64, 32, True)
    need = int(ds41.load().ds41_tree_attn_workspace_bytes(1, 1, 1, 700, 8, 2, 64, 0, 1))
    want = ds41.tree_attn_fwd(*a)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # whatever it holds
    assert torch.equal(ds41.tree_attn_fwd(*a, ws=ws), want)
    with pytest.raises(ValueError):
        ds41.tree_attn_fwd(*a, ws=ws[:need - 1])
    assert ds41.load().ds41_tree_attn_workspace_bytes(1, 1, 1, 700, 8, 3, 64, 0, 1) == 0


def test_binding_refuses_wrong_tensors():
    g = gen(77)
    q, cache, table, lens, c, mq, ml, scale = tree_inputs(g, [70], [2], 8, 2, 64, 32, True)
    for bad in (dict(q=q[:, :, :48]), dict(q=q.float()), dict(table=table.long()),
                dict(lens=lens.long()), dict(cache=cache._replace(v_scales=None)),
                dict(cache=cache._replace(k_scales=cache.k_scales[:1])),
                dict(cache=cache._replace(v=cache.v[:1])), dict(c=c.cpu())):
        x = dict(q=q, cache=cache, table=table, lens=lens, c=c) | bad
        with pytest.raises(ValueError):
            ds41.tree_attn_fwd(x["q"], x["cache"], x["table"], x["lens"], x["c"], mq, ml, scale)
    with pytest.raises(ValueError):
        ds41.tree_attn_fwd(q, cache, table, lens, c, mq, ml, scale, o=torch.empty_like(q)[:1])
    with pytest.raises(ValueError):
        ds41.tree_attn_fwd(q, cache, table, lens, c, mq, ml, scale,
                           mask=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ds41.DS41Error) as e:
        ds41.tree_attn_fwd(q, cache, table, lens, c, mq, ml, scale, window=1)
    assert e.value.code == 1
    k = randn(g, 5, 2, 64)
    with pytest.raises(ValueError):
        ds41.kv_cache_write(cache, k, k[:4], torch.zeros(5, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ds41.kv_cache_write(cache, k, k, torch.zeros(5, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ds41.prompt_attn_fwd(q, k, k[:, :1], c, c, 2, 0.1)
    # a broadcast of one head is no layout of heads
    with pytest.raises(ds41.DS41Error) as e:
        ds41.prompt_attn_fwd(q, k[:, :1].expand(5, 2, 64), k, c, c, 2, 0.1)
    assert e.value.code == 1
