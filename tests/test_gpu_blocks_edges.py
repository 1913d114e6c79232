"""Where block attention, its selection, the pages and beam search could go wrong beside the
plain cases: keys that are no numbers in other tokens' blocks, scores of any size, long
lists, tables in pieces, offsets past 2^31, two streams, equal offers in masses."""
import math

import pytest
import torch

import blocks_ref as br
import dense_ref as ref
import test_gpu_blocks as blocks
from compressed_sparse_attention_window_gb300 import ds41
from test_gpu_blocks import DEV, cu, filled_cache, gen, ints, randn, random_lists, sequence, tables
from test_gpu_dense_attention_edges import aligned, close_by_weight, packed_cache
from test_gpu_pages import check_beam, filled_keys

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


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_keys_of_other_tokens_blocks_may_be_anything(what, hd):
    """Token 5 lists a block whose keys are no numbers, its neighbours in the tile do not:
    theirs are what they would be without it."""
    g = gen(1)
    n, block, kvh, nh = 40, 16, 2, 8
    q, k, v = randn(g, n, nh, hd), randn(g, 100, kvh, hd), randn(g, 100, kvh, hd)
    lists = [[[0, (60 + t) // block]] * kvh for t in range(n)]
    lists[5] = [[0, 2, 65 // block]] * kvh
    idx = ints([[x + [-1] * (3 - len(x)) for x in rows] for rows in lists])
    w = br.attend(q, k.double(), v.double(), lists, 60, block, 0.1, None)
    k[32:48] = what
    o, lse = torch.empty_like(q), torch.empty(n, nh, device=DEV)
    ds41.block_prompt_attn_fwd(q, k, v, cu([n]), cu([100]), n, 100, idx, block, 0.1, o=o, lse=lse)
    keep = torch.arange(n, device=DEV) != 5
    ref.close(o[keep], lse[keep], *(x[keep] for x in w))


@pytest.mark.parametrize("size", [2.0 ** -40, 1.0, 2.0 ** 22, 2.0 ** 60])
@pytest.mark.parametrize("hd", [64, 128])
def test_scores_of_any_size(size, hd):
    """Scores that are whole multiples of a large or small number, worked out exactly: all weight is
    on the largest (size 2^22 and up), even (2^-40), or as the definition has it."""
    g = gen(2)
    n, block, kvh, nh, m = 9, 32, 1, 2, 300
    step = (torch.arange(m, device=DEV) * 7 % 13).float()
    k = torch.zeros(m, kvh, hd, device=DEV)
    k[:, 0, 3] = step
    q = torch.zeros(n, nh, hd, device=DEV)
    q[:, :, 3] = 1.0
    q, k, v = q.bfloat16(), k.bfloat16(), randn(g, m, kvh, hd)
    lists = [[[1, 4, (m - n + t) // block]] for t in range(n)]
    idx = ints(lists)
    o, lse = torch.empty_like(q), torch.empty(n, nh, device=DEV)
    ds41.block_prompt_attn_fwd(q, k, v, cu([n]), cu([m]), n, m, idx, block, size, o=o, lse=lse)
    cache = ds41.make_kv_cache(12, kvh, block, hd, e4m3=False)
    ds41.kv_cache_write(cache, k, v, torch.arange(m, device=DEV))
    table = torch.arange(12, dtype=torch.int32, device=DEV)[None]
    o2, lse2 = torch.empty_like(q), torch.empty(n, nh, device=DEV)
    ds41.block_attn_fwd(q, cache, table, ints([m]), cu([n]), n, idx, size, o=o2, lse=lse2)
    for t in range(n):
        seen = [j for j in range(m - n + t + 1) if j // block in lists[t][0]]
        x = step[seen].double() * size
        p = torch.softmax(x, 0)
        want = p @ v[seen, 0].double()
        # weights to bf16, the output to bf16, the exponential and the scores' scale in f32
        tol = (p @ v[seen, 0].double().abs()) * (2.0 ** -8 + 2.0 ** -18) + want.abs() * 2.0 ** -8
        top = torch.logsumexp(x, 0).item()
        for a, b in ((o, lse), (o2, lse2)):
            assert ((a[t].double() - want).abs() <= tol).all()
            assert (b[t].double() - top).abs().max().item() <= 2.0 ** -20 * max(1.0, abs(top))


@pytest.mark.parametrize("nh,kvh,block,m,n", [(1, 1, 16, 17000, 300), (2, 1, 16, 40000, 5), (3, 3, 256, 3000, 130)])
def test_prompt_over_many_blocks(nh, kvh, block, m, n):
    """More blocks than the plan's table of masks holds at a time; masks of up to 256 tokens."""
    g = gen(m)
    hd, topk = 64, 40
    idx, lists = random_lists(g, [m], [n], kvh, block, topk)
    q, k, v = randn(g, n, nh, hd), randn(g, m, kvh, hd), randn(g, m, kvh, hd)
    o, lse = torch.empty_like(q), torch.empty(n, nh, device=DEV)
    ds41.block_prompt_attn_fwd(q, k, v, cu([n]), cu([m]), n, m, idx, block, 0.125, o=o, lse=lse)
    ref.close(o, lse, *br.attend(q, k.double(), v.double(), lists, m - n, block, 0.125, None))
    # the same bits again
    o2, lse2 = torch.empty_like(q), torch.empty(n, nh, device=DEV)
    ds41.block_prompt_attn_fwd(q, k, v, cu([n]), cu([m]), n, m, idx, block, 0.125, o=o2, lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("topk", [129, 300, 1024])
def test_long_lists(topk, e4m3):
    g = gen(topk)
    n, page, kvh, hd, nh = 16 * topk + 37, 16, 2, 64, 6
    n_pages, rows = tables(g, [n], page)
    cache = filled_cache(g, n_pages, kvh, page, hd, e4m3)
    idx, lists = random_lists(g, [n], [3], kvh, page, topk)
    q = randn(g, 3, 3 * nh, hd)[:, nh:2 * nh]  # (strided)
    k, v, vs = sequence(cache, rows[0], n, page)
    o, lse = torch.empty(3, nh, hd, dtype=torch.bfloat16, device=DEV), torch.empty(3, nh, device=DEV)
    ds41.block_attn_fwd(q, cache, ints(rows), ints([n]), cu([3]), 3, idx, 0.125, o=o, lse=lse)
    ref.close(o, lse, *br.attend(q, k, v, lists, n - 3, page, 0.125, None, vs))


def test_offsets_past_31_bits():
    """Pages whose rows lie more than 2^31 elements into the cache: copied, summed into
    block keys, attended to."""
    n_pages, kvh, page, hd = 33000, 8, 64, 128
    g = gen(3)
    cache = ds41.make_kv_cache(n_pages, kvh, page, hd)
    keys = ds41.make_block_keys(n_pages, kvh, hd)
    small = filled_cache(g, 3, kvh, page, hd, True)
    far = [n_pages - 1, n_pages - 2, n_pages - 3]
    for i, p in enumerate(far):
        for t, s in zip(cache, small):
            t[p].copy_(s[i]) if t.dtype == torch.float32 else t.view(torch.uint8)[p].copy_(s.view(torch.uint8)[i])
    table = ints([far])
    ds41.kv_block_keys(cache, keys, table, ints([150]), 150)
    want = ds41.make_block_keys(3, kvh, hd)
    ds41.kv_block_keys(small, want, ints([[0, 1, 2]]), ints([150]), 150)
    for a, b in zip(keys, want):
        assert torch.equal(a[far], b)
    q = randn(g, 1, 16, hd)
    one, idx = cu([1]), ints([[[0, 1, 2]] * kvh])
    o = ds41.block_attn_fwd(q, cache, table, ints([150]), one, 1, idx, 0.1)
    assert torch.equal(o, ds41.block_attn_fwd(q, small, ints([[0, 1, 2]]), ints([150]), one, 1, idx, 0.1))
    ds41.kv_pages_copy(cache, ints(far), ints([5, 6, 7]), keys=keys)
    ds41.kv_pages_copy(cache, ints([5, 6]), ints([32990, 32991]), keys=keys)
    near = ds41.block_attn_fwd(q, cache, ints([[32990, 32991, 7]]), ints([150]), one, 1, idx, 0.1)
    assert torch.equal(o, near)
    got = ds41.block_select(q, keys, page, ints([[32990, 32991, 7]]), ints([150]), one, 1, 150, 2, 0, 1)
    assert torch.equal(got, ds41.block_select(q, want, page, ints([[0, 1, 2]]), ints([150]), one, 1, 150, 2, 0, 1))


def test_two_streams_at_once():
    """Calls of the same kind on two streams, each with scratch of its own."""
    g = gen(4)
    page, kvh, hd, nh = 16, 2, 64, 8
    jobs = []
    for i in range(2):
        n = 500 + 300 * i
        n_pages, rows = tables(g, [n], page)
        cache = filled_cache(g, n_pages, kvh, page, hd, True)
        idx, _ = random_lists(g, [n], [64], kvh, page, 9)
        x = torch.randn(2, 4, 30000 + i, generator=g, device=DEV)
        jobs.append((randn(g, 64, nh, hd), cache, ints(rows), ints([n]), idx, randn(g, n, kvh, hd), x, n))

    def run(job):
        q, cache, table, lens, idx, k, x, n = job
        out = [ds41.block_attn_fwd(q, cache, table, lens, cu64, 64, idx, 0.1),
               ds41.block_prompt_attn_fwd(q, k, k, cu64, job_cu[n], 64, n, idx, page, 0.1)]
        return out + list(ds41.beam_select(x, zero, 4))
    cu64, zero = cu([64]), torch.zeros(2, 4, device=DEV)
    job_cu = {job[-1]: cu([job[-1]]) for job in jobs}
    want = [run(job) for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(5):
        for i, (s, job) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i].append(run(job))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_alike_in_masses(dtype):
    """More equal offers than are ranked at once, in a beam and over the beams."""
    x = torch.zeros(1, 16, 9000, device=DEV, dtype=dtype)
    scores = torch.zeros(1, 16, device=DEV)
    check_beam(x, scores, 128)
    scores[0, 7] = 1.0
    check_beam(x, scores, 128)
    x[0, :, 4000:] = -math.inf
    check_beam(x, scores, 100)
    # beams that are copies of one another, in rows of every alignment
    g = gen(5)
    one = torch.randn(1, 1, 8191, generator=g, device=DEV).to(dtype)
    check_beam(one.expand(2, 9, 8191).contiguous(), torch.zeros(2, 9, device=DEV), 18)


def test_beam_many_lists():
    """Long rows in few searches: more lists than a merging thread has keys in registers."""
    g = gen(6)
    for B, W, V, k in ((1, 40, 60000, 32), (1, 3, 1000003, 128), (300, 1, 5000, 7)):
        x = torch.randn(B, W, V, generator=g, device=DEV).bfloat16()
        check_beam(x, torch.zeros(B, W, device=DEV), k)


def test_captured_reordering():
    """A beam step's selection and reordering as a graph, replayed: as eagerly."""
    g = gen(7)
    B, W, V, page, kvh, hd, P = 2, 3, 500, 16, 1, 32, 60
    lens = ints([20, 20, 37, 40, 40, 5])
    need = [2, 2, 3, 3, 3, 1]
    rows, at = [], 0
    for n in need:
        rows.append(list(range(at, at + n)) + [-1] * (4 - n))
        at += n
    cache, keys = filled_cache(g, P, kvh, page, hd, True), filled_keys(g, P, kvh, hd)
    refs = ints([1] * at + [0] * (P - at))
    tables_ = [ints(rows), torch.empty(6, 4, dtype=torch.int32, device=DEV)]
    lens_ = [lens.clone(), torch.empty_like(lens)]
    x, scores = torch.zeros(B, W, V, device=DEV), torch.zeros(B, W, device=DEV)

    def step():
        s, parents, tokens = ds41.beam_select(x, scores, W)
        ds41.kv_pages_fork(cache, refs, tables_[0], lens_[0], parents.view(-1), tables_[1], lens_[1], replace=True,
                           keys=keys)
        tables_[0].copy_(tables_[1])
        lens_[0].copy_(lens_[1])
        scores.copy_(s)
        return tokens
    state = [refs, tables_[0], lens_[0], scores] + [t.view(torch.uint8) for t in cache] + list(keys)
    begin = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = step()
    inputs = [torch.randn(B, W, V, generator=g, device=DEV) for _ in range(4)]

    def play(once):
        for t, b in zip(state, begin):
            t.copy_(b)
        out = []
        for y in inputs:
            x.copy_(y)
            out.append(once().clone())
        return out + [t.clone() for t in state]

    def replay():
        graph.replay()
        return tokens
    for a, b in zip(play(step), play(replay)):
        assert torch.equal(a, b)
    held = [p for row, n in zip(tables_[0].tolist(), lens_[0].tolist()) for p in row[:-(-n // page)]]
    assert refs.tolist() == [held.count(p) for p in range(P)]


@pytest.mark.parametrize("lens,news,nh,kvh,hd,page,topk,first,local", [
    ([9000, 40], [3, 1], 5, 1, 80, 16, 20, 1, 2), ([33000], [1], 8, 1, 128, 16, 50, 0, 1),
    ([20011, 0, 17000], [4, 0, 2], 6, 2, 64, 16, 9, 1, 1), ([16384], [2], 80, 1, 64, 16, 200, 2, 2),
    ([9000], [6], 4, 1, 128, 16, 90, 1, 2)])
def test_select_over_many_blocks(lens, news, nh, kvh, hd, page, topk, first, local):
    """More than 512 blocks, by clusters where the tokens are few; scores that repeat."""
    g = gen(sum(lens))
    n_pages, rows = tables(g, lens, page)
    keys = filled_keys(g, n_pages, kvh, hd)
    keys.scales.add_(0.01)
    keys.codes[n_pages // 2:] = keys.codes[:n_pages - n_pages // 2].clone()
    keys.scales[n_pages // 2:] = keys.scales[:n_pages - n_pages // 2].clone()
    q = randn(g, sum(news), nh, hd)
    got = ds41.block_select(q, keys, page, ints(rows), ints(lens), cu(news), max(news), max(lens), topk, first, local).tolist()
    codes, scales = keys.codes.double(), keys.scales.double()
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        mine = torch.tensor(rows[b][:-(-n // page)], device=DEV, dtype=torch.long)
        for i in range(m):
            for h in range(kvh):
                w = br.picks(q[at + i, h * nh // kvh:(h + 1) * nh // kvh], codes[mine, h], scales[mine, h], n - m + i,
                             page, topk, first, local)
                assert got[at + i][h] == w + [-1] * (topk - len(w)), (b, i, h)
        at += m


def test_select_equal_scores_of_many_blocks():
    """Thousands of blocks alike, or in two kinds: the lowest are taken."""
    page, kvh, hd, topk, n = 16, 1, 64, 70, 60000
    NB = n // page
    table = torch.arange(NB, dtype=torch.int32, device=DEV)[None]
    keys = ds41.make_block_keys(NB, kvh, hd)
    keys.codes.fill_(3)
    keys.scales.fill_(0.5)
    q = torch.ones(1, 2, hd, dtype=torch.bfloat16, device=DEV)
    for k in (topk, 20):
        got = ds41.block_select(q, keys, page, table, ints([n]), cu([1]), 1, n, k, 1, 2)
        assert got[0, 0].tolist() == list(range(k - 2)) + [NB - 2, NB - 1]
    keys.scales[1000:1005] = 1.0
    got = ds41.block_select(q, keys, page, table, ints([n]), cu([1]), 1, n, 20, 1, 2)
    assert got[0, 0].tolist() == list(range(13)) + list(range(1000, 1005)) + [NB - 2, NB - 1]


@pytest.mark.parametrize("behind", [[-7, -5, -3], [-(1 << 31), -(1 << 30), -(1 << 29)], [1 << 30, -(1 << 30), 0], [-2, -1, 0]])
def test_entries_behind_a_lists_end_may_be_anything(behind):
    """Entries below 0 that rise, or far outside the table, behind the one that ends the list."""
    g = gen(21)
    n, page = 100, 16
    n_pages, rows = tables(g, [n], page)
    cache = filled_cache(g, n_pages, 1, page, 64, False)
    q = randn(g, 1, 4, 64)
    k, v, _ = sequence(cache, rows[0], n, page)
    w = br.attend(q, k, v, [[[2]]], n - 1, page, 0.1, None)
    i = ints([[[2] + behind]])
    o, lse = torch.empty_like(q), torch.empty(1, 4, device=DEV)
    ds41.block_attn_fwd(q, cache, ints(rows), ints([n]), cu([1]), 1, i, 0.1, o=o, lse=lse)
    assert ds41.device_status() == 4
    ref.close(o, lse, *w)
    ds41.block_prompt_attn_fwd(q, k.bfloat16(), v.bfloat16(), cu([1]), cu([n]), 1, n, i, page, 0.1, o=o, lse=lse)
    assert ds41.device_status() == 4
    ref.close(o, lse, *w)


def test_beam_scores_in_place():
    """out_scores may be scores: a search's are read before they are written."""
    g = gen(22)
    x, scores = randn(g, 30, 6, 9000).float(), -torch.rand(30, 6, generator=g, device=DEV)
    want = [t.clone() for t in ds41.beam_select(x, scores, 6)]
    for _ in range(3):
        s = scores.clone()
        got = ds41.beam_select(x, s, 6, out_scores=s)
        assert got[0] is s and all(torch.equal(a, b) for a, b in zip(got, want))


def test_beam_offers_that_f32_does_not_hold():
    """-3e38 - 3e38 is no f32: such offers are none, whichever beam they are of."""
    x = torch.zeros(1, 3, 10, device=DEV)
    x[0, 0, 4:] = -3e38
    s = torch.tensor([[-3e38, -math.inf, -1.0]], device=DEV)
    ended = torch.tensor([[False, False, True]], device=DEV)
    out, parents, tokens = ds41.beam_select(x, s, 8, ended=ended, end_token=7)
    assert parents.tolist() == [[2, 0, 0, 0, 0, -1, -1, -1]] and tokens.tolist() == [[7, 0, 1, 2, 3, -1, -1, -1]]
    assert out[0, 0] == -1 and (out[0, 5:] == -math.inf).all()
    assert torch.allclose(out[0, 1:5], torch.tensor(-3e38, device=DEV), rtol=2.0 ** -23)


def test_nothing_to_do():
    """No sequences, no tokens, no children: nothing happens, and parents without children
    give their pages back."""
    g = gen(23)
    cache, keys = filled_cache(g, 6, 2, 16, 64, True), filled_keys(g, 6, 2, 64)
    before = [t.clone().view(torch.uint8) for t in list(cache) + list(keys)]
    refs, none, table = ints([1, 1, 0, 2, 0, 0]), ints([]), ints([[0, 1, 3]])
    ds41.kv_pages_take(refs, table[:0], none, none, 16)
    ds41.kv_pages_free(refs, table[:0], none, 16)
    out, lens = ds41.kv_pages_fork(cache, refs, table, ints([40]), none, keys=keys)
    assert out.shape == (0, 3) and lens.shape == (0,)
    ds41.kv_pages_copy(cache, none, none, keys=keys)
    out, lens = ds41.kv_pages_fork(cache, refs, table[:0], none, ints([-1, -1]), keys=keys)
    assert out.tolist() == [[-1] * 3] * 2 and lens.tolist() == [0, 0]
    assert refs.tolist() == [1, 1, 0, 2, 0, 0]
    ds41.kv_pages_fork(cache, refs, table, ints([40]), none, replace=True, keys=keys)
    assert refs.tolist() == [0, 0, 0, 1, 0, 0]
    ds41.kv_block_keys(cache, keys, table, ints([40]), 0, starts=ints([40]))
    q = randn(g, 0, 4, 64)
    idx = ds41.block_select(q, keys, 16, table, ints([40]), cu([0]), 1, 48, 3, first=1, local=1)
    assert idx.shape == (0, 2, 3)
    assert ds41.block_attn_fwd(q, cache, table, ints([40]), cu([0]), 1, idx, 0.1).shape == q.shape
    k = randn(g, 0, 2, 64)
    assert ds41.block_prompt_attn_fwd(q, k, k, cu([0]), cu([0]), 0, 0, idx, 16, 0.1).shape == q.shape
    s, p, t = ds41.beam_select(randn(g, 0, 2, 9), torch.zeros(0, 2, device=DEV), 4)
    assert s.shape == p.shape == t.shape == (0, 4)
    for a, b in zip(list(cache) + list(keys), before):
        assert torch.equal(a.view(torch.uint8), b)


def test_keys_without_values():
    """Prompts whose keys are none but whose queries are: refused sequence by sequence, outputs
    as they were."""
    g = gen(24)
    q, k = randn(g, 3, 4, 64), randn(g, 0, 2, 64)
    o, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device=DEV)
    ds41.block_prompt_attn_fwd(q, k, k, cu([3]), cu([0]), 3, 16, ints([[[0]] * 2] * 3), 16, 0.1, o=o, lse=lse)
    assert ds41.device_status() == 4
    assert (o == 7).all() and (lse == 7).all()


def some_blocks(g, d, n, page, share):
    """Lists for d tokens at n - d .. n - 1, alike for all heads: a token's own block and `share`
    of the others; what each sees of the n rows."""
    lists, seen = [], torch.zeros(d, n, dtype=torch.bool)
    for t in range(d):
        cur = (n - d + t) // page
        keep = torch.rand(cur, generator=g, device=DEV).tolist()
        lists.append([x for x in range(cur) if keep[x] < share] + [cur])
        for x in lists[-1]:
            seen[t, x * page:min((x + 1) * page, n - d + t + 1)] = True
    width = max(map(len, lists))
    return [x + [-1] * (width - len(x)) for x in lists], seen.to(DEV)


def run_tokens(g, q, cache, table, n, kvh, page, share, sink=None):
    d, nh, hd = q.shape
    lists, seen = some_blocks(g, d, n, page, share)
    idx = ints([[x] * kvh for x in lists])
    o, lse = torch.empty_like(q), torch.empty(d, nh, device=DEV)
    ds41.block_attn_fwd(q, cache, table, ints([n]), cu([d]), d, idx, hd ** -0.5, sink=sink, o=o, lse=lse)
    close_by_weight(q, cache, table, n, seen, (o, lse), sink)


TILES = [(2, 8, 2), (3, 8, 1), (2, 18, 2), (1, 20, 1)]  # tokens, heads: 4, 8, 9 and 20 of a group


@pytest.mark.parametrize("spread", [6, 20, 50])
@pytest.mark.parametrize("d,nh,kvh", TILES)
@pytest.mark.parametrize("n,share", [(64, 1.0), (3000, 0.5)])
def test_tokens_value_scales_far_apart(n, share, d, nh, kvh, spread):
    g = gen(n + spread + nh)
    q, k, v = randn(g, d, nh, 128), randn(g, n, kvh, 128) * 3.0, randn(g, n, kvh, 128)
    cache, table = packed_cache(k, v, 64, True)
    e = torch.randint(-spread, spread + 1, cache.v_scales.shape, generator=g, device=DEV)
    cache.v_scales.mul_(torch.exp2(e.float()))
    for sink in (None, torch.randn(nh, generator=g, device=DEV)):
        run_tokens(g, q, cache, table, n, kvh, 64, share, sink)


@pytest.mark.parametrize("gain", [2.0 ** 8, 2.0 ** 20, 2.0 ** 40])
@pytest.mark.parametrize("d,nh,kvh", TILES)
@pytest.mark.parametrize("hd", [64, 128])
def test_tokens_large_value_row_of_little_weight(hd, d, nh, kvh, gain):
    q, k, v = aligned(gen(hd + nh), d, nh, 800, kvh, hd)
    k[300, :, 0] = -300.0
    v[300] *= gain
    cache, table = packed_cache(k, v, 32, True)
    run_tokens(gen(1), q, cache, table, 800, kvh, 32, 1.0)


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -60, 2.0 ** 60, 2.0 ** 96])
@pytest.mark.parametrize("d,nh,kvh", TILES)
def test_tokens_values_all_small_or_all_large(d, nh, kvh, size):
    g = gen(nh)
    q, k, v = randn(g, d, nh, 64), randn(g, 900, kvh, 64), randn(g, 900, kvh, 64) * size
    v[5] = 0.0
    cache, table = packed_cache(k, v, 128, True)
    run_tokens(g, q, cache, table, 900, kvh, 128, 0.8)


@pytest.mark.parametrize("d,nh,kvh", TILES)
def test_tokens_queries_with_outliers(d, nh, kvh):
    """A channel 1000 times the rest, a zero query, one next to nothing."""
    g = gen(nh + 1)
    q, k, v = randn(g, d, nh, 128), randn(g, 700, kvh, 128), randn(g, 700, kvh, 128)
    q[:, :, 5] *= 1000.0
    q[0, 1] = 0.0
    q[0, 2] *= 2.0 ** -90
    cache, table = packed_cache(k, v, 16, True)
    run_tokens(g, q, cache, table, 700, kvh, 16, 0.7)


@pytest.mark.parametrize("lens,nh,block", [
    ([70, 3, 0, 41], 16, 16), ([600, 3, 700], 128, 32), ([0, 0, 530], 128, 64), ([17] * 64, 32, 16),
    ([x * 7 % 31 for x in range(64)], 16, 32), ([x * 5 % 23 for x in range(65)], 16, 16),
    ([x % 4 for x in range(300)], 64, 16)])
def test_prompt_of_many_sequences(lens, nh, block):
    """Pairs of tiles of all sequences, the latest first, or sequence by sequence; some empty."""
    blocks.test_prompt(lens, 20, nh, 1, 32, block, 3, True)


def test_prompt_with_sequences_that_are_skipped():
    """Sequences that break their limits between others, whose results are as without them."""
    g = gen(25)
    lens, nh, kvh, hd, block = [40, 90, 33, 7], 16, 2, 64, 16
    q, k = randn(g, sum(lens), nh, hd), randn(g, sum(lens), kvh, hd)
    idx = ints([[[0, min(3, t // block)][:1 + (t >= block)] + [-1] * (t < block)] * kvh for n in lens for t in range(n)])
    o, want = torch.full_like(q, 7.0), torch.empty_like(q)
    ds41.block_prompt_attn_fwd(q, k, k, cu(lens), cu(lens), 90, 90, idx, block, 0.1, o=want)
    ds41.block_prompt_attn_fwd(q, k, k, cu(lens), cu(lens), 89, 90, idx, block, 0.1, o=o)
    assert ds41.device_status() == 4
    assert (o[40:130] == 7).all() and torch.equal(o[:40], want[:40]) and torch.equal(o[130:], want[130:])
