"""What is measured of the operators of sparse serving: attention over blocks of the
paged cache that a cheap score selects for each query (block keys and selection, single
tokens over pages, packed prompts), the cache's pages (forked with their last rows
copied, freed, compacted), and beam search's selection over beams and vocabulary.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, calls the framework's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
STEPS = 127  # of a block key's codes to either side
TINY = 2.0 ** -126


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one sequence's beam step, a small vocabulary: latency
        dict(name="beam_one", op="beam", batch=1, beams=4, vocab=32000, k=8, fmt="f32", ended=False, shape=1),
        # the beams of a batch over a large vocabulary of odd size, some of them ended
        dict(name="beam_batch", op="beam", batch=64, beams=8, vocab=129281, k=16, fmt="bf16", ended=True, shape=2),
        # a beam step's reordering: every beam of 16 searches goes on from one of its search's beams
        dict(name="fork_beams", op="fork", batch=64, groups=16, children=64, max_len=2000, kvh=8, hd=128, page=64, fmt="e4m3", replace=True, shape=3),
        # prompts forked into the samples that are drawn from each, and the samples freed
        dict(name="fork_samples", op="fork", batch=8, groups=8, children=256, max_len=16383, kvh=8, hd=128, page=64, fmt="bf16", replace=False, shape=4),
        # a small pool after most of its sequences have ended
        dict(name="compact_small", op="compact", pages=300, live=0.3, kvh=2, hd=128, page=16, fmt="e4m3", shape=5),
        # a large pool, to be cut to what lives
        dict(name="compact_large", op="compact", pages=4099, live=0.6, kvh=8, hd=128, page=64, fmt="bf16", shape=6),
        # a decode step's selection: the new rows' block keys, then 64 blocks of up to 512 for each token
        dict(name="select_step", op="select", batch=24, max_q=1, max_len=32768, nh=32, kvh=8, hd=128, page=64, fmt="e4m3", topk=64, first=1, local=2, shape=7),
        # a prompt chunk's selection behind earlier rows
        dict(name="select_chunk", op="select", batch=1, max_q=8192, max_len=32768, nh=32, kvh=8, hd=128, page=64, fmt="bf16", topk=32, first=1, local=2, shape=8),
        # one sequence's next token over a few small blocks: latency
        dict(name="tokens_one", op="tokens", batch=1, max_q=1, max_len=5000, nh=16, kvh=2, hd=64, page=16, fmt="bf16", topk=12, sink=False, shape=9),
        # the next tokens of a batch over long caches
        dict(name="tokens_batch", op="tokens", batch=16, max_q=1, max_len=32768, nh=64, kvh=8, hd=128, page=64, fmt="e4m3", topk=64, sink=True, shape=10),
        # prompts of odd lengths, packed, each token with blocks of its own
        dict(name="prompt_packed", op="prompt", batch=6, max_len=2001, prior=0, nh=16, kvh=2, hd=64, page=32, topk=12, alike=1, sink=True, shape=11),
        # a chunk of a long prompt behind earlier rows, neighbours' blocks mostly alike
        dict(name="prompt_chunk", op="prompt", batch=1, max_len=8192, prior=24576, nh=32, kvh=8, hd=128, page=64, topk=32, alike=32, sink=False, shape=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["beam", "fork", "compact", "select", "tokens", "tokens", "prompt", "prompt"])
    shape = rng.randrange(1 << 30)
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _log(rng, 500, 160000)
        batch = min(_log(rng, 1, 64), max(1, 64 * 8 * 129281 // (beams * vocab) // 2))
        return dict(op=op, batch=batch, beams=beams, vocab=vocab, k=beams * rng.choice([1, 2]), fmt=rng.choice(["f32", "bf16", "bf16"]),
                    ended=rng.random() < 0.5, shape=shape)
    kvh = rng.choice([1, 2, 4, 8])
    hd = rng.choice([64, 128, 128, 80, 96])
    page, fmt = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "e4m3", "bf16"])
    if op == "fork":
        groups = _log(rng, 1, 16)
        batch = groups * rng.choice([1, 2, 4])
        return dict(op=op, batch=batch, groups=groups, children=_log(rng, 1, 256), max_len=_log(rng, 1, 8000), kvh=kvh, hd=hd, page=page,
                    fmt=fmt, replace=rng.random() < 0.5, shape=shape)
    if op == "compact":
        return dict(op=op, pages=_log(rng, 16, 4000), live=rng.choice([0.1, 0.3, 0.6, 0.9]), kvh=kvh, hd=hd, page=min(page, 64), fmt=fmt, shape=shape)
    nh = kvh * rng.choice([1, 2, 4, 5, 8] if kvh < 8 else [1, 4, 8])
    topk = _log(rng, 4, 64)
    if op == "select":
        max_q = rng.choice([1, 1, _log(rng, 2, 2000)])
        max_len = _log(rng, max(64, max_q), 32768)
        batch = min(_log(rng, 1, 24), max(1, 100000 // max_len), max(1, 3000 // max_q))
        return dict(op=op, batch=batch, max_q=max_q, max_len=max_len, nh=nh, kvh=kvh, hd=hd, page=page, fmt=fmt, topk=topk,
                    first=rng.choice([0, 1]), local=rng.choice([1, 2, 3]), shape=shape)
    if op == "tokens":
        max_q = rng.choice([1, 1, 1, _log(rng, 2, 8)])
        max_len = _log(rng, 64, 32768)
        batch = min(_log(rng, 1, 48), max(1, 250000 // max_len), max(1, 500000 // (max_q * topk * page)))
        return dict(op=op, batch=batch, max_q=max_q, max_len=max_len, nh=nh, kvh=kvh, hd=hd, page=page, fmt=fmt, topk=topk,
                    sink=rng.random() < 0.5, shape=shape)
    max_len = _log(rng, 1, 6000)
    batch = min(_log(rng, 1, 16), max(1, 6000 // max_len))
    return dict(op=op, batch=batch, max_len=max_len, prior=rng.choice([0, 0, _log(rng, 1, 8000)]), nh=nh, kvh=kvh, hd=hd, page=page,
                topk=topk, alike=rng.choice([1, 8, 32]), sink=rng.random() < 0.5, shape=shape)


def _lens(c):
    """The sequences' lengths: the longest is max_len, the others are spread below it."""
    r = random.Random(c["shape"])
    lo = max(c.get("max_q", 1), c["max_len"] // 8, 1)
    return [c["max_len"]] + [r.randint(lo, c["max_len"]) for _ in range(c["batch"] - 1)]


def _queries(c):
    """The new tokens of each sequence: max_q for the first, the others at least half of that."""
    r = random.Random(c["shape"] + 1)
    return [c["max_q"]] + [r.randint((c["max_q"] + 1) // 2, c["max_q"]) for _ in range(c["batch"] - 1)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _ints(at)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _keys(g, *shape):
    """Keys as trained models have them: a few channels larger than the rest."""
    k = _randn(g, *shape)
    k[..., :4] *= 3.0
    return k


def _quantise(x):
    """x [..., hd] to e4m3 with one scale for each row."""
    x = x.float()
    s = x.abs().amax(-1).clamp_min(E4M3_MAX * TINY) / E4M3_MAX
    return (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn), s


def _cache(g, c, n_pages):
    """A cache that holds rows already: [page, head, row of the page, hd], K and V, and the scales."""
    shape = (n_pages, c["kvh"], c["page"], c["hd"])
    k, v = _keys(g, *shape), _randn(g, *shape)
    if c["fmt"] == "bf16":
        return dict(k=k.bfloat16(), v=v.bfloat16(), k_scales=None, v_scales=None)
    (kc, ks), (vc, vs) = _quantise(k.bfloat16()), _quantise(v.bfloat16())
    return dict(k=kc, v=vc, k_scales=ks, v_scales=vs)


def _pages(g, c, lens):
    """Each sequence's pages, in no order, among some that belong to nobody."""
    need = [-(-n // c["page"]) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return n_pages, table


def _listed_blocks(g, c, cur, alike):
    """For each token and head ascending block numbers up to its own block `cur` [T], -1 behind them: the first block, the last
    two, others at random, mostly the same ones for `alike` tokens one after another."""
    T, kvh, topk = len(cur), c["kvh"], c["topk"]
    n = int(cur.max()) + 1
    x = torch.rand(T, kvh, n, generator=g, device=DEV)
    if alike > 1:
        shared = torch.rand(-(-T // alike), kvh, n, generator=g, device=DEV).repeat_interleave(alike, 0)[:T]
        x = shared + 0.05 * x
    b = torch.arange(n, device=DEV)
    x = torch.where(((b == 0) | (b > cur[:, None] - 2))[:, None], 3.0, x)
    x = torch.where((b > cur[:, None])[:, None], -1.0, x)
    if n < topk:
        x = torch.cat([x, x.new_full((T, kvh, topk - n), -1.0)], 2)
    best, at = x.topk(topk, -1)
    at = torch.where(best < 0, 1 << 30, at).sort(-1).values
    return torch.where(at == 1 << 30, -1, at).to(torch.int32)


def _pool(c):
    """The sequences of a fork: each group's share the pages of a common beginning, and have the rest for themselves.
    Returns their lengths, pages, the parents of the children and the pool's size."""
    r = random.Random(c["shape"])
    per, page = c["batch"] // c["groups"], c["page"]
    lens, owned, used = [], [], 0
    for gr in range(c["groups"]):
        n = c["max_len"] if gr == 0 else r.randint(max(1, c["max_len"] // 8), c["max_len"])
        need, shared = -(-n // page), 0
        if per > 1:
            shared = r.randint(n // page // 2, n // page)
        common = list(range(used, used + shared))
        used += shared
        for _ in range(per):
            owned.append(common + list(range(used, used + need - shared)))
            used += need - shared
            lens.append(n)
    if c["children"] == c["batch"]:  # every beam from one of its own group
        parents = [i // per * per + r.randrange(per) for i in range(c["children"])]
    else:
        parents = [i * c["batch"] // c["children"] if c["children"] > c["batch"] else r.randrange(c["batch"]) for i in range(c["children"])]
    return lens, owned, parents, used + c["children"] + 5


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + c["shape"] % 1000)
    if c["op"] == "beam":
        B, W, V = c["batch"], c["beams"], c["vocab"]
        logits = _randn(g, B, W, V) * 2.5
        logits += 8.0 * (torch.rand(B, W, V, generator=g, device=DEV) < 6.0 / V)  # the few tokens that fit
        scores = -(torch.rand(B, W, generator=g, device=DEV) * 2.0).cumsum(1) - 5.0
        ended = torch.rand(B, W, generator=g, device=DEV) < 0.2 if c["ended"] else None
        return dict(c=c, logits=logits if c["fmt"] == "f32" else logits.bfloat16(), scores=scores, ended=ended)
    if c["op"] == "fork":
        lens, owned, parents, n_pages = _pool(c)
        order = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        width = max(len(p) for p in owned) + 1
        table = _ints([[order[p] for p in pages] + [-1] * (width - len(pages)) for pages in owned])
        count = [0] * n_pages
        for pages in owned:
            for p in pages:
                count[order[p]] += 1
        out = torch.full((c["children"], width), -1, dtype=torch.int32, device=DEV)
        return dict(c=c, cache=_cache(g, c, n_pages), refs=_ints(count), refs_before=_ints(count), table=table, lens=_ints(lens),
                    parents=_ints(parents), out=out, out_lens=torch.zeros(c["children"], dtype=torch.int32, device=DEV))
    if c["op"] == "compact":
        r = random.Random(c["shape"])
        P, page = c["pages"], c["page"]
        n_live = max(1, min(P, int(P * c["live"])))
        lens, left = [], n_live
        while left:
            n = min(left, r.randint(1, max(1, n_live // 4)))
            lens.append((n - 1) * page + r.randint(1, page))
            left -= n
        order = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
        need = [-(-n // page) for n in lens]
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        refs[order[:n_live].long()] = 1
        return dict(c=c, cache=_cache(g, c, P), refs=refs.clone(), refs_before=refs, table=table.clone(), table_before=table, lens=_ints(lens))
    if c["op"] == "prompt":
        lens = _lens(c)
        lens_k = [n + c["prior"] for n in lens]
        q = _randn(g, sum(lens), c["nh"], c["hd"]).bfloat16()
        k = _keys(g, sum(lens_k), c["kvh"], c["hd"]).bfloat16()
        v = _randn(g, sum(lens_k), c["kvh"], c["hd"]).bfloat16()
        cur = torch.cat([torch.arange(n, device=DEV) + c["prior"] for n in lens]) // c["page"]
        return dict(c=c, q=q, k=k, v=v, cu_q=_cu(lens), cu_k=_cu(lens_k), max_q=max(lens), max_k=max(lens_k), lens=lens, scale=c["hd"] ** -0.5,
                    sink=_randn(g, c["nh"]) if c["sink"] else None, idx=_listed_blocks(g, c, cur, c["alike"]))
    lens, news = _lens(c), _queries(c)
    n_pages, table = _pages(g, c, lens)
    s = dict(c=c, cache=_cache(g, c, n_pages), table=table, lens=_ints(lens), cu_q=_cu(news), max_q=max(news), max_len=max(lens))
    s["q"] = _randn(g, sum(news), c["nh"], c["hd"]).bfloat16()
    if c["op"] == "select":
        s["starts"] = _ints([n - m for n, m in zip(lens, news)])
        s["keys"] = dict(codes=torch.zeros(n_pages, c["kvh"], c["hd"], dtype=torch.int8, device=DEV),
                         scales=torch.zeros(n_pages, c["kvh"], device=DEV))
        _plain_keys(s, torch.zeros_like(s["starts"]), max(lens))  # those of the earlier rows
        return s
    cur = torch.cat([torch.arange(n - m, n, device=DEV) for n, m in zip(lens, news)]) // c["page"]
    return s | dict(scale=c["hd"] ** -0.5, sink=_randn(g, c["nh"]) if c["sink"] else None, idx=_listed_blocks(g, c, cur, 1))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["c"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _ds41():
    from compressed_sparse_attention_window_gb300 import ds41
    return ds41


def _own_beam(s):
    scores, parents, tokens = _ds41().beam_select(s["logits"], s["scores"], s["c"]["k"], ended=s["ended"], end_token=2)
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _own_fork(s):
    d = _ds41()
    cache = d.KvCache(**s["cache"])
    if s["c"]["replace"]:
        s["refs"].copy_(s["refs_before"])  # so that the pass can be repeated
        d.kv_pages_fork(cache, s["refs"], s["table"], s["lens"], s["parents"], s["out"], s["out_lens"], replace=True)
        return s["cache"] | {"refs": s["refs"], "table": s["out"], "lens": s["out_lens"]}
    d.kv_pages_fork(cache, s["refs"], s["table"], s["lens"], s["parents"], s["out"], s["out_lens"])
    d.kv_pages_free(s["refs"], s["out"], s["out_lens"], s["c"]["page"])
    return s["cache"] | {"refs": s["refs"], "table": s["out"], "lens": s["out_lens"]}


def _own_compact(s):
    d = _ds41()
    s["refs"].copy_(s["refs_before"])  # so that the pass can be repeated
    s["table"].copy_(s["table_before"])
    live = d.kv_pages_compact(d.KvCache(**s["cache"]), s["refs"], s["table"], s["lens"])
    return s["cache"] | {"refs": s["refs"], "table": s["table"], "live": live}


def _own_select(s):
    d, c = _ds41(), s["c"]
    keys = d.BlockKeys(**s["keys"])
    d.kv_block_keys(d.KvCache(**s["cache"]), keys, s["table"], s["lens"], s["max_q"], starts=s["starts"])
    idx = d.block_select(s["q"], keys, c["page"], s["table"], s["lens"], s["cu_q"], s["max_q"], s["max_len"], c["topk"],
                         first=c["first"], local=c["local"])
    return s["keys"] | {"idx": idx}


def _own_tokens(s):
    d = _ds41()
    lse = torch.empty(s["q"].shape[:2], device=DEV)
    o = d.block_attn_fwd(s["q"], d.KvCache(**s["cache"]), s["table"], s["lens"], s["cu_q"], s["max_q"], s["idx"], s["scale"],
                         sink=s["sink"], lse=lse)
    return {"o": o, "lse": lse}


def _own_prompt(s):
    lse = torch.empty(s["q"].shape[:2], device=DEV)
    o = _ds41().block_prompt_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], s["idx"], s["c"]["page"],
                                      s["scale"], sink=s["sink"], lse=lse)
    return {"o": o, "lse": lse}


def _plain_beam(s):
    k = s["c"]["k"]
    x = s["logits"].double()  # candidates next to each other differ by less than 32 bits hold
    B, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    x = s["scores"].double().unsqueeze(-1) + (x - lse)
    if s["ended"] is not None:  # an ended beam goes on as it is, under the end token
        x = torch.where(s["ended"].unsqueeze(-1), -math.inf, x)
        x[..., 2] = torch.where(s["ended"], s["scores"].double(), x[..., 2])
    best, at = x.view(B, W * V).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    if best.shape[1] < k:
        best = torch.cat([best, best.new_full((B, k - best.shape[1]), -math.inf)], 1)
        at = torch.cat([at, at.new_zeros(B, k - at.shape[1])], 1)
    real = best > -math.inf
    parents = torch.where(real, at // V + W * torch.arange(B, device=DEV)[:, None], -1)
    return {"scores": best.float(), "parents": parents.to(torch.int32), "tokens": torch.where(real, at % V, -1).to(torch.int32)}


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_fork(s):
    c, cache = s["c"], s["cache"]
    page, replace = c["page"], c["replace"]
    if replace:
        s["refs"].copy_(s["refs_before"])
    refs, table, parents = s["refs"], s["table"], s["parents"].long()
    B, width = table.shape
    lens = s["lens"].long()
    i = torch.arange(width, device=DEV)
    whole, part = lens // page, lens % page  # whole pages, and rows of the last one
    born = torch.zeros(B, dtype=torch.long, device=DEV).index_add_(0, parents, torch.ones_like(parents))
    # the first child of a parent that is replaced takes its last page over
    ids = torch.arange(len(parents), device=DEV)
    first = torch.full((B,), len(parents), dtype=torch.long, device=DEV).scatter_reduce_(0, parents, ids, "amin")
    heir = (first[parents] == ids) if replace else torch.zeros_like(ids, dtype=torch.bool)
    change = torch.where(i < whole[:, None], born[:, None] - int(replace), 0)
    if replace:
        change -= ((i == whole[:, None]) & (part > 0)[:, None] & (born == 0)[:, None]).long()
    refs.index_add_(0, table.long().clamp_min(0).view(-1), change.view(-1).to(torch.int32))
    needy = (part[parents] > 0) & ~heir
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)  # the free pages first, in order
    fresh = free[(needy.cumsum(0) - 1).clamp_min(0)]
    last = table.long()[parents, whole[parents].clamp_max(width - 1)].clamp_min(0)
    to = torch.where(needy, fresh, last)
    refs.index_add_(0, fresh, needy.to(torch.int32))
    which = torch.nonzero(needy)[:, 0]
    src, dst, rows = last[which], fresh[which], part[parents][which]
    copied = torch.arange(page, device=DEV) < rows[:, None]  # [copies, page]
    for name in ("k", "v", "k_scales", "v_scales"):
        if cache[name] is not None:
            t = _bytes_of(cache[name])
            t[dst] = torch.where(copied[:, None, :, None] if t.dim() == 4 else copied[:, None], t[src], t[dst])
    wp = whole[parents][:, None]
    s["out"].copy_(torch.where(i < wp, table[parents], torch.where((i == wp) & (part[parents] > 0)[:, None], to[:, None].to(torch.int32), -1)))
    s["out_lens"].copy_(s["lens"][parents])
    if not replace:  # the samples end
        used = i < (-(-s["out_lens"].long() // page))[:, None]
        refs.index_add_(0, s["out"].long().clamp_min(0).view(-1), -used.view(-1).to(torch.int32))
    return cache | {"refs": refs, "table": s["out"], "lens": s["out_lens"]}


def _plain_compact(s):
    c, cache = s["c"], s["cache"]
    s["refs"].copy_(s["refs_before"])
    s["table"].copy_(s["table_before"])
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n = live.sum()
    p = torch.arange(len(refs), device=DEV)
    src, dst = torch.nonzero(live & (p >= n))[:, 0], torch.nonzero(~live & (p < n))[:, 0]
    for name in ("k", "v", "k_scales", "v_scales"):
        if cache[name] is not None:
            t = _bytes_of(cache[name])
            t[dst] = t[src]
    to = p.to(torch.int32)
    to[src] = dst.to(torch.int32)
    refs[dst] = refs[src]
    refs[src] = 0
    used = torch.arange(table.shape[1], device=DEV) < (-(-s["lens"].long() // c["page"]))[:, None]
    table.copy_(torch.where(used, to[table.long().clamp_min(0)], table))
    return cache | {"refs": refs, "table": table, "live": n.to(torch.int32).view(1)}


def _rows_of(x, scales, at, off):
    """Cache rows [..., kvh, hd] as 32-bit values: page `at`, row `off` of the page."""
    if scales is None:
        return x[at, :, off].float()
    return x.view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).float() * scales[at, :, off].unsqueeze(-1)


def _int8(x):
    """Rows [..., hd] in 32 bits -> codes of -127 .. 127 and the scales; a row that is not finite: codes of 0, the scale NaN."""
    s = x.abs().amax(-1).clamp_min(STEPS * TINY) * (1.0 / STEPS)
    bad = ~torch.isfinite(x).all(-1)
    codes = torch.where(bad.unsqueeze(-1), 0.0, torch.round(x / s.unsqueeze(-1)))
    return codes, torch.where(bad, math.nan, s)


def _plain_keys(s, starts, max_new):
    """The block keys of the pages from row starts[b] on: the mean of a page's rows, summed in their order."""
    c, cache, page = s["c"], s["cache"], s["c"]["page"]
    lens = s["lens"].long()
    i = torch.arange(max_new // page + 2, device=DEV)
    pi = torch.minimum((starts.long() // page)[:, None] + i, ((lens - 1) // page)[:, None])  # (the last one more than once)
    at = torch.gather(s["table"].long(), 1, pi)
    n = (lens[:, None] - pi * page).clamp_max(page)
    total = torch.zeros(*at.shape, c["kvh"], c["hd"], device=DEV)
    for r in range(page):
        total = total + torch.where((r < n)[..., None, None], _rows_of(cache["k"], cache["k_scales"], at, r), 0.0)
    codes, scales = _int8(total / n[..., None, None].float())
    s["keys"]["codes"][at] = codes.to(torch.int8)
    s["keys"]["scales"][at] = scales


def _padded(cu, width):
    """Rows of a packed tensor for [B, width], the last one where a sequence is shorter, and which of them are real."""
    first, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    i = torch.arange(width, device=DEV)
    return (first[:, None] + i).clamp_max(cu[-1].long() - 1), i < n[:, None], n


def _plain_select(s):
    c, page, topk = s["c"], s["c"]["page"], s["c"]["topk"]
    _plain_keys(s, s["starts"], s["max_q"])
    rows, real, n = _padded(s["cu_q"], s["max_q"])
    B, Q = rows.shape
    NB = -(-s["max_len"] // page)
    kvh, hd, G = c["kvh"], c["hd"], c["nh"] // c["kvh"]
    qc, qs = _int8(s["q"][rows].float())
    qc = qc.view(B, Q, kvh, G, hd).permute(0, 2, 1, 3, 4).reshape(B, kvh, Q * G, hd)
    at = s["table"].long()[:, :NB]
    dots = qc @ s["keys"]["codes"][at].float().permute(0, 2, 3, 1)  # whole numbers below 2^24: exact
    x = dots.view(B, kvh, Q, G, NB).mul_(qs.view(B, Q, kvh, G).permute(0, 2, 1, 3).unsqueeze(-1))
    x = x.mul_(s["keys"]["scales"][at].permute(0, 2, 1)[:, :, None, None])
    x = torch.where(x.isnan(), -math.inf, x).amax(3)  # [B, kvh, Q, NB]
    cur = ((s["lens"].long() - n)[:, None] + torch.arange(Q, device=DEV)) // page
    b, cur = torch.arange(NB, device=DEV), cur[:, None, :, None]
    x = x.double().clamp(-1e300, 1e300)  # below, and above, any score: the blocks that are out and those that are in
    x = torch.where((b < c["first"]) | (b > cur - c["local"]), math.inf, x)
    x = torch.where(b > cur, -math.inf, x)
    if NB < topk:
        x = torch.cat([x, x.new_full((B, kvh, Q, topk - NB), -math.inf)], 3)
    best, at = x.sort(dim=-1, descending=True, stable=True)
    at = torch.where(best[..., :topk] == -math.inf, 1 << 30, at[..., :topk]).sort(-1).values
    idx = torch.where(at == 1 << 30, -1, at).to(torch.int32).permute(0, 2, 1, 3)
    return s["keys"] | {"idx": idx[real]}


def _attend(q, k, v, visible, scale, sink):
    """q [..., G, hd], k and v [..., L, hd] in 32 bits, visible broadcast to [..., G, L] -> o [..., G, hd] and the log of the
    denominators [..., G]; sink broadcast to [..., G] or None."""
    x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~visible, -math.inf)
    top = x.amax(-1) if sink is None else torch.maximum(x.amax(-1), sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top.unsqueeze(-1)).exp_()
    den = p.sum(-1) if sink is None else p.sum(-1) + (sink - top).exp()
    o = p @ v
    return torch.where(den.unsqueeze(-1) > 0, o / den.unsqueeze(-1), 0.0), top + den.log()


def _positions(s):
    """For each query token: its sequence and its position."""
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    T = len(s["q"])
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=T)
    return seq, s["lens"].long()[seq] - n[seq] + torch.arange(T, device=DEV) - s["cu_q"].long()[seq]


def _plain_tokens(s):
    c, cache, page = s["c"], s["cache"], s["c"]["page"]
    T, nh, hd = s["q"].shape
    kvh = c["kvh"]
    seq, pos = _positions(s)
    idx = s["idx"].long()  # [T, kvh, topk]
    pg = s["table"].long()[seq[:, None, None], idx.clamp_min(0)]
    h = torch.arange(kvh, device=DEV)[None, :, None]

    def rows(x, scales):
        if scales is None:
            return x[pg, h].float().reshape(T, kvh, -1, hd)
        x = x.view(torch.uint8)[pg, h].view(torch.float8_e4m3fn).float() * scales[pg, h].unsqueeze(-1)
        return x.reshape(T, kvh, -1, hd)

    j = idx.unsqueeze(-1) * page + torch.arange(page, device=DEV)
    visible = ((idx >= 0).unsqueeze(-1) & (j <= pos[:, None, None, None])).view(T, kvh, 1, -1)
    sink = None if s["sink"] is None else s["sink"].view(1, kvh, -1)
    o, lse = _attend(s["q"].float().view(T, kvh, nh // kvh, hd), rows(cache["k"], cache["k_scales"]), rows(cache["v"], cache["v_scales"]),
                     visible, s["scale"], sink)
    return {"o": o.view(T, nh, hd).bfloat16(), "lse": lse.view(T, nh)}


def _plain_prompt(s):
    c, page = s["c"], s["c"]["page"]
    nh, hd, kvh = c["nh"], c["hd"], c["kvh"]
    G = nh // kvh
    o, lse = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV), torch.empty(s["q"].shape[:2], device=DEV)
    at_q = at_k = 0
    for n in s["lens"]:
        m = n + c["prior"]
        NB = -(-m // page)
        j = torch.arange(m, device=DEV)
        past = j <= torch.arange(n, device=DEV)[:, None] + c["prior"]
        for h in range(kvh):
            idx = s["idx"][at_q:at_q + n, h].long()
            taken = torch.zeros(n, NB + 1, dtype=torch.bool, device=DEV).scatter_(1, torch.where(idx < 0, NB, idx), True)
            visible = taken[:, j // page] & past
            q = s["q"][at_q:at_q + n, h * G:(h + 1) * G].float().transpose(0, 1)
            sink = None if s["sink"] is None else s["sink"][h * G:(h + 1) * G, None]
            oh, lh = _attend(q, s["k"][at_k:at_k + m, h].float(), s["v"][at_k:at_k + m, h].float(), visible, s["scale"], sink)
            o[at_q:at_q + n, h * G:(h + 1) * G] = oh.transpose(0, 1).bfloat16()
            lse[at_q:at_q + n, h * G:(h + 1) * G] = lh.T
        at_q, at_k = at_q + n, at_k + m
    return {"o": o, "lse": lse}


_OWN = {"beam": _own_beam, "fork": _own_fork, "compact": _own_compact, "select": _own_select, "tokens": _own_tokens, "prompt": _own_prompt}
_PLAIN = {"beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact, "select": _plain_select, "tokens": _plain_tokens,
          "prompt": _plain_prompt}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _row_bytes(c):
    """Bytes of one cache row, K and V of every head."""
    return 2 * c["kvh"] * (2 * c["hd"] if c["fmt"] == "bf16" else c["hd"] + 4)


def work(case):
    c = case
    if c["op"] == "beam":
        n = c["batch"] * c["beams"] * c["vocab"]
        return {"bytes": n * (4 if c["fmt"] == "f32" else 2) + 12 * c["batch"] * c["k"], "flops": 3 * n}
    if c["op"] == "fork":
        lens, owned, parents, n_pages = _pool(c)
        seen, rows = set(), 0
        for p in parents:
            if lens[p] % c["page"] and not (c["replace"] and p not in seen):
                rows += lens[p] % c["page"]
            seen.add(p)
        tables = sum(len(owned[p]) for p in parents) + sum(len(x) for x in owned)
        return {"bytes": 2 * rows * _row_bytes(c) + 4 * tables + 8 * n_pages, "flops": 0}
    if c["op"] == "compact":
        n_live = max(1, min(c["pages"], int(c["pages"] * c["live"])))
        moved = n_live * (c["pages"] - n_live) / c["pages"]  # as many as are expected above the border
        return {"bytes": 2 * moved * c["page"] * _row_bytes(c) + 8 * c["pages"] + 8 * n_live, "flops": 0}
    lens, page = _lens(c), c["page"]
    if c["op"] == "prompt":
        rows = sum(lens) + c["prior"] * len(lens)
        keys = sum(min(i + c["prior"] + 1, c["topk"] * page - (page - 1 - (i + c["prior"]) % page)) for n in lens for i in range(n))
        return {"bytes": sum(lens) * (c["nh"] * (4 * c["hd"] + 4) + 4 * c["kvh"] * c["topk"]) + 4 * rows * c["kvh"] * c["hd"],
                "flops": 4 * c["hd"] * c["nh"] * keys}
    news = _queries(c)
    if c["op"] == "tokens":
        rows = sum(min(n, c["topk"] * page) for n in lens)  # (of one token of each sequence: the others' may be the same)
        keys = sum(m * min(n, c["topk"] * page) for n, m in zip(lens, news))
        return {"bytes": rows * _row_bytes(c) + sum(news) * (c["nh"] * (4 * c["hd"] + 4) + 4 * c["kvh"] * c["topk"]),
                "flops": 4 * c["hd"] * c["nh"] * keys}
    blocks = [-(-n // page) for n in lens]
    fresh = sum(n - (n - m) // page * page for n, m in zip(lens, news))  # rows of the pages that get new block keys
    pairs = sum(m * (n - m // 2) // page for n, m in zip(lens, news))
    return {"bytes": sum(blocks) * c["kvh"] * (c["hd"] + 4) + fresh * _row_bytes(c) // 2
            + sum(news) * (2 * c["nh"] * c["hd"] + 4 * c["kvh"] * c["topk"]), "flops": 2 * c["hd"] * c["nh"] * pairs}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _f32(x):
    return x.float().double()  # what the definition rounds to 32 bits


def _exact_int8(x):
    """x in 64 bits (values of 32): the codes and the scale, whose roundings to 32 bits are part of the definition."""
    s = _f32(x.abs().max(dim=-1).values.clamp_min(STEPS * TINY) * _f32(torch.tensor(1.0 / STEPS, dtype=torch.float64, device=DEV)))
    return torch.round(_f32(x / s[..., None])), s


def _exact_rows(cache, name):
    """The cache's values [page, head, row, hd] in 64 bits."""
    x = cache[name].double()
    return x if cache[name + "_scales"] is None else x * cache[name + "_scales"].double()[..., None]


def _exact_beam(s):
    c = s["c"]
    scores, parents, tokens = [], [], []
    for b in range(c["batch"]):
        x = s["logits"][b].double()
        x = s["scores"][b].double()[:, None] + torch.log_softmax(x, -1)
        if s["ended"] is not None:
            for w in torch.nonzero(s["ended"][b])[:, 0].tolist():
                x[w] = -math.inf
                x[w, 2] = s["scores"][b, w].double()
        flat = x.flatten()
        least = flat.topk(min(c["k"], flat.numel())).values[-1]
        at = torch.nonzero(flat >= least)[:, 0].tolist()  # ties with the last one among them
        at = sorted(at, key=lambda i: (-flat[i].item(), i))[:c["k"]]
        at = [i for i in at if flat[i].item() > -math.inf]
        none = c["k"] - len(at)
        scores.append([flat[i].item() for i in at] + [-math.inf] * none)
        parents.append([b * c["beams"] + i // c["vocab"] for i in at] + [-1] * none)
        tokens.append([i % c["vocab"] for i in at] + [-1] * none)
    return {"scores": torch.tensor(scores, dtype=torch.float64, device=DEV), "parents": _ints(parents), "tokens": _ints(tokens)}


def _exact_select(s):
    c, page, news = s["c"], s["c"]["page"], _queries(s["c"])
    kvh, G, topk = c["kvh"], c["nh"] // c["kvh"], c["topk"]
    codes, scales = s["keys"]["codes"].clone(), s["keys"]["scales"].double()
    out, at_q = [], 0
    for b, (n, m) in enumerate(zip(_lens(c), news)):
        for i in range((n - m) // page, (n - 1) // page + 1):
            p, r = int(s["table"][b, i]), min(page, n - i * page)
            x = s["cache"]["k"][p, :, :r].double()
            if s["cache"]["k_scales"] is not None:
                x = _f32(x * s["cache"]["k_scales"][p, :, :r].double()[..., None])
            total = torch.zeros(kvh, c["hd"], dtype=torch.float64, device=DEV)
            for y in range(r):
                total = _f32(total + x[:, y])
            k8, ks = _exact_int8(_f32(total / r))
            codes[p], scales[p] = k8.to(torch.int8), ks
        NB = -(-n // page)
        pages = s["table"][b, :NB].long()
        q8, qs = _exact_int8(s["q"][at_q:at_q + m].double())  # [m, nh, hd], [m, nh]
        cur = (torch.arange(n - m, n, device=DEV) // page)[:, None]
        blocks = torch.arange(NB, device=DEV)
        rows = torch.full((m, kvh, topk), -1, dtype=torch.int64, device=DEV)
        for h in range(kvh):
            x = torch.einsum("mgd,bd->mgb", q8[:, h * G:(h + 1) * G], codes[pages, h].double())
            x = _f32(_f32(x * qs[:, h * G:(h + 1) * G, None]) * scales[pages, h]).max(dim=1).values
            # rank: how many blocks come before this one
            x = torch.where((blocks < c["first"]) | (blocks > cur - c["local"]), 1e300, x)
            x = torch.where(blocks > cur, -1e300, x)
            order = torch.argsort(-x, dim=1, stable=True)
            rank = torch.empty_like(order).scatter_(1, order, blocks.expand(m, NB).contiguous())
            keep = (rank < topk) & (blocks <= cur)
            place = keep.cumsum(1) - 1
            t, j = torch.nonzero(keep, as_tuple=True)
            rows[t, h, place[t, j]] = j
        out.append(rows)
        at_q += m
    return {"codes": codes, "scales": scales, "idx": torch.cat(out).to(torch.int32)}


def _exact_softmax(q, k, v, visible, scale, sink):
    """One head: q [n, hd], k and v [L, hd], visible [n, L]."""
    x = torch.where(visible, (q.double() @ k.double().T) * scale, -math.inf)
    if sink is not None:
        x = torch.cat([x, sink.double().expand(len(x), 1)], 1)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p[:, :len(k)] @ v.double(), lse


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None  # nothing there is computed
    if c["op"] == "prompt" and sum(_lens(c)) * (c["max_len"] + c["prior"]) * c["nh"] * c["hd"] > 1.2e12:
        return None
    s = prepare(case, seed)
    if c["op"] == "beam":
        return _exact_beam(s)
    if c["op"] == "select":
        return _exact_select(s)
    nh, kvh, hd, page = c["nh"], c["kvh"], c["hd"], c["page"]
    G = nh // kvh
    o = torch.empty(len(s["q"]), nh, hd, dtype=torch.float64, device=DEV)
    lse = torch.empty(len(s["q"]), nh, dtype=torch.float64, device=DEV)
    at_q = at_k = 0
    if c["op"] == "tokens":
        ks, vs = _exact_rows(s["cache"], "k"), _exact_rows(s["cache"], "v")
    for b, n in enumerate(_lens(c)):
        m = n + c["prior"] if c["op"] == "prompt" else n
        d = n if c["op"] == "prompt" else _queries(c)[b]
        pos = torch.arange(m - d, m, device=DEV)
        for h in range(kvh):
            idx = s["idx"][at_q:at_q + d, h].long()
            if c["op"] == "prompt":
                k, v = s["k"][at_k:at_k + m, h], s["v"][at_k:at_k + m, h]
            else:
                pages = s["table"][b, :-(-n // page)].long()
                k, v = ks[pages, h].flatten(0, 1)[:n], vs[pages, h].flatten(0, 1)[:n]
            own_block = torch.arange(m, device=DEV) // page
            visible = torch.zeros(d, m, dtype=torch.bool, device=DEV)
            for x in range(idx.shape[1]):
                visible |= own_block == idx[:, x, None]
            visible &= torch.arange(m, device=DEV) <= pos[:, None]
            for g in range(G):
                sink = None if s["sink"] is None else s["sink"][h * G + g]
                o[at_q:at_q + d, h * G + g], lse[at_q:at_q + d, h * G + g] = _exact_softmax(
                    s["q"][at_q:at_q + d, h * G + g], k, v, visible, s["scale"], sink)
        at_q, at_k = at_q + d, at_k + m
    return {"o": o, "lse": lse}
