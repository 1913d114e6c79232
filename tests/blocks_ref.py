"""Block keys, the selection of blocks, attention over them, pages and beam selection written
out plainly: Python integers and 64 bits.  The roundings to f32 that are part of the
definition of block keys and scores are made as such (one operation on f32 values in 64
bits, rounded to f32, is that operation's correctly rounded result: 53 >= 2 * 24 + 2
bits), so codes, scales and picks have to be equal.  The attention's tolerances are those
of dense_ref.attend."""
from __future__ import annotations

import math

import torch

import dense_ref as ref

INV = torch.tensor(1.0 / 127.0, dtype=torch.float32).double().item()


def f32(x):
    return x.float().double()


def int8(x):
    """Rows [..., hd] in 64 bits (f32 values): codes and scales in 64 bits."""
    s = f32(x.abs().amax(-1).clamp_min(127 * 2.0 ** -126) * INV)
    bad = ~torch.isfinite(x).all(-1)
    codes = torch.round(f32(x / s[..., None]))
    return torch.where(bad[..., None], 0.0, codes), torch.where(bad, math.nan, s)


def block_key(rows):
    """rows [n, hd] in 64 bits (f32 values) -> codes [hd], scale."""
    total = torch.zeros(rows.shape[1], dtype=torch.float64, device=rows.device)
    for r in rows:
        total = f32(total + r)
    return int8(f32(total / len(rows)))


def key_rows(cache, page, h):
    """The K rows [page, hd] of a page and head as f32 values in 64 bits."""
    k = cache.k[page, h].double()
    return k if cache.k_scales is None else f32(k * cache.k_scales[page, h].double()[:, None])


def picks(q, codes, scales, p, page, topk, first, local):
    """One token and key/value head: q [G, hd], codes [NB, hd], scales [NB] (64 bits) ->
    the ascending list of blocks."""
    cur = p // page
    qc, qs = int8(q.double())
    s = f32(f32((qc @ codes[:cur + 1].T) * qs[:, None]) * scales[:cur + 1])
    s = torch.where(s.isnan(), -math.inf, s).amax(0).tolist()
    order = sorted(range(cur + 1), key=lambda j: (not (j < first or j > cur - local), -s[j], j))
    return sorted(order[:topk])


def attend(q, k, v, lists, p0, block, scale, sink, vs=None):
    """One sequence: q [n, nh, hd], k and v [L, kvh, hd] (64 bits), lists[t][h] block
    numbers, token t at p0 + t.  As dense_ref.attend."""
    n, nh, _ = q.shape
    L, kvh = k.shape[:2]
    G = nh // kvh
    j = torch.arange(L, device=q.device)
    outs = []
    for h in range(kvh):
        vis = torch.zeros(n, L, dtype=torch.bool, device=q.device)
        for t in range(n):
            for x in lists[t][h]:
                vis[t] |= j // block == x
            vis[t] &= j <= p0 + t
        outs.append(ref.attend(q[:, h * G:(h + 1) * G], k[:, h:h + 1], v[:, h:h + 1], vis, scale,
                               None if sink is None else sink[h * G:(h + 1) * G],
                               None if vs is None else vs[:, h:h + 1]))
    return [torch.cat([x[i] for x in outs], 1) for i in range(4)]


# ---------------------------------------------------------------------------
# Pages: plain lists
# ---------------------------------------------------------------------------
class Pool:
    def __init__(self, refs):
        self.refs = list(refs)

    def take(self):
        for p, r in enumerate(self.refs):
            if r == 0:
                self.refs[p] = 1
                return p
        return -1


def fork(refs, table, lens, parents, page, replace):
    """-> refs, table_out, lens_out, copies [(src, dst, rows)], in order."""
    pool = Pool(refs)
    width = len(table[0]) if table else 0
    born = [sum(p == b for p in parents) for b in range(len(lens))]
    for b, n in enumerate(lens):
        whole, part = divmod(n, page)
        for x in range(whole):
            pool.refs[table[b][x]] += born[b] - int(replace)
        if part and replace and not born[b]:
            pool.refs[table[b][whole]] -= 1
    out, out_lens, copies, seen = [], [], [], set()
    for p in parents:
        if p < 0:
            out.append([-1] * width)
            out_lens.append(0)
            continue
        whole, part = divmod(lens[p], page)
        row = table[p][:whole]
        if part:
            if replace and p not in seen:
                row.append(table[p][whole])
            else:
                d = pool.take()
                if d >= 0:
                    copies.append((table[p][whole], d, part))
                row.append(d)
            seen.add(p)
        out.append(row + [-1] * (width - len(row)))
        out_lens.append(lens[p])
    return pool.refs, out, out_lens, copies


def compact(refs, table, lens, page):
    """-> refs, table, live, moves [(src, dst)]."""
    live = sum(r != 0 for r in refs)
    src = [p for p, r in enumerate(refs) if r != 0 and p >= live]
    dst = [p for p, r in enumerate(refs) if r == 0 and p < live]
    to = dict(zip(src, dst))
    refs = list(refs)
    for s, d in to.items():
        refs[d], refs[s] = refs[s], 0
    table = [[to.get(p, p) if x < -(-n // page) else p for x, p in enumerate(row)]
             for row, n in zip(table, lens)]
    return refs, table, live, list(to.items())


# ---------------------------------------------------------------------------
# Beam search
# ---------------------------------------------------------------------------
def beam(logits, scores, k, ended=None, end_token=0):
    """[B, W, V], [B, W] -> per search a list of (score, b W + w, token), best first, the
    scores in 64 bits."""
    B, W, V = logits.shape
    out = []
    for b in range(B):
        offers = []
        for w in range(W):
            s = float(scores[b, w])
            if not -math.inf < s < math.inf:
                continue
            if ended is not None and bool(ended[b, w]):
                offers.append((-s, w, 0.0, end_token, s))
                continue
            x = logits[b, w].double().cpu()
            if bool(x.isnan().any()) or bool((x == math.inf).any()) or not bool((x > -math.inf).any()):
                continue
            L = torch.logsumexp(x, 0).item()
            # the row's best k: by logit, then by token
            for t in torch.sort(x, descending=True, stable=True).indices[:k].tolist():
                if x[t].item() > -math.inf:
                    offers.append((-(s + (x[t].item() - L)), w, -x[t].item(), t, s + (x[t].item() - L)))
        offers.sort(key=lambda o: o[:4])
        out.append([(o[4], b * W + o[1], o[3]) for o in offers[:k]])
    return out
