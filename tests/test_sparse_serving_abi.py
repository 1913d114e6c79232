"""The entry points of pages, beam search and block attention reject bad arguments on the
host, before any device work (no GPU needed), and the binding rejects bad tensors."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_window_gb300 import build as ds41_build
from compressed_sparse_attention_window_gb300 import ds41

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced: validation fails first
FAR = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 20) + 8)
OFF = ctypes.c_void_p((1 << 20) + 2)
F = ctypes.c_float
ARG, RANGE, WS = 1, 2, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    ds41_build.build()
    return ds41.load()


def take(lib, refs=FAKE, n_pages=4, page=16, table=FAKE, mp=2, lens=FAKE, new=FAKE, B=1, ws=FAKE, size=BIG):
    return lib.ds41_kv_pages_take(refs, n_pages, page, table, mp, lens, new, B, ws, size, None)


def free(lib, refs=FAKE, n_pages=4, page=16, table=FAKE, mp=2, lens=FAKE, B=1):
    return lib.ds41_kv_pages_free(refs, n_pages, page, table, mp, lens, B, None)


def fork(lib, k=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, codes=None, kscales=None, refs=FAKE,
         table=FAKE, mp=2, lens=FAKE, B=1, parents=FAKE, n=2, replace=0, out=FAR, out_lens=FAR, ws=FAKE, size=BIG):
    return lib.ds41_kv_pages_fork(k, FAKE, ks, FAKE, fmt, n_pages, page, kvh, hd, codes, kscales, refs, table, mp,
                                  lens, B, parents, n, replace, out, out_lens, ws, size, None)


def copy(lib, k=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, codes=None, kscales=None, src=FAKE,
         dst=FAKE, rows=None, n=2):
    return lib.ds41_kv_pages_copy(k, FAKE, ks, FAKE, fmt, n_pages, page, kvh, hd, codes, kscales, src, dst, rows, n,
                                  None)


def compact(lib, k=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, codes=None, kscales=None, refs=FAKE,
            table=FAKE, mp=2, lens=FAKE, B=1, live=FAKE, ws=FAKE, size=BIG):
    return lib.ds41_kv_pages_compact(k, FAKE, ks, FAKE, fmt, n_pages, page, kvh, hd, codes, kscales, refs, table, mp,
                                     lens, B, live, ws, size, None)


def keys(lib, k=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, table=FAKE, mp=2, lens=FAKE, starts=None,
         B=1, new=3, codes=FAKE, kscales=FAKE):
    return lib.ds41_kv_block_keys(k, ks, fmt, n_pages, page, kvh, hd, table, mp, lens, starts, B, new, codes, kscales,
                                  None)


def select(lib, q=FAKE, q_tok=512, q_head=128, codes=FAKE, kscales=FAKE, n_pages=4, page=16, kvh=2, hd=128,
           table=FAKE, mp=2, lens=FAKE, cu=FAKE, B=1, Tq=4, max_q=4, max_len=32, nh=4, topk=2, first=1, local=1,
           idx=FAKE):
    return lib.ds41_block_select(q, q_tok, q_head, codes, kscales, n_pages, page, kvh, hd, table, mp, lens, cu, B, Tq,
                                 max_q, max_len, nh, topk, first, local, idx, None)


def tokens(lib, q=FAKE, q_tok=512, k=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, table=FAKE, mp=2, lens=FAKE, cu=FAKE,
           idx=FAKE, topk=2, B=1, Tq=4, max_q=4, nh=4, kvh=2, hd=128, scale=0.1, o=FAKE):
    return lib.ds41_block_attn_fwd(q, q_tok, 128, k, FAKE, ks, FAKE, fmt, n_pages, page, table, mp, lens, cu, idx,
                                   topk, B, Tq, max_q, nh, kvh, hd, F(scale), None, o, None, None)


def prompt(lib, q=FAKE, q_tok=512, k=FAKE, k_tok=256, cu=FAKE, idx=FAKE, topk=2, block=16, B=1, Tq=4, Tk=4, max_q=4,
           max_k=4, nh=4, kvh=2, hd=128, scale=0.1, o=FAKE, ws=FAKE, size=BIG):
    return lib.ds41_block_prompt_attn_fwd(q, q_tok, 128, k, k_tok, 128, FAKE, 256, 128, cu, FAKE, idx, topk, block, B,
                                          Tq, Tk, max_q, max_k, nh, kvh, hd, F(scale), None, o, None, ws, size, None)


def beam(lib, x=FAKE, fmt=0, bs=40, ws_=10, scores=FAKE, ended=None, end=0, B=1, W=4, V=10, k=4, out=FAKE, ws=FAKE,
         size=BIG):
    return lib.ds41_beam_select(x, fmt, bs, ws_, scores, ended, end, B, W, V, k, out, FAKE, FAKE, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(page=24), ARG), (dict(page=8), ARG), (dict(page=512), ARG), (dict(n_pages=0), ARG),
    (dict(B=-1), RANGE), (dict(mp=-1), RANGE), (dict(refs=None), ARG), (dict(refs=OFF), ARG), (dict(table=None), ARG),
    (dict(lens=None), ARG)])
def test_pools_are_checked(lib, kw, code):
    for call in (take, free, fork, compact):
        assert call(lib, **kw) == code, call.__name__


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), ARG), (dict(page=24), ARG), (dict(kvh=0), ARG), (dict(hd=72), ARG), (dict(hd=144), ARG),
    (dict(k=None), ARG), (dict(k=ODD), ARG), (dict(ks=None), ARG), (dict(codes=FAKE), ARG), (dict(kscales=FAKE), ARG),
    (dict(codes=ODD, kscales=FAKE), ARG)])
def test_caches_are_checked(lib, kw, code):
    for call in (fork, copy, compact):
        assert call(lib, **kw) == code, call.__name__


def test_pages_refuse(lib):
    assert take(lib, new=None) == ARG
    assert take(lib, ws=None) == WS and take(lib, size=15) == WS
    assert fork(lib, parents=None) == ARG and fork(lib, out=None) == ARG and fork(lib, out_lens=OFF) == ARG
    assert fork(lib, n=-1) == RANGE
    assert fork(lib, ws=None) == WS and fork(lib, size=63) == WS
    assert fork(lib, out=FAKE) == ARG                                        # the table itself
    assert fork(lib, out=ctypes.c_void_p((1 << 20) + 4)) == ARG              # or in it
    assert fork(lib, out_lens=FAKE) == ARG
    assert b"table_out" in lib.ds41_last_error()
    assert copy(lib, src=None) == ARG and copy(lib, dst=OFF) == ARG and copy(lib, rows=OFF) == ARG
    assert copy(lib, n=-1) == RANGE
    assert compact(lib, live=None) == ARG and compact(lib, ws=ODD) == WS and compact(lib, size=60) == WS
    # nothing to do
    assert take(lib, B=0) == 0 and free(lib, B=0) == 0 and copy(lib, n=0) == 0 and fork(lib, n=0, B=0) == 0
    assert lib.ds41_kv_pages_fork_workspace_bytes(4, 1, 3) == 64
    assert lib.ds41_kv_pages_fork_workspace_bytes(0, 1, 3) == 0
    assert lib.ds41_kv_pages_compact_workspace_bytes(5) == 3 * 32 + 16


@pytest.mark.parametrize("kw", [dict(n=65536), dict(B=65536), dict(n=1 << 29), dict(B=1 << 29), dict(n=0, B=65536, replace=1)])
def test_forks_of_masses_are_refused(lib, kw):
    """Every child and parent looks through all children: 2^20 of them would be 2^41 reads, minutes in one launch."""
    far = dict(out=ctypes.c_void_p(1 << 50), out_lens=ctypes.c_void_p(1 << 51))
    assert fork(lib, **far, **kw) == RANGE
    assert b"65536" in lib.ds41_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=3), ARG), (dict(page=20), ARG), (dict(k=ODD), ARG), (dict(codes=None), ARG), (dict(codes=ODD), ARG),
    (dict(kscales=None), ARG), (dict(table=None), ARG), (dict(lens=OFF), ARG), (dict(starts=OFF), ARG),
    (dict(B=65536), RANGE), (dict(new=-1), RANGE), (dict(hd=8), ARG)])
def test_keys_refuse(lib, kw, code):
    assert keys(lib, **kw) == code
    assert keys(lib, B=0) == 0 and keys(lib, new=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(nh=3), ARG), (dict(kvh=0), ARG), (dict(hd=24), ARG), (dict(page=20), ARG), (dict(n_pages=0), ARG),
    (dict(topk=0), ARG), (dict(topk=1025), ARG), (dict(first=-1), ARG), (dict(local=0), ARG),
    (dict(first=2, local=1), ARG), (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(codes=ODD), ARG),
    (dict(idx=None), ARG), (dict(q_tok=500), ARG), (dict(q_head=64), ARG), (dict(B=-1), RANGE), (dict(Tq=-1), RANGE),
    (dict(max_q=-1), RANGE), (dict(max_len=32768 * 16 + 1), RANGE), (dict(mp=-1), RANGE)])
def test_select_refuses(lib, kw, code):
    assert select(lib, **kw) == code
    assert lib.ds41_last_error().startswith(b"ds41_block_select")
    assert select(lib, B=0) == 0 and select(lib, Tq=0) == 0 and select(lib, max_q=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), ARG), (dict(page=24), ARG), (dict(nh=3), ARG), (dict(hd=24), ARG), (dict(ks=None), ARG),
    (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(o=None), ARG), (dict(idx=None), ARG), (dict(idx=OFF), ARG),
    (dict(topk=0), ARG), (dict(topk=1025), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(q_tok=500), ARG), (dict(B=-1), RANGE), (dict(Tq=1 << 31), RANGE), (dict(max_q=-1), RANGE),
    (dict(mp=-1), RANGE)])
def test_tokens_refuse(lib, kw, code):
    assert tokens(lib, **kw) == code
    assert tokens(lib, B=0) == 0 and tokens(lib, Tq=0) == 0 and tokens(lib, max_q=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(block=24), ARG), (dict(block=512), ARG), (dict(nh=3), ARG), (dict(hd=24), ARG), (dict(q=None), ARG),
    (dict(q=ODD), ARG), (dict(k=None), ARG), (dict(k_tok=12), ARG), (dict(o=None), ARG), (dict(idx=None), ARG),
    (dict(topk=0), ARG), (dict(topk=1025), ARG), (dict(scale=-1.0), ARG), (dict(B=-1), RANGE), (dict(Tk=-1), RANGE),
    (dict(max_q=-1), RANGE), (dict(max_k=32768 * 16 + 1), RANGE), (dict(ws=None), WS), (dict(size=10), WS),
    (dict(ws=ODD), WS)])
def test_prompt_refuses(lib, kw, code):
    assert prompt(lib, **kw) == code
    assert prompt(lib, B=0) == 0 and prompt(lib, Tq=0) == 0 and prompt(lib, max_q=0) == 0


def test_prompt_workspace(lib):
    size = lib.ds41_block_prompt_attn_workspace_bytes
    # 4 tokens of 2 groups of 2 heads: one pair of tiles at most and one for the batch; a record of
    # 8 units of 16 keys with masks of 128 tokens, three of them
    assert size(1, 4, 4, 4, 2, 16, 4, 2) == 2 * (64 + 3 * 8 * (1 + 4) * 4)
    assert size(1, 4, 4, 4, 2, 24, 4, 2) == 0 and size(1, 4, 4, 4, 2, 16, 3, 2) == 0 and size(0, 4, 4, 4, 2, 16, 4, 2) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), ARG), (dict(k=0), ARG), (dict(k=129), ARG), (dict(x=None), ARG), (dict(x=OFF), ARG),
    (dict(scores=None), ARG), (dict(out=None), ARG), (dict(out=OFF), ARG), (dict(ws_=9), ARG),
    (dict(ended=FAKE, end=10), ARG), (dict(ended=FAKE, end=-1), ARG), (dict(B=-1), RANGE), (dict(W=0), RANGE),
    (dict(W=1025), RANGE), (dict(V=0), RANGE), (dict(V=(1 << 22) + 1), RANGE), (dict(B=20000), RANGE),
    (dict(ws=None), WS), (dict(ws=ODD), WS), (dict(size=7), WS)])
def test_beam_refuses(lib, kw, code):
    assert beam(lib, **kw) == code
    assert beam(lib, B=0) == 0
    assert lib.ds41_beam_select_workspace_bytes(1, 4, 10, 0) == 0
    assert lib.ds41_beam_select_workspace_bytes(1, 4, 10, 4) == 4 * 4 * 8 + 4 * 8


def test_binding_refuses_tensors():
    """Wrong types, shapes and devices: ValueError or TypeError, no call."""
    t = torch.zeros
    i32 = dict(dtype=torch.int32)
    kv = ds41.make_kv_cache(4, 2, 16, 64, device="cpu")
    bk = ds41.make_block_keys(4, 2, 64, device="cpu")
    cpu = "CUDA tensors"
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_pages_take(t(4, **i32), t(1, 2, **i32), t(1, **i32), t(1, **i32), 16)
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_pages_free(t(4, **i32), t(1, 2, **i32), t(1, **i32), 16)
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_pages_fork(kv, t(4, **i32), t(1, 2, **i32), t(1, **i32), t(1, **i32))
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_pages_copy(kv, t(1, **i32), t(1, **i32))
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_pages_compact(kv, t(4, **i32), t(1, 2, **i32), t(1, **i32))
    with pytest.raises(ValueError, match=cpu):
        ds41.beam_select(t(1, 2, 8), t(1, 2), 2)
    with pytest.raises(ValueError, match=cpu):
        ds41.kv_block_keys(kv, bk, t(1, 2, **i32), t(1, **i32), 4)
    q = t(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=cpu):
        ds41.block_select(q, bk, 16, t(1, 2, **i32), t(1, **i32), t(2, **i32), 1, 32, 2)
    with pytest.raises(ValueError, match=cpu):
        ds41.block_attn_fwd(q, kv, t(1, 2, **i32), t(1, **i32), t(2, **i32), 1, t(1, 2, 2, **i32), 0.1)
    with pytest.raises(ValueError, match=cpu):
        ds41.block_prompt_attn_fwd(q, q, q, t(2, **i32), t(2, **i32), 1, 1, t(1, 4, 2, **i32), 16, 0.1)
    with pytest.raises(TypeError):
        ds41.beam_select(None, t(1, 2), 2)
    with pytest.raises(TypeError):
        ds41.kv_pages_take(t(4, **i32), None, t(1, **i32), t(1, **i32), 16)
