"""The dense attention entry points reject bad arguments on the host, before
any device work (no GPU needed), and the binding rejects bad tensors."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_window_gb300 import build as ds41_build
from compressed_sparse_attention_window_gb300 import ds41

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)
F = ctypes.c_float
ARG, RANGE = 1, 2


@pytest.fixture(scope="module")
def lib():
    ds41_build.build()
    return ds41.load()


def write(lib, k=FAKE, k_stride=256, v=FAKE, v_stride=256, slots=FAKE, kc=FAKE, vc=FAKE, ks=FAKE,
          vs=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, n=3):
    return lib.ds41_kv_cache_write(k, k_stride, v, v_stride, slots, kc, vc, ks, vs, fmt, n_pages,
                                   page, kvh, hd, n, None)


def read(lib, kc=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, kvh=2, hd=128, table=FAKE, mp=2,
         cu=FAKE, B=1, k=FAKE, rows=3):
    return lib.ds41_kv_cache_read(kc, FAKE, ks, FAKE, fmt, n_pages, page, kvh, hd, table, mp, cu,
                                  None, B, k, FAKE, rows, None)


def prompt(lib, q=FAKE, q_tok=512, q_head=128, k=FAKE, k_tok=256, k_head=128, v_tok=256, cu=FAKE,
           B=1, Tq=4, Tk=4, max_q=4, nh=4, kvh=2, hd=128, scale=0.1, window=0, o=FAKE, lse=None):
    return lib.ds41_prompt_attn_fwd(q, q_tok, q_head, k, k_tok, k_head, FAKE, v_tok, 128, cu, FAKE,
                                    B, Tq, Tk, max_q, nh, kvh, hd, F(scale), window, None, o, lse,
                                    None)


def tree(lib, q=FAKE, q_tok=512, kc=FAKE, ks=FAKE, fmt=1, n_pages=4, page=16, table=FAKE,
         lens=FAKE, mask=None, words=0, B=1, Tq=4, max_q=4, max_len=32, nh=4, kvh=2, hd=128,
         scale=0.1, window=0, o=FAKE):
    return lib.ds41_tree_attn_fwd(q, q_tok, 128, kc, FAKE, ks, FAKE, fmt, n_pages, page, table, 2,
                                  lens, FAKE, mask, words, B, Tq, max_q, max_len, nh, kvh, hd,
                                  F(scale), window, None, o, None, FAKE, 1 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), ARG), (dict(page=24), ARG), (dict(page=8), ARG), (dict(page=512), ARG),
    (dict(kvh=0), ARG), (dict(hd=72), ARG), (dict(hd=144), ARG), (dict(hd=0), ARG),
    (dict(n_pages=0), ARG), (dict(kc=None), ARG), (dict(kc=ODD), ARG), (dict(ks=None), ARG)])
def test_cache_layout_is_checked(lib, kw, code):
    for call in (write, read, tree):
        assert call(lib, **kw) == code, call.__name__


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), ARG), (dict(k=ODD), ARG), (dict(slots=None), ARG),
    (dict(slots=ctypes.c_void_p((1 << 20) + 4)), ARG), (dict(k_stride=128), ARG),
    (dict(v_stride=260), ARG), (dict(n=-1), RANGE)])
def test_write_refuses(lib, kw, code):
    assert write(lib, **kw) == code
    assert lib.ds41_last_error().startswith(b"ds41_kv_cache_write")


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), ARG), (dict(cu=None), ARG), (dict(k=None), ARG), (dict(k=ODD), ARG),
    (dict(rows=-1), RANGE), (dict(B=-1), RANGE), (dict(mp=-1), RANGE)])
def test_read_refuses(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(o=None), ARG), (dict(cu=None), ARG),
    (dict(nh=3), ARG), (dict(kvh=0), ARG), (dict(hd=24), ARG), (dict(hd=256), ARG),
    (dict(q_tok=500), ARG), (dict(q_head=64), ARG), (dict(k_tok=12), ARG), (dict(k=None), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(window=-1), ARG), (dict(B=-1), RANGE),
    (dict(Tq=1 << 31), RANGE), (dict(max_q=-1), RANGE)])
def test_prompt_refuses(lib, kw, code):
    assert prompt(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(o=ODD), ARG),
    (dict(nh=5), ARG), (dict(q_tok=100), ARG), (dict(mask=FAKE, words=0), ARG),
    (dict(mask=FAKE, words=5), ARG), (dict(mask=FAKE, words=1, max_q=65), ARG),
    (dict(max_q=257), RANGE), (dict(window=3), ARG), (dict(max_len=-1), RANGE),
    (dict(scale=0.0), ARG)])
def test_tree_refuses(lib, kw, code):
    assert tree(lib, **kw) == code


def test_nothing_to_do_is_no_error(lib):
    assert write(lib, n=0, k=None, v=None, slots=None) == 0
    assert read(lib, rows=0) == 0 and read(lib, B=0) == 0
    assert prompt(lib, Tq=0) == 0 and prompt(lib, B=0) == 0 and prompt(lib, max_q=0) == 0
    assert tree(lib, Tq=0) == 0 and tree(lib, B=0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    c = ds41.KvCache(*(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    with pytest.raises(ValueError):
        ds41.prompt_attn_fwd(x, x, x, i, i, 4, 0.1)
    with pytest.raises(ValueError):
        ds41.kv_cache_write(c, x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        ds41.kv_cache_read(c, i.view(1, 2), i, 4)
    with pytest.raises(ValueError):
        ds41.tree_attn_fwd(x, c, i.view(1, 2), i[:1], i, 1, 4, 0.1)


def test_binding_refuses_what_is_no_tensor_or_cache():
    x = torch.zeros(1, 1, 16, dtype=torch.bfloat16)
    cache = ds41.make_kv_cache(1, 1, 16, 16, device="cpu")
    idx = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ds41.kv_cache_write(cache, None, x, idx),
                 lambda: ds41.kv_cache_write(cache, x, 3, idx),
                 lambda: ds41.kv_cache_read(cache, [[0]], idx, 1),
                 lambda: ds41.kv_cache_read(cache, idx[None], None, 1),
                 lambda: ds41.prompt_attn_fwd(x, x, "v", idx, idx, 1, 1.0),
                 lambda: ds41.tree_attn_fwd(None, cache, idx[None], idx, idx, 1, 1, 1.0)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("window", [1 << 31, (1 << 63) - 257, (1 << 63) - 1])
def test_workspace_of_a_window_larger_than_any_sequence(lib, window):
    """As without a window: the sum of the window and the tokens must not wrap."""
    for nh, max_q in ((8, 1), (8, 40), (64, 40)):
        sizes = [lib.ds41_tree_attn_workspace_bytes(8, 8 * max_q, max_q, 32768, nh, 2, 128, w, 1)
                 for w in (0, window)]
        assert sizes[0] == sizes[1] > 0


@pytest.mark.parametrize("kw", [
    dict(hd=144), dict(hd=24), dict(nh=8192), dict(kvh=2048, nh=2048), dict(B=65536),
    dict(max_q=257), dict(window=3), dict(fmt=2), dict(fmt=-1), dict(max_len=1 << 30),
    dict(Tq=1 << 31), dict(B=0), dict(max_len=-1), dict(window=-1)])
def test_workspace_of_sizes_that_are_refused_is_zero(lib, kw):
    """What the call refuses, or has nothing to do for, needs no scratch."""
    size = dict(B=1, Tq=4, max_q=4, max_len=32, nh=4, kvh=2, hd=128, window=0, fmt=1)
    names = list(size)
    assert lib.ds41_tree_attn_workspace_bytes(*size.values()) > 0
    size |= kw
    assert lib.ds41_tree_attn_workspace_bytes(*(size[n] for n in names)) == 0


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scale_that_overflows_in_units_of_log2_is_refused(lib, scale):
    """scale * log2(e) is what the kernels take."""
    assert prompt(lib, scale=scale) == ARG and tree(lib, scale=scale) == ARG
    assert b"scale" in lib.ds41_last_error()
