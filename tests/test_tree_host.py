"""Host-only checks of the speculative-decoding entry points: bad arguments are
refused before a device is touched, and by the binding before a pointer is
taken.  No kernel is launched here."""
import ctypes
import os

import pytest
import torch

from mla_latent_kv_23_b200 import mla

INVALID, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mla.LIB_PATH):
        from mla_latent_kv_23_b200 import build
        build.build()
    return mla.lib()


def tree(**kw):
    base = dict(q=16, kv_cache=32, block_table=48, seqlens=64, cu_q=80, tree_mask=96, u=112, lse=128, B=2, T=9,
                n_h=128, d_c=512, d_R=64, page_size=64, max_pages_per_seq=4, num_pages=8, softmax_scale=0.07,
                dtype=mla.MLA_DTYPE_BF16, num_splits=0, u_fp32=0)
    base.update(kw)
    return mla.TreeParams(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(n_h=0), INVALID), (dict(n_h=129), UNSUPPORTED),
    (dict(d_c=12), INVALID), (dict(d_c=1024), UNSUPPORTED), (dict(d_R=7), INVALID), (dict(d_R=-8), INVALID),
    (dict(d_R=128), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(page_size=96), INVALID),
    (dict(max_pages_per_seq=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 26), UNSUPPORTED),
    (dict(max_pages_per_seq=1 << 26), UNSUPPORTED), (dict(softmax_scale=float("nan")), INVALID),
    (dict(softmax_scale=0.0), INVALID), (dict(softmax_scale=float("inf")), INVALID), (dict(dtype=7), INVALID),
    (dict(num_splits=-1), INVALID), (dict(num_splits=70000), UNSUPPORTED), (dict(T=1 << 25), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(kv_cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(seqlens=None), INVALID), (dict(cu_q=None), INVALID), (dict(tree_mask=None), INVALID),
    (dict(u=None), INVALID), (dict(q=18), INVALID), (dict(lse=132), INVALID), (dict(tree_mask=104), INVALID),
])
def test_tree_refuses(lib, kw, want):
    p = tree(**kw)
    n = ctypes.c_size_t(0)
    assert lib.mla_decode_tree(ctypes.byref(p), None, 0, None) == want
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want


def test_tree_null_and_empty(lib):
    assert lib.mla_decode_tree(None, None, 0, None) == INVALID
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(tree()), None) == INVALID
    for kw in (dict(B=0), dict(T=0)):
        p = tree(q=None, kv_cache=None, u=None, block_table=None, seqlens=None, cu_q=None, tree_mask=None, **kw)
        assert lib.mla_decode_tree(ctypes.byref(p), None, 0, None) == OK


def tables(**kw):
    # buffers far apart: overlaps are refused
    names = ("ctx_lens", "new_lens", "block_table", "free_pages", "free_used", "free_used_out", "seqlens", "cu_new",
             "seq_ids", "pos", "slots")
    base = {n: 4096 * (i + 1) for i, n in enumerate(names)}
    base.update(pages_held=None, pages_held_out=None, parents=None, tree_mask=None, B=3, max_pages_per_seq=4,
                n_free=5, max_tokens=20, page_size=64, num_pages=8)
    base.update(kw)
    return mla.TablesParams(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(B=16385), UNSUPPORTED), (dict(max_tokens=-1), INVALID), (dict(n_free=-1), INVALID),
    (dict(page_size=0), INVALID), (dict(max_pages_per_seq=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 26), UNSUPPORTED), (dict(max_pages_per_seq=1 << 26), UNSUPPORTED),
    (dict(ctx_lens=None), INVALID), (dict(new_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(free_pages=None), INVALID), (dict(free_used=None), INVALID), (dict(free_used_out=None), INVALID),
    (dict(seqlens=None), INVALID), (dict(cu_new=None), INVALID), (dict(seq_ids=None), INVALID),
    (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(parents=1 << 20), INVALID),
    (dict(tree_mask=1 << 20), INVALID), (dict(pages_held=1 << 20), INVALID), (dict(pages_held_out=1 << 20), INVALID),
    (dict(slots=(1 << 20) + 4), INVALID),
    (dict(free_used_out=4096 * 5), INVALID),          # free_used in place
    (dict(seqlens=4096), INVALID),                    # ctx_lens in place
    (dict(pos=4096 * 4 + 16), INVALID),               # inside the free list
    (dict(parents=1 << 20, tree_mask=(1 << 20) + 64), INVALID),
])
def test_tables_refuses(lib, kw, want):
    assert lib.mla_build_tables(ctypes.byref(tables(**kw)), None) == want


def test_tables_null(lib):
    assert lib.mla_build_tables(None, None) == INVALID


def accept(**kw):
    base = dict(kv_cache=16, block_table=32, seqlens=48, cu_q=64, tree_mask=80, accepted=96, seqlens_out=112,
                path=128, B=2, T=9, width=576, page_size=64, max_pages_per_seq=4, num_pages=8,
                dtype=mla.MLA_DTYPE_BF16)
    base.update(kw)
    return mla.AcceptParams(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(width=0), INVALID), (dict(width=12), INVALID),
    (dict(dtype=3), INVALID), (dict(page_size=0), INVALID), (dict(max_pages_per_seq=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 26), UNSUPPORTED), (dict(kv_cache=None), INVALID),
    (dict(block_table=None), INVALID), (dict(seqlens=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(tree_mask=None), INVALID), (dict(accepted=None), INVALID), (dict(seqlens_out=None), INVALID),
    (dict(path=None), INVALID), (dict(path=136), INVALID),
])
def test_accept_refuses(lib, kw, want):
    assert lib.mla_accept_tree(ctypes.byref(accept(**kw)), None) == want


def test_accept_null_and_empty(lib):
    assert lib.mla_accept_tree(None, None) == INVALID
    assert lib.mla_accept_tree(ctypes.byref(accept(B=0, kv_cache=None)), None) == OK


@pytest.mark.parametrize("args,want", [
    ((16, 32, 48, 64, 80, 96, 8, 4, 256, 512, 64, 1e4, 9, None), INVALID),      # dtype
    ((16, 32, 48, 64, 80, 96, 8, -1, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, 48, 64, 80, 96, 0, 4, 256, 512, 64, 1e4, 0, None), INVALID),      # cache rows
    ((16, 32, 48, 64, 80, 96, 8, 4, 256, 510, 64, 1e4, 0, None), INVALID),      # d_c
    ((16, 32, 48, 64, 80, 96, 8, 4, 256, 512, 60, 1e4, 0, None), INVALID),      # d_R
    ((16, 32, 48, 64, 80, 96, 8, 4, 256, 512, 64, -1.0, 0, None), INVALID),
    ((None, 32, 48, 64, 80, 96, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, None, 48, 64, 80, 96, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, None, 64, 80, 96, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, 48, None, 80, 96, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, 48, 64, None, 96, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, 48, 64, 80, None, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),
    ((16, 32, 48, 64, 80, 100, 8, 4, 256, 512, 64, 1e4, 0, None), INVALID),     # alignment
    ((None, None, None, None, None, None, 8, 0, 256, 512, 64, 1e4, 0, None), OK),
])
def test_append_slots_refuses(lib, args, want):
    assert lib.mla_append_latent_slots(*args) == want


def test_binding_refuses():
    # wrong types and shapes, and host tensors, never reach the library
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, cache, u = torch.zeros((4, 2, 576)), torch.zeros((128, 576)), torch.zeros((4, 2, 512))
    good = dict(q=q, kv_cache=cache, block_table=i(2, 1), seqlens=i(2), cu_q=i(3),
                tree_mask=torch.zeros(4, dtype=torch.int64), u=u, lse=None, page_size=64, d_R=64, softmax_scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        mla.tree_params(**good)
    for kw, err in ((dict(tree_mask=i(4)), TypeError), (dict(cu_q=i(2)), ValueError),
                    (dict(block_table=i(3, 1)), ValueError), (dict(u=u[:3]), ValueError),
                    (dict(u=u.double()), TypeError), (dict(kv_cache=cache.double()), TypeError),
                    (dict(kv_cache=torch.zeros((100, 576))), ValueError),
                    (dict(lse=torch.zeros((4, 2), dtype=torch.float64)), ValueError),
                    (dict(seqlens=torch.zeros(2, dtype=torch.int64)), TypeError)):
        with pytest.raises(err):
            mla.tree_params(**{**good, **kw})
    with pytest.raises(ValueError):
        mla.tables_params(i(2), i(3), i(2, 4), i(5), i(1), i(1), i(2), i(3), i(9), i(9), i(9), 64, 8)
    with pytest.raises(TypeError):
        mla.tables_params(i(2), i(2), i(2, 4), i(5), i(1), i(1), i(2), i(3), i(9), i(9), i(9), 64, 8, parents=i(9), tree_mask=i(9))
    with pytest.raises(ValueError):
        mla.accept_params(cache, i(2, 1), i(2), i(3), torch.zeros(4, dtype=torch.int64), i(3), i(2), i(4), 64)
    h, w = torch.zeros((4, 64)), torch.zeros((512, 64))
    with pytest.raises(ValueError):
        mla.mla_append_latent_slots(h, w, torch.zeros((64, 32)), i(4), i(4), cache)
    with pytest.raises(TypeError):
        mla.mla_append_latent_slots(h, w, torch.zeros((64, 64)), i(4), i(4), cache.double())
    with pytest.raises(TypeError):
        mla.mla_append_latent_slots(h, w, torch.zeros((64, 64)), i(4).long(), i(4), cache)
