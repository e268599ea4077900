"""Argument checks of the calls for trees of drafted tokens, made before any
GPU work (no GPU needed)."""
import ctypes

import pytest

import paged_kv_cache_262_gb300 as pa
from paged_kv_cache_262_gb300 import build as pbuild

P = 4096  # an address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load()


def desc(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=10,
             max_blocks_per_seq=4, max_context_len=64, scale=0.1)
    d.update(kw)
    return pa.DecodeDesc(**d)


def attend(lib, d, q=P, k=P, v=P, bt=P, ctx=P, cu=P, parents=P, most=8, total=10, out=P, ws=None, n=0):
    return lib.pa_paged_attention_decode_tree(None if d is None else ctypes.byref(d), q, k, v, bt, ctx, cu, parents,
                                              most, total, out, ws, n, None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(head_dim=96), pa.PA_ERR_UNSUPPORTED), (dict(block_size=8), pa.PA_ERR_UNSUPPORTED),
    (dict(num_q_heads=34), pa.PA_ERR_UNSUPPORTED), (dict(num_q_heads=7), pa.PA_ERR_INVALID),
    (dict(num_seqs=-1), pa.PA_ERR_INVALID), (dict(num_seqs=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(num_blocks=0), pa.PA_ERR_INVALID), (dict(max_context_len=-1), pa.PA_ERR_INVALID),
])
def test_attention_desc(lib, kw, expect):
    assert attend(lib, desc(**kw)) == expect
    if expect == pa.PA_ERR_INVALID or "num_seqs" not in kw:
        assert lib.pa_decode_tree_workspace_bytes(ctypes.byref(desc(**kw)), 8) == 0


def test_attention_arguments(lib):
    d = desc()
    assert attend(lib, None) == pa.PA_ERR_INVALID
    for name in ("q", "k", "v", "bt", "ctx", "cu", "parents", "out"):
        assert attend(lib, d, **{name: None}) == pa.PA_ERR_INVALID, name
    for name in ("q", "k", "v", "out"):
        assert attend(lib, d, **{name: P + 8}) == pa.PA_ERR_INVALID, name
    assert attend(lib, d, most=0) == pa.PA_ERR_INVALID
    assert attend(lib, d, most=257) == pa.PA_ERR_UNSUPPORTED
    assert attend(lib, d, total=-1) == pa.PA_ERR_INVALID
    for most in (0, -3, 257):
        assert lib.pa_decode_tree_workspace_bytes(ctypes.byref(d), most) == 0
    # nothing to do: no pointer is looked at
    none = dict(q=None, k=None, v=None, bt=None, ctx=None, cu=None, parents=None, out=None)
    assert attend(lib, desc(num_seqs=0), **none) == pa.PA_OK
    assert attend(lib, d, total=0, **none) == pa.PA_OK


def verify(lib, logits=P, kind=0, stride=100, V=100, tokens=P, parents=P, cu=P, S=2, most=8, total=10, targets=P,
           path=P, lens=P, nexts=P):
    return lib.pa_verify_tree(logits, kind, stride, V, tokens, parents, cu, S, most, total, targets, path, lens, nexts,
                              None, None)


def test_verify_arguments(lib):
    for name in ("logits", "tokens", "parents", "cu", "targets", "path", "lens", "nexts"):
        assert verify(lib, **{name: None}) == pa.PA_ERR_INVALID, name
    assert verify(lib, kind=2) == pa.PA_ERR_INVALID
    assert verify(lib, stride=99) == pa.PA_ERR_INVALID
    assert verify(lib, V=0) == pa.PA_ERR_INVALID
    assert verify(lib, S=-1) == pa.PA_ERR_INVALID
    assert verify(lib, S=65536) == pa.PA_ERR_UNSUPPORTED
    assert verify(lib, most=0) == pa.PA_ERR_INVALID
    assert verify(lib, most=257) == pa.PA_ERR_UNSUPPORTED
    assert verify(lib, total=-1) == pa.PA_ERR_INVALID
    assert verify(lib, logits=P + 1) == pa.PA_ERR_INVALID
    assert verify(lib, logits=P + 2, kind=1) == pa.PA_ERR_INVALID
    none = dict(logits=None, tokens=None, parents=None, cu=None, targets=None, path=None, lens=None, nexts=None)
    assert verify(lib, S=0, **none) == pa.PA_OK


def commit(lib, d, k=(P,), v=(P,), L=1, bt=P, ctx=P, path=P, lens=P, most=8, new=1 << 20):
    arr = lambda x: None if x is None else (ctypes.c_void_p * len(x))(*x)  # noqa: E731
    return lib.pa_commit_tree(None if d is None else ctypes.byref(d), arr(k), arr(v), L, bt, ctx, path, lens, most, new,
                              None, None)


def test_commit_arguments(lib):
    d = desc()
    assert commit(lib, None) == pa.PA_ERR_INVALID
    for name in ("k", "v", "bt", "ctx", "path", "lens", "new"):
        assert commit(lib, d, **{name: None}) == pa.PA_ERR_INVALID, name
    assert commit(lib, d, L=0) == pa.PA_ERR_INVALID
    assert commit(lib, d, k=(P,) * 257, v=(P,) * 257, L=257) == pa.PA_ERR_INVALID
    assert commit(lib, d, k=(P, None), v=(P, P), L=2) == pa.PA_ERR_INVALID
    assert commit(lib, d, k=(P, P), v=(P, P + 8), L=2) == pa.PA_ERR_INVALID
    assert commit(lib, d, most=0) == pa.PA_ERR_INVALID
    assert commit(lib, d, most=257) == pa.PA_ERR_UNSUPPORTED
    assert commit(lib, desc(block_size=64)) == pa.PA_ERR_UNSUPPORTED
    base = 1 << 20
    for name, words in (("ctx", 2), ("lens", 2), ("path", 16), ("bt", 8)):  # new_lens over an input
        for at in (base, base - 4 * (words - 1), base + 4):
            assert commit(lib, d, **{name: at}) == pa.PA_ERR_INVALID, (name, at)
    assert commit(lib, desc(num_seqs=0), bt=None, ctx=None, path=None, lens=None, new=None) == pa.PA_OK


def test_flag_bits(lib):
    bits = [pa.DEVERR_CTX, pa.DEVERR_PAGE, pa.DEVERR_SLOT, pa.DEVERR_PAIR, pa.DEVERR_TIMEOUT, pa.DEVERR_ROW,
            pa.DEVERR_TREE]
    assert sorted(bits) == [1 << i for i in range(7)]
