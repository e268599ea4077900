"""Outputs of the calls on trees that lie over one another or over an input, and
pools given twice: refused before anything is launched."""
import ctypes

import pytest

import paged_kv_cache_262_gb300 as pa
from paged_kv_cache_262_gb300 import build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load()


# verify: 2 trees of up to 8 nodes, 10 nodes, 100 bf16 logits a row of 104
WORDS = dict(logits=(9 * 104 + 100) // 2, tokens=10, parents=10, cu=3, targets=10, path=16, lens=2, nexts=2)
OUT = ("targets", "path", "lens", "nexts")


def verify(lib, at):
    return lib.pa_verify_tree(at["logits"], 0, 104, 100, at["tokens"],
                              at["parents"], at["cu"], 2, 8, 10, *(at[k] for k in OUT), None, None)


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("other", sorted(WORDS))
def test_verify_outputs_lie_apart(lib, out, other):
    if out == other:
        return
    at = {k: (i + 1) << 20 for i, k in enumerate(sorted(WORDS))}
    for shift in {0, -(WORDS[out] - 1), WORDS[other] - 1}:  # the same place, and one word in common at either end
        assert verify(lib, {**at, out: at[other] + 4 * shift}) == pa.PA_ERR_INVALID


def commit(lib, k, v):
    d = pa.DecodeDesc(2, 8, 8, 64, 16, 4, 4, 64, 1.0)
    arr = lambda x: (ctypes.c_void_p * len(x))(*x)  # noqa: E731
    return lib.pa_commit_tree(ctypes.byref(d), arr(k), arr(v), len(k), 16, 1 << 12, 1 << 13, 1 << 14, 8, 1 << 15, None,
                              None)


def test_commit_pools_lie_apart(lib):
    base, size = 1 << 24, 4 * 8 * 16 * 64 * 2
    p = [base + i * size for i in range(6)]
    assert commit(lib, p[:3], [p[3], p[4], p[0]]) == pa.PA_ERR_INVALID
    assert commit(lib, [p[0], p[1], p[1]], p[3:]) == pa.PA_ERR_INVALID
    assert commit(lib, p[:1], p[:1]) == pa.PA_ERR_INVALID
    assert commit(lib, p[:3], [p[3], p[4], p[5] - 16]) == pa.PA_ERR_INVALID
