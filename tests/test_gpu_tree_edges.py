"""Calls on trees of drafted tokens at the edges of what is allowed, on the GPU:
the largest sizes, other streams, two calls at once, the quick way from Python
and the one through ctypes."""
import ctypes
import math
import random
import threading

import pytest

import gpu_util
import tree_ref as tr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return gpu_util.need_gpu()


@pytest.fixture(scope="module")
def pa(torch):
    import paged_kv_cache_262_gb300 as pa
    return pa


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_verify_largest_vocabulary(pa, torch):
    """Indices of the row's last words are just below 2^31."""
    V = 2**31 - 1
    x = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    args = (i32(torch, [0]), i32(torch, [-1]), i32(torch, [0, 1]))
    for at in (V - 1, V - 8, V - 9, 0):
        x[0, at] = 1
        got = pa.verify_tree(x, *args, max_tree_nodes=1)
        assert [t.flatten().tolist() for t in got] == [[at], [0], [1], [at]]
        x[0, at] = -1
