"""Block-sparse decode and eviction: every refusal that needs no GPU, by the
C calls (before any launch) and by the binding, and the wrappers' marshalling
against a recording stand-in for the library."""
import ctypes

import pytest

import paged_kv_cache_262_gb300 as pa
from paged_kv_cache_262_gb300 import build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load()


def _desc(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=10,
             max_blocks_per_seq=4, max_context_len=64, scale=0.1)
    d.update(kw)
    return ctypes.byref(pa.DecodeDesc(**d))


BAD_DESC = [(dict(head_dim=96), pa.PA_ERR_UNSUPPORTED), (dict(block_size=8), pa.PA_ERR_UNSUPPORTED),
            (dict(num_q_heads=6, num_kv_heads=4), pa.PA_ERR_INVALID), (dict(num_seqs=-1), pa.PA_ERR_INVALID),
            (dict(num_q_heads=34, num_kv_heads=2), pa.PA_ERR_UNSUPPORTED)]


def bounds(lib, d, k=16, bt=16, ctx=16, start=16, new=64, out=16):
    return lib.pa_block_key_bounds(d, k, bt, ctx, start, new, out, None, None)


def select(lib, d, q=16, b=16, bt=16, ctx=16, k=4, sink=1, recent=1, sel=16, ws=16, n=1 << 20):
    return lib.pa_select_blocks(d, q, b, bt, ctx, k, sink, recent, sel, ws, n, None, None)


def sparse(lib, d, q=16, kp=16, vp=16, bt=16, ctx=16, sel=16, k=4, out=16, ws=None, n=0):
    return lib.pa_paged_attention_decode_sparse(d, q, kp, vp, bt, ctx, sel, k, out, ws, n, None, None)


def weights(lib, d, q=16, kp=16, vp=16, bt=16, ctx=16, w=16, wo=16, rows=None, nr=2, mt=64, out=16, ws=16, n=1 << 30):
    return lib.pa_paged_attention_decode_weights(d, q, kp, vp, bt, ctx, w, wo, rows, nr, mt, out, ws, n, None, None)


def evict(lib, d, kp=16, vp=16, bt=16, dst=None, ctx=16, keep=16, mk=8, sink=1, recent=1, w=16, wo=16, rows=None,
          nr=2, mt=64, kept=16, new=32):
    return lib.pa_evict_tokens(d, kp, vp, bt, dst, ctx, keep, mk, sink, recent, w, wo, rows, nr, mt, kept, new, None,
                               None)


@pytest.mark.parametrize("call", [bounds, select, sparse, weights, evict])
@pytest.mark.parametrize("kw,expect", BAD_DESC)
def test_bad_descs(lib, call, kw, expect):
    assert call(lib, _desc(**kw)) == expect


@pytest.mark.parametrize("call", [bounds, select, sparse, weights, evict])
def test_null_desc_and_no_sequences(lib, call):
    assert call(lib, None) == pa.PA_ERR_INVALID
    assert call(lib, _desc(num_seqs=0)) == pa.PA_OK  # nothing to launch


def test_no_workspace_for_a_bad_desc(lib):
    bad = _desc(head_dim=96)
    assert lib.pa_select_blocks_workspace_bytes(bad) == 0
    assert lib.pa_decode_sparse_workspace_bytes(bad, 4) == 0
    assert lib.pa_decode_weights_workspace_bytes(bad) == 0
    assert lib.pa_decode_sparse_workspace_bytes(_desc(), 0) == 0


INVALID = pa.PA_ERR_INVALID


@pytest.mark.parametrize("call,kw", [
    (bounds, dict(k=None)), (bounds, dict(bt=None)), (bounds, dict(ctx=None)), (bounds, dict(out=None)),
    (bounds, dict(k=18)), (bounds, dict(out=24)), (bounds, dict(new=-1)),
    (select, dict(q=None)), (select, dict(b=None)), (select, dict(bt=None)), (select, dict(ctx=None)),
    (select, dict(sel=None)), (select, dict(q=18)), (select, dict(b=24)), (select, dict(k=0)), (select, dict(k=-1)),
    (select, dict(sink=-1)), (select, dict(recent=-1)), (select, dict(sink=3, recent=2)),
    (select, dict(sink=2**31 - 1, recent=2**31 - 1)),
    (sparse, dict(q=None)), (sparse, dict(kp=None)), (sparse, dict(vp=None)), (sparse, dict(bt=None)),
    (sparse, dict(ctx=None)), (sparse, dict(sel=None)), (sparse, dict(out=None)), (sparse, dict(q=18)),
    (sparse, dict(out=24)), (sparse, dict(k=0)), (sparse, dict(k=-3)),
    (weights, dict(q=None)), (weights, dict(w=None)), (weights, dict(wo=None)), (weights, dict(out=None)),
    (weights, dict(ctx=None)), (weights, dict(w=20)), (weights, dict(wo=24)), (weights, dict(mt=63)),
    (weights, dict(nr=1)), (weights, dict(nr=-1, rows=16)),
    (evict, dict(kp=None)), (evict, dict(vp=None)), (evict, dict(bt=None)), (evict, dict(ctx=None)),
    (evict, dict(keep=None)), (evict, dict(w=None)), (evict, dict(wo=None)), (evict, dict(kept=None)),
    (evict, dict(new=None)), (evict, dict(kp=18)), (evict, dict(w=20)), (evict, dict(mk=0)), (evict, dict(sink=-1)),
    (evict, dict(recent=-1)), (evict, dict(mt=63)), (evict, dict(nr=1)), (evict, dict(new=16)),
    # (2 rows x 2 heads x 64 tokens x 4 bytes = 1024: arrays less than that apart overlap)
    (evict, dict(w=4096, wo=4096 + 1008)), (evict, dict(w=4096 + 16, wo=4096)),
    (weights, dict(w=4096, wo=4096 + 1008)), (weights, dict(w=4096 + 16, wo=4096)),
])
def test_bad_arguments(lib, call, kw):
    assert call(lib, _desc(), **kw) == INVALID


def test_workspaces_are_checked(lib):
    # (the selection's plan needs no device; the others ask the GPU for its SM count first)
    need = lib.pa_select_blocks_workspace_bytes(_desc())
    assert need > 0
    assert select(lib, _desc(), ws=None) == pa.PA_ERR_WORKSPACE
    assert select(lib, _desc(), n=need - 1) == pa.PA_ERR_WORKSPACE
    assert select(lib, _desc(), ws=24) == pa.PA_ERR_WORKSPACE
    assert sparse(lib, _desc(), k=256 * 512 + 1) == pa.PA_ERR_UNSUPPORTED


class _Lib:
    capturing = False

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("workspace_bytes") else 0
        return f


@pytest.fixture
def fake(monkeypatch):
    """CPU tensors through the wrappers: the device checks and torch.cuda's
    stream calls faked, the library a recorder."""
    import torch
    from paged_kv_cache_262_gb300 import _binding as b
    lib = _Lib()

    def need(t, dtype, name, ndim=None):  # _need without the device check
        if t.dtype != dtype:
            raise TypeError(name)
        if not t.is_contiguous() or (ndim is not None and t.dim() != ndim):
            raise ValueError(name)

    T = b._Torch()
    T.device = lambda: -1  # a host tensor's get_device()
    T.stream = lambda device: 7
    T.capturing = lambda: lib.capturing
    T.empty = lambda *a, **k: torch.empty(*a, **{x: y for x, y in k.items() if x != "device"})
    monkeypatch.setattr(b, "_T", T)
    monkeypatch.setattr(b, "_FAST", False)
    monkeypatch.setattr(b, "_LIB", lib)
    monkeypatch.setattr(b, "_need", need)
    monkeypatch.setattr(b, "_ws", lambda w: None if w is None else w.data_ptr())
    monkeypatch.setattr(b, "_cached_ws", lambda cache, n, device, stream: cache.setdefault(
        (device.index, 7), torch.empty(n, dtype=torch.uint8)))
    lib.capturing = False
    lib.T = T
    lib.caches = {}
    for name in ("_WS_SELECT", "_WS_SPARSE", "_WS_WEIGHTS"):
        lib.caches[name] = {}
        monkeypatch.setattr(b, name, lib.caches[name])
    return lib


def _tensors():
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    S, HQ, HKV, D, B, NB, MB = 4, 8, 2, 128, 16, 32, 6
    t = dict(q=torch.zeros(S, HQ, D, dtype=bf), kp=torch.zeros(NB, HKV, B, D, dtype=bf),
             bt=torch.zeros(S, MB, dtype=i32), ctx=torch.full((S,), 40, dtype=i32),
             bounds=torch.zeros(NB, HKV, 2, D, dtype=bf), sel=torch.zeros(S, HKV, 3, dtype=i32),
             w=torch.zeros(S, HKV, MB * B), keep=torch.full((S,), 8, dtype=i32))
    t["vp"] = t["kp"].clone()
    return t


def test_wrappers_marshal_their_calls(fake):
    t = _tensors()
    assert pa.block_key_bounds(t["kp"], t["bounds"], t["bt"], t["ctx"]) is t["bounds"]
    sel = pa.select_blocks(t["q"], t["bounds"], t["bt"], t["ctx"], 3, block_size=16, max_context_len=80)
    assert tuple(sel.shape) == (4, 2, 3)
    out = pa.paged_attention_decode_sparse(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], sel)
    assert out.shape == t["q"].shape
    out, w = pa.paged_attention_decode_weights(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"])
    assert w is t["w"]
    kept, new = pa.evict_tokens(t["kp"], t["vp"], t["bt"], t["ctx"], t["keep"], t["w"], max_keep_len=9, sink_tokens=1,
                                recent_tokens=2)
    assert tuple(kept.shape) == (4, 2, 9) and tuple(new.shape) == (4,)
    args = {n: a for n, a in fake.calls}
    d = args["pa_block_key_bounds"][0]._obj
    assert (d.num_q_heads, d.num_kv_heads, d.head_dim, d.block_size, d.num_blocks, d.max_blocks_per_seq,
            d.max_context_len) == (2, 2, 128, 16, 32, 6, 96)
    assert args["pa_block_key_bounds"][4:6] == (None, 96)
    d = args["pa_select_blocks"][0]._obj
    assert (d.num_seqs, d.num_q_heads, d.num_kv_heads, d.max_context_len) == (4, 8, 2, 80)
    assert args["pa_select_blocks"][5:8] == (3, 1, 1)
    assert args["pa_paged_attention_decode_sparse"][7] == 3
    assert args["pa_paged_attention_decode_weights"][8:11] == (None, 4, 96)
    assert args["pa_evict_tokens"][7:10] == (9, 1, 2)
    assert args["pa_evict_tokens"][10] == args["pa_evict_tokens"][11] == t["w"].data_ptr()
    assert [len(c) for c in fake.caches.values()] == [1, 1, 1]  # one workspace per (device, stream)


def test_captured_calls_take_no_cached_workspace(fake):
    t = _tensors()
    fake.capturing = True
    pa.select_blocks(t["q"], t["bounds"], t["bt"], t["ctx"], 3, block_size=16)
    pa.paged_attention_decode_weights(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"])
    assert [len(c) for c in fake.caches.values()] == [0, 0, 0]


def _refused(fake, exc, f, *a, **k):
    n = len(fake.calls)
    with pytest.raises(exc):
        f(*a, **k)
    assert all(name.endswith("workspace_bytes") for name, _ in fake.calls[n:])


def test_wrappers_refuse_what_the_pointers_cannot_show(fake):
    import torch
    t = _tensors()
    V = ValueError
    _refused(fake, V, pa.block_key_bounds, t["kp"], t["bounds"][:-1], t["bt"], t["ctx"])
    _refused(fake, V, pa.block_key_bounds, t["kp"], t["bounds"], t["bt"][:3], t["ctx"])
    _refused(fake, V, pa.block_key_bounds, t["kp"], t["bounds"], t["bt"], t["ctx"], t["ctx"][:3])
    _refused(fake, TypeError, pa.block_key_bounds, t["kp"], t["bounds"].float(), t["bt"], t["ctx"])
    _refused(fake, V, pa.select_blocks, t["q"][:, :, :64].contiguous(), t["bounds"], t["bt"], t["ctx"], 3,
             block_size=16)
    _refused(fake, V, pa.select_blocks, t["q"], t["bounds"], t["bt"], t["ctx"][:2], 3, block_size=16)
    _refused(fake, V, pa.select_blocks, t["q"], t["bounds"], t["bt"], t["ctx"], 3, block_size=16,
             selected=torch.zeros(4, 2, 4, dtype=torch.int32))
    _refused(fake, V, pa.paged_attention_decode_sparse, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["sel"][:3])
    _refused(fake, V, pa.paged_attention_decode_sparse, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"],
             t["sel"][:, :1].contiguous())
    _refused(fake, V, pa.paged_attention_decode_sparse, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"],
             t["sel"].transpose(0, 1))  # strided
    w = pa.paged_attention_decode_weights
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"][:3].contiguous())
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"][:, :, :95].contiguous())
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"][:, :1].contiguous())
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"], weights_out=t["w"][:3].contiguous())
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"],
             weight_rows=torch.zeros(3, dtype=torch.int32))
    _refused(fake, TypeError, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"].double())
    both = torch.zeros(5, 2, 96)
    _refused(fake, V, w, t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], both[:4], weights_out=both[1:])  # overlap
    e = pa.evict_tokens
    ok = (t["kp"], t["vp"], t["bt"], t["ctx"])
    _refused(fake, V, e, *ok, t["keep"], t["w"], max_keep_len=0)
    _refused(fake, V, e, *ok, t["keep"][:3], t["w"], max_keep_len=8)
    _refused(fake, V, e, *ok, t["keep"], t["w"][:3].contiguous(), max_keep_len=8)
    _refused(fake, V, e, *ok, t["keep"], t["w"], max_keep_len=8, dst_tables=t["bt"][:, :5].contiguous())
    _refused(fake, V, e, *ok, t["keep"], t["w"], max_keep_len=8, dst_tables=t["bt"][:3])
    _refused(fake, V, e, *ok, t["keep"], t["w"], max_keep_len=8, kept=torch.zeros(4, 2, 9, dtype=torch.int32))
    _refused(fake, V, e, *ok, t["keep"], t["w"], max_keep_len=8, new_lens=t["ctx"])
    _refused(fake, V, e, t["kp"], t["vp"][:-1], t["bt"], t["ctx"], t["keep"], t["w"], max_keep_len=8)


def test_wrappers_refuse_host_tensors(monkeypatch):
    import torch
    t = _tensors()
    from paged_kv_cache_262_gb300 import _binding as b
    T = b._Torch()
    T.device = lambda: 0
    monkeypatch.setattr(b, "_T", T)
    with pytest.raises(TypeError):
        pa.block_key_bounds(t["kp"], t["bounds"], t["bt"], t["ctx"])
    with pytest.raises(TypeError):
        pa.select_blocks(t["q"], t["bounds"], t["bt"], t["ctx"], 3, block_size=16)
    with pytest.raises(TypeError):
        pa.paged_attention_decode_weights(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"])
    with pytest.raises(TypeError):
        pa.evict_tokens(t["kp"], t["vp"], t["bt"], t["ctx"], t["keep"], t["w"], max_keep_len=8)
    assert isinstance(t["q"], torch.Tensor)


def test_wrappers_refuse_what_is_no_tensor_or_on_another_device(fake):
    t = _tensors()
    with pytest.raises((TypeError, AttributeError)):
        pa.block_key_bounds(t["kp"], t["bounds"], t["bt"].tolist(), t["ctx"])
    fake.T.device = lambda: 1
    for call in (lambda: pa.block_key_bounds(t["kp"], t["bounds"], t["bt"], t["ctx"]),
                 lambda: pa.select_blocks(t["q"], t["bounds"], t["bt"], t["ctx"], 3, block_size=16),
                 lambda: pa.paged_attention_decode_sparse(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["sel"]),
                 lambda: pa.paged_attention_decode_weights(t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"]),
                 lambda: pa.evict_tokens(t["kp"], t["vp"], t["bt"], t["ctx"], t["keep"], t["w"], max_keep_len=8)):
        _refused(fake, ValueError, call)


def test_the_quick_way_leaves_everything_unusual_to_the_other(lib):
    """The extension module, where it is built: None, without a launch and
    without an error, for host tensors, for what is no tensor, for a wrong
    number of arguments -- and for anything at all where there is no GPU."""
    from paged_kv_cache_262_gb300 import _binding as b
    F = b._FAST if b._FAST is not None else b._fast()
    if not F:
        pytest.skip("the extension module is not built")
    t = _tensors()
    calls = [(F.bounds, (t["kp"], t["bounds"], t["bt"], t["ctx"], None, None, None, None)),
             (F.select, (t["q"], t["bounds"], t["bt"], t["ctx"], 3, 16, 1, 1, None, None, {})),
             (F.sparse, (t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["sel"], None, None, None, {})),
             (F.weights, (t["q"], t["kp"], t["vp"], t["bt"], t["ctx"], t["w"], None, None, None, None, None, {})),
             (F.evict, (t["kp"], t["vp"], t["bt"], t["ctx"], t["keep"], t["w"], 8, 0, 0, None, None, None, None,
                        None))]
    for f, args in calls:
        assert f(*args) is None
        assert f(*args[:-1]) is None and f() is None
        for i in range(len(args)):
            for x in (None, "q", 1.5, [1], 2**40, -2**40, object()):
                assert f(*args[:i], x, *args[i + 1:]) is None
    with pytest.raises(TypeError):
        F.bind(1, 2)


# (2 sequences, 2 kv heads, 4 blocks a table, max_keep_len 8: new_lens 8 bytes, kept 128, a table 32)
APART = dict(bt=4096, ctx=8192, keep=12288, kept=16384, new=20480)


@pytest.mark.parametrize("kw", [
    dict(new=8192), dict(new=8196), dict(new=8188), dict(new=12288), dict(new=12292), dict(new=12284),
    dict(new=4096), dict(new=4124), dict(rows=24576, new=24576), dict(rows=24576, new=24580),
    dict(dst=28672, new=28672), dict(dst=28672, new=28700), dict(new=16384), dict(new=16508), dict(new=16380),
    dict(kept=8192), dict(kept=8068), dict(kept=12288), dict(kept=4096 + 28), dict(kept=4096 - 124),
    dict(rows=24576, kept=24576), dict(dst=28672, kept=28672 - 124),
])
def test_outputs_of_an_eviction_that_overlap_what_it_reads(lib, kw):
    """Another kv head's CTA may still have to read what the first one
    writes: refused, whole or in part."""
    assert evict(lib, _desc(), **{**APART, **kw}) == INVALID


@pytest.mark.parametrize("kw", [dict(), dict(new=8200), dict(new=8184), dict(new=4128), dict(new=16512),
                                dict(rows=24576, new=24584), dict(dst=28672, kept=28672 - 128), dict(dst=4096)])
def test_outputs_of_an_eviction_beside_what_it_reads(lib, kw):
    """Not refused: the call goes on to ask for the GPU (and, having one,
    would launch, so only where there is none)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory")
    assert evict(lib, _desc(), **{**APART, **kw}) == pa.PA_ERR_CUDA


def test_the_wrapper_refuses_outputs_that_overlap(fake):
    import torch
    t = _tensors()
    ok = (t["kp"], t["vp"], t["bt"], t["ctx"])

    def refused(**kw):
        args = dict(keep_lens=t["keep"])
        args.update(kw)
        keep = args.pop("keep_lens")
        _refused(fake, ValueError, pa.evict_tokens, *ok, keep, t["w"], max_keep_len=8, **args)

    both = torch.zeros(7, dtype=torch.int32)  # [0:4] and [3:7]
    rows = torch.arange(4, dtype=torch.int32)
    refused(new_lens=t["keep"])
    refused(keep_lens=both[:4], new_lens=both[3:])
    refused(new_lens=rows, weight_rows=rows)
    refused(new_lens=t["bt"].view(-1)[:4])
    flat = torch.zeros(4 * 2 * 8 + 4, dtype=torch.int32)
    refused(kept=flat[:64].view(4, 2, 8), new_lens=flat[60:64])
    dst = torch.zeros(64 + 24, dtype=torch.int32)
    refused(kept=dst[:64].view(4, 2, 8), dst_tables=dst[63:87].view(4, 6))
    # side by side: taken
    one = torch.zeros(64 + 4 + 4, dtype=torch.int32)
    kept, new = pa.evict_tokens(*ok, one[64:68], t["w"], max_keep_len=8, kept=one[:64].view(4, 2, 8),
                                new_lens=one[68:])
    assert fake.calls[-1][0] == "pa_evict_tokens" and kept.data_ptr() == one.data_ptr()
