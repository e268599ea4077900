"""The long-context calls at their edges: logits and values that are not
finite, refused sequences, calls from several host threads, launches that
fail."""
import math

import pytest

import paged_kv_cache_262_gb300 as pa
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def _ref():
    import long_context_ref
    return long_context_ref


def err_of(torch):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------ values that are not finite
NOT_FINITE = ["nan_key", "nan_query", "inf_key", "all_nan", "nan_value"]
#: (query heads, kv heads, head_dim, block), contexts, PA_PARTITION_PAGES: one
#: CTA a (sequence, kv head), clusters, and several clusters joined
SPLITS = [((8, 2, 64, 16), [1, 40, 1000, 300], None), ((8, 2, 128, 16), [1, 40, 1000, 300], "1"),
          ((16, 1, 64, 32), [1, 40, 1000, 300], "3"), ((6, 2, 128, 32), [1, 40, 1000, 300], "512"),
          ((4, 1, 64, 16), [30000, 20], None), ((20, 2, 128, 16), [9000, 20], None)]


def not_finite_case(torch, what, shape, lens):
    """Caches and queries with such a value in every sequence but the second."""
    R = _ref()
    Hq, Hkv, D, B = shape
    c = R.make_cache(lens, Hkv, D, B, seed=81, junk=float("nan"))
    q = torch.randn(len(lens), Hq, D, device="cuda",
                    generator=torch.Generator(device="cuda").manual_seed(82)).to(torch.bfloat16)
    for s, n in enumerate(lens):
        if s == 1:
            continue
        j = n // 2
        blk, at = int(c["bt"][s, j // B]), j % B
        if what == "nan_key":
            c["k"][blk, Hkv - 1, at, 3] = math.nan
        elif what == "nan_query":
            q[s, Hq - 1, 5] = math.nan
        elif what == "inf_key":  # +infinity for some heads, -infinity for others
            c["k"][blk, 0, at, 7] = math.inf
        elif what == "all_nan":
            c["k"][c["bt"][s, :-(-n // B)].long(), 0] = math.nan
        else:
            c["v"][blk, 0, at, 9] = math.nan
    return c, q


def as_wanted(torch, got, want, tol):
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and bool(((got - want).abs() <= tol)[~nan].all())


@pytest.mark.parametrize("what", NOT_FINITE)
@pytest.mark.parametrize("shape,lens,pp", SPLITS)
def test_sparse_reports_what_is_not_finite(torch, monkeypatch, what, shape, lens, pp):
    """A NaN or +infinite logit makes its head's row NaN, however the list is
    split; -infinity weighs nothing."""
    R = _ref()
    monkeypatch.delenv("PA_PARTITION_PAGES", raising=False)
    if pp:
        monkeypatch.setenv("PA_PARTITION_PAGES", pp)
    Hq, Hkv, D, B = shape
    G = Hq // Hkv
    c, q = not_finite_case(torch, what, shape, lens)
    k = max(-(-n // B) for n in lens)
    sel = torch.full((len(lens), Hkv, k), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        sel[s, :, :-(-n // B)] = torch.arange(-(-n // B), dtype=torch.int32, device="cuda")
    err = err_of(torch)
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel, err_flag=err)
    assert int(err) == 0
    for s, n in enumerate(lens):
        for h in range(Hkv):
            _, want, tol, _ = R.ref_attend_any(q[s, h * G:(h + 1) * G], R.rows(c["k"], c["bt"][s], n, B, h),
                                               R.rows(c["v"], c["bt"][s], n, B, h), 1 / math.sqrt(D))
            assert as_wanted(torch, out[s, h * G:(h + 1) * G].double(), want, tol), (s, h)


@pytest.mark.parametrize("what", NOT_FINITE)
@pytest.mark.parametrize("shape,lens,pp", SPLITS)
@pytest.mark.parametrize("with_rows", [False, True])
def test_weights_report_what_is_not_finite(torch, monkeypatch, what, shape, lens, pp, with_rows):
    """The same for decode with weights; the weights of a kv head with such a
    row are NaN, by one launch and by two (with_rows)."""
    R = _ref()
    monkeypatch.delenv("PA_PARTITION_PAGES", raising=False)
    if pp:
        monkeypatch.setenv("PA_PARTITION_PAGES", pp)
    Hq, Hkv, D, B = shape
    G = Hq // Hkv
    c, q = not_finite_case(torch, what, shape, lens)
    rows = torch.arange(len(lens), dtype=torch.int32, device="cuda") if with_rows else None
    w, err = torch.zeros(len(lens), Hkv, c["mb"] * B, device="cuda"), err_of(torch)
    out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w, weight_rows=rows,
                                               max_context_len=max(lens), err_flag=err)
    assert int(err) == 0
    for s, n in enumerate(lens):
        for h in range(Hkv):
            p, want, tol, tp = R.ref_attend_any(q[s, h * G:(h + 1) * G], R.rows(c["k"], c["bt"][s], n, B, h),
                                                R.rows(c["v"], c["bt"][s], n, B, h), 1 / math.sqrt(D))
            assert as_wanted(torch, out[s, h * G:(h + 1) * G].double(), want, tol), (s, h)
            # (the tolerance of the weights: their probabilities', and 2^-24 an addition)
            assert as_wanted(torch, w[s, h, :n].double(), p.sum(0), tp.sum(0) + 2.0**-20 * p.sum(0)), (s, h)
            assert bool((w[s, h, n:] == 0).all())


# ---------------------------------------------------------- refused sequences
@pytest.mark.parametrize("S,Hkv,D", [(2, 2, 64), (3, 8, 128), (40, 8, 128)])
@pytest.mark.parametrize("blocks", [4, 9])
def test_evict_refuses_a_context_past_its_table(torch, S, Hkv, D, blocks):
    """max_keep_len above the table's capacity, and in the last row a context
    past it: refused, and nothing behind the tables' rows is read (tables that
    end their allocation; every form of the row kernel)."""
    R = _ref()
    B = 16
    lens = [blocks * B - s % 7 for s in range(S)]
    c = R.make_cache(lens, Hkv, D, B, seed=86)
    bt = c["bt"][:, :blocks].contiguous()
    dst, ctx = bt.clone(), c["ctx"].clone()
    ctx[S - 1] = 5000
    max_keep, keep = 4096, torch.full((S,), 20, dtype=torch.int32, device="cuda")
    keep[S - 1] = 4096
    k0, v0 = c["k"].clone(), c["v"].clone()
    w0 = torch.rand(S, Hkv, 5000, device="cuda")
    w, err = w0.clone(), err_of(torch)
    kept, new = pa.evict_tokens(c["k"], c["v"], bt, ctx, keep, w, max_keep_len=max_keep, dst_tables=dst,
                                max_context_len=5000, err_flag=err)
    assert int(err) == pa.DEVERR_CTX and new.tolist() == [20] * (S - 1) + [5000]
    assert bool((kept[S - 1] == -1).all()) and torch.equal(w[S - 1], w0[S - 1])
    for s, n in enumerate(lens[:-1]):
        for h in range(Hkv):
            at = R.ref_evict(w0[s, h, :n], 20, 0, 0, n)
            assert torch.equal(kept[s, h, :20].long(), at) and bool((kept[s, h, 20:] == -1).all())
            i = torch.arange(20, device="cuda")
            src, to = bt[s].long()[at // B], bt[s].long()[i // B]
            for pool, old in ((c["k"], k0), (c["v"], v0)):
                assert torch.equal(pool[to, h, i % B], old[src, h, at % B])
    last = bt[S - 1].long()
    assert torch.equal(c["k"][last], k0[last]) and torch.equal(c["v"][last], v0[last])


# ------------------------------------------------------ several host threads
def test_small_and_large_grids_from_several_threads(torch, monkeypatch):
    """Launches of one kernel with unlike amounts of shared memory, made at
    the same time: a grid of a wave asks for more than a larger one does."""
    import ctypes
    import threading

    R = _ref()
    monkeypatch.setenv("PA_PARTITION_PAGES", "1")  # three parts a list
    Hkv, Hq, D, B = 2, 8, 128, 16
    c = R.make_cache([48], Hkv, D, B, seed=83)
    lib, stream = pa.load(), torch.cuda.current_stream().cuda_stream
    calls, outs, want, keep = [], [], [], []
    for S in (1, 120, 2, 90):  # 6, 720, 12 and 540 CTAs
        q = torch.randn(S, Hq, D, device="cuda").to(torch.bfloat16)
        sel = torch.arange(3, dtype=torch.int32, device="cuda").expand(S, Hkv, 3).contiguous()
        bt, ctx, out = c["bt"].expand(S, -1).contiguous(), c["ctx"].expand(S).contiguous(), torch.empty_like(q)
        want.append(pa.paged_attention_decode_sparse(q, c["k"], c["v"], bt, ctx, sel))
        desc = pa.DecodeDesc(S, Hq, Hkv, D, B, c["k"].shape[0], bt.shape[1], 48, D**-0.5)
        assert lib.pa_decode_sparse_workspace_bytes(ctypes.byref(desc), 3) == 0
        calls.append((ctypes.byref(desc), q.data_ptr(), c["k"].data_ptr(), c["v"].data_ptr(), bt.data_ptr(),
                      ctx.data_ptr(), sel.data_ptr(), 3, out.data_ptr(), None, 0, None, stream))
        outs.append(out)
        keep.append((q, sel, bt, ctx))
    torch.cuda.synchronize()
    start, status = threading.Barrier(len(calls)), [set() for _ in calls]

    def run(i):
        f, args, seen = lib.pa_paged_attention_decode_sparse, calls[i], status[i]
        start.wait(60)
        for _ in range(4000):  # (the interpreter lock is free while the C call runs)
            seen.add(f(*args))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{pa.PA_OK}] * len(calls), status
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("with_rows", [True, False])
def test_weights_calls_of_several_threads_share_a_workspace(torch, with_rows):
    """C calls from threads that share a stream and a workspace: two kernels
    each (with rows, or for the long context), of which no other thread's call
    comes between."""
    import ctypes
    import threading

    R = _ref()
    Hq, Hkv, D, B, lens = 8, 2, 64, 16, [40000, 900, 40]
    c = R.make_cache(lens, Hkv, D, B, seed=87)
    lib, stream = pa.load(), torch.cuda.current_stream().cuda_stream
    rows = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda") if with_rows else None
    desc = pa.DecodeDesc(3, Hq, Hkv, D, B, c["k"].shape[0], c["mb"], max(lens), D**-0.5)
    n = int(lib.pa_decode_weights_workspace_bytes(ctypes.byref(desc)))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    width, N, T = c["mb"] * B, 150, 4

    def arrays():
        return [(torch.zeros(3, Hkv, width, device="cuda"), torch.empty(3, Hq, D, dtype=torch.bfloat16, device="cuda"))
                for _ in range(T)]

    qs = [torch.randn(3, Hq, D, device="cuda").to(torch.bfloat16) for _ in range(T)]

    def call(i, w, out):
        return lib.pa_paged_attention_decode_weights(
            ctypes.byref(desc), qs[i].data_ptr(), c["k"].data_ptr(), c["v"].data_ptr(), c["bt"].data_ptr(),
            c["ctx"].data_ptr(), w.data_ptr(), w.data_ptr(), None if rows is None else rows.data_ptr(), 3, width,
            out.data_ptr(), ws.data_ptr(), n, None, stream)

    want, got = arrays(), arrays()
    for i in range(T):
        for _ in range(N):
            assert call(i, *want[i]) == pa.PA_OK
    torch.cuda.synchronize()
    start, status = threading.Barrier(T), [set() for _ in range(T)]

    def run(i):
        start.wait(60)
        for _ in range(N):
            status[i].add(call(i, *got[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(T)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{pa.PA_OK}] * T
    for x, y in zip(want, got):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


# ------------------------------------------------------- launches that fail
def test_a_call_that_failed_is_not_made_again(torch, monkeypatch):
    """Every call by the extension module against a library whose calls fail
    as a launch does (the first of two kernels may be on its way by then): the
    failure is raised, and no call is made twice."""
    import ctypes

    from paged_kv_cache_262_gb300 import _binding as b
    R = _ref()
    F = b._FAST if b._FAST is not None else b._fast()
    assert F, "the extension module is not built"
    lib = pa.load()
    names = ("pa_block_key_bounds", "pa_select_blocks_workspace_bytes", "pa_select_blocks",
             "pa_decode_sparse_workspace_bytes", "pa_paged_attention_decode_sparse",
             "pa_decode_weights_workspace_bytes", "pa_paged_attention_decode_weights", "pa_evict_tokens")
    made, keep = [], []

    def failing(name):
        def call(*_):
            made.append(name)
            return pa.PA_ERR_CUDA
        f = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(lib, name).argtypes)(call)
        keep.append(f)
        return f

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes") or name == "pa_status_string":
                return getattr(lib, name)
            return made.append(name) or (lambda *_: 0)

    c = R.make_cache([100, 40], 2, 64, 16, seed=84)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    bd = torch.zeros(c["k"].shape[0], 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    sel = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 2, c["mb"] * 16, device="cuda")
    cache = (c["k"], c["v"], c["bt"], c["ctx"])
    calls = [("pa_block_key_bounds", lambda: pa.block_key_bounds(c["k"], bd, c["bt"], c["ctx"])),
             ("pa_select_blocks", lambda: pa.select_blocks(q, bd, c["bt"], c["ctx"], 3, block_size=16)),
             ("pa_paged_attention_decode_sparse", lambda: pa.paged_attention_decode_sparse(q, *cache, sel)),
             ("pa_paged_attention_decode_weights", lambda: pa.paged_attention_decode_weights(q, *cache, w)),
             ("pa_evict_tokens", lambda: pa.evict_tokens(*cache, torch.full_like(c["ctx"], 8), w, max_keep_len=8))]
    for _, call in calls:
        call()  # (so that the default workspaces are there)
    real = [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names]
    F.bind(*(a if n.endswith("_bytes") else ctypes.cast(failing(n), ctypes.c_void_p).value
             for n, a in zip(names, real)))
    try:
        monkeypatch.setattr(b, "_LIB", Lib())
        for name, call in calls:
            made.clear()
            with pytest.raises(pa.PaError) as e:
                call()
            assert made == [name] and e.value.status == pa.PA_ERR_CUDA and name in str(e.value)
    finally:
        F.bind(*real)
    monkeypatch.undo()
    for _, call in calls:
        call()


# ------------------------------------------------ table entries of the ends
@pytest.mark.parametrize("entry", ["above", -1, -2**31])
@pytest.mark.parametrize("where", ["sink", "recent", "short", "all_listed"])
@pytest.mark.parametrize("blocks", [40, 9000])
def test_selection_reports_every_unreadable_block(torch, entry, where, blocks):
    """A block with an entry outside the pool is reported also where it is
    listed whatever its score: a sink, a recent block, any block of a context
    with no more of them than the list has places."""
    R = _ref()
    Hkv, G, D, B, k = 2, 2, 64, 16, 12
    lens = [blocks * B, 9 * B - 3, k * B]
    g = torch.Generator(device="cuda").manual_seed(85)
    b = torch.randn(blocks, Hkv, 2, D, generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    bt = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)[None].expand(3, -1).contiguous()
    bt[1, 9:], bt[2, k:] = blocks + 1, -1  # past a context: not looked at
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(3, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    want, err = R.ref_select(q, b, bt, lens, B, G, k, 2, 3), err_of(torch)
    got = pa.select_blocks(q, b, bt, ctx, k, block_size=B, sink_blocks=2, recent_blocks=3, err_flag=err)
    assert torch.equal(got, want) and int(err) == 0
    s, i = {"sink": (0, 1), "recent": (0, blocks - 2), "short": (1, 8), "all_listed": (2, 5)}[where]
    bt[s, i] = blocks if entry == "above" else entry
    got = pa.select_blocks(q, b, bt, ctx, k, block_size=B, sink_blocks=2, recent_blocks=3, err_flag=err)
    assert torch.equal(got, want) and int(err) == pa.DEVERR_PAGE
