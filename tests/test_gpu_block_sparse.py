"""Block-sparse decode on the GPU: key bounds, block selection and attention
over the selected blocks against plain 64-bit implementations."""
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


def same_bits(torch, a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


SHAPES = [(4, 4, 64, 16), (8, 2, 64, 32), (32, 8, 128, 16), (64, 8, 128, 16), (6, 2, 128, 32), (16, 1, 128, 16),
          (10, 2, 64, 16), (3, 1, 128, 32)]
ids = lambda s: "q%dkv%dd%db%d" % s  # noqa: E731
LENS = [1, 2, 15, 16, 17, 31, 32, 33, 100, 257, 513, 1000, 1999]


# ------------------------------------------------------------------ key bounds
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_bounds_of_whole_contexts(torch, shape, junk):
    R = _ref()
    _, Hkv, D, B = shape
    c = R.make_cache(LENS, Hkv, D, B, seed=3, junk=junk)
    before = torch.full((c["k"].shape[0], Hkv, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    b, err = before.clone(), err_of(torch)
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"], err_flag=err)
    want = before.double()
    for blk, x in R.ref_bounds(c).items():
        want[blk] = x
    assert torch.equal(b.double(), want) and int(err) == 0


@pytest.mark.parametrize("new", [1, 2, 17, 40])
def test_bounds_of_the_last_tokens(torch, new):
    R = _ref()
    c = R.make_cache([n for n in LENS if n >= new], 3, 64, 16, seed=4, junk=float("nan"))
    start = [n - new for n in c["lens"]]
    b, err = torch.full((c["k"].shape[0], 3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"), err_of(torch)
    want = b.double()
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"], torch.tensor(start, dtype=torch.int32, device="cuda"),
                        max_new_tokens=new, err_flag=err)
    for blk, x in R.ref_bounds(c, start).items():
        want[blk] = x
    assert torch.equal(b.double(), want) and int(err) == 0


def test_bounds_with_nan_keys_and_signed_zeros(torch):
    R = _ref()
    c = R.make_cache([20, 33], 2, 64, 16, seed=5)
    blk = int(c["bt"][0, 0])
    c["k"][blk, 1, 3, 10] = float("nan")
    c["k"][blk, 0, :, 5] = 0.0
    c["k"][blk, 0, 4, 5] = -0.0
    c["k"][blk, 0, 0, 6] = float("inf")
    c["k"][blk, 0, 1, 6] = float("-inf")
    b = torch.zeros(c["k"].shape[0], 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"])
    assert torch.isnan(b[blk, 1, :, 10]).all() and int(torch.isnan(b).sum()) == 2
    assert (b[blk, 0, :, 5] == 0).all()
    assert b[blk, 0, 0, 6] == -math.inf and b[blk, 0, 1, 6] == math.inf


def test_bounds_refusals_on_the_device(torch):
    """Bad contexts, starts and table entries: the flag, and nothing written."""
    R = _ref()
    c = R.make_cache([40, 40, 40, 40, 40, 40], 2, 64, 16, seed=6)
    ctx = torch.tensor([0, -3, 40, 40, 1000, 40], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 0, 41, -1, 0, 38], dtype=torch.int32, device="cuda")
    b = torch.full((c["k"].shape[0], 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    want, err = b.double(), err_of(torch)
    pa.block_key_bounds(c["k"], b, c["bt"], ctx, start, max_new_tokens=40, err_flag=err)
    c["lens"] = [0, 0, 0, 0, 0, 40]
    for blk, x in R.ref_bounds(c, [0, 0, 0, 0, 0, 38]).items():
        want[blk] = x
    assert torch.equal(b.double(), want) and int(err) == pa.DEVERR_CTX
    # more new tokens than the bound
    b2, err = torch.full_like(b, 7.0), err_of(torch)
    pa.block_key_bounds(c["k"], b2, c["bt"], c["ctx"], max_new_tokens=39, err_flag=err)
    assert int(err) == pa.DEVERR_CTX and bool((b2 == 7).all())
    # a table entry outside the pool: that block is skipped
    bt, err = c["bt"].clone(), err_of(torch)
    bt[0, 1], bt[1, 0] = c["k"].shape[0], -1
    b3 = torch.full_like(b, 7.0)
    pa.block_key_bounds(c["k"], b3, bt, c["ctx"], err_flag=err)
    assert int(err) == pa.DEVERR_PAGE
    touched = {int(x) for s in range(6) for i, x in enumerate(c["bt"][s, :3].tolist()) if (s, i) not in ((0, 1), (1, 0))}
    assert {i for i in range(b3.shape[0]) if not bool((b3[i] == 7).all())} == touched


# ------------------------------------------------------------------- selection
def select_case(torch, shape, lens, seed):
    R = _ref()
    Hq, Hkv, D, B = shape
    c = R.make_cache(lens, Hkv, D, B, seed=seed)
    b = torch.zeros(c["k"].shape[0], Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"])
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(len(lens), Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    return c, b, q, Hq // Hkv


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("k,sink,recent", [(1, 0, 0), (1, 0, 1), (2, 1, 1), (5, 1, 2), (8, 0, 0), (16, 4, 4), (40, 1, 1)])
def test_select_ragged(torch, shape, k, sink, recent):
    R = _ref()
    c, b, q, G = select_case(torch, shape, LENS, seed=11)
    err = err_of(torch)
    got = pa.select_blocks(q, b, c["bt"], c["ctx"], k, block_size=c["B"], sink_blocks=sink, recent_blocks=recent,
                           err_flag=err)
    assert torch.equal(got, R.ref_select(q, b, c["bt"], c["lens"], c["B"], G, k, sink, recent)) and int(err) == 0


@pytest.mark.parametrize("n", [129, 1000, 8191, 8194, 8195, 9001, 20000])
@pytest.mark.parametrize("k", [2, 77, 500])
def test_select_long_contexts(torch, n, k):
    """More blocks than a CTA scores, and than its shared memory keeps."""
    R = _ref()
    g = torch.Generator(device="cuda").manual_seed(n)
    lens, Hkv, G, D, B = [n * 16 - 3, n * 16 // 2], 2, 3, 64, 16
    x = torch.randn(n + 5, Hkv, 2, D, generator=g, device="cuda")
    b = x.sort(dim=2).values.to(torch.bfloat16)
    bt = torch.stack([torch.randperm(n + 5, generator=g, device="cuda")[:n] for _ in lens]).to(torch.int32)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(2, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    got = pa.select_blocks(q, b, bt, ctx, k, block_size=B, sink_blocks=1, recent_blocks=1)
    assert torch.equal(got, R.ref_select(q, b, bt, lens, B, G, k, 1, 1))


@pytest.mark.parametrize("n,distinct", [(40, 1), (300, 3), (700, 2), (700, 100), (9000, 5)])
def test_select_ties_go_to_the_lowest_index(torch, n, distinct):
    """Blocks with the same bounds tie exactly, in any number."""
    R = _ref()
    g = torch.Generator(device="cuda").manual_seed(n)
    b = torch.randn(distinct, 2, 2, 128, generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    b = b[torch.randint(distinct, (n,), generator=g, device="cuda")].contiguous()
    bt = torch.arange(n, device="cuda", dtype=torch.int32)[None].contiguous()
    ctx = torch.tensor([n * 32], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    for k, sink, recent in ((4, 1, 1), (n // 2, 0, 1), (n - 1, 2, 0)):
        got = pa.select_blocks(q, b, bt, ctx, k, block_size=32, sink_blocks=sink, recent_blocks=recent)
        assert torch.equal(got, R.ref_select(q, b, bt, [n * 32], 32, 4, k, sink, recent))
    zero = pa.select_blocks(torch.zeros_like(q), b, bt, ctx, 5, block_size=32, sink_blocks=1, recent_blocks=1)
    assert zero.tolist() == [[[0, 1, 2, 3, n - 1]] * 2]


def test_select_near_ties(torch):
    """Scores that differ by less than an fp32 sum can tell: the exact sums
    decide.  Channel 0 carries a large common part, the last ones differences
    of its last bits."""
    R = _ref()
    n, D = 600, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    b = torch.zeros(n, 1, 2, D, device="cuda")
    b[:, :, :, :8] = 1e4
    b[:, 0, 1, 8:] = torch.randint(0, 3, (n, D - 8), generator=g, device="cuda") * 2.0**-10
    b = b.to(torch.bfloat16)
    q = torch.ones(1, 1, D, device="cuda", dtype=torch.bfloat16)
    bt = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    ctx = torch.tensor([n * 16], dtype=torch.int32, device="cuda")
    for k in (2, 10, 300):
        got = pa.select_blocks(q, b, bt, ctx, k, block_size=16, sink_blocks=0, recent_blocks=0)
        assert torch.equal(got, R.ref_select(q, b, bt, [n * 16], 16, 1, k, 0, 0))


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e20])
def test_select_at_the_ends_of_the_range(torch, size):
    R = _ref()
    c, b, q, G = select_case(torch, (8, 2, 128, 16), [2000, 333], seed=15)
    b = (b.float() * size).to(torch.bfloat16)
    for scale in (1.0, 1e-6):
        x = (q.float() * scale).to(torch.bfloat16)
        got = pa.select_blocks(x, b, c["bt"], c["ctx"], 9, block_size=16, sink_blocks=1, recent_blocks=1)
        assert torch.equal(got, R.ref_select(x, b, c["bt"], c["lens"], 16, G, 9, 1, 1))


@pytest.mark.parametrize("what", ["inf_bound", "nan_bound", "inf_query", "nan_query", "overflow", "minus"])
def test_select_with_values_that_are_not_finite(torch, what):
    R = _ref()
    c, b, q, G = select_case(torch, (4, 2, 64, 16), [640, 333, 48], seed=13)
    blk = c["bt"][:, 7].long()
    if what == "inf_bound":
        b[blk[0], 0, 1, 3], b[blk[1], 1, 0, 5] = math.inf, -math.inf
    elif what == "nan_bound":
        b[blk[0], 0, :, 3] = math.nan
        q[0, 0, 3] = 0.0  # head 1 of the group still sees it
    elif what == "inf_query":
        q[0, 1, 2], q[1, 3, 4] = math.inf, -math.inf
    elif what == "nan_query":
        q[0, 1, 2] = math.nan
    elif what == "overflow":
        b *= 1e30
        q *= 1e20
    else:
        b[blk[0], 0, 0, 3] = -math.inf
        b[blk[0], 0, 1, 3] = torch.finfo(torch.bfloat16).min
    got = pa.select_blocks(q, b, c["bt"], c["ctx"], 6, block_size=16, sink_blocks=1, recent_blocks=1)
    assert torch.equal(got, R.ref_select(q, b, c["bt"], c["lens"], 16, G, 6, 1, 1))


def test_select_refusals_on_the_device(torch):
    R = _ref()
    c, b, q, G = select_case(torch, (8, 2, 64, 16), [640, 640, 640, 640], seed=14)
    ctx = torch.tensor([0, 640, 700, -1], dtype=torch.int32, device="cuda")
    err = err_of(torch)
    got = pa.select_blocks(q, b, c["bt"], ctx, 6, block_size=16, max_context_len=640, err_flag=err)
    want = R.ref_select(q, b, c["bt"], c["lens"], 16, G, 6, 1, 1)
    assert int(err) == pa.DEVERR_CTX and torch.equal(got[1], want[1]) and bool((got[[0, 2, 3]] == -1).all())
    # entries outside the pool rank below all
    bt, err = c["bt"].clone(), err_of(torch)
    top = int(want[0, 0, 3])
    bt[0, top] = c["k"].shape[0] + 3
    got = pa.select_blocks(q, b, bt, c["ctx"], 6, block_size=16, err_flag=err)
    assert int(err) == pa.DEVERR_PAGE and top not in got[0, 0].tolist() and torch.equal(got[1:], want[1:])
    for entry in (-1, -2, -3, -2**31, 2**31 - 1):
        bt[0, top] = entry
        err.zero_()
        assert torch.equal(pa.select_blocks(q, b, bt, c["ctx"], 6, block_size=16, err_flag=err), got)
        assert int(err) == pa.DEVERR_PAGE, entry
    # fewer readable blocks than asked for: all of them, then the first unreadable ones
    bt = c["bt"].clone()
    bt[0, 3:37] = -5
    got = pa.select_blocks(q, b, bt, c["ctx"], 10, block_size=16)
    assert got[0].tolist() == [[0, 1, 2, 3, 4, 5, 6, 37, 38, 39]] * 2


# -------------------------------------------------------- attention over a list
def check_sparse(torch, c, q, sel, out, scale, once=False):
    R = _ref()
    G = q.shape[1] // c["Hkv"]
    B = c["B"]
    for s, n in enumerate(c["lens"]):
        for h in range(c["Hkv"]):
            toks = [j for i in sel[s, h].tolist() if 0 <= i < -(-n // B) for j in range(i * B, min(n, i * B + B))]
            at = torch.tensor(toks, dtype=torch.long, device="cuda")
            k, v = R.rows(c["k"], c["bt"][s], n, B, h)[at], R.rows(c["v"], c["bt"][s], n, B, h)[at]
            _, want, tol, _ = R.ref_attend(q[s, h * G:(h + 1) * G], k, v, scale, once)
            got = out[s, h * G:(h + 1) * G].double()
            assert bool(((got - want).abs() <= tol).all()), (s, h, float((got - want).abs().max()))


def random_lists(torch, c, S, k, seed, shuffled):
    g = torch.Generator().manual_seed(seed)
    sel = torch.full((S, c["Hkv"], k), -1, dtype=torch.int32)
    for s in range(S):
        n = -(-c["lens"][s] // c["B"])
        for h in range(c["Hkv"]):
            at = torch.randperm(n, generator=g)[:k].to(torch.int32)
            sel[s, h, :len(at)] = at if shuffled else at.sort().values
            if shuffled:  # -1 anywhere
                sel[s, h] = sel[s, h][torch.randperm(k, generator=g)]
    return sel.cuda()


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("k", [1, 3, 40])
@pytest.mark.parametrize("pp", [None, 1, 3])
def test_sparse_ragged(torch, monkeypatch, shape, k, pp):
    R = _ref()
    monkeypatch.delenv("PA_PARTITION_PAGES", raising=False)
    if pp:
        monkeypatch.setenv("PA_PARTITION_PAGES", str(pp))
    Hq, Hkv, D, B = shape
    c = R.make_cache(LENS, Hkv, D, B, seed=21, junk=float("nan"))
    q = torch.randn(len(LENS), Hq, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(torch.bfloat16)
    sel = random_lists(torch, c, len(LENS), k, 5, shuffled=pp == 3)
    err = err_of(torch)
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel, err_flag=err)
    check_sparse(torch, c, q, sel, out, 1 / math.sqrt(D))
    assert int(err) == 0


def test_sparse_over_every_block_is_attention_over_the_context(torch):
    """A list of the whole context: both it and decode are within tolerance of
    the definition."""
    R = _ref()
    c = R.make_cache([500, 77, 1], 2, 128, 16, seed=22)
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    sel = torch.full((3, 2, 32), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(c["lens"]):
        sel[s, :, :-(-n // 16)] = torch.arange(-(-n // 16), device="cuda", dtype=torch.int32)
    check_sparse(torch, c, q, sel, pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel),
                 128**-0.5)
    out = pa.paged_attention_decode(q, c["k"], c["v"], c["bt"], c["ctx"], max_context_len=500)
    check_sparse(torch, c, q, sel, out, 128**-0.5, once=True)


def test_sparse_empty_lists_and_refusals(torch):
    R = _ref()
    c = R.make_cache([100, 100, 100, 100, 100], 2, 64, 16, seed=23, junk=float("nan"))
    q = torch.randn(5, 4, 64, device="cuda").to(torch.bfloat16)
    sel = torch.full((5, 2, 4), -1, dtype=torch.int32, device="cuda")
    err = err_of(torch)
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel,
                                           torch.full_like(q, float("nan")), err_flag=err)
    assert bool((out == 0).all()) and int(err) == 0  # empty lists: zeros, no error
    sel[:, :, 0] = 2
    sel[1, 0, 1], sel[2, 1, 1], sel[2, 1, 2] = 7, -2, 2**31 - 1  # the context has blocks 0 .. 6
    ctx = c["ctx"].clone()
    ctx[3], ctx[4] = 0, 10**6
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], ctx, sel, err_flag=err)
    assert int(err) == (pa.DEVERR_PAGE | pa.DEVERR_CTX) and bool((out[3:] == 0).all())
    c["lens"] = c["lens"][:3]
    check_sparse(torch, c, q[:3], sel[:3], out[:3], 1 / 8)
    # a table entry outside the pool is left out
    bt, err = c["bt"].clone(), err_of(torch)
    bt[0, 2] = -9
    sel[0, :, 1] = 3
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], bt, c["ctx"], sel, err_flag=err)
    assert int(err) == pa.DEVERR_PAGE
    one = torch.full_like(sel, -1)
    one[0, :, 1] = 3
    c["lens"] = [100]
    check_sparse(torch, c, q[:1], one[:1], out[:1], 1 / 8)


def test_sparse_a_block_listed_twice_counts_twice(torch):
    R = _ref()
    c = R.make_cache([64], 1, 64, 16, seed=24)
    q = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    sel = torch.tensor([[[1, 3, 1, 1]]], dtype=torch.int32, device="cuda")
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel)
    check_sparse(torch, c, q, sel, out, 1 / 8)


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
def test_sparse_scales(torch, scale):
    R = _ref()
    c = R.make_cache([300, 5], 2, 64, 16, seed=25)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    sel = random_lists(torch, c, 2, 6, 3, shuffled=False)
    out = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel, scale=scale)
    check_sparse(torch, c, q, sel, out, scale)


# ----------------------------------------------------- streams, graphs, offsets
def test_a_step_of_select_and_attend_in_graphs_and_on_streams(torch):
    """The three calls as a decode step: eager, on another stream, captured
    twice (two graphs, replayed in turn with new queries) -- the same bits."""
    R = _ref()
    c = R.make_cache([900, 40, 333, 2000], 2, 128, 16, seed=31)
    qs = [torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(3)]
    q = torch.empty_like(qs[0])
    b = torch.zeros(c["k"].shape[0], 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    err = err_of(torch)

    def step(x, stream=None):
        pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"], err_flag=err, stream=stream)
        sel = pa.select_blocks(x, b, c["bt"], c["ctx"], 9, block_size=16, err_flag=err, stream=stream)
        return sel, pa.paged_attention_decode_sparse(x, c["k"], c["v"], c["bt"], c["ctx"], sel, err_flag=err,
                                                     stream=stream)

    want = [step(x) for x in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(qs[0], side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0][0]) and same_bits(torch, got[1], want[0][1])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step(q)
        graphs.append((g, r))
    for i in (0, 1, 2, 1):
        for g, r in graphs:
            q.copy_(qs[i])
            g.replay()
            step(qs[2 - i if i < 3 else 0])  # an eager call in between shares nothing with the graph
            torch.cuda.synchronize()
            assert torch.equal(r[0], want[i][0]) and same_bits(torch, r[1], want[i][1])
    # the queries made in the graph, by other kernels between the calls
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = [step(q * 1 + 0) for _ in range(3)]
    for i in (2, 0, 1):
        q.copy_(qs[i])
        g.replay()
        torch.cuda.synchronize()
        for x in r:
            assert torch.equal(x[0], want[i][0]) and same_bits(torch, x[1], want[i][1])
    assert int(err) == 0


def test_long_rows_in_a_graph(torch):
    """Rows that go through the workspace and its arrival counters: replays,
    and eager calls on the same workspace between them."""
    R = _ref()
    n, Hkv, G, D, B = 9000, 2, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    b = torch.randn(n, Hkv, 2, D, generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    bt = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].expand(3, -1).contiguous()
    lens = [n * B, 300, 5000 * B]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [torch.randn(3, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [R.ref_select(x, b, bt, lens, B, G, 50, 1, 1) for x in qs]
    desc = pa.DecodeDesc(3, Hkv * G, Hkv, D, B, n, n, n * B, 1.0)
    import ctypes
    ws = torch.full((int(pa.load().pa_select_blocks_workspace_bytes(ctypes.byref(desc))),), 255, dtype=torch.uint8,
                    device="cuda")
    q, sel = qs[0].clone(), torch.empty(3, Hkv, 50, dtype=torch.int32, device="cuda")
    call = lambda: pa.select_blocks(q, b, bt, ctx, 50, block_size=B, workspace=ws, selected=sel)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for i in (0, 1, 1, 0):
        q.copy_(qs[i])
        graph.replay()
        assert torch.equal(sel, want[i])
        sel.zero_()
        call()
        assert torch.equal(sel, want[i])


def test_calls_on_two_streams_at_once(torch):
    """Default workspaces belong to their stream: two steps in flight at the
    same time do not meet."""
    R = _ref()
    c = R.make_cache([4000, 1500], 4, 128, 16, seed=33)
    b = torch.zeros(c["k"].shape[0], 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"])
    qs = [torch.randn(2, 16, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    w = [torch.zeros(2, 4, c["mb"] * 16, device="cuda") for _ in range(2)]

    def step(x, w):
        sel = pa.select_blocks(x, b, c["bt"], c["ctx"], 130, block_size=16)
        out, _ = pa.paged_attention_decode_weights(x, c["k"], c["v"], c["bt"], c["ctx"], w)
        return sel, pa.paged_attention_decode_sparse(x, c["k"], c["v"], c["bt"], c["ctx"], sel), out

    want = [step(x, y) for x, y in zip(qs, w)]
    once = [y.clone() for y in w]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for r in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                w[i].zero_()
                got[i].append(step(qs[i], w[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(w[i], once[i])
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quick", [True, False])
def test_the_first_call_of_a_thread(torch, monkeypatch, D, quick):
    """A new host thread has no context of its own yet."""
    import threading

    if not quick:
        monkeypatch.setattr(pa._binding, "_FAST", False)
    c = _ref().make_cache([300, 40], 2, D, 16, seed=35)
    q = torch.randn(2, 8, D, device="cuda").to(torch.bfloat16)
    b = torch.zeros(c["k"].shape[0], 2, 2, D, dtype=torch.bfloat16, device="cuda")
    pa.block_key_bounds(c["k"], b, c["bt"], c["ctx"])
    fresh = torch.zeros_like(b)
    w = [torch.zeros(2, 2, c["mb"] * 16, device="cuda") for _ in range(2)]
    sel = pa.select_blocks(q, b, c["bt"], c["ctx"], 6, block_size=16)
    calls = [
        lambda i: pa.block_key_bounds(c["k"], fresh if i else b, c["bt"], c["ctx"]),
        lambda i: pa.select_blocks(q, b, c["bt"], c["ctx"], 6, block_size=16),
        lambda i: pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel),
        lambda i: pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w[i])[0],
        lambda i: pa.paged_attention_decode(q, c["k"], c["v"], c["bt"], c["ctx"]),
    ]
    for f in calls:
        want, got = f(0), []

        def run():
            try:
                got.append(f(1))
            except Exception as e:  # noqa: BLE001
                got.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        assert isinstance(got[0], torch.Tensor) and torch.equal(got[0], want), got
    assert torch.equal(w[0], w[1])


def test_calls_from_two_threads_on_one_stream(torch):
    """The two launches of a call with weights share a default workspace with
    every other such call on the stream: no other thread's come between them."""
    import threading

    R = _ref()
    c = R.make_cache([5000, 900, 40], 2, 64, 16, seed=34)
    rows = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")  # a shared row: by two launches
    qs = [torch.randn(3, 8, 64, device="cuda").to(torch.bfloat16) for _ in range(2)]

    def step(x, w, out):
        return pa.paged_attention_decode_weights(x, c["k"], c["v"], c["bt"], c["ctx"], w, out, weight_rows=rows)

    def zeros():
        return torch.zeros(2, 2, c["mb"] * 16, device="cuda")

    want = [zeros() for _ in qs]
    outs = [step(x, w, None)[0] for x, w in zip(qs, want)]
    torch.cuda.synchronize()
    ws = [[zeros() for _ in range(200)] for _ in qs]
    got = [[torch.empty_like(x) for _ in range(200)] for x in qs]
    start = threading.Barrier(2)
    failed = []

    def run(i):
        try:
            start.wait(60)
            for n, (w, out) in enumerate(zip(ws[i], got[i])):
                if n % 2:
                    step(qs[i], w, out)  # the way through ctypes
                else:
                    out.copy_(step(qs[i], w, None)[0])
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert all(torch.equal(w, want[i]) for w in ws[i])
        assert all(torch.equal(o, outs[i]) for o in got[i])


def test_offsets_beyond_32_bits(torch):
    """Blocks at the end of a pool of more than 2^31 elements."""
    R = _ref()
    lens, Hkv, D, B = [100, 33], 8, 128, 16
    c = R.make_cache(lens, Hkv, D, B, seed=41)
    n = c["k"].shape[0]
    nblk = (2**31 + 2**28) // (Hkv * D * B)
    kp = torch.empty(nblk, Hkv, B, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty(nblk, Hkv, B, D, dtype=torch.bfloat16, device="cuda")
    kp[-n:], vp[-n:] = c["k"], c["v"]
    bt = c["bt"] + (nblk - n)
    q = torch.randn(2, 16, D, device="cuda").to(torch.bfloat16)
    small = torch.zeros(n, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    big = torch.empty(nblk, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    big[-n:] = 0
    res = []
    for k, v, b, t in ((c["k"], c["v"], small, c["bt"]), (kp, vp, big, bt)):
        pa.block_key_bounds(k, b, t, c["ctx"], max_context_len=100)
        sel = pa.select_blocks(q, b, t, c["ctx"], 3, block_size=B, max_context_len=100)
        res.append((b[-n:], sel, pa.paged_attention_decode_sparse(q, k, v, t, c["ctx"], sel, max_context_len=100)))
    w, keep = [torch.zeros(2, Hkv, 112, device="cuda") for _ in range(2)], torch.full((2,), 20, dtype=torch.int32,
                                                                                      device="cuda")
    for (k, v, t), x in zip(((c["k"], c["v"], c["bt"]), (kp, vp, bt)), w):
        pa.paged_attention_decode_weights(q, k, v, t, c["ctx"], x, max_context_len=100)
        pa.evict_tokens(k, v, t, c["ctx"], keep, x, max_keep_len=20, max_context_len=100)
    assert torch.equal(w[0], w[1]) and same_bits(torch, c["k"], kp[-n:]) and same_bits(torch, c["v"], vp[-n:])
    assert same_bits(torch, res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert same_bits(torch, res[0][2], res[1][2])


# ------------------------------------------------- the two ways into the calls
def test_both_ways_into_the_calls_agree(torch, monkeypatch):
    """Every call by the extension module and by the Python beside it: the
    same bits, the same refusals; the extension module was built here and
    takes the common form."""
    from paged_kv_cache_262_gb300 import _binding as b
    R = _ref()
    F = b._FAST if b._FAST is not None else b._fast()
    assert F, "the extension module is not built"
    c = R.make_cache([700, 33, 1], 2, 128, 16, seed=71)
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    keep = torch.tensor([300, 20, 5], dtype=torch.int32, device="cuda")
    w0 = torch.rand(3, 2, c["mb"] * 16, device="cuda")
    rows = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    k0, v0 = c["k"].clone(), c["v"].clone()

    def all_calls():
        c["k"].copy_(k0), c["v"].copy_(v0)
        w, err = w0.clone(), err_of(torch)
        bd = torch.zeros(k0.shape[0], 2, 2, 128, dtype=torch.bfloat16, device="cuda")
        pa.block_key_bounds(c["k"], bd, c["bt"], c["ctx"], c["ctx"] - 1, max_new_tokens=1, err_flag=err)
        pa.block_key_bounds(c["k"], bd, c["bt"], c["ctx"])
        sel = pa.select_blocks(q, bd, c["bt"], c["ctx"], 5, block_size=16, sink_blocks=2, recent_blocks=1,
                               max_context_len=700, err_flag=err)
        o1 = pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"], sel, scale=0.125)
        o2, w2 = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w, weight_rows=rows,
                                                   max_context_len=700, err_flag=err)
        assert w2 is w
        o3, w3 = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w,
                                                   weights_out=torch.zeros_like(w))
        kept, new = pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], keep, w, max_keep_len=300, sink_tokens=1,
                                    recent_tokens=2, weight_rows=rows, err_flag=err)
        assert int(err) == 0
        return [bd, sel, o1, o2, o3, w3, kept, new, w, c["k"].clone(), c["v"].clone()]

    def refusals():
        got = []
        for f in (lambda: pa.block_key_bounds(c["k"], w0, c["bt"], c["ctx"]),
                  lambda: pa.block_key_bounds(c["k"], torch.zeros_like(c["k"]), c["bt"], c["ctx"]),
                  lambda: pa.select_blocks(q, torch.zeros(9, 2, 2, 64, dtype=torch.bfloat16, device="cuda"), c["bt"],
                                           c["ctx"], 5, block_size=16),
                  lambda: pa.select_blocks(q, torch.zeros(9, 2, 2, 128, dtype=torch.bfloat16, device="cuda"), c["bt"],
                                           c["ctx"], 5, block_size=8),
                  lambda: pa.select_blocks(q, torch.zeros(9, 2, 2, 128, dtype=torch.bfloat16, device="cuda"), c["bt"],
                                           c["ctx"], 2, block_size=16, sink_blocks=2),
                  lambda: pa.paged_attention_decode_sparse(q, c["k"], c["v"][:-1], c["bt"], c["ctx"], rows),
                  lambda: pa.paged_attention_decode_sparse(q, c["k"], c["v"], c["bt"], c["ctx"].cpu(),
                                                           torch.zeros(3, 2, 4, dtype=torch.int32, device="cuda")),
                  lambda: pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w0[:2]),
                  lambda: pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w0[:, :, ::2]),
                  lambda: pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], keep, w0, max_keep_len=0),
                  lambda: pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], keep, w0, max_keep_len=8,
                                          sink_tokens=-1)):
            with pytest.raises((TypeError, ValueError, pa.PaError)) as e:
                f()
            got.append((type(e.value), str(e.value)))
        return got

    quick, said = all_calls(), refusals()
    assert F.sparse(q, c["k"], c["v"], c["bt"], c["ctx"], quick[1], None, None, None, b._WS_SPARSE) is not None
    monkeypatch.setattr(b, "_FAST", False)
    assert all(torch.equal(x, y) for x, y in zip(quick, all_calls()))
    assert said == refusals()
