"""Decode attention of trees of drafted tokens on the GPU, against plain 64-bit
operations."""
import math
import random

import pytest

import gpu_util
import long_context_ref as lc
import tree_ref as tr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return gpu_util.need_gpu()


@pytest.fixture(scope="module")
def pa(torch):
    import paged_kv_cache_262_gb300 as pa
    return pa


def call(pa, torch, c, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw.setdefault("max_tree_nodes", c["most"])
    kw.setdefault("scale", c["scale"])
    out = torch.full_like(c["q"], 7.0)
    got = pa.paged_attention_decode_tree(c["q"], c["k"], c["v"], c["bt"], c["ctx"], c["cu"], c["parents"], out,
                                         err_flag=err, **kw)
    assert got is out
    torch.cuda.synchronize()
    return out, int(err.item())


def whole(pa, torch, c, **kw):
    out, err = call(pa, torch, c, **kw)
    assert err == 0
    tr.check(out, tr.ref_tree(c))
    assert bool((out[c["cu_host"][-1]:] == 7.0).all())  # rows behind the last tree


SHAPES = [
    # contexts, nodes, Hq, Hkv, D, B, kind
    ([0], [1], 1, 1, 64, 16, "chain"),
    ([1], [1], 8, 8, 128, 32, "chain"),
    ([0, 0, 0], [2, 1, 3], 4, 4, 128, 16, "roots"),
    ([5, 16, 17, 31, 32, 33], [1, 2, 3, 4, 5, 6], 8, 2, 128, 16, "any"),
    ([127, 128, 129, 126], [1, 1, 1, 4], 12, 4, 64, 32, "star"),
    ([100, 0, 1000], [0, 0, 0], 8, 2, 128, 16, "any"),
    ([100, 3, 250], [0, 7, 0], 8, 2, 128, 16, "any"),
    ([300, 200, 1], [26, 13, 26], 21, 3, 128, 16, "any"),
    ([300, 200, 1], [26, 13, 26], 20, 4, 64, 16, "any"),
    ([511], [64], 8, 1, 128, 32, "any"),
    ([77, 700], [64, 33], 16, 2, 128, 16, "chain"),
    ([250, 3], [128, 100], 2, 2, 128, 16, "any"),
    ([250, 3], [256, 199], 1, 1, 64, 32, "chain"),
    ([100], [256], 16, 1, 128, 16, "any"),
    ([640], [20], 26, 2, 128, 32, "any"),
    ([3000, 10, 900], [8, 8, 8], 24, 8, 64, 32, "any"),
    ([129] * 40, [3] * 40, 8, 2, 128, 16, "chain"),
]


@pytest.mark.parametrize("ctx,nodes,hq,hkv,d,b,kind", SHAPES)
def test_small(pa, torch, ctx, nodes, hq, hkv, d, b, kind):
    whole(pa, torch, tr.make_case(ctx, nodes, hq, hkv, d, b, kind, seed=len(ctx) + hq))


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("b", [16, 32])
def test_unwritten_slots_do_not_reach_the_output(pa, torch, junk, b):
    whole(pa, torch, tr.make_case([100, 13, 127, 0, 250], [5, 3, 1, 2, 20], 8, 2, 128, b, seed=3, junk=junk))
    whole(pa, torch, tr.make_case([100, 13, 127], [70, 3, 2], 8, 2, 128, b, seed=3, junk=junk))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [12, 60, 140])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
def test_values_that_are_not_finite_reach_only_the_nodes_that_attend_them(pa, torch, d, nodes, bad, which):
    c = tr.make_case([90, 130], [nodes, 5], 8, 2, d, 16, "any", seed=nodes)
    pos = 90 + 3  # node 3 of the first tree, one channel
    block, off = int(c["bt"][0, pos // 16]), pos % 16
    c[which][block, :, off, 5] = bad
    c[which][block, 1, off, 6] = -bad
    whole(pa, torch, c)


def test_logits_of_minus_infinity(pa, torch):
    c = tr.make_case([0, 40], [3, 4], 8, 2, 128, 16, "roots", seed=5)
    c["q"][:, :, 0] = 1.0
    for s, p in ((0, 0), (0, 1), (0, 2), (1, 7), (1, 41)):
        c["k"][int(c["bt"][s, p // 16]), :, p % 16, 0] = -math.inf
    out, err = call(pa, torch, c)
    assert err == 0 and bool((out[:3] == 0).all())
    tr.check(out, tr.ref_tree(c))


def test_large_logits(pa, torch):
    c = tr.make_case([600, 33], [40, 9], 8, 2, 128, 16, seed=6)
    c["k"] *= 30
    c["q"] *= 3
    whole(pa, torch, c)


def test_growing_logits_rescale(pa, torch):
    """Keys whose logits grow along the context: every key tile has a new maximum."""
    for nodes in (9, 60):
        c = tr.make_case([900], [nodes], 8, 2, 128, 16, "chain", seed=8)
        n = 900 + nodes
        at = torch.arange(n, device="cuda")
        blocks, off = c["bt"][0, at // 16].long(), at % 16
        c["k"][blocks, :, off] = (torch.randn(n, 2, 128, device="cuda") + 0.02 * at[:, None, None]).to(torch.bfloat16)
        c["q"] = c["q"].abs()
        whole(pa, torch, c)


@pytest.mark.parametrize("ctx,nodes,hq,hkv,d,b", [
    ([40000], [4], 8, 1, 128, 16),
    ([20011], [33], 16, 2, 128, 32),
    ([9000, 17000, 100], [64, 50, 64], 16, 2, 128, 16),
    ([33000, 5], [61, 61], 14, 2, 64, 16),
])
def test_long_contexts(pa, torch, ctx, nodes, hq, hkv, d, b):
    c = tr.make_case(ctx, nodes, hq, hkv, d, b, seed=1)
    out, err = call(pa, torch, c, max_context_len=max(x + y for x, y in zip(ctx, nodes)))
    assert err == 0
    tr.check(out, tr.ref_tree(c, nodes=[0, 1, 2, 31, 32, 49, 60, 63]))


def test_ragged_batch(pa, torch):
    rng = random.Random(4)
    nodes = [rng.choice((0, 1, 2, 5, 17, 31)) for _ in range(70)]
    ctx = [rng.choice((0, 1, 15, 100, 400, 1500)) for _ in range(70)]
    whole(pa, torch, tr.make_case(ctx, nodes, 8, 2, 64, 16, seed=9))


def test_a_chain_is_decode_token_by_token(pa, torch):
    """A chain's node i is the decode step with the nodes up to i in the context."""
    c = tr.make_case([200, 31], [5, 5], 8, 2, 128, 16, "chain", seed=11)
    out, err = call(pa, torch, c)
    assert err == 0
    ref = tr.ref_tree(c)
    for i in range(5):
        rows = [c["cu_host"][s] + i for s in range(2)]
        one = pa.paged_attention_decode(c["q"][rows].contiguous(), c["k"], c["v"], c["bt"],
                                        c["ctx"] + i + 1, scale=c["scale"])
        for s, r in enumerate(rows):
            # both are within their tolerance of the same sum (decode rounds the probabilities once: 2^-8)
            o, tol = ref[r]
            assert bool(((one[s].double() - out[r].double()).abs() <= 2 * tol + 2.0**-7 * (1 + o.abs())).all())


def test_bad_sequences_are_zeros_and_the_others_stay(pa, torch):
    ctx, nodes = [50, 60, 70, 80, 90], [4, 5, 6, 7, 8]
    c = tr.make_case(ctx, nodes, 8, 2, 128, 16, seed=12)
    ref = tr.ref_tree(c)
    cap = c["bt"].shape[1] * 16
    for s, value in ((1, -1), (2, cap - 5), (3, 2**31 - 1), (0, -2**31)):
        d = dict(c, ctx=c["ctx"].clone())
        d["ctx"][s] = value
        out, err = call(pa, torch, d)
        assert err == pa.DEVERR_CTX
        n0, n1 = c["cu_host"][s], c["cu_host"][s + 1]
        assert bool((out[n0:n1] == 0).all())
        tr.check(out, {r: x for r, x in ref.items() if not n0 <= r < n1})
    out, err = call(pa, torch, c, max_context_len=90)  # 80 + 7 fits, 90 + 8 does not
    assert err == pa.DEVERR_CTX and bool((out[c["cu_host"][4]:c["cu_host"][5]] == 0).all())
    tr.check(out, {r: x for r, x in ref.items() if r < c["cu_host"][4]})


def test_bad_node_ranges(pa, torch):
    c = tr.make_case([50, 60, 70], [4, 5, 6], 8, 2, 128, 16, seed=13)
    ref = tr.ref_tree(c)
    out, err = call(pa, torch, c, max_tree_nodes=5)  # the last tree has six
    assert err == pa.DEVERR_TREE and bool((out[9:15] == 0).all())
    tr.check(out, {r: x for r, x in ref.items() if r < 9})
    for cu in ([0, 4, 9, 19], [0, 4, 9, 8], [0, 4, 9, -1]):
        d = dict(c, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        out, err = call(pa, torch, d)
        assert err == pa.DEVERR_TREE and bool((out[9:] == 7.0).all())
        tr.check(out, {r: x for r, x in ref.items() if r < 9})


def test_bad_parents(pa, torch):
    for t in (9, 70):
        c = tr.make_case([50, 60], [t, 4], 8, 2, 128, 16, "chain", seed=14)
        for node, parent in ((3, 3), (3, 5), (3, -2), (3, 2**31 - 1), (0, 0), (3, -2**31)):
            d = dict(c, parents=c["parents"].clone(), trees=[list(x) for x in c["trees"]])
            d["parents"][node] = parent
            d["trees"][0][node] = parent
            out, err = call(pa, torch, d)
            assert err == pa.DEVERR_TREE
            assert bool((out[node:t] == 0).all())  # it and what hangs on it
            tr.check(out, tr.ref_tree(d))


@pytest.mark.parametrize("nodes", [4, 60])
def test_pages_outside_the_pool_are_left_out(pa, torch, nodes):
    c = tr.make_case([200, 40], [nodes, 3], 8, 2, 128, 16, seed=15, junk=math.nan)
    ref = tr.ref_tree(c, drop=((0, 2), (0, 7), (0, 13)))
    c["bt"][0, 2], c["bt"][0, 7], c["bt"][0, 13] = -1, c["k"].shape[0], 2**31 - 1
    out, err = call(pa, torch, c)
    assert err == pa.DEVERR_PAGE
    tr.check(out, ref)


def test_every_page_outside_the_pool(pa, torch):
    c = tr.make_case([100], [3], 8, 2, 128, 16, seed=16)
    c["bt"].fill_(-1)
    out, err = call(pa, torch, c)
    assert err == pa.DEVERR_PAGE and bool((out[:3] == 0).all())


def test_pool_past_32_bit_offsets(pa, torch):
    """Blocks whose values lie past 2^32 bytes and 2^31 elements."""
    hkv, d, b = 8, 128, 32
    nblk = (1 << 31) // (hkv * d * b) + 40
    c = tr.make_case([70], [5], 16, hkv, d, b, seed=17)
    k = torch.empty(nblk, hkv, b, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    bt = c["bt"].clone()
    for i in range(3):
        to = nblk - 1 - 7 * i
        k[to], v[to] = c["k"][int(bt[0, i])], c["v"][int(bt[0, i])]
        bt[0, i] = to
    whole(pa, torch, dict(c, k=k, v=v, bt=bt))


def test_graph_replays_with_new_contexts(pa, torch):
    c = tr.make_case([500, 90], [20, 20], 8, 2, 128, 16, seed=18)
    other = tr.make_case([300, 290], [20, 20], 8, 2, 128, 16, seed=19)
    for x in (c, other):  # room for either case's table
        wide = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
        wide[:, :x["bt"].shape[1]] = x["bt"]
        x["bt"] = wide
    n = max(c["k"].shape[0], other["k"].shape[0])
    bufs = {}
    for name in ("q", "bt", "ctx", "cu", "parents"):
        bufs[name] = c[name].clone()
    for name in ("k", "v"):
        bufs[name] = torch.zeros(n, *c[name].shape[1:], dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    graphs, outs = [], []

    def make():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(pa.paged_attention_decode_tree(
                bufs["q"], bufs["k"], bufs["v"], bufs["bt"], bufs["ctx"], bufs["cu"], bufs["parents"],
                max_tree_nodes=20, scale=c["scale"], max_context_len=1000))
        graphs.append(g)

    with torch.cuda.stream(s):
        pa.paged_attention_decode_tree(bufs["q"], bufs["k"], bufs["v"], bufs["bt"], bufs["ctx"], bufs["cu"],
                                       bufs["parents"], max_tree_nodes=20, scale=c["scale"], max_context_len=1000)
    make()
    make()  # two graphs, their workspaces apart
    for x in (c, other, c):
        for name in ("q", "bt", "ctx", "cu", "parents"):
            bufs[name].copy_(x[name])
        for name in ("k", "v"):
            bufs[name][:x[name].shape[0]].copy_(x[name])
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        ref = tr.ref_tree(x)
        for o in outs:
            tr.check(o, ref)
        assert torch.equal(outs[0][:40], outs[1][:40])


def test_two_streams_and_repeats_are_alike(pa, torch):
    cases = [tr.make_case([3000, 64], [9, 40], 16, 2, 128, 16, seed=20 + i) for i in range(2)]
    alone = [call(pa, torch, c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [torch.full_like(c["q"], 7.0) for c in cases]
        torch.cuda.synchronize()
        for c, st, o in zip(cases, streams, outs):
            pa.paged_attention_decode_tree(c["q"], c["k"], c["v"], c["bt"], c["ctx"], c["cu"], c["parents"], o,
                                           max_tree_nodes=c["most"], scale=c["scale"], stream=st)
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o, a)


def test_given_workspace(pa, torch):
    import ctypes
    c = tr.make_case([3000, 64], [9, 40], 16, 2, 128, 16, seed=22)
    desc = pa.make_desc(c["q"], c["k"], c["bt"], num_seqs=2)
    need = pa.load().pa_decode_tree_workspace_bytes(ctypes.byref(desc), c["most"])
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    whole(pa, torch, c, workspace=ws)
    if need:
        with pytest.raises(pa.PaError) as e:
            call(pa, torch, c, workspace=ws[:need - 1])
        assert e.value.status == pa.PA_ERR_WORKSPACE


def test_refusals(pa, torch):
    c = tr.make_case([50, 60], [4, 5], 8, 2, 128, 16, seed=23)
    args = [c["q"], c["k"], c["v"], c["bt"], c["ctx"], c["cu"], c["parents"]]
    kw = dict(max_tree_nodes=5)

    def refused(i, x, exc=(TypeError, ValueError), **more):
        a = list(args)
        a[i] = x
        with pytest.raises(exc):
            pa.paged_attention_decode_tree(*a, **{**kw, **more})

    refused(0, c["q"].float())
    refused(0, c["q"].cpu())
    refused(0, c["q"][:, :, :64])
    refused(1, c["k"][:-1])
    refused(2, c["v"].float())
    refused(3, c["bt"][:1])
    refused(3, c["bt"].long())
    refused(5, c["cu"][:2])
    refused(5, c["cu"].long())
    refused(6, c["parents"][:3])
    refused(6, None)
    for most in (0, -1, 257):
        refused(0, c["q"], max_tree_nodes=most)
    with pytest.raises(ValueError):
        pa.paged_attention_decode_tree(*args, torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), **kw)
    # no sequences, no nodes: nothing to do
    none = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert pa.paged_attention_decode_tree(none, c["k"], c["v"], c["bt"], c["ctx"][:0], c["cu"][:1],
                                          c["parents"][:0], **kw).shape[0] == 0
