"""Decode with accumulated attention weights, and eviction by them, on the
GPU against plain 64-bit implementations; the two together with the block
manager and block-sparse decode."""
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


def random_q(torch, *shape, seed=2):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(torch.bfloat16)


def random_weights(torch, rows, Hkv, width, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(2 * torch.randn(rows, Hkv, width, generator=g, device="cuda") - 4)


def check_weights(torch, c, q, out, w0, w1, scale, rows=None, w_out_before=None):
    """out and the sums; a sum's tolerance is its probabilities' (ref_attend)
    and one rounding, 2^-24 of it, an addition."""
    R = _ref()
    G = q.shape[1] // c["Hkv"]
    want, tol = w0.double(), torch.zeros_like(w0, dtype=torch.float64)
    reached = torch.zeros(w0.shape[0], dtype=torch.long)
    for s, n in enumerate(c["lens"]):
        r = s if rows is None else rows[s]
        if n <= 0 or r < 0 or r >= w0.shape[0]:
            continue
        reached[r] = max(int(reached[r]), n)
        for h in range(c["Hkv"]):
            k, v = R.rows(c["k"], c["bt"][s], n, c["B"], h), R.rows(c["v"], c["bt"][s], n, c["B"], h)
            p, o, t, tp = R.ref_attend(q[s, h * G:(h + 1) * G], k, v, scale)
            got = out[s, h * G:(h + 1) * G].double()
            assert bool(((got - o).abs() <= t).all()), (s, h, float((got - o).abs().max()))
            want[r, h, :n] += p.sum(0)
            tol[r, h, :n] += tp.sum(0)
    before = (w0 if w_out_before is None else w_out_before).double()
    for r in range(w0.shape[0]):
        n = int(reached[r])
        assert torch.equal(w1[r, :, n:].double(), before[r, :, n:])  # past every context: as it was
        bad = (w1[r, :, :n].double() - want[r, :, :n]).abs() - (tol[r, :, :n] + 2.0**-22 * want[r, :, :n].abs())
        assert bool((bad <= 0).all()), (r, float(bad.max()))


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("pp", [None, 1, 3])
@pytest.mark.parametrize("in_place", [True, False])
def test_weights_ragged(torch, monkeypatch, shape, pp, in_place):
    R = _ref()
    monkeypatch.delenv("PA_PARTITION_PAGES", raising=False)
    if pp:
        monkeypatch.setenv("PA_PARTITION_PAGES", str(pp))
    Hq, Hkv, D, B = shape
    c = R.make_cache(LENS, Hkv, D, B, seed=51, junk=float("nan"))
    q = random_q(torch, len(LENS), Hq, D)
    w0 = random_weights(torch, len(LENS) + 1, Hkv, c["mb"] * B + 5)
    w, other, err = w0.clone(), torch.full_like(w0, -3.0), err_of(torch)
    out, w1 = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w,
                                                weights_out=None if in_place else other, err_flag=err)
    assert (w1 is w) == in_place and int(err) == 0
    check_weights(torch, c, q, out, w0, w1, 1 / math.sqrt(D),
                  w_out_before=None if in_place else torch.full_like(w0, -3.0))
    if not in_place:
        assert torch.equal(w, w0)


def test_weights_of_a_row_sum_to_its_heads(torch):
    R = _ref()
    c = R.make_cache([700, 33, 1, 2000], 2, 128, 16, seed=52)
    q = random_q(torch, 4, 8, 128)
    w = torch.zeros(4, 2, c["mb"] * 16, device="cuda")
    pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w)
    # every query head gives 1 in all: G a row, to the fp32 sum's 2^-24 a term
    # on values summing to G, and 2^-21 of each probability
    for s, n in enumerate(c["lens"]):
        total = w[s, :, :n].double().sum(1)
        assert bool(((total - 4).abs() <= 4 * 2.0**-20).all()), total
    assert bool((w[0, :, 700:] == 0).all())


@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (16, 1, 64, 32), (3, 1, 64, 16)], ids=ids)
@pytest.mark.parametrize("lens", [[1], [700], [1500, 3, 40], [9000], [30000, 100]])
def test_weights_by_one_launch_and_by_two(torch, shape, lens):
    """Few sequences of every length: units of one CTA, clusters, splits
    through the workspace, the weights added by the CTAs and (with rows) by
    the second kernel -- both within tolerance, and each its own bits again."""
    R = _ref()
    Hq, Hkv, D, B = shape
    c = R.make_cache(lens, Hkv, D, B, seed=57, junk=float("nan"))
    q = random_q(torch, len(lens), Hq, D)
    w0 = random_weights(torch, len(lens), Hkv, c["mb"] * B)
    rows = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    outs = []
    for r in (None, rows):
        again = []
        for _ in range(2):
            w, err = w0.clone(), err_of(torch)
            out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w, weight_rows=r,
                                                       max_context_len=max(lens), err_flag=err)
            assert int(err) == 0
            again.append(w)
        check_weights(torch, c, q, out, w0, w, 1 / math.sqrt(D))
        assert torch.equal(*again)
        outs.append(out)
    assert same_bits(torch, *outs)


def test_weights_summed_over_steps(torch):
    """Steps accumulate; a token added by a step starts from the zeros
    behind the context."""
    R = _ref()
    c = R.make_cache([48, 100], 2, 64, 16, seed=53)
    w = torch.zeros(2, 2, c["mb"] * 16, device="cuda")
    want = w.double()
    for step, lens in enumerate(([45, 97], [46, 98], [48, 100])):
        c["lens"] = lens
        ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = random_q(torch, 2, 8, 64, seed=step)
        pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], ctx, w, max_context_len=100)
        for s, n in enumerate(lens):
            for h in range(2):
                p = R.ref_attend(q[s, h * 4:h * 4 + 4], R.rows(c["k"], c["bt"][s], n, 16, h),
                                 R.rows(c["v"], c["bt"][s], n, 16, h), 1 / 8)[0]
                want[s, h, :n] += p.sum(0)
    assert bool(((w.double() - want).abs() <= want * 2.0**-12).all())  # (12 probabilities: ref_attend's 2e-4 each)


def test_weights_rows(torch):
    """Rows in any order, rows that no sequence names, one row named by many
    (a window of queries over one prompt, each with its own context), rows out
    of range."""
    R = _ref()
    base = R.make_cache([300, 50], 2, 64, 16, seed=54)
    W = 21
    lens = [300 - W + 1 + i for i in range(W)] + [50]
    c = dict(base, lens=lens, bt=base["bt"][[0] * W + [1]].contiguous(),
             ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = random_q(torch, W + 1, 4, 64)
    rows = [3] * W + [1]
    w0 = random_weights(torch, 5, 2, c["mb"] * 16)
    got = []
    for _ in range(3):
        w, err = w0.clone(), err_of(torch)
        out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w,
                                                   weight_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"),
                                                   err_flag=err)
        assert int(err) == 0
        got.append(w)
    check_weights(torch, c, q, out, w0, got[0], 1 / 8, rows=rows)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])  # one order, whatever the timing
    rows = [3] * W + [5]
    w, err = w0.clone(), err_of(torch)
    out2, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w,
                                                weight_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"),
                                                err_flag=err)
    assert int(err) == pa.DEVERR_ROW and same_bits(torch, out, out2)
    assert torch.equal(w[:3], w0[:3]) and torch.equal(w[3], got[0][3]) and torch.equal(w[4], w0[4])


def test_weights_many_sequences_one_row(torch):
    """More sequences than a CTA has threads name the row."""
    R = _ref()
    base = R.make_cache([40], 1, 64, 16, seed=55)
    S = 600
    lens = [1 + i % 40 for i in range(S)]
    c = dict(base, lens=lens, bt=base["bt"].expand(S, -1).contiguous(),
             ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = random_q(torch, S, 1, 64)
    rows = [0 if i % 3 else 1 for i in range(S)]
    w0 = torch.zeros(2, 1, c["mb"] * 16, device="cuda")
    w = w0.clone()
    out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w, max_context_len=40,
                                               weight_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    want = torch.zeros_like(w0, dtype=torch.float64)
    for s in range(S):
        p = R.ref_attend(q[s], R.rows(c["k"], c["bt"][s], lens[s], 16, 0), R.rows(c["v"], c["bt"][s], lens[s], 16, 0),
                         1 / 8)[0]
        want[rows[s], 0, :lens[s]] += p[0]
    # up to 400 additions of 2^-24 each on the running sum, probabilities within 2^-12
    assert bool(((w.double() - want).abs() <= want * (400 * 2.0**-24 + 2.0**-12)).all())


def test_weights_refusals_on_the_device(torch):
    R = _ref()
    c = R.make_cache([100, 100, 100, 100], 2, 64, 16, seed=56)
    q = random_q(torch, 4, 4, 64)
    ctx = torch.tensor([100, 0, 101, 100], dtype=torch.int32, device="cuda")
    bt = c["bt"].clone()
    bt[3, 2] = c["k"].shape[0]  # a block outside the pool: its keys weigh nothing
    w0, err = random_weights(torch, 4, 2, 128), err_of(torch)
    w = w0.clone()
    out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], bt, ctx, w, max_context_len=100, err_flag=err)
    assert int(err) == (pa.DEVERR_CTX | pa.DEVERR_PAGE)
    assert torch.equal(w[1:3], w0[1:3]) and bool((out[1:3] == 0).all())
    assert torch.equal(w[3, :, 32:48], w0[3, :, 32:48])
    added = (w[3].double() - w0[3].double())[:, :100].sum(1)
    assert bool(((added - 2).abs() < 1e-4).all())
    # a context with no readable block
    bt[3] = -1
    w = w0.clone()
    out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], bt, c["ctx"], w, max_context_len=100)
    assert torch.equal(w[3], w0[3]) and bool((out[3] == 0).all())


# -------------------------------------------------------------------- eviction
def dst_tables(torch, c, ns, replace):
    """Tables whose entry i < ceil(n / B) is the sequence's own block, or a
    free one where `replace` says so."""
    free, dst = list(c["free"]), c["bt"].clone()
    for s, n in enumerate(ns):
        for i in range(-(-n // c["B"])):
            if replace(s, i):
                dst[s, i] = free.pop()
    return dst


def check_evict(torch, c, before, got, w0, w1, keep, sink, recent, dst, max_keep, rows=None, wo_before=None):
    R = _ref()
    kept, new = got
    k0, v0 = before
    B, Hkv = c["B"], c["Hkv"]
    wantk, wantv = k0.clone(), v0.clone()
    wantw = (w0 if wo_before is None else wo_before).clone()
    for s, ctx in enumerate(c["lens"]):
        n, r = min(keep[s], ctx), s if rows is None else rows[s]
        assert int(new[s]) == n
        for h in range(Hkv):
            at = R.ref_evict(w0[r, h, :ctx], n, sink, recent, ctx)
            assert torch.equal(kept[s, h, :n].long(), at), (s, h)
            assert bool((kept[s, h, n:] == -1).all())
            i = torch.arange(n, device="cuda")
            sb, db = c["bt"][s].long()[at // B], dst[s].long()[i // B]
            wantk[db, h, i % B] = k0[sb, h, at % B]
            wantv[db, h, i % B] = v0[sb, h, at % B]
            wantw[r, h, :n] = w0[r, h][at]
            wantw[r, h, n:ctx] = 0
    assert tuple(kept.shape) == (len(c["lens"]), Hkv, max_keep)
    assert same_bits(torch, c["k"], wantk) and same_bits(torch, c["v"], wantv)
    assert torch.equal(w1.nan_to_num(nan=-7.0), wantw.nan_to_num(nan=-7.0))


def run_evict(torch, shape, lens, keep, sink, recent, dst=None, seed=61, in_place=True, weights=None, spare=200):
    R = _ref()
    _, Hkv, D, B = shape
    c = R.make_cache(lens, Hkv, D, B, seed=seed, spare=spare)
    w0 = random_weights(torch, len(lens), Hkv, c["mb"] * B + 3, seed=seed)
    if weights is not None:
        weights(w0)
    before = (c["k"].clone(), c["v"].clone())
    d = None if dst is None else dst_tables(torch, c, [min(k, n) for k, n in zip(keep, lens)], dst)
    w, wo, err = w0.clone(), torch.full_like(w0, -5.0), err_of(torch)
    got = pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], torch.tensor(keep, dtype=torch.int32, device="cuda"), w,
                          max_keep_len=max(keep), sink_tokens=sink, recent_tokens=recent, dst_tables=d,
                          weights_out=None if in_place else wo, err_flag=err)
    assert int(err) == 0
    check_evict(torch, c, before, got, w0, w if in_place else wo, keep, sink, recent, c["bt"] if d is None else d,
                max(keep), wo_before=None if in_place else torch.full_like(w0, -5.0))
    if not in_place:
        assert torch.equal(w.view(torch.int32), w0.view(torch.int32))


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (16, 4, 4), (31, 0, 31), (64, 0, 0), (500, 4, 32)])
def test_evict_in_place(torch, shape, keep, sink, recent):
    run_evict(torch, shape, LENS, [keep] * len(LENS), sink, recent)


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4]], ids=ids)
@pytest.mark.parametrize("which", ["all", "leading", "odd"])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_into_other_blocks(torch, shape, which, in_place):
    pick = {"all": lambda s, i: True, "leading": lambda s, i: i < 2, "odd": lambda s, i: (s + i) % 2 == 1}[which]
    run_evict(torch, shape, LENS, [50 + 7 * s for s in range(len(LENS))], 2, 5, dst=pick, in_place=in_place)


@pytest.mark.parametrize("ctx,keep", [(5000, 4999), (5000, 4096), (20000, 10001), (49000, 300), (60001, 30000)])
def test_evict_long_contexts(torch, ctx, keep):
    """Many stretches of rows in place; more weights than shared memory holds."""
    run_evict(torch, (2, 2, 64, 16), [ctx, ctx // 2], [keep, keep // 2], 4, 64)


def test_evict_many_long_rows(torch):
    """Rows enough to fill the GPU without clusters."""
    lens = [4200 + 37 * i for i in range(40)]
    run_evict(torch, (8, 8, 64, 16), lens, [3000 + 11 * i for i in range(40)], 3, 40)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_a_row_longer_than_any_shared_memory(torch, in_place):
    run_evict(torch, (1, 1, 64, 32), [200001, 9], [120000, 9], 1, 64, in_place=in_place)


@pytest.mark.parametrize("fill", ["_ties", "_zeros", "_odd", "_same", "_steps"])
@pytest.mark.parametrize("ctx,keep", [(5000, 77), (9999, 9000), (33000, 16001)])
def test_evict_weights_of_every_kind_in_clusters(torch, fill, ctx, keep):
    run_evict(torch, (1, 1, 64, 16), [ctx, ctx - 640], [keep, keep // 2], 1, 2, weights=globals()[fill])


@pytest.mark.parametrize("ctx,keep,sink,recent", [(3500, 2000, 3, 1500), (3500, 2000, 0, 2000), (9000, 8000, 1, 5000),
                                                  (60000, 40000, 2, 30000), (700, 600, 600, 0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_with_long_ends(torch, ctx, keep, sink, recent, in_place):
    run_evict(torch, (2, 2, 64, 16), [ctx, ctx // 2 + 11], [keep, keep], sink, recent, in_place=in_place)


def _ties(w):
    w.copy_((w * 40).round() / 40)  # few values


def _zeros(w):
    w.zero_()
    w[:, :, ::7] = -0.0
    w[:, :, 5::11] = 1e-20


def _same(w):
    w.fill_(0.25)


def _steps(w):  # a few values that differ in their last bits, in blocks
    n = w.shape[2]
    i = w.new_tensor(range(n)).long()
    w.copy_((1.0 + (i // 700 * 5 % 7) * 2.0**-23).expand_as(w))


def _odd(w):
    w[:, :, 3::13] = math.nan
    w[:, :, 4::17] = math.inf
    w[:, :, 5::19] = -math.inf
    w[:, :, 6::5] *= -1
    w[:, :, 7::29] = 3.4e38
    w[:, :, 8::23] = 1e-42


@pytest.mark.parametrize("fill", [_ties, _zeros, _odd])
@pytest.mark.parametrize("keep", [3, 40, 300])
def test_evict_weights_of_every_kind(torch, fill, keep):
    run_evict(torch, (4, 2, 64, 16), LENS, [keep] * len(LENS), 1, 2, weights=fill, in_place=False)


def test_evict_refusals_on_the_device(torch):
    """Every refused sequence stays as it is, the others do not notice."""
    R = _ref()
    lens = [100] * 8
    c = R.make_cache(lens, 2, 64, 16, seed=62)
    w0 = random_weights(torch, 8, 2, 128)
    ctx = torch.tensor([0, -1, 101, 100, 100, 100, 100, 100], dtype=torch.int32, device="cuda")
    keep = torch.tensor([20, 20, 20, 0, 41, 9, 20, 20], dtype=torch.int32, device="cuda")
    before = (c["k"].clone(), c["v"].clone())
    w, err = w0.clone(), err_of(torch)
    kept, new = pa.evict_tokens(c["k"], c["v"], c["bt"], ctx, keep, w, max_keep_len=40, sink_tokens=4,
                                recent_tokens=6, max_context_len=100, err_flag=err)
    assert int(err) == pa.DEVERR_CTX
    assert new.tolist() == [0, -1, 101, 100, 100, 100, 20, 20] and bool((kept[:6] == -1).all())
    assert torch.equal(w[:6], w0[:6])
    c2 = dict(c, lens=[100, 100], bt=c["bt"][6:].contiguous())
    check_evict(torch, c2, before, (kept[6:], new[6:]), w0[6:], w[6:], [20, 20], 4, 6, c2["bt"], 40)
    # rows out of range, and one that two sequences name: the first has it
    rows = torch.tensor([7, 8, -1, 2, 7, 0, 1, 3], dtype=torch.int32, device="cuda")
    c = R.make_cache(lens, 2, 64, 16, seed=63)
    before = (c["k"].clone(), c["v"].clone())
    w, err = w0.clone(), err_of(torch)
    kept, new = pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], torch.full_like(keep, 30), w, max_keep_len=40,
                                weight_rows=rows, err_flag=err, max_context_len=100)
    assert int(err) == pa.DEVERR_ROW and new.tolist() == [30, 100, 100, 30, 100, 30, 30, 30]
    assert bool((kept[[1, 2, 4]] == -1).all())
    live = [0, 3, 5, 6, 7]
    c2 = dict(c, lens=[100] * 5, bt=c["bt"][live].contiguous())
    check_evict(torch, c2, before, (kept[live], new[live]), w0, w, [30] * 5, 0, 0, c2["bt"], 40,
                rows=[int(rows[i]) for i in live])


def test_evict_blocks_outside_the_pool_are_not_touched(torch):
    R = _ref()
    c = R.make_cache([100, 100], 2, 64, 16, seed=64)
    bt = c["bt"].clone()
    bt[0, 3] = c["k"].shape[0]
    bt[0, 5] = -1
    before = (c["k"].clone(), c["v"].clone())
    w0, err = random_weights(torch, 2, 2, 128), err_of(torch)
    w = w0.clone()
    kept, _ = pa.evict_tokens(c["k"], c["v"], bt, c["ctx"], torch.tensor([70, 70], dtype=torch.int32, device="cuda"),
                              w, max_keep_len=70, max_context_len=100, err_flag=err)
    assert int(err) == pa.DEVERR_PAGE
    k = before[0].clone()
    for s in range(2):
        for h in range(2):
            for i, j in enumerate(kept[s, h].tolist()):
                sb, db = int(bt[s, j // 16]), int(bt[s, i // 16])
                if 0 <= sb < k.shape[0] and 0 <= db < k.shape[0]:
                    k[db, h, i % 16] = before[0][sb, h, j % 16]
    assert same_bits(torch, c["k"], k)


def test_evict_in_a_graph_and_on_a_stream(torch):
    R = _ref()
    c = R.make_cache([900, 300, 41], 2, 128, 16, seed=65)
    w0 = random_weights(torch, 3, 2, c["mb"] * 16)
    keep = torch.tensor([400, 299, 20], dtype=torch.int32, device="cuda")
    k0, v0 = c["k"].clone(), c["v"].clone()
    w = w0.clone()
    q = random_q(torch, 3, 8, 128)

    def step(stream=None):
        out, _ = pa.paged_attention_decode_weights(q, c["k"], c["v"], c["bt"], c["ctx"], w, max_context_len=900,
                                                   stream=stream)
        kept, new = pa.evict_tokens(c["k"], c["v"], c["bt"], c["ctx"], keep, w, max_keep_len=400, sink_tokens=1,
                                    recent_tokens=8, max_context_len=900, stream=stream)
        return out, kept, new

    def reset():
        c["k"].copy_(k0), c["v"].copy_(v0), w.copy_(w0)

    def state(r):
        return [x.clone() for x in (*r, c["k"], c["v"], w)]

    want = state(step())
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(state(r), want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step()
        graphs.append((g, r))
    for _ in range(2):
        for g, r in graphs:
            reset()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(state(r), want))


# ------------------------------------------------------------------- together
def test_long_context_loop(torch):
    """A serving loop over the block manager: two samples of one prompt decode
    with accumulated weights, one is evicted (its shared blocks replaced, the
    other sample untouched), its bounds are brought up to date, and it goes
    on with block-sparse steps.  Every step against the definition over the
    tokens that the bookkeeping says are cached."""
    R = _ref()
    B, Hkv, D, G = 16, 2, 64, 4
    bm = pa.BlockManager(64, B)
    g = torch.Generator(device="cuda").manual_seed(9)
    kp = torch.zeros(64, Hkv, B, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    bounds = torch.zeros(64, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    err = err_of(torch)
    MB, MAXTOK = 24, 24 * B
    w = torch.zeros(4, Hkv, MAXTOK, device="cuda")
    rows = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    n0 = 213
    bm.add_seq(0, n0)
    tok = lambda n: torch.randn(n, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ks, vs = tok(n0), tok(n0)
    t = bm.block_table(0)
    pa.reshape_and_cache(ks, vs, kp, vp, torch.tensor([t[j // B] * B + j % B for j in range(n0)], device="cuda"),
                         err_flag=err)
    bm.fork(0, 1)
    # per (sequence, kv head): what is cached, in slot order
    cache = {s: [[(ks[j, h], vs[j, h]) for j in range(n0)] for h in range(Hkv)] for s in (0, 1)}
    sums = torch.zeros(4, Hkv, MAXTOK, dtype=torch.float64, device="cuda")
    scale = 1 / math.sqrt(D)

    def tables(seqs):
        bt, lens = bm.block_tables(seqs, MB)
        return (torch.as_tensor(bt, dtype=torch.int32).cuda().contiguous(),
                torch.as_tensor(lens, dtype=torch.int32).cuda())

    def append(seqs):
        slots, cows = bm.append_batch(seqs)
        cows = torch.as_tensor(cows, dtype=torch.int64).reshape(-1, 2)
        cows = cows[cows[:, 0] >= 0]
        if len(cows):
            pa.copy_blocks([kp], [vp], cows.cuda().contiguous(), err_flag=err)
        nk, nv = tok(len(seqs)), tok(len(seqs))
        pa.reshape_and_cache(nk, nv, kp, vp, torch.as_tensor(slots, dtype=torch.int64).cuda(), err_flag=err)
        for i, s in enumerate(seqs):
            for h in range(Hkv):
                cache[s][h].append((nk[i, h], nv[i, h]))

    def check(s, out, lists=None):
        for h in range(Hkv):
            n = len(cache[s][h])
            at = range(n) if lists is None else [j for i in lists[h].tolist() if i >= 0
                                                 for j in range(i * B, min(n, i * B + B))]
            k = torch.stack([cache[s][h][j][0] for j in at]).double()
            v = torch.stack([cache[s][h][j][1] for j in at]).double()
            p, o, tol, _ = R.ref_attend(q[s, h * G:h * G + G], k, v, scale)
            assert bool(((out[h * G:h * G + G].double() - o).abs() <= tol).all())
            if lists is None:
                sums[int(rows[s]), h, :n] += p.sum(0)

    for step in range(4):
        append([0, 1])
        bt, lens = tables([0, 1])
        q = torch.randn(2, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
        out, _ = pa.paged_attention_decode_weights(q, kp, vp, bt, lens, w, weight_rows=rows, err_flag=err)
        check(0, out[0])
        check(1, out[1])
    assert bool(((w.double() - sums).abs() <= sums * 2.0**-11).all())
    # sequence 1 goes down to 96 tokens; the prompt's whole blocks are shared with sequence 0
    bt, lens = tables([1])
    dst = bm.evict(1, 96)
    assert sum(d != int(bt[0, i]) for i, d in enumerate(dst)) == len(dst)
    dt = torch.zeros(1, MB, dtype=torch.int32)
    dt[0, :len(dst)] = torch.tensor(dst)
    kept, new = pa.evict_tokens(kp, vp, bt, lens, torch.tensor([96], dtype=torch.int32, device="cuda"), w,
                                max_keep_len=96, sink_tokens=4, recent_tokens=16, dst_tables=dt.cuda(),
                                weight_rows=rows[1:].contiguous(), max_context_len=MAXTOK, err_flag=err)
    assert new.tolist() == [96] == [bm.seq_len(1)]
    for h in range(Hkv):
        cache[1][h] = [cache[1][h][j] for j in kept[0, h].tolist()]
    bt, lens = tables([0, 1])
    pa.block_key_bounds(kp, bounds, bt, lens, err_flag=err)
    for step in range(20):
        append([0, 1])
        bt, lens = tables([0, 1])
        pa.block_key_bounds(kp, bounds, bt, lens, lens - 1, max_new_tokens=1, err_flag=err)
        q = torch.randn(2, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
        sel = pa.select_blocks(q, bounds, bt, lens, 5, block_size=B, err_flag=err)
        assert torch.equal(sel, R.ref_select(q, bounds, bt, lens.tolist(), B, G, 5, 1, 1))
        out = pa.paged_attention_decode_sparse(q, kp, vp, bt, lens, sel, err_flag=err)
        for s in (0, 1):
            check(s, out[s], sel[s])
    assert int(err) == 0


@pytest.mark.parametrize("max_blocks", [40, 64])
def test_several_sequences_of_a_block_manager_in_one_eviction(torch, max_blocks):
    """Samples of one prompt and other sequences, shortened together: every
    kept row comes from its sequence's blocks as they were before the call."""
    R = _ref()
    B, Hkv, D, N = 16, 2, 128, 150
    bm = pa.BlockManager(N, B)
    bm.add_seq(0, 300)
    bm.fork(0, 1)
    bm.fork(0, 2)
    bm.append_batch([1, 2])
    bm.add_seq(3, 500)
    bm.add_seq(4, 40)
    bm.fork(4, 5)
    ids, keep = [3, 1, 0, 2, 5], [200, 150, 299, 301, 17]
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(N, Hkv, B, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    bt, lens = bm.block_tables(ids, max_blocks)
    dst, new = bm.evict_batch(ids, keep, max_blocks)
    assert new.tolist() == [200, 150, 299, 301, 17] and lens.tolist() == [500, 301, 300, 301, 40]
    c = dict(k=k, v=v, bt=torch.as_tensor(bt).cuda(), ctx=torch.as_tensor(lens).cuda(), lens=lens.tolist(), B=B, D=D,
             Hkv=Hkv, mb=max_blocks)
    w0 = random_weights(torch, len(ids), Hkv, max_blocks * B)
    w, before, err = w0.clone(), (k.clone(), v.clone()), err_of(torch)
    dt = torch.as_tensor(dst).cuda()
    got = pa.evict_tokens(k, v, c["bt"], c["ctx"], torch.as_tensor(keep, dtype=torch.int32).cuda(), w, max_keep_len=301,
                          sink_tokens=2, recent_tokens=9, dst_tables=dt, err_flag=err)
    assert int(err) == 0 and got[1].tolist() == new.tolist()
    check_evict(torch, c, before, got, w0, w, keep, 2, 9, dt, 301)
