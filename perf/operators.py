"""Measured cases of the long-context decode operators: block-sparse decode
(key bounds of every block, selection of blocks by them, attention over the
selected blocks) and cache eviction by accumulated attention weight (decode
that accumulates the weights, eviction of the tokens with the smallest sums).

`run` computes a case in plain torch operations, or, with `own` set, through
the library's calls.
"""
import math
import random

import torch

own = False

OPS = ("bounds", "select", "sparse", "weights", "evict")


def listed():
    return [
        # every block of eight 32K-token prompts, as after their prefill
        _case("bounds", "bounds_prompts_32k", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, B=16, new=32768),
        # one new token per sequence of a 64-sequence batch: the last block of each
        _case("bounds", "bounds_step_batch64", S=64, lo=128, hi=2048, Hq=32, Hkv=8, D=128, B=16, new=1),
        # 128 of 2048 blocks for each (sequence, kv head) of eight 32K-token contexts
        _case("select", "select_32k", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, B=16, k=128),
        # a ragged batch of ordinary contexts: up to 32 of at most 128 blocks, some contexts shorter than that
        _case("select", "select_batch64", S=64, lo=128, hi=2048, Hq=32, Hkv=8, D=128, B=16, k=32),
        # one sequence alone, where the latency of the calls counts
        _case("select", "select_single_8k", S=1, lo=8191, hi=8191, Hq=24, Hkv=8, D=64, B=32, k=33),
        # attention over those 128 blocks of each 32K-token context
        _case("sparse", "sparse_32k", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, B=16, k=128),
        # a large ragged batch with 32-token blocks and short lists
        _case("sparse", "sparse_batch240", S=240, lo=64, hi=4096, Hq=32, Hkv=8, D=128, B=32, k=24),
        # the whole cache read with the weights summed, long contexts
        _case("weights", "weights_32k", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, B=16),
        # the same for an ordinary decode batch
        _case("weights", "weights_batch64", S=64, lo=128, hi=2048, Hq=32, Hkv=8, D=128, B=16),
        # the smallest call: four short sequences without grouped heads
        _case("weights", "weights_tiny", S=4, lo=1, hi=100, Hq=4, Hkv=4, D=64, B=16),
        # eight 32K-token caches cut to half
        _case("evict", "evict_32k", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, B=16, keep=16384),
        # an ordinary batch cut to 512 tokens; the shorter sequences stay as they are
        _case("evict", "evict_batch64", S=64, lo=128, hi=2048, Hq=32, Hkv=8, D=128, B=16, keep=512),
    ]


def _case(op, name=None, **sizes):
    c = dict(op=op, **sizes)
    if name:
        c["name"] = name
    return c


#: Keys of the largest listed cases over all sequences and kv heads, times head_dim.
MOST = 8 * 32768 * 8 * 128


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    D, B = rng.choice((64, 128)), rng.choice((16, 32))
    Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    S, hi = _log(rng, 1, 240), _log(rng, 1, 32768)
    while S * (hi + B) * Hkv * D > MOST // 2 or S * hi * Hkv * G > MOST // 32:
        S, hi = (S + 1) // 2, max(1, (hi * 3) // 4)
    lo = rng.choice((hi, 1 + hi // 16, 1 + hi // 2))
    c = dict(S=S, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, B=B)
    n = -(-hi // B)
    if op == "bounds":
        c["new"] = rng.choice((1, hi, _log(rng, 1, hi)))
    elif op in ("select", "sparse"):
        c["k"] = max(2, _log(rng, 1, max(2, n // 2)))
    elif op == "evict":
        c["keep"] = max(2, _log(rng, 1, max(2, hi - hi // 8)))
    return _case(op, **c)


def _lens(case):
    """Context lengths: the case's own, whatever the seed."""
    r = random.Random("%d %d %d" % (case["S"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]


def _blocks(case):
    return [-(-n // case["B"]) for n in _lens(case)]


def _ends(case):
    """Leading and trailing blocks (tokens, for the eviction) that are always kept."""
    most = case["k"] if "k" in case else case["keep"]
    sink = min(4, most // 4) if "keep" in case else min(1, most // 2)
    return sink, max(1, min(32, most // 8)) if "keep" in case else max(1, most // 8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, Hkv, D, B = case["S"], case["Hkv"], case["D"], case["B"]
    lens, nblk = _lens(case), _blocks(case)
    mb = max(nblk)
    dst = [min(case["keep"], n) for n in lens] if case["op"] == "evict" else [0] * S
    ndst = [-(-n // B) for n in dst]
    used = sum(nblk) + sum(ndst)
    num_blocks = used + max(4, used // 4)
    ids = torch.randperm(num_blocks, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)

    def tables(counts, first):
        n = torch.tensor(counts, device="cuda")
        at = first + torch.cumsum(n, 0) - n
        i = torch.arange(mb, device="cuda")
        t = ids[(at[:, None] + i).clamp(max=num_blocks - 1)]
        return torch.where(i < n[:, None], t, torch.zeros_like(t)).contiguous()

    st = dict(case=case, B=B, G=case["Hq"] // Hkv, scale=1.0 / math.sqrt(D), max_ctx=max(lens), mb=mb)
    st["tables"] = tables(nblk, 0)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    # keys with a part that a block's tokens share, and channels of unlike sizes
    k = normal(num_blocks, Hkv, B, D)
    k += normal(num_blocks, Hkv, 1, D) * 0.5
    k *= 0.5 + torch.rand(Hkv, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    st["q"] = normal(S, case["Hq"], D)
    op = case["op"]
    if op == "bounds":
        st["k"] = k
        st["bounds"] = torch.zeros(num_blocks, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
        st["start"] = (st["lens"] - case["new"]).clamp(min=0)
    elif op == "select":
        bounds = torch.empty(num_blocks, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
        # of whole blocks: a partly filled last block's bounds may be of fewer keys, which changes nothing here
        torch.amin(k, 2, out=bounds[:, :, 0])
        torch.amax(k, 2, out=bounds[:, :, 1])
        st["bounds"] = bounds
    else:
        st["k"], st["v"] = k, normal(num_blocks, Hkv, B, D)
    if op == "sparse":
        n = torch.tensor(nblk, device="cuda")[:, None, None]
        i = torch.arange(mb, device="cuda").expand(S, Hkv, mb)
        rank = torch.rand(S, Hkv, mb, generator=g, device="cuda")
        sink, recent = _ends(case)
        rank = torch.where((i < sink) | (i >= n - recent), torch.full_like(rank, 2.0), rank)
        rank = torch.where(i < n, rank, torch.full_like(rank, -1.0))
        kk = min(case["k"], mb)
        top, at = torch.topk(rank, kk, dim=2)
        at = torch.where(top >= 0, at, torch.full_like(at, mb)).sort(dim=2).values
        sel = torch.full((S, Hkv, case["k"]), -1, dtype=torch.int32, device="cuda")
        sel[:, :, :kk] = torch.where(at < mb, at, torch.full_like(at, -1)).to(torch.int32)
        st["selected"] = sel
    if op in ("weights", "evict"):
        # the sums of the first few steps: uneven, of the size of one step's weights
        w = torch.exp(2.0 * torch.randn(S, Hkv, mb * B, generator=g, device="cuda") - 1.0)
        w *= st["G"] / st["lens"][:, None, None]
        j = torch.arange(mb * B, device="cuda")
        st["weights"] = torch.where(j < st["lens"][:, None, None], w, torch.zeros_like(w))
        st["weights_out"] = torch.zeros_like(w)
    if op == "evict":
        st["dst"] = tables(ndst, sum(nblk))
        st["keep"] = torch.full((S,), case["keep"], dtype=torch.int32, device="cuda")
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


# ------------------------------------------------------------ the library's calls
def _own_bounds(st):
    import paged_kv_cache_262_gb300 as pa
    return pa.block_key_bounds(st["k"], st["bounds"], st["tables"], st["lens"], st["start"],
                               max_new_tokens=st["case"]["new"], max_context_len=st["max_ctx"], err_flag=st["err"])


def _own_select(st):
    import paged_kv_cache_262_gb300 as pa
    sink, recent = _ends(st["case"])
    return pa.select_blocks(st["q"], st["bounds"], st["tables"], st["lens"], st["case"]["k"], block_size=st["B"],
                            sink_blocks=sink, recent_blocks=recent, max_context_len=st["max_ctx"], err_flag=st["err"])


def _own_sparse(st):
    import paged_kv_cache_262_gb300 as pa
    return pa.paged_attention_decode_sparse(st["q"], st["k"], st["v"], st["tables"], st["lens"], st["selected"],
                                            scale=st["scale"], max_context_len=st["max_ctx"], err_flag=st["err"])


def _own_weights(st):
    import paged_kv_cache_262_gb300 as pa
    return pa.paged_attention_decode_weights(st["q"], st["k"], st["v"], st["tables"], st["lens"], st["weights"],
                                             weights_out=st["weights_out"], scale=st["scale"],
                                             max_context_len=st["max_ctx"], err_flag=st["err"])


def _own_evict(st):
    import paged_kv_cache_262_gb300 as pa
    sink, recent = _ends(st["case"])
    kept, new_lens = pa.evict_tokens(st["k"], st["v"], st["tables"], st["lens"], st["keep"], st["weights"],
                                     max_keep_len=st["case"]["keep"], sink_tokens=sink, recent_tokens=recent,
                                     dst_tables=st["dst"], weights_out=st["weights_out"],
                                     max_context_len=st["max_ctx"], err_flag=st["err"])
    return kept, new_lens, st["weights_out"], st["k"], st["v"]


_OWN = dict(bounds=_own_bounds, select=_own_select, sparse=_own_sparse, weights=_own_weights, evict=_own_evict)


# ------------------------------------------------------------ the plain forms
def _pages(pool, tables):
    """Rows of the table's blocks, one sequence and head after another: [S][Hkv][blocks * B][D], 32 bits."""
    x = pool[tables.long()]
    S, n, H, B, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(S, H, n * B, D).float()


def _plain_bounds(st):
    k, B, lens = st["k"], st["B"], st["lens"].long()
    first = st["start"].long() // B
    span = min(st["mb"], (st["case"]["new"] + B - 1) // B + 1)
    i = first[:, None] + torch.arange(span, device=k.device)
    live = i * B < lens[:, None]
    i = torch.where(live, i, ((lens - 1) // B)[:, None])  # the last block again instead of one past it
    phys = st["tables"].long().gather(1, i)
    x = k[phys].float()
    there = (i[:, :, None] * B + torch.arange(B, device=k.device)) < lens[:, None, None]
    there = there[:, :, None, :, None]
    lo = torch.where(there, x, torch.full_like(x, math.inf)).amin(3)
    hi = torch.where(there, x, torch.full_like(x, -math.inf)).amax(3)
    st["bounds"][phys] = torch.stack((lo, hi), 3).to(torch.bfloat16)
    return st["bounds"]


def _plain_select(st):
    S, Hkv, B, k = st["case"]["S"], st["case"]["Hkv"], st["B"], st["case"]["k"]
    q = st["q"].double().view(S, Hkv, st["G"], -1)
    b = st["bounds"][st["tables"].long()].permute(0, 2, 3, 4, 1).double()  # [S][Hkv][2][D][blocks]
    score = (q.clamp(min=0) @ b[:, :, 1] + q.clamp(max=0) @ b[:, :, 0]).amax(2)
    n = ((st["lens"].long() + B - 1) // B)[:, None, None]
    i = torch.arange(st["mb"], device=q.device)
    sink, recent = _ends(st["case"])
    score = torch.where((i < sink) | (i >= n - recent), torch.full_like(score, math.inf), score)
    score = torch.where(i < n, score, torch.full_like(score, -math.inf))
    at = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :k]
    at = torch.where(at < n, at, torch.full_like(at, st["mb"])).sort(dim=2).values
    at = torch.where(at < st["mb"], at, torch.full_like(at, -1)).to(torch.int32)
    return torch.nn.functional.pad(at, (0, k - at.shape[2]), value=-1)


def _attend(q, k, v, seen, scale):
    s = (q @ k.transpose(-1, -2)) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return p, p @ v


def _plain_sparse(st):
    S, Hkv, B, D = st["case"]["S"], st["case"]["Hkv"], st["B"], st["case"]["D"]
    sel = st["selected"].long()
    phys = st["tables"].long()[:, None, :].expand(S, Hkv, st["mb"]).gather(2, sel.clamp(min=0))
    h = torch.arange(Hkv, device=sel.device)[:, None]
    k = st["k"][phys, h].reshape(S, Hkv, -1, D).float()
    v = st["v"][phys, h].reshape(S, Hkv, -1, D).float()
    j = sel[..., None] * B + torch.arange(B, device=sel.device)
    seen = (sel[..., None] >= 0) & (j < st["lens"].long()[:, None, None, None])
    q = st["q"].float().view(S, Hkv, st["G"], D)
    _, o = _attend(q, k, v, seen.reshape(S, Hkv, 1, -1), st["scale"])
    return o.reshape(S, -1, D).to(torch.bfloat16)


def _plain_weights(st):
    S, Hkv, D = st["case"]["S"], st["case"]["Hkv"], st["case"]["D"]
    k, v = _pages(st["k"], st["tables"]), _pages(st["v"], st["tables"])
    j = torch.arange(k.shape[2], device=k.device)
    seen = j < st["lens"].long()[:, None, None, None]
    q = st["q"].float().view(S, Hkv, st["G"], D)
    p, o = _attend(q, k, v, seen, st["scale"])
    st["weights_out"].copy_(torch.where(seen[:, :, 0], st["weights"] + p.sum(2), st["weights_out"]))
    return o.reshape(S, -1, D).to(torch.bfloat16), st["weights_out"]


def _plain_evict(st):
    case, B, w = st["case"], st["B"], st["weights"]
    Hkv, keep = case["Hkv"], case["keep"]
    lens = st["lens"].long()[:, None, None]
    n = torch.minimum(st["keep"].long()[:, None, None], lens)
    j = torch.arange(w.shape[2], device=w.device)
    sink, recent = _ends(case)
    rank = torch.where((j < sink) | (j >= lens - recent), torch.full_like(w, math.inf), w)
    rank = torch.where(j < lens, rank, torch.full_like(w, -math.inf))
    at = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    i = torch.arange(at.shape[2], device=w.device)
    at = torch.where(i < n, at, torch.full_like(at, w.shape[2])).sort(dim=2).values
    kept = torch.where(i < n, at, torch.full_like(at, -1)).to(torch.int32)
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[2]), value=-1)
    # past the kept tokens: the first one once more, to its own place
    src, to = torch.where(i < n, at, at[:, :, :1]), torch.where(i < n, i, torch.zeros_like(i))
    sphys = st["tables"].long()[:, None, :].expand(-1, Hkv, -1).gather(2, src // B)
    dphys = st["dst"].long()[:, None, :].expand(-1, Hkv, -1).gather(2, to // B)
    h = torch.arange(Hkv, device=w.device)[:, None]
    st["k"][dphys, h, to % B] = st["k"][sphys, h, src % B]
    st["v"][dphys, h, to % B] = st["v"][sphys, h, src % B]
    moved = torch.nn.functional.pad(w.gather(2, src), (0, w.shape[2] - src.shape[2]))
    moved = torch.where(j < n, moved, torch.zeros_like(w))
    st["weights_out"].copy_(torch.where(j < lens, moved, st["weights_out"]))
    return kept, n[:, 0, 0].to(torch.int32), st["weights_out"], st["k"], st["v"]


_PLAIN = dict(bounds=_plain_bounds, select=_plain_select, sparse=_plain_sparse, weights=_plain_weights,
              evict=_plain_evict)


# ------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, nblk, op = _lens(case), _blocks(case), case["op"]
    S, Hq, Hkv, D, B = case["S"], case["Hq"], case["Hkv"], case["D"], case["B"]
    G = Hq // Hkv
    plan = 4 * sum(nblk) + 4 * S  # table entries and lengths
    if op == "bounds":
        touched = [(max(0, n - case["new"]) // B * B, n) for n in lens]
        keys = sum(b - a for a, b in touched)
        blocks = sum(-(-b // B) - a // B for a, b in touched)
        return {"bytes": Hkv * (keys * D * 2 + blocks * D * 4) + 4 * blocks + 8 * S, "flops": 2 * Hkv * keys * D}
    if op == "select":
        read = sum(n for n in nblk if n > case["k"])
        return {"bytes": Hkv * read * D * 4 + S * Hq * D * 2 + 4 * S * Hkv * case["k"] + plan,
                "flops": 4 * Hkv * read * G * D}
    if op == "sparse":
        tokens = sum(min(n, case["k"]) * B - (-c % B) for c, n in zip(lens, nblk))
        return {"bytes": Hkv * tokens * D * 4 + 4 * S * Hq * D + 4 * S * Hkv * case["k"] + plan,
                "flops": 4 * Hkv * tokens * G * D}
    if op == "weights":
        return {"bytes": Hkv * sum(lens) * (D * 4 + 8) + 4 * S * Hq * D + plan, "flops": 4 * Hkv * sum(lens) * G * D}
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": Hkv * (8 * sum(lens) + 4 * S * case["keep"] + 8 * D * kept) + plan + 4 * sum(
        -(-min(n, case["keep"]) // B) for n in lens) + 8 * S, "flops": Hkv * sum(lens)}


# ------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, lens, nblk = case["op"], _lens(case), _blocks(case)
    Hkv, D, B, G = case["Hkv"], case["D"], case["B"], st["G"]
    tables = st["tables"].long()

    def rows(pool, s):  # [Hkv][ctx][D] of sequence s
        return pool[tables[s, :nblk[s]]].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[s]].double()

    def softmax(s, k, scale):
        z = torch.einsum("hgd,hjd->hgj", st["q"][s].double().view(Hkv, G, D), k) * scale
        return torch.softmax(z, -1)

    if op == "bounds":
        out = st["bounds"].double()
        for s in range(case["S"]):
            first = max(0, lens[s] - case["new"]) // B
            k = rows(st["k"], s)[:, first * B:]
            left = k.shape[1] // B * B
            full = tables[s, first:first + left // B]
            whole = k[:, :left].reshape(Hkv, -1, B, D)
            out[full] = torch.stack((whole.amin(2), whole.amax(2)), 2).transpose(0, 1)
            if left < k.shape[1]:
                out[tables[s, nblk[s] - 1]] = torch.stack((k[:, left:].amin(1), k[:, left:].amax(1)), 1)
        return out
    if op == "select":
        out = torch.full((case["S"], Hkv, case["k"]), -1, dtype=torch.int32)
        sink, recent = _ends(case)
        for s in range(case["S"]):
            n = nblk[s]
            if n <= case["k"]:
                out[s, :, :n] = torch.arange(n, dtype=torch.int32)
                continue
            b = st["bounds"][tables[s, :n]].double()  # [blocks][Hkv][2][D]
            best = None
            for g in range(G):
                x = st["q"][s].double().view(Hkv, G, D)[:, g]
                one = torch.maximum(x * b[:, :, 0], x * b[:, :, 1]).sum(-1)
                best = one if best is None else torch.maximum(best, one)
            best = best[sink:n - recent].t()
            some = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["k"] - sink - recent] + sink
            ends = torch.cat((torch.arange(sink), torch.arange(n - recent, n))).to(some.device)
            out[s] = torch.cat((some, ends.expand(Hkv, -1)), 1).sort(1).values.to(torch.int32).cpu()
        return out
    if op == "sparse":
        out = torch.empty(case["S"], Hkv * G, D, dtype=torch.float64)
        for s in range(case["S"]):
            j = st["selected"][s].long()[:, :, None] * B + torch.arange(B, device="cuda")
            j = torch.where(j < 0, torch.full_like(j, 1 << 40), j).flatten(1)
            count = int((j[0] < lens[s]).sum())
            j = j.sort(1).values[:, :count]
            take = j[:, :, None].expand(-1, -1, D)
            k, v = rows(st["k"], s).gather(1, take), rows(st["v"], s).gather(1, take)
            out[s] = torch.einsum("hgj,hjd->hgd", softmax(s, k, st["scale"]), v).reshape(-1, D).cpu()
        return out
    if op == "weights":
        out = torch.empty(case["S"], Hkv * G, D, dtype=torch.float64)
        sums = st["weights_out"].double()
        for s in range(case["S"]):
            p = softmax(s, rows(st["k"], s), st["scale"])
            out[s] = torch.einsum("hgj,hjd->hgd", p, rows(st["v"], s)).reshape(-1, D).cpu()
            sums[s, :, :lens[s]] = st["weights"][s, :, :lens[s]].double() + p.sum(1)
        return out, sums
    kept = torch.full((case["S"], Hkv, case["keep"]), -1, dtype=torch.int32)
    sums = st["weights_out"].double()
    sink, recent = _ends(case)
    for s in range(case["S"]):
        c, n = lens[s], min(lens[s], case["keep"])
        if n == c:
            at = torch.arange(c, device="cuda").expand(Hkv, -1)
        else:
            mid = st["weights"][s, :, sink:c - recent].double()
            some = torch.sort(mid, dim=1, descending=True, stable=True).indices[:, :n - sink - recent] + sink
            ends = torch.cat((torch.arange(sink), torch.arange(c - recent, c))).to(some.device)
            at = torch.cat((some, ends.expand(Hkv, -1)), 1).sort(1).values
        kept[s, :, :n] = at.to(torch.int32).cpu()
        sums[s, :, :n] = st["weights"][s].double().gather(1, at)
    return kept, torch.tensor([min(n, case["keep"]) for n in lens], dtype=torch.int32), sums, None, None
