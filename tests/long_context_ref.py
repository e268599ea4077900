"""Block-sparse decode and eviction in plain 64-bit torch operations, one
(sequence, kv head) at a time, and the makings of their test cases."""
import math

import torch

LOG2E = 1.4426950408889634


def make_cache(lens, Hkv, D, B, seed, device="cuda", spare=7, junk=None):
    """A pool whose blocks belong to sequences of these lengths in shuffled
    order, with `junk` in every slot past a context and in the spare blocks."""
    g = torch.Generator(device=device).manual_seed(seed)
    nblk = [-(-n // B) if n > 0 else 0 for n in lens]
    total = sum(nblk) + spare
    mb = max(max(nblk), 1) + 2
    perm = torch.randperm(total, generator=g, device=device).to(torch.int32).cpu()
    bt = torch.full((len(lens), mb), -1, dtype=torch.int32)  # entries past a context are never read
    at = 0
    for s, n in enumerate(nblk):
        bt[s, :n] = perm[at:at + n]
        at += n
    k = torch.randn(total, Hkv, B, D, generator=g, device=device).to(torch.bfloat16)
    v = torch.randn(total, Hkv, B, D, generator=g, device=device).to(torch.bfloat16)
    if junk is not None:
        used = torch.zeros(total, B, dtype=torch.bool)
        for s, n in enumerate(nblk):
            for i in range(n):
                used[bt[s, i], :min(B, lens[s] - i * B)] = True
        hole = ~used.to(device)[:, None, :, None].expand_as(k)
        k[hole] = junk
        v[hole] = junk
    free = perm[at:].tolist()
    return dict(k=k, v=v, bt=bt.to(device), ctx=torch.tensor(lens, dtype=torch.int32, device=device), lens=list(lens),
                free=free, B=B, D=D, Hkv=Hkv, mb=mb)


def rows(pool, bt, n, B, h):
    """[n][D] of one sequence and head."""
    blocks = bt[:-(-n // B)].long()
    return pool[blocks, h].reshape(-1, pool.shape[-1])[:n].double()


def ref_bounds(c, start=None):
    """{physical block: [Hkv][2][D]} of the blocks from `start` on."""
    out = {}
    for s, n in enumerate(c["lens"]):
        if n <= 0:
            continue
        for i in range((start[s] if start else 0) // c["B"], -(-n // c["B"])):
            b = int(c["bt"][s, i])
            x = c["k"][b, :, :min(c["B"], n - i * c["B"])].double()
            out[b] = torch.stack((x.amin(1), x.amax(1)), 1)
    return out


def ref_scores(q, bounds, bt, n, h, G):
    """Exact scores of n blocks of one sequence for kv head h."""
    x = q[h * G:(h + 1) * G].double()[:, None, :]
    b = bounds[bt[:n].long(), h].double()  # [n][2][D]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    term = torch.where(x > 0, x * b[None, :, 1], torch.where(x < 0, x * b[None, :, 0], torch.where(x == 0, zero, x)))
    sc = term.sum(-1)
    return torch.where(torch.isnan(sc), torch.full_like(sc, math.inf), sc).amax(0)


def ref_take(score, want):
    """Indices of the largest `want`, ties to the lowest index, increasing."""
    return torch.sort(torch.sort(score, descending=True, stable=True).indices[:want]).values


def ref_select(q, bounds, bt, lens, B, G, k, sink, recent):
    S, Hkv = q.shape[0], bounds.shape[1]
    out = torch.full((S, Hkv, k), -1, dtype=torch.int32, device=q.device)
    for s in range(S):
        n = -(-lens[s] // B)
        for h in range(Hkv):
            if n <= k:
                out[s, h, :n] = torch.arange(n)
                continue
            sc = ref_scores(q[s], bounds, bt[s], n, h, G)[sink:n - recent]
            mid = ref_take(sc, k - sink - recent) + sink
            out[s, h] = torch.cat((torch.arange(sink, device=q.device), mid,
                                   torch.arange(n - recent, n, device=q.device))).to(torch.int32)
    return out


def ref_attend(q, k, v, scale, once=False):
    """Softmax weights, outputs and their tolerances for [G][D] queries over
    [n][D] keys.

    The kernel takes each probability p as a bf16 value and a bf16 remainder,
    which leave at most 2^-16 of it, and divides by the sum of the unrounded
    ones: the output moves by at most 2^-16 A, A = sum p |v|.  (`once`: rounded
    once, by 2^-8 each, and divided by the sum of the rounded ones: at most
    2^-8 sum p |v - out| <= 2^-8 (A + |out|).)  The output's own rounding is at
    most 2^-8 |out|.  The values and products are of fp32: the logits x (base
    2) are off by e_x (below), which moves p by 2 ln2 e_x relative, ex2 by
    2^-22, the sums by n terms cut at 2^-23 on the partial sums, covered by
    2^-12 of A + |out|.
    """
    x = (q.double() @ k.T) * scale
    if x.shape[1] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        return x, z, z, x
    p = torch.softmax(x, -1)
    out = p @ v
    A = p @ v.abs()
    # A 16-wide MMA adds 17 terms, each cut at 2^-23 of the largest of them or
    # better; D/16 of them in a row: within 17 (D/16) 2^-23 of sum |q k|.
    ex = (q.double().abs() @ k.abs().T) * (abs(scale) * LOG2E * 17 * (q.shape[1] // 16) * 2.0**-23)
    ex = ex + x.abs() * LOG2E * 2.0**-22
    rel = 2 * math.log(2) * ex.amax(-1, keepdim=True)
    tol = ((2.0**-8 if once else 2.0**-16) + 2.0**-12 + rel) * (A + out.abs()) + 2.0**-8 * out.abs() + 1e-30
    return p, out, tol, p * (rel + 2.0**-19)


def ref_attend_any(q, k, v, scale):
    """ref_attend for any keys: a head with a NaN or +infinite logit has NaN
    weights and a NaN row, a key of -infinity weighs nothing (a head that has
    no others gives zeros)."""
    x = (q.double() @ k.T) * scale
    p, tp = torch.zeros_like(x), torch.zeros_like(x)
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for g in range(q.shape[0]):
        if bool((torch.isnan(x[g]) | (x[g] == math.inf)).any()):
            p[g], out[g] = math.nan, math.nan
            continue
        live = x[g] != -math.inf
        r = ref_attend(q[g:g + 1], k[live], v[live], scale)
        p[g, live], out[g], tol[g], tp[g, live] = (y[0] for y in r)
    return p, out, tol, tp


def ref_evict(w, n, sink, recent, ctx):
    """Kept tokens of one row of weights [ctx]."""
    if n >= ctx:
        return torch.arange(ctx, device=w.device)
    key = torch.where(torch.isnan(w), torch.full_like(w, math.inf), w.double() if w.dtype != torch.float64 else w)
    nan_first = torch.isnan(w)[sink:ctx - recent]
    mid = key[sink:ctx - recent]
    # NaN above +infinity: ranked in two strokes, each in index order
    order = torch.sort(mid, descending=True, stable=True).indices
    order = torch.cat((order[nan_first[order]], order[~nan_first[order]]))
    some = torch.sort(order[:n - sink - recent]).values + sink
    return torch.cat((torch.arange(sink, device=w.device), some, torch.arange(ctx - recent, ctx, device=w.device)))
