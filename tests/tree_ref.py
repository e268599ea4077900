"""Decoding with trees of drafted tokens in plain 64-bit operations, one node
and kv head at a time, and the makings of its test cases."""
import math
import random

import torch

import long_context_ref as lc


def make_tree(t, kind, rng):
    """Parents of t nodes: a chain, a star around node 0, only roots, or any earlier node."""
    if kind == "chain":
        return [i - 1 for i in range(t)]
    if kind == "star":
        return [min(i, 1) - 1 for i in range(t)]
    if kind == "roots":
        return [-1] * t
    return [rng.randrange(-1, i) if i else -1 for i in range(t)]


def chain_of(parents, i):
    """Node i's chain of ancestors, itself first; None if it meets a bad parent."""
    out = []
    while i >= 0:
        out.append(i)
        p = parents[i]
        if not -1 <= p < i:
            return None
        i = p
    return out


def make_case(ctx, nodes, Hq, Hkv, D, B, kind="any", seed=0, junk=None, spare_rows=3, device="cuda"):
    """A cache of contexts and trees, queries for every node (and `spare_rows`
    rows behind the last tree)."""
    rng = random.Random(seed)
    c = lc.make_cache([a + b for a, b in zip(ctx, nodes)], Hkv, D, B, seed, device=device, junk=junk)
    cu = [0]
    for t in nodes:
        cu.append(cu[-1] + t)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    trees = [make_tree(t, kind, rng) for t in nodes]
    flat = [p for tree in trees for p in tree] + [-1] * spare_rows
    c.update(q=torch.randn(cu[-1] + spare_rows, Hq, D, generator=g, device=device).to(torch.bfloat16), trees=trees,
             cu_host=cu, nodes=list(nodes), contexts=list(ctx), Hq=Hq, G=Hq // Hkv,
             cu=torch.tensor(cu, dtype=torch.int32, device=device),
             parents=torch.tensor(flat, dtype=torch.int32, device=device),
             ctx=torch.tensor(list(ctx), dtype=torch.int32, device=device),
             most=max(max(nodes), 1), scale=D**-0.5)
    return c


def attend(q, k, v, scale, once):
    """lc.ref_attend for any keys: a query head with a NaN or +infinite logit
    has a NaN row, a key of -infinity weighs nothing."""
    x = (q.double() @ k.T) * scale
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    plain = bool(torch.isfinite(x).all())
    if plain:
        _, out, tol, _ = lc.ref_attend(q, k, v, scale, once)
        return out, tol
    for g in range(q.shape[0]):
        if bool((torch.isnan(x[g]) | (x[g] == math.inf)).any()):
            out[g] = math.nan
            continue
        live = x[g] != -math.inf
        _, o, tl, _ = lc.ref_attend(q[g:g + 1], k[live], v[live], scale, once)
        out[g], tol[g] = o[0], tl[0]
    return out, tol


def ref_tree(c, sequences=None, nodes=None, drop=()):
    """{row: (out [Hq][D], tolerance)} of the listed sequences' nodes (all).
    `drop`: (sequence, logical block) whose keys are left out.

    The kernel rounds each probability to bf16 once, by at most 2^-8 of it,
    and divides by the sum of the unrounded ones: the output moves by at most
    2^-8 A, A = sum p |v|, within lc.ref_attend's bound for `once`."""
    once = True
    got = {}
    for s in sequences if sequences is not None else range(len(c["nodes"])):
        n0, B, ctx, t = c["cu_host"][s], c["B"], c["contexts"][s], c["nodes"][s]
        if t == 0:
            continue
        keys = [lc.rows(c["k"], c["bt"][s], ctx + t, B, h) for h in range(c["Hkv"])]
        vals = [lc.rows(c["v"], c["bt"][s], ctx + t, B, h) for h in range(c["Hkv"])]
        for i in nodes if nodes is not None else range(t):
            if i >= t:
                continue
            chain = chain_of(c["trees"][s], i)
            out = torch.zeros(c["Hq"], c["D"], dtype=torch.float64, device=c["q"].device)
            tol = torch.zeros_like(out)
            if chain is not None:
                at = [j for j in list(range(ctx)) + [ctx + a for a in sorted(chain)] if (s, j // B) not in drop]
                at = torch.tensor(at, dtype=torch.int64, device=c["q"].device)
                for h in range(c["Hkv"]):
                    g = slice(h * c["G"], (h + 1) * c["G"])
                    out[g], tol[g] = attend(c["q"][n0 + i, g], keys[h][at], vals[h][at], c["scale"], once)
            got[n0 + i] = (out, tol)
    return got


def check(got, ref):
    """Every reference row within its tolerance; NaN and infinite values where the reference has values that are not finite."""
    for row, (out, tol) in ref.items():
        g = got[row].double()
        fine = torch.isfinite(out)
        assert bool((torch.isfinite(g) == fine).all()), f"row {row}: finite values in other places"
        off = (g - out).abs()
        bad = fine & ~(off <= tol)
        assert not bool(bad.any()), f"row {row}: {int(bad.sum())} values off, worst {float((off / tol)[bad].max()):.3g} of the tolerance"


def ref_verify(logits, tokens, trees, cu, V):
    """(targets, paths, next tokens) in plain Python."""
    x = logits[:, :V].double().cpu()
    targets = []
    for row in x:
        nan = torch.isnan(row)
        best = nan if bool(nan.any()) else row == row.max()
        targets.append(int(torch.nonzero(best)[0, 0]))
    paths, nexts = [], []
    for s, tree in enumerate(trees):
        path, node = [], 0 if tree and tree[0] == -1 else None
        while node is not None:
            path.append(node)
            said = targets[cu[s] + node]
            node = next((i for i in range(node + 1, len(tree)) if tree[i] == node and tokens[cu[s] + i] == said), None)
        paths.append(path)
        nexts.append(targets[cu[s] + path[-1]] if path else -1)
    return targets, paths, nexts
