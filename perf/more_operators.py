"""Measured cases of decoding with trees of drafted tokens: attention of every
drafted token over the paged cache and its own ancestors, verification of the
trees against the model's logits, and the compaction of the accepted paths'
keys and values in the cache.

`run` computes a case in plain torch operations, or, with `own` set, through
the library's calls.
"""
import math
import random

import torch

own = False

OPS = ("tree", "verify", "commit")


def listed():
    return [
        # one sequence alone with a small tree, where the latency of the call counts
        _case("tree", "tree_single", S=1, lo=1000, hi=1000, tlo=8, thi=8, Hq=24, Hkv=8, D=64, B=32),
        # an ordinary decode batch, each sequence with a chain of five drafted tokens
        _case("tree", "tree_chain_batch64", S=64, lo=128, hi=2048, tlo=5, thi=5, Hq=32, Hkv=8, D=128, B=16, deep=5),
        # a batch of longer contexts with trees of up to 32 tokens: at most 128 query rows a kv head
        _case("tree", "tree_batch32", S=32, lo=512, hi=8192, tlo=16, thi=32, Hq=32, Hkv=8, D=128, B=16),
        # ragged in everything: an empty context, trees of one token, seven heads a kv head, 32-token blocks
        _case("tree", "tree_ragged", S=9, lo=0, hi=5000, tlo=1, thi=61, Hq=28, Hkv=4, D=128, B=32),
        # eight 32K-token contexts with trees of 64: 512 query rows a kv head, the most arithmetic
        _case("tree", "tree_64_32k", S=8, lo=32768, hi=32768, tlo=64, thi=64, Hq=64, Hkv=8, D=128, B=16),
        # one small tree against a 32000-token vocabulary
        _case("verify", "verify_single", S=1, tlo=8, thi=8, V=32000, bits=16),
        # fp32 logits of a vocabulary whose rows are aligned to nothing
        _case("verify", "verify_fp32_odd", S=16, tlo=1, thi=40, V=50001, bits=32),
        # a batch of 64 trees of 26 against a 128000-token vocabulary
        _case("verify", "verify_batch64", S=64, tlo=26, thi=26, V=128000, bits=16),
        # one sequence's accepted path, all layers of a 32-layer model
        _case("commit", "commit_single", S=1, lo=100, hi=100, tlo=16, thi=16, Hkv=8, D=128, B=16, L=32),
        # the accepted paths of a batch, all layers
        _case("commit", "commit_batch64", S=64, lo=20, hi=200, tlo=26, thi=26, Hkv=8, D=128, B=16, L=32),
        # long paths in large trees, few layers
        _case("commit", "commit_long", S=8, lo=1, hi=500, tlo=200, thi=256, Hkv=4, D=64, B=32, L=6, deep=100),
    ]


def _case(op, name=None, **sizes):
    c = dict(op=op, **sizes)
    if name:
        c["name"] = name
    return c


#: Most of the listed cases: keys times head_dim over all sequences and kv heads, multiply-adds, logits' bytes, pools' values.
MOST = 8 * 32768 * 8 * 128
MOST_FLOPS = 4 * MOST * 512
MOST_LOGITS = 64 * 26 * 128000 * 2
MOST_POOL = 1 << 29


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    thi = _log(rng, 1, 256 if op == "commit" else 64)
    tlo = rng.choice((thi, 1, max(1, thi // 2)))
    if op == "verify":
        S, V, bits = _log(rng, 1, 128), _log(rng, 1000, 160000), rng.choice((16, 32))
        while S * thi * V * bits // 8 > MOST_LOGITS:
            S, V = (S + 1) // 2, max(1000, V * 3 // 4)
        return _case(op, S=S, tlo=tlo, thi=thi, V=V, bits=bits)
    D, B, Hkv = rng.choice((64, 128)), rng.choice((16, 32)), rng.choice((1, 2, 4, 8))
    if op == "commit":
        S, hi, L = _log(rng, 1, 64), _log(rng, 1, 1000), _log(rng, 1, 64)
        while S * (hi + thi + 2 * B) * Hkv * D * L > MOST_POOL // 2:
            S, L, hi = (S + 1) // 2, (L + 1) // 2, max(1, hi * 3 // 4)
        return _case(op, S=S, lo=rng.choice((0, hi, 1 + hi // 2)), hi=hi, tlo=tlo, thi=thi, Hkv=Hkv, D=D, B=B, L=L)
    G = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    S, hi = _log(rng, 1, 128), _log(rng, 1, 32768)
    while S * (hi + thi + B) * Hkv * D > MOST // 2 or 4 * S * (hi + thi) * Hkv * D * thi * G > MOST_FLOPS // 2:
        S, hi = (S + 1) // 2, max(1, hi * 3 // 4)
    c = _case(op, S=S, lo=rng.choice((hi, 0, 1 + hi // 2)), hi=hi, tlo=tlo, thi=thi, Hq=Hkv * G, Hkv=Hkv, D=D, B=B)
    if rng.random() < 0.25:
        c["deep"] = thi  # chains
    return c


# ------------------------------------------------------------ the sizes of a case, whatever the seed
def _sizes(case):
    """Context lengths before the tree and numbers of nodes."""
    r = random.Random("%(S)d %(tlo)d %(thi)d" % case + " %d" % case.get("hi", 0))
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])] if "hi" in case else [0] * case["S"]
    if "hi" in case and case["S"] > 1:
        lens[:2] = case["lo"], case["hi"]
    return lens, [r.randint(case["tlo"], case["thi"]) for _ in range(case["S"])]


def _paths(case):
    """(accepted nodes, leading ones of them on the tree's first chain) of every sequence of a commit."""
    r = random.Random("path %(S)d %(thi)d" % case)
    out = []
    for t in _sizes(case)[1]:
        deep = _deep(case, t)
        k, m = (r.randint(1, deep), r.random()) if out else (deep, 0.0)  # the first one leaves its chain at the root
        out.append((k, max(1 + int(m * k), k - (t - deep))))
    return out


def _deep(case, t):
    """Length of a tree's longest chain."""
    return min(t, case.get("deep", 6))


def _parents(case, rng):
    """Parents of every sequence's nodes.  A drafter's tree: its most likely
    chain first, then branches off earlier nodes, none deeper than the chain."""
    out = []
    for t in _sizes(case)[1]:
        deep = _deep(case, t)
        parents, depth = [], []
        for i in range(t):
            p = i - 1
            while i >= deep:
                p = rng.randrange(i)
                if depth[p] + 1 < deep:
                    break
            parents.append(p)
            depth.append(0 if p < 0 else depth[p] + 1)
        out.append(parents)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, S = case["op"], case["S"]
    lens, nodes = _sizes(case)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0]
    for t in nodes:
        cu.append(cu[-1] + t)
    st = dict(case=case, lens_host=lens, nodes_host=nodes, cu_host=cu, cu=i32(cu), most=max(nodes))
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    if op != "commit":
        st["parents_host"] = _parents(case, rng)
        st["parents"] = i32([p for tree in st["parents_host"] for p in tree])
    if op == "verify":
        V, N = case["V"], cu[-1]
        x = torch.randn(N, V, generator=g, device="cuda", dtype=torch.bfloat16) * 3
        st["logits"] = x if case["bits"] == 16 else x.float() + 0.01 * torch.randn(N, V, generator=g, device="cuda")
        # about half of the drafted tokens are what the model says after their parent
        best = st["logits"].argmax(1)
        parent = torch.tensor([c + max(p, 0) for c, tree in zip(cu, st["parents_host"]) for p in tree], device="cuda")
        guess = torch.randint(0, V, (N,), generator=g, device="cuda")
        right = torch.rand(N, generator=g, device="cuda") < 0.5
        st["tokens"] = torch.where(right, best[parent], guess).to(torch.int32)
        return st
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    nblk = [-(-(c + t) // B) for c, t in zip(lens, nodes)]
    mb = max(nblk)
    num_blocks = sum(nblk) + max(4, sum(nblk) // 4)
    ids = torch.randperm(num_blocks, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    n = torch.tensor(nblk, device="cuda")
    i = torch.arange(mb, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + i
    st["tables"] = torch.where(i < n[:, None], ids[at.clamp(max=num_blocks - 1)], torch.zeros_like(ids[:1])).contiguous()
    st["lens"] = i32(lens)
    st["max_ctx"] = max(c + t for c, t in zip(lens, nodes))
    if op == "commit":
        L = case["L"]
        st["k"], st["v"] = normal(L, num_blocks, Hkv, B, D), normal(L, num_blocks, Hkv, B, D)
        st["k_pools"], st["v_pools"] = list(st["k"].unbind(0)), list(st["v"].unbind(0))
        paths = []
        for (k, m), t in zip(_paths(case), nodes):
            paths.append(list(range(m)) + sorted(rng.sample(range(_deep(case, t), t), k - m)))
        st["path_host"] = paths
        st["path"] = i32([p + [-1] * (st["most"] - len(p)) for p in paths])
        st["path_lens"] = i32([len(p) for p in paths])
        return st
    k = normal(num_blocks, Hkv, B, D)
    k *= 0.5 + torch.rand(Hkv, 1, D, generator=g, device="cuda").to(torch.bfloat16)  # channels of unlike sizes
    st["k"], st["v"] = k, normal(num_blocks, Hkv, B, D)
    st["q"] = normal(cu[-1], case["Hq"], D)
    st["scale"] = 1.0 / math.sqrt(D)
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


# ------------------------------------------------------------ the library's calls
def _own_tree(st):
    import paged_kv_cache_262_gb300 as pa
    return pa.paged_attention_decode_tree(st["q"], st["k"], st["v"], st["tables"], st["lens"], st["cu"], st["parents"],
                                          max_tree_nodes=st["most"], scale=st["scale"], max_context_len=st["max_ctx"],
                                          err_flag=st["err"])


def _own_verify(st):
    import paged_kv_cache_262_gb300 as pa
    return pa.verify_tree(st["logits"], st["tokens"], st["parents"], st["cu"], max_tree_nodes=st["most"],
                          err_flag=st["err"])


def _own_commit(st):
    import paged_kv_cache_262_gb300 as pa
    new_lens = pa.commit_tree(st["k_pools"], st["v_pools"], st["tables"], st["lens"], st["path"], st["path_lens"],
                              err_flag=st["err"])
    return new_lens, st["k"], st["v"]


_OWN = dict(tree=_own_tree, verify=_own_verify, commit=_own_commit)


# ------------------------------------------------------------ the plain forms
def _chains(parents, cu, most, deep):
    """[N][most]: whether a tree's node is on the node's own chain, none of which is longer than `deep`."""
    n = torch.arange(parents.shape[0], device=parents.device)
    first = cu[:-1].long()[torch.bucketize(n, cu[1:].long(), right=True)]
    at = n - first
    j = torch.arange(most, device=parents.device)
    seen = torch.zeros(parents.shape[0], most, dtype=torch.bool, device=parents.device)
    for _ in range(deep):
        seen |= at[:, None] == j
        at = torch.where(at >= 0, parents.long()[first + at.clamp(min=0)], at)
    return seen


def _plain_tree(st):
    case, B, D = st["case"], st["case"]["B"], st["case"]["D"]
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    out = torch.empty_like(st["q"])
    deep = max(_deep(case, t) for t in st["nodes_host"])
    chain = _chains(st["parents"], st["cu"], st["most"], deep)
    for s, (c, t) in enumerate(zip(st["lens_host"], st["nodes_host"])):
        n0, n1, n = st["cu_host"][s], st["cu_host"][s + 1], c + t
        blocks = st["tables"][s, :-(-n // B)].long()
        k = st["k"][blocks].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float()
        v = st["v"][blocks].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float()
        q = st["q"][n0:n1].float().view(t, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, t * G, D)
        x = (q @ k.transpose(1, 2)) * st["scale"]
        x = x.view(Hkv, t, G, n)
        x[..., c:] = torch.where(chain[n0:n1, None, :t], x[..., c:], torch.full_like(x[..., c:], -math.inf))
        x = torch.exp(x - x.amax(-1, keepdim=True))
        o = (x / x.sum(-1, keepdim=True)).view(Hkv, t * G, n) @ v
        out[n0:n1] = o.view(Hkv, t, G, D).permute(1, 0, 2, 3).reshape(t, Hkv * G, D).to(torch.bfloat16)
    return out


def _plain_verify(st):
    S, most = st["case"]["S"], st["most"]
    deep = max(_deep(st["case"], t) for t in st["nodes_host"])
    x, cu, parents = st["logits"], st["cu"].long(), st["parents"].long()
    best = x.amax(1, keepdim=True)
    v = torch.arange(x.shape[1], device=x.device, dtype=torch.int32)
    targets = torch.where(x == best, v, torch.full_like(v, x.shape[1])).amin(1)
    # the trees side by side, [S][most]
    i = torch.arange(most, device=x.device)
    there = i < (cu[1:] - cu[:-1])[:, None]
    n = (cu[:-1, None] + i).clamp(max=x.shape[0] - 1)
    par, tok, tgt = parents[n], st["tokens"][n], targets[n]
    node = torch.zeros(S, dtype=torch.int64, device=x.device)
    live = there[:, 0]
    path, count, last = [], torch.zeros_like(node), torch.full_like(tgt[:, 0], -1)
    for _ in range(deep):
        path.append(torch.where(live, node, torch.full_like(node, -1)))
        count += live
        said = tgt.gather(1, node[:, None])
        last = torch.where(live, said[:, 0], last)
        fits = there & (par == node[:, None]) & (tok == said) & live[:, None]
        nxt = torch.where(fits, i, torch.full_like(i, most)).amin(1)
        live = nxt < most
        node = torch.where(live, nxt, node)
    path = torch.nn.functional.pad(torch.stack(path, 1), (0, most - deep), value=-1)
    return targets, path.to(torch.int32), count.to(torch.int32), last


def _plain_commit(st):
    B, c, path = st["case"]["B"], st["lens"].long()[:, None], st["path"].long()
    i = torch.arange(path.shape[1], device=path.device)
    live = i < st["path_lens"].long()[:, None]
    # past the path: the first node once more, to its own place
    src = torch.where(live, path, path[:, :1]) + c
    to = torch.where(live, i, path[:, :1]) + c
    t = st["tables"].long()
    sb, db = t.gather(1, src // B), t.gather(1, to // B)
    for pool in (st["k"], st["v"]):
        pool[:, db, :, to % B] = pool[:, sb, :, src % B]
    return (st["lens"] + st["path_lens"]).to(torch.int32), st["k"], st["v"]


_PLAIN = dict(tree=_plain_tree, verify=_plain_verify, commit=_plain_commit)


# ------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, nodes = _sizes(case)
    S, N = case["S"], sum(nodes)
    if case["op"] == "verify":
        V, width = case["V"], case["bits"] // 8
        return {"bytes": N * V * width + 12 * N + 4 * (S + 1) + 4 * S * max(nodes) + 8 * S, "flops": N * V}
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    if case["op"] == "commit":
        moved = sum(k - m for k, m in _paths(case))
        rows = sum(k for k, _ in _paths(case))
        return {"bytes": 2 * case["L"] * Hkv * moved * 2 * D * 2 + 8 * rows + 12 * S, "flops": 0}
    keys = sum(lens) + N
    blocks = sum(-(-(c + t) // B) for c, t in zip(lens, nodes))
    seen = sum(t * (c + 1) for c, t in zip(lens, nodes))
    return {"bytes": Hkv * keys * D * 4 + 4 * N * case["Hq"] * D + 4 * blocks + 4 * N + 8 * S,
            "flops": 4 * D * case["Hq"] * seen}


# ------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, lens, nodes, cu = case["op"], st["lens_host"], st["nodes_host"], st["cu_host"]
    if op == "commit":
        return torch.tensor([c + len(p) for c, p in zip(lens, st["path_host"])], dtype=torch.int32), None, None
    if op == "verify":
        x = st["logits"].double().cpu()
        targets = torch.stack([torch.nonzero(row == row.max())[0, 0] for row in x]).to(torch.int32)
        path = torch.full((case["S"], st["most"]), -1, dtype=torch.int32)
        count, last = [], []
        tokens = st["tokens"].cpu().tolist()
        for s, tree in enumerate(st["parents_host"]):
            node, k = 0, 0
            while node is not None:
                path[s, k] = node
                k += 1
                said = int(targets[cu[s] + node])
                node = next((i for i, p in enumerate(tree) if p == node and tokens[cu[s] + i] == said), None)
            count.append(k)
            last.append(said)
        return targets, path, torch.tensor(count, dtype=torch.int32), torch.tensor(last, dtype=torch.int32)
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    out = torch.empty(cu[-1], Hq, D, dtype=torch.float64)
    for s, tree in enumerate(st["parents_host"]):
        c, n = lens[s], lens[s] + nodes[s]
        blocks = st["tables"][s, :-(-n // B)].long()
        chains = []
        for p in range(len(tree)):
            row = [False] * len(tree)
            while p >= 0:
                row[p] = True
                p = tree[p]
            chains.append(row)
        hidden = ~torch.tensor(chains, device="cuda")
        for h in range(Hkv):
            k = st["k"][blocks, h].reshape(-1, D)[:n].double()
            v = st["v"][blocks, h].reshape(-1, D)[:n].double()
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = (st["q"][cu[s]:cu[s + 1], g].double() @ k.t()) * st["scale"]
                z[:, c:].masked_fill_(hidden, -math.inf)
                out[cu[s]:cu[s + 1], g] = (torch.softmax(z, -1) @ v).cpu()
    return out
