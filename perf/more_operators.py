"""What the operators of speculative decoding cost, and what they have to give.

A step verifies a small tree of drafted tokens per sequence over the paged
cache.  Node 0 of a tree is the sequence's newest token, every other node
names an earlier one as its parent; the nodes' keys and values stand behind the
context in the cache, in the tree's order.  Four operators:

  norm     each head's q and k normalised (RMS), rotary positions on one or
           more axes, keys and values written to their cache slots (16-bit or E4M3)
  tree     attention of the tree's nodes: each sees the context, its ancestors
           and itself
  accept   the longest path of drafted tokens that the model agrees with
  commit   the accepted path's rows close up behind the context, in the caches
           of all layers

``listed`` and ``draw`` give cases, ``prepare`` the inputs of one, ``run`` one
pass: in plain torch operations, or with ``own`` through the library.  All
sizes of a case follow from the case alone; the seed sets the values, the
shapes of the trees and which of their nodes are accepted.
"""
import math

import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_E4M3_MAX = 448.0
_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences: few rows, so the call itself is what is paid
        dict(name="norm decode step", op="norm", dtype="bf16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, tokens=64, far=2048, rotary=128, axes=1, cyclic=False,
             interleaved=False, base=1000000.0, padding=0),
        # packed prompts with images: time, height and width turn a share of the pairs each
        dict(name="norm image prompts", op="norm", dtype="bf16", fp8=False, heads=64, kv_heads=8,
             head_dim=128, block=16, tokens=8192, far=32768, rotary=128, axes=3, cyclic=False,
             interleaved=False, base=1000000.0, padding=0),
        # interleaved pairs over half of the head, an E4M3 cache, an odd count with padding rows
        dict(name="norm partial e4m3", op="norm", dtype="fp16", fp8=True, heads=32, kv_heads=8,
             head_dim=128, block=32, tokens=5001, far=8192, rotary=64, axes=2, cyclic=True,
             interleaved=True, base=10000.0, padding=13),
        # a handful of short contexts and small trees: latency
        dict(name="tree few short", op="tree", dtype="fp16", fp8=False, heads=6, kv_heads=2,
             head_dim=64, block=16, seqs=3, low=20, high=250, nodes=7, chain=False),
        # the usual serving batch
        dict(name="tree 64 ragged", op="tree", dtype="bf16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=64, low=128, high=2048, nodes=16, chain=False),
        # large trees on eight query heads to a KV head: 512 rows meet every key
        dict(name="tree 16 wide", op="tree", dtype="fp16", fp8=False, heads=64, kv_heads=8,
             head_dim=128, block=16, seqs=16, low=2048, high=8192, nodes=64, chain=False),
        # few long contexts
        dict(name="tree 4 long", op="tree", dtype="bf16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=4, low=32768, high=50000, nodes=60, chain=False),
        # a line of drafted tokens over an E4M3 cache, eight query heads to a KV head
        dict(name="tree 32 e4m3 line", op="tree", dtype="fp16", fp8=True, heads=64, kv_heads=8,
             head_dim=128, block=32, seqs=32, low=4096, high=4096, nodes=8, chain=True),
        # one sequence's small tree
        dict(name="accept one", op="accept", seqs=1, nodes=26, chain=False),
        # a large batch of large trees
        dict(name="accept 256", op="accept", seqs=256, nodes=64, chain=False),
        # one layer's cache of the usual batch
        dict(name="commit one layer", op="commit", dtype="fp16", fp8=False, kv_heads=8, head_dim=128,
             block=16, layers=1, seqs=64, low=128, high=2048, nodes=16),
        # every layer's cache of a smaller one
        dict(name="commit 32 layers", op="commit", dtype="bf16", fp8=False, kv_heads=8, head_dim=128,
             block=16, layers=32, seqs=16, low=64, high=512, nodes=26),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["norm", "tree", "tree", "accept", "commit"])
    if op == "accept":
        return dict(op=op, seqs=_spread(rng, 1, 256), nodes=_spread(rng, 1, 128),
                    chain=rng.random() < 0.3)
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), head_dim=rng.choice([64, 128, 128]),
             block=rng.choice([16, 32]))
    kv = rng.choice([1, 2, 4, 8])
    c.update(kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]))
    c["fp8"] = c["head_dim"] == 128 and rng.random() < 0.3
    if op == "norm":
        tokens = _spread(rng, 1, 8192)
        axes = rng.choice([1, 1, 2, 3, 4])
        c.update(tokens=tokens, far=max(tokens, _spread(rng, 256, 131072)),
                 rotary=rng.choice([r for r in (32, 48, 64, 96, 128) if r <= c["head_dim"]]),
                 axes=axes, cyclic=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                 base=rng.choice([10000.0, 1000000.0]),
                 padding=rng.choice([0, 0, rng.randrange(tokens)]))
        return c
    if op == "tree":
        seqs, nodes = _spread(rng, 1, 64), _spread(rng, 1, 128)
        most = min(50000, 160000 // seqs, 500_000_000 // (seqs * c["heads"] * nodes))
        high = _spread(rng, 17, max(18, most))
        c.update(seqs=seqs, low=rng.randrange(0, high + 1), high=high, nodes=nodes,
                 chain=rng.random() < 0.3)
        return c
    del c["heads"]
    layers, seqs = _spread(rng, 1, 32), _spread(rng, 1, 64)
    high = _spread(rng, 17, max(18, min(4096, 140000 // (layers * seqs))))
    c.update(layers=layers, seqs=seqs, low=rng.randrange(0, high + 1), high=high,
             nodes=_spread(rng, 1, 128))
    return c


def _lens(case):
    """The batch's context lengths, the drafted nodes among them: even steps from low to high."""
    n, low, high = case["seqs"], case["low"], case["high"]
    return [high if n == 1 else low + (high - low) * i // (n - 1) for i in range(n)]


def _nodes(case, lens=None):
    """Nodes of each sequence's tree: a little less for every other sequence."""
    n = case["nodes"]
    sizes = [max(1, n - (i % 2) * (n // 8)) for i in range(case["seqs"])]
    return sizes if lens is None else [min(s, most) for s, most in zip(sizes, lens)]


def _path_len(i, nodes):
    """Length of sequence i's accepted path in a commit: one to five nodes, now and then none."""
    return 0 if i % 17 == 16 else min(nodes, 1 + i % 5)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    e = 1 if case.get("fp8") else 2
    if case["op"] == "accept":
        nodes = sum(_nodes(case))
        return {"bytes": nodes * (8 + 8 + 4) + case["seqs"] * (4 * case["nodes"] + 4 + 4 + 8), "flops": 0}
    hkv, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "norm":
        t, live, hq = case["tokens"], case["tokens"] - case["padding"], case["heads"]
        return {"bytes": t * (2 * hq * d * 2 + 8 * case["axes"] + 8) + live * 2 * hkv * d * (2 + e),
                "flops": t * hq * (4 * d + case["rotary"] * 3) + live * hkv * (4 * d + case["rotary"] * 3)}
    lens = _lens(case)
    nodes = _nodes(case, lens)
    if case["op"] == "tree":
        hq = case["heads"]
        pairs = sum(c * (n - c) + c for c, n in zip(nodes, lens))       # the context, and itself
        return {"bytes": sum(lens) * hkv * 2 * d * e + 2 * sum(nodes) * hq * d * 2,
                "flops": 4 * pairs * hq * d}
    # node 0 leads every path and stays where it is; most of the others move
    moved = sum(max(0, _path_len(i, n) - 1) for i, n in enumerate(nodes))
    return {"bytes": case["layers"] * moved * 2 * 2 * hkv * d * e + case["seqs"] * (4 * case["nodes"] + 16),
            "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pool(case, blocks, gen, dev):
    """A cache that has been in use: every slot holds something."""
    shape = (blocks, case["block"], case["kv_heads"], case["head_dim"])
    if case["fp8"]:
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
        return (x * 8).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(_DTYPES[case["dtype"]])


def _tables(lens, block, gen, dev):
    """Scattered block tables of the lengths, and the pool's blocks."""
    need = [-(-n // block) for n in lens]
    width, total = max(1, max(need)), max(1, sum(need))
    blocks = total + total // 10 + 1
    order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    start = torch.tensor([0] + need, device=dev).cumsum(0)
    at = torch.arange(width, device=dev)[None, :]
    held = at < (start[1:] - start[:-1])[:, None]
    return torch.where(held, order[(start[:-1, None] + at).clamp(max=blocks - 1)],
                       torch.zeros((), dtype=torch.int32, device=dev)).contiguous(), blocks


def _trees(case, nodes, gen, dev):
    """(first node of each tree in the batch, parents inside the tree): every node but the first
    hangs below any earlier one, or below the one before it in a chain."""
    start = torch.tensor([0] + nodes, device=dev).cumsum(0).to(torch.int32)
    at = torch.arange(sum(nodes), device=dev)
    which = torch.repeat_interleave(torch.arange(len(nodes), device=dev), torch.tensor(nodes, device=dev))
    place = at - start[which]
    if case["chain"]:
        return start, (place - 1).to(torch.int32)
    u = torch.rand(sum(nodes), generator=gen, device=dev)
    parents = torch.minimum((u * place).long(), place - 1)
    return start, parents.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case, k_scale=5 / 32, v_scale=3 / 32)
    if case["op"] == "accept":
        nodes = _nodes(case)
        s["start"], s["parents"] = _trees(case, nodes, gen, dev)
        n = sum(nodes)
        # the model agrees with four drafted tokens of five
        s["target"] = torch.randint(0, 32000, (n,), generator=gen, device=dev)
        first = torch.repeat_interleave(s["start"][:-1].long(), torch.tensor(nodes, device=dev))
        wanted = s["target"][first + s["parents"].clamp(min=0)]
        other = torch.randint(0, 32000, (n,), generator=gen, device=dev)
        s["draft"] = torch.where(torch.rand(n, generator=gen, device=dev) < 0.8, wanted, other)
        return s
    dt = _DTYPES[case["dtype"]]
    hkv, d, block = case["kv_heads"], case["head_dim"], case["block"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    if case["op"] == "norm":
        t, hq, half = case["tokens"], case["heads"], case["rotary"] // 2
        blocks = -(-t // block) + 2
        # one projection's output, tokens and heads of different size
        qkv = normal(t, hq + 2 * hkv, d) * torch.exp(0.7 * normal(t, hq + 2 * hkv, 1))
        q, k, v = qkv.to(dt).view(t, -1).split([hq * d, hkv * d, hkv * d], dim=1)
        slots = torch.randperm(blocks * block, generator=gen, device=dev)[:t]
        if case["padding"]:
            slots[t - case["padding"]:] = -1
        # text runs on along every axis; the middle half is an image of rows of 64 patches
        begin = torch.randint(0, case["far"] - t + 1, (1,), generator=gen, device=dev)
        at = begin + torch.arange(t, device=dev)
        image = (torch.arange(t, device=dev) >= t // 4) & (torch.arange(t, device=dev) < t - t // 4)
        corner = begin + t // 4
        patch = (at - corner).clamp(min=0)
        axes = [at, corner + patch // 64, corner + patch % 64, corner + patch % 7][:case["axes"]]
        if case["axes"] > 1:
            axes[0] = torch.where(image, corner.expand(t), at)
        axes = [axes[0]] + [torch.where(image, a, at) for a in axes[1:]]
        pair = torch.arange(half, device=dev)
        s.update(q=q.view(t, hq, d), k=k.view(t, hkv, d), v=v.view(t, hkv, d), slots=slots,
                 positions=torch.stack(axes) if case["axes"] > 1 else at,
                 axes=(pair % case["axes"] if case["cyclic"] else pair * case["axes"] // half).to(torch.int32)
                 if case["axes"] > 1 else None,
                 inv_freq=(case["base"] ** (-pair.double() * 2 / case["rotary"])).float(),
                 q_weight=(1 + 0.3 * normal(d)).to(dt), k_weight=(1 + 0.3 * normal(d)).to(dt),
                 k_cache=_pool(case, blocks, gen, dev), v_cache=_pool(case, blocks, gen, dev))
        return s
    lens = _lens(case)
    nodes = _nodes(case, lens)
    s["tables"], blocks = _tables(lens, block, gen, dev)
    s.update(lens=torch.tensor(lens, dtype=torch.int32, device=dev), longest=max(lens),
             largest=max(1, max(nodes)))
    if case["op"] == "tree":
        s["start"], s["parents"] = _trees(case, nodes, gen, dev)
        s.update(q=normal(sum(nodes), case["heads"], d).to(dt), scale=1 / math.sqrt(d),
                 k_cache=_pool(case, blocks, gen, dev), v_cache=_pool(case, blocks, gen, dev))
        return s
    shape = (case["layers"], 2, blocks, block, hkv, d)
    s["caches"] = torch.empty(shape, dtype=torch.uint8 if case["fp8"] else dt, device=dev)
    for layer in range(case["layers"]):
        for kind in range(2):
            s["caches"][layer, kind] = _pool(case, blocks, gen, dev)
    s["k_caches"] = [s["caches"][layer, 0] for layer in range(case["layers"])]
    s["v_caches"] = [s["caches"][layer, 1] for layer in range(case["layers"])]
    s["start"] = torch.tensor([0] + nodes, device=dev).cumsum(0).to(torch.int32)
    # paths: node 0 and later nodes in the tree's order
    s["path_lens"] = torch.tensor([_path_len(i, n) for i, n in enumerate(nodes)], dtype=torch.int32, device=dev)
    at = torch.arange(s["largest"], device=dev)
    sizes = torch.tensor(nodes, device=dev)[:, None]
    rank = torch.rand((len(nodes), s["largest"]), generator=gen, device=dev)
    rank = torch.where(at == 0, rank - 1, rank + 2 * (at >= sizes))
    chosen = rank.argsort(dim=1)
    on = at < s["path_lens"][:, None]
    path = torch.where(on, chosen, torch.full_like(chosen, 1 << 20)).sort(dim=1).values
    s["path"] = torch.where(on, path, torch.full_like(path, -1)).to(torch.int32)
    s["new_lens"] = torch.zeros_like(s["lens"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"norm": _norm, "tree": _tree, "accept": _accept, "commit": _commit}[c["op"]](s, c)


def _own(s, c):
    from paged_kv_cache_226_gb300 import lib

    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if c.get("fp8") else {}
    if c["op"] == "norm":
        q = lib.norm_rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                                    s["k_cache"], s["v_cache"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=_EPS, axes=s["axes"],
                                    interleaved=c["interleaved"], **scales)
        return _written(s, c, q=q)
    if c["op"] == "tree":
        return {"out": lib.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                          s["start"], s["parents"], s["scale"], s["largest"],
                                          s["longest"], **scales)}
    if c["op"] == "accept":
        path, path_lens, following = lib.accept_tree(s["draft"], s["target"], s["parents"], s["start"],
                                                     c["nodes"])
        return {"path": path, "path_lens": path_lens, "next": following}
    new_lens = lib.commit_path(s["k_caches"], s["v_caches"], s["tables"], s["lens"], s["start"],
                               s["path"], s["path_lens"], new_lens=s["new_lens"])
    return {"caches": _numbered(s["caches"], c), "new_lens": new_lens}


def _numbered(cache, c):
    """E4M3 codes as the numbers they stand for."""
    return cache.view(torch.float8_e4m3fn) if c["fp8"] else cache


def _written(s, c, **more):
    return dict(more, k_cache=_numbered(s["k_cache"], c), v_cache=_numbered(s["v_cache"], c))


def _normed(x, weight):
    x = x.float()
    return x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * weight.float()


def _rotated(x, cos, sin, rotary, interleaved):
    turned, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rotary // 2], turned[..., rotary // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _norm(s, c):
    positions = s["positions"].double()
    place = positions[s["axes"].long()].T if s["axes"] is not None else positions[:, None]
    angle = place * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q = _rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["rotary"], c["interleaved"]).to(s["q"].dtype)
    k, v = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["rotary"], c["interleaved"]), s["v"]
    if c["fp8"]:
        k = (k / s["k_scale"]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / s["v_scale"]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    live = s["slots"] >= 0
    s["k_cache"].view(-1, c["kv_heads"], c["head_dim"])[s["slots"][live]] = k.to(s["k_cache"].dtype)[live]
    s["v_cache"].view(-1, c["kv_heads"], c["head_dim"])[s["slots"][live]] = v[live]
    return _written(s, c, q=q)


def _gathered(cache, s, c, scale):
    """[B][Hkv][tokens][D] in 32 bits through the block tables."""
    x = cache[s["tables"].long()].flatten(1, 2)
    if c["fp8"]:
        x = x.view(torch.float8_e4m3fn).float() * scale
    return x.float().transpose(1, 2)


def _padded(s, most):
    """(row of node i of sequence b in the batch, whether the sequence has it, its parent): [B][most]."""
    first, last = s["start"][:-1].long()[:, None], s["start"][1:].long()[:, None]
    at = first + torch.arange(most, device=first.device)
    live = at < last
    at = torch.where(live, at, torch.zeros_like(at))
    parent = torch.where(live, s["parents"][at].long(), torch.full_like(at, -1))
    return at, live, parent


def _ancestors(parent):
    """[B][n][n]: whether node j is node i or above it.  With P the matrix of parents, the sum of
    all its powers, as the inverse of I - P (whole numbers, no sum over 1)."""
    n = parent.shape[1]
    eye = torch.eye(n, device=parent.device)
    above = (parent[..., None] == torch.arange(n, device=parent.device)).float()
    return torch.linalg.solve_triangular(eye - above, eye.expand_as(above), upper=False, unitriangular=True) > 0.5


def _tree(s, c):
    g, d, n = c["heads"] // c["kv_heads"], c["head_dim"], s["largest"]
    if s["q"].shape[0] == 0:
        return {"out": torch.zeros_like(s["q"])}
    at, live, parent = _padded(s, n)
    k = _gathered(s["k_cache"], s, c, s["k_scale"])
    q = s["q"][at].float().view(c["seqs"], n, c["kv_heads"], g, d).permute(0, 2, 1, 3, 4)
    scores = (q.reshape(c["seqs"], c["kv_heads"], n * g, d) @ k.transpose(2, 3)) * s["scale"]
    scores = scores.view(c["seqs"], c["kv_heads"], n, g, -1)
    # context tokens, and of the tree's own the node's line
    base = (s["lens"].long() - (s["start"][1:] - s["start"][:-1]))[:, None, None]
    place = torch.arange(k.shape[2], device=k.device) - base
    line = _ancestors(parent).gather(2, place.clamp(0, n - 1).expand(-1, n, -1))
    seen = (place < 0) | ((place < n) & line)
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    e = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    p = (e / e.sum(dim=-1, keepdim=True)).view(c["seqs"], c["kv_heads"], n * g, -1)
    out = (p @ _gathered(s["v_cache"], s, c, s["v_scale"])).view(c["seqs"], c["kv_heads"], n, g, d)
    return {"out": out.permute(0, 2, 1, 3, 4)[live].reshape(s["q"].shape).to(s["q"].dtype)}


def _accept(s, c):
    n = c["nodes"]
    at, live, parent = _padded(s, n)
    draft, target = s["draft"][at], s["target"][at]
    place = torch.arange(n, device=at.device)
    agreed = torch.where(parent < 0, place == 0, draft == target.gather(1, parent.clamp(min=0)))
    line = _ancestors(parent)
    reached = live & ~(line & ~agreed[:, None, :]).any(dim=2)
    length = torch.where(reached, line.sum(dim=2), torch.zeros_like(at))
    best = (length * n + (n - 1 - place)).argmax(dim=1, keepdim=True)         # the first of the longest
    path_lens = length.gather(1, best)
    on = line.gather(1, best[..., None].expand(-1, 1, n))[:, 0]
    order = torch.sort(~on, dim=1, stable=True).indices
    path = torch.where(place < path_lens, order, torch.full_like(order, -1))
    following = torch.where(path_lens > 0, target.gather(1, best), torch.full_like(best, -1))[:, 0]
    return {"path": path.to(torch.int32), "path_lens": path_lens[:, 0].to(torch.int32), "next": following}


def _commit(s, c):
    block = c["block"]
    base = s["lens"].long() - (s["start"][1:] - s["start"][:-1])
    place = torch.arange(s["path"].shape[1], device=base.device)
    seq, nth = torch.nonzero(place < s["path_lens"][:, None], as_tuple=True)
    frm, to = base[seq] + s["path"][seq, nth], base[seq] + nth
    src = s["tables"][seq, frm // block].long() * block + frm % block
    dst = s["tables"][seq, to // block].long() * block + to % block
    rows = s["caches"].view(2 * c["layers"], -1, c["kv_heads"] * c["head_dim"])
    rows[:, dst] = rows[:, src]
    s["new_lens"].copy_(base + s["path_lens"])
    return {"caches": _numbered(s["caches"], c), "new_lens": s["new_lens"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "tree": _exact_tree, "accept": _exact_accept,
            "commit": _exact_commit}[case["op"]](s, case)


def _numbers(cache, fp8):
    return (cache.view(torch.float8_e4m3fn) if fp8 else cache).double()


def _exact_norm(s, c):
    r, t = c["rotary"], c["tokens"]
    f = s["inv_freq"].double()
    if s["axes"] is None:
        angle = torch.outer(s["positions"].double(), f)
    else:
        angle = torch.stack([s["positions"][a].double() * f[i] for i, a in enumerate(s["axes"].tolist())], dim=1)
    turn = torch.polar(torch.ones_like(angle), angle)

    def turned(x, weight):
        x = x.double()
        y = x * (x.square().sum(dim=2, keepdim=True) / c["head_dim"] + _EPS).rsqrt() * weight.double()
        real, imag = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(y[:, :, real], y[:, :, imag]) * turn[:, None, :]
        y[:, :, real], y[:, :, imag] = z.real, z.imag
        return y

    caches = {}
    for name, new, scale in (("k_cache", turned(s["k"], s["k_weight"]), s["k_scale"]),
                             ("v_cache", s["v"].double(), s["v_scale"])):
        y = _numbers(s[name], c["fp8"])
        flat = y.view(-1, c["kv_heads"], c["head_dim"])
        if c["fp8"]:
            new = (new / scale).clamp(-_E4M3_MAX, _E4M3_MAX)
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat[s["slots"][live]] = new[live]
        caches[name] = y
    return dict(caches, q=turned(s["q"], s["q_weight"]))


def _lines(parents):
    """Each node's own line, as lists of nodes from the root."""
    lines = []
    for i, p in enumerate(parents):
        lines.append((lines[p] if p >= 0 else []) + [i])
    return lines


def _exact_tree(s, c):
    g, d = c["heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    start, parents = s["start"].tolist(), s["parents"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        first, last = start[b], start[b + 1]
        if first == last:
            continue
        blocks = s["tables"][b, :-(-n // c["block"])].long()
        k, v = (_numbers(x[blocks], c["fp8"]).flatten(0, 1)[:n] * (scale if c["fp8"] else 1.0)
                for x, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        hidden = torch.ones((last - first, n), dtype=torch.bool)
        hidden[:, :n - (last - first)] = False
        for i, line in enumerate(_lines(parents[first:last])):
            hidden[i, [n - (last - first) + j for j in line]] = False
        hidden = hidden.to(k.device)
        for h in range(c["heads"]):
            scores = s["q"][first:last, h].double() @ k[:, h // g].T * s["scale"]
            out[first:last, h] = torch.softmax(scores.masked_fill(hidden, -math.inf), dim=1) @ v[:, h // g]
    return {"out": out}


def _exact_accept(s, c):
    start, parents = s["start"].tolist(), s["parents"].tolist()
    draft, target = s["draft"].tolist(), s["target"].tolist()
    paths, lengths, following = [], [], []
    for b in range(c["seqs"]):
        first, last = start[b], start[b + 1]
        best = []
        for line in _lines(parents[first:last]):
            right = line[0] == 0 and all(draft[first + j] == target[first + i] for i, j in zip(line, line[1:]))
            if right and len(line) > len(best):
                best = line
        paths.append(best + [-1] * (c["nodes"] - len(best)))
        lengths.append(len(best))
        following.append(target[first + best[-1]] if best else -1)
    return {"path": torch.tensor(paths, dtype=torch.int32), "path_lens": torch.tensor(lengths, dtype=torch.int32),
            "next": torch.tensor(following)}


def _exact_commit(s, c):
    """Nothing is computed here but copies: the same rows, one at a time."""
    block, caches = c["block"], _numbers(s["caches"], c["fp8"])
    rows = caches.view(2 * c["layers"], -1, c["kv_heads"] * c["head_dim"])
    tables, start = s["tables"].cpu(), s["start"].tolist()
    new_lens = []
    for b, n in enumerate(s["lens"].tolist()):
        base, count = n - (start[b + 1] - start[b]), int(s["path_lens"][b])
        for to, frm in enumerate(s["path"][b, :count].tolist()):
            src, dst = ((int(tables[b, (base + x) // block]) * block + (base + x) % block) for x in (frm, to))
            rows[:, dst] = rows[:, src].clone()
        new_lens.append(base + count)
    return {"caches": caches, "new_lens": torch.tensor(new_lens, dtype=torch.int32)}
