"""What the bounded-cache operators cost, and what they have to give.

Four operators keep a paged KV cache within a budget of tokens:

  rope      rotary positions on the new tokens' queries and keys, the keys and
            values written to their cache slots (16-bit or E4M3 cache)
  decode    one query token per sequence over the paged cache, which also adds
            to every cached token the attention weight that the query gave it
  prefill   the attention weights that a chunk's queries (all of them, or the
            last `window`) give to the cached tokens, added up per token
  evict     per (sequence, KV head): keep the first and the newest tokens and
            those of the largest weight, drop the rest, and close the gaps

``listed`` and ``draw`` give cases, ``prepare`` the inputs of one, ``run`` one
pass: in plain torch operations, or with ``own`` through the library.  All
sizes of a case follow from the case alone; the seed sets the values.
"""
import math

import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences: few rows, so the call itself is what is paid
        dict(name="rope decode step", op="rope", dtype="fp16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, tokens=64, far=2048, rotary=128, interleaved=False,
             base=10000.0, stretch=1.0, padding=0),
        # packed prompts of a long-context model (angles stretched, positions to 131072), q, k
        # and v being slices of one projection's output
        dict(name="rope packed prompts", op="rope", dtype="bf16", fp8=False, heads=64, kv_heads=8,
             head_dim=128, block=16, tokens=8192, far=131072, rotary=128, interleaved=False,
             base=500000.0, stretch=8.0, padding=0),
        # interleaved pairs over half of the head, an E4M3 cache, an odd count with padding rows
        dict(name="rope partial e4m3", op="rope", dtype="bf16", fp8=True, heads=32, kv_heads=8,
             head_dim=128, block=32, tokens=5001, far=8192, rotary=64, interleaved=True,
             base=10000.0, stretch=1.0, padding=13),
        # a handful of short contexts: latency
        dict(name="decode few short", op="decode", dtype="fp16", fp8=False, heads=8, kv_heads=2,
             head_dim=64, block=16, seqs=4, low=1, high=250),
        # the usual serving batch
        dict(name="decode 64 ragged", op="decode", dtype="fp16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=64, low=128, high=2048),
        # few long contexts
        dict(name="decode 8 long", op="decode", dtype="bf16", fp8=False, heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=8, low=32768, high=50000),
        # the same operator over an E4M3 cache, eight query heads to a KV head
        dict(name="decode 32 e4m3", op="decode", dtype="fp16", fp8=True, heads=64, kv_heads=8,
             head_dim=128, block=16, seqs=32, low=4096, high=4096),
        # short odd chunks, three query heads to a KV head
        dict(name="prefill short odd", op="prefill", dtype="fp16", heads=6, kv_heads=2,
             head_dim=64, block=16, seqs=3, low=20, high=250, chunk=19, window=0),
        # large chunks, one a whole prompt and one behind a long context, every query counted
        dict(name="prefill large chunks", op="prefill", dtype="bf16", heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=2, low=2048, high=16384, chunk=2048, window=0),
        # the last queries of each prompt judge the whole prompt
        dict(name="prefill last window", op="prefill", dtype="fp16", heads=32, kv_heads=8,
             head_dim=128, block=16, seqs=16, low=2048, high=8192, chunk=512, window=32),
        # the cut after the prompts: every sequence down to 1024 tokens
        dict(name="evict after prompts", op="evict", dtype="bf16", fp8=False, heads=32,
             kv_heads=8, head_dim=128, block=16, seqs=16, low=2048, high=8192, budget=1024,
             sinks=4, recent=256, known=False),
        # decoding at the budget: a block's worth of new tokens, as many to go
        dict(name="evict while decoding", op="evict", dtype="fp16", fp8=False, heads=32,
             kv_heads=8, head_dim=128, block=16, seqs=64, low=1040, high=1040, budget=1024,
             sinks=4, recent=256, known=True),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["rope", "decode", "prefill", "evict"])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), head_dim=rng.choice([64, 128, 128]),
             block=rng.choice([16, 32]))
    kv = rng.choice([1, 2, 4, 8])
    c.update(kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]))
    if op != "prefill":
        c["fp8"] = c["head_dim"] == 128 and rng.random() < 0.3
    if op == "rope":
        tokens = _spread(rng, 1, 8192)
        c.update(tokens=tokens, far=max(tokens, _spread(rng, 256, 131072)),
                 rotary=rng.choice([r for r in (32, 48, 64, 96, 128) if r <= c["head_dim"]]),
                 interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                 stretch=rng.choice([1.0, 4.0, 8.0]),
                 padding=rng.choice([0, 0, rng.randrange(tokens)]))
        return c
    if op == "decode":
        seqs = _spread(rng, 1, 64)
        high = _spread(rng, 17, max(18, min(50000, 400000 // seqs)))
        c.update(seqs=seqs, low=rng.randrange(0, high + 1), high=high)
        return c
    if op == "prefill":
        seqs = _spread(rng, 1, 8)
        high = _spread(rng, 17, max(18, min(16384, 32768 // seqs)))
        chunk = min(high, _spread(rng, 2, max(3, 65536 // (seqs * max(32, c["heads"])))))
        c.update(seqs=seqs, low=rng.randrange(0, high + 1), high=high, chunk=chunk,
                 window=rng.choice([0, 0, 1, 16, 32, 64]))
        return c
    seqs = _spread(rng, 1, 64)
    high = _spread(rng, 64, max(65, min(32768, 131072 // seqs)))
    budget = rng.randrange(16, high + 1)
    sinks = rng.randrange(0, 5)
    c.update(seqs=seqs, low=rng.randrange(0, high + 1), high=high, budget=budget, sinks=sinks,
             recent=rng.randrange(0, budget - sinks + 1), known=rng.random() < 0.5)
    return c


def _lens(case):
    """The batch's context lengths: even steps from low to high."""
    n, low, high = case["seqs"], case["low"], case["high"]
    return [high if n == 1 else low + (high - low) * i // (n - 1) for i in range(n)]


def _chunks(case, lens):
    """New tokens of each sequence: the chunk, a little less for every other sequence."""
    return [min(n, max(1, case["chunk"] - (i % 2) * (case["chunk"] // 16))) for i, n in enumerate(lens)]


def work(case):
    """Bytes and operations that one pass cannot do without."""
    e = 1 if case.get("fp8") else 2
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        t, live = case["tokens"], case["tokens"] - case["padding"]
        return {"bytes": t * (2 * hq * d * 2 + 8 + 8) + live * 2 * hkv * d * (2 + e),
                "flops": t * hq * case["rotary"] * 3 + live * hkv * case["rotary"] * 3}
    lens = _lens(case)
    total = sum(lens)
    if case["op"] == "decode":
        return {"bytes": total * hkv * (2 * d * e + 8) + 2 * case["seqs"] * hq * d * 2,
                "flops": 4 * total * hq * d}
    if case["op"] == "prefill":
        chunks = _chunks(case, lens)
        counted = [min(c, case["window"]) if case["window"] else c for c in chunks]
        pairs = sum(w * n - w * (w - 1) // 2 for w, n in zip(counted, lens))
        return {"bytes": total * hkv * (d * 2 + 8) + sum(counted) * hq * d * 2,
                "flops": 2 * pairs * hq * d}
    kept = [min(n, case["budget"]) for n in lens]
    moved = 0.0
    for n, k in zip(lens, kept):
        newest = min(case["recent"], n)
        rest = max(1, n - newest - case["sinks"])
        # of the tokens kept for their weight, those past the budget move; the newest all do,
        # but where the order is that of earlier cuts only the tokens added since
        past = (n - k) if case["known"] else max(0, n - max(k, n - newest))
        share = max(0, k - newest - case["sinks"]) * max(0, n - k - past) / rest
        moved += min(n - k, past + share) if n > k else 0
    return {"bytes": hkv * (sum(lens) * 4 + (sum(lens) * 4 if case["known"] else 0) + sum(kept) * 8 +
                            moved * 2 * 2 * d * e), "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inverse_frequencies(case):
    """1 / base^(2i/R), the slow half of them divided by `stretch` for long contexts."""
    half = case["rotary"] // 2
    f = case["base"] ** (-torch.arange(half, dtype=torch.float64) * 2 / case["rotary"])
    slow = torch.arange(half) >= half // 2
    return torch.where(slow, f / case["stretch"], f).float()


def _pool(case, blocks, gen, dev):
    """A cache that has been in use: every slot holds something."""
    shape = (blocks, case["block"], case["kv_heads"], case["head_dim"])
    if case.get("fp8"):
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


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = dict(case=case, k_scale=5 / 32, v_scale=3 / 32)
    if case["op"] == "rope":
        t, block = case["tokens"], case["block"]
        blocks = -(-t // block) + 2
        qkv = normal(t, (hq + 2 * hkv) * d)          # one projection's output
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        slots = torch.randperm(blocks * block, generator=gen, device=dev)[:t]
        if case["padding"]:
            slots[t - case["padding"]:] = -1
        start = torch.randint(0, case["far"] - t + 1, (1,), generator=gen, device=dev)
        s.update(q=q.view(t, hq, d), k=k.view(t, hkv, d), v=v.view(t, hkv, d), slots=slots,
                 positions=start + torch.arange(t, device=dev),
                 inv_freq=_inverse_frequencies(case).to(dev),
                 factor=1.0 if case["stretch"] == 1 else 0.1 * math.log(case["stretch"]) + 1,
                 k_cache=_pool(case, blocks, gen, dev), v_cache=_pool(case, blocks, gen, dev))
        return s
    lens = _lens(case)
    tables, blocks = _tables(lens, case["block"], gen, dev)
    width = tables.shape[1] * case["block"]
    context_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    s.update(tables=tables, lens=context_lens, longest=max(lens), scale=1 / math.sqrt(d),
             k_cache=_pool(case, blocks, gen, dev))
    # attention weights gathered so far: a few heavy tokens, many light ones, some at zero
    seen = torch.randn((case["seqs"], hkv, width), generator=gen, device=dev, dtype=torch.float32)
    s["weights"] = torch.where(seen < -1.5, torch.zeros_like(seen), torch.exp(2 * seen))
    s["weights_out"] = torch.zeros_like(s["weights"])
    if case["op"] == "prefill":
        chunks = _chunks(case, lens)
        s.update(q=normal(sum(chunks), hq, d), longest_chunk=max(chunks),
                 query_start=torch.tensor([0] + chunks, device=dev).cumsum(0).to(torch.int32))
        return s
    s["v_cache"] = _pool(case, blocks, gen, dev)
    if case["op"] == "decode":
        s["q"] = normal(case["seqs"], hq, d)
        return s
    s["positions"] = torch.zeros(s["weights"].shape, dtype=torch.int32, device=dev)
    s["positions_out"] = torch.zeros_like(s["positions"])
    s["new_lens"] = torch.zeros_like(context_lens)
    s["known_lens"], s["seen_lens"] = None, context_lens.clone()
    if case["known"]:
        # earlier cuts left the tokens up to the last block in the order in which gaps were
        # closed: some of the first 3 L positions, the newest among them
        added = torch.minimum(context_lens, torch.full_like(context_lens, case["block"]))
        s["known_lens"] = context_lens - added
        s["seen_lens"] = 3 * context_lens + added
        old = 3 * context_lens
        places = 3 * max(1, max(lens))
        at = torch.arange(places, device=dev)
        rank = torch.rand((case["seqs"], hkv, places), generator=gen, device=dev)
        rank += 2 * (at >= (old - case["recent"])[:, None, None]).float()
        rank -= 9 * (at >= old[:, None, None]).float()
        picked = rank.argsort(dim=2, descending=True)[:, :, :width]
        known = s["known_lens"][:, None, None]
        inside = torch.arange(width, device=dev) < known
        mix = torch.rand(s["weights"].shape, generator=gen, device=dev)[:, :, :picked.shape[2]]
        mixed = torch.where(inside[:, :, :picked.shape[2]], mix, mix + 2).argsort(dim=2)
        s["positions"][:, :, :picked.shape[2]] = picked.gather(2, mixed).to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"rope": _rope, "decode": _decode, "prefill": _prefill, "evict": _evict}[c["op"]](s, c)


def _own(s, c):
    from paged_kv_cache_226_gb300 import lib

    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if c.get("fp8") else {}
    if c["op"] == "rope":
        q = lib.rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                               s["k_cache"], s["v_cache"], interleaved=c["interleaved"],
                               factor=s["factor"], **scales)
        return _written(s, c, q=q)
    if c["op"] == "decode":
        out, weights = lib.decode_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                          s["scale"], s["longest"], weights=s["weights"],
                                          weights_out=s["weights_out"], **scales)
        return {"out": out, "weights": weights}
    if c["op"] == "prefill":
        return {"weights": lib.prefill_weights(
            s["q"], s["k_cache"], s["tables"], s["lens"], s["query_start"], s["scale"],
            s["longest_chunk"], s["longest"], window=c["window"], weights=s["weights"],
            weights_out=s["weights_out"])}
    new_lens, weights, positions = lib.evict(
        s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["seen_lens"], c["budget"],
        s["weights"], s["positions"], known_lens=s["known_lens"], sinks=c["sinks"],
        recent=c["recent"], weights_out=s["weights_out"], positions_out=s["positions_out"],
        new_lens=s["new_lens"])
    return _written(s, c, new_lens=new_lens, weights=weights, positions=positions)


def _written(s, c, **more):
    """The caches beside the other outputs; E4M3 codes as the numbers they stand for."""
    k, v = s["k_cache"], s["v_cache"]
    if c["fp8"]:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return dict(more, k_cache=k, v_cache=v)


def _rotated(x, cos, sin, rotary, interleaved):
    x = x.float()
    turned, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rotary // 2], turned[..., rotary // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _rope(s, c):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos = (angle.cos() * s["factor"]).float()[:, None, :]
    sin = (angle.sin() * s["factor"]).float()[:, None, :]
    q = _rotated(s["q"], cos, sin, c["rotary"], c["interleaved"]).to(s["q"].dtype)
    k, v = _rotated(s["k"], cos, sin, c["rotary"], c["interleaved"]), s["v"]
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
    if c.get("fp8"):
        x = x.view(torch.float8_e4m3fn).float() * scale
    return x.float().transpose(1, 2)


def _shares(scores, seen):
    """softmax over the last axis of what is seen; rows that see nothing are zero."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(dim=-1, keepdim=True).clamp(min=1e-30)


def _added(s, new, first_new):
    """weights_out: what was there before the new tokens, plus `new`, up to each length."""
    at = torch.arange(new.shape[2], device=new.device)
    before = torch.where(at < first_new[:, None, None], s["weights"], torch.zeros_like(new))
    s["weights_out"].copy_(torch.where(at < s["lens"][:, None, None], before + new, s["weights_out"]))
    return s["weights_out"]


def _decode(s, c):
    b, g = c["seqs"], c["heads"] // c["kv_heads"]
    k = _gathered(s["k_cache"], s, c, s["k_scale"])
    q = s["q"].float().view(b, c["kv_heads"], g, c["head_dim"])
    seen = torch.arange(k.shape[2], device=k.device) < s["lens"][:, None, None, None]
    p = _shares((q @ k.transpose(2, 3)) * s["scale"], seen)
    out = p @ _gathered(s["v_cache"], s, c, s["v_scale"])
    return {"out": out.to(s["q"].dtype).view(b, c["heads"], c["head_dim"]),
            "weights": _added(s, p.sum(dim=2), s["lens"] - 1)}


def _prefill(s, c):
    b, g, d = c["seqs"], c["heads"] // c["kv_heads"], c["head_dim"]
    first, last = s["query_start"][:-1].long(), s["query_start"][1:].long()
    rows = min(c["window"], s["longest_chunk"]) if c["window"] else s["longest_chunk"]
    back = torch.arange(rows, device=first.device)              # 0: a chunk's last query
    at = last[:, None] - 1 - back                               # [B][rows]
    live = at >= first[:, None]
    q = s["q"][at.clamp(min=0)].float().view(b, rows, c["kv_heads"], g, d).permute(0, 2, 3, 1, 4)
    k = _gathered(s["k_cache"], s, c, 1.0)
    key = torch.arange(k.shape[2], device=k.device)
    seen = (key <= (s["lens"][:, None] - 1 - back)[..., None]) & live[..., None]
    scores = q.reshape(b, c["kv_heads"], g * rows, d) @ k.transpose(2, 3)
    p = _shares(scores.view(b, c["kv_heads"], g, rows, -1) * s["scale"], seen[:, None, None])
    return {"weights": _added(s, p.sum(dim=(2, 3)), s["lens"] - (last - first))}


def _evict(s, c):
    b, hkv, d, block = c["seqs"], c["kv_heads"], c["head_dim"], c["block"]
    w, lens, width = s["weights"], s["lens"][:, None, None], s["weights"].shape[2]
    at = torch.arange(width, device=w.device).expand(b, hkv, width)
    known = s["known_lens"][:, None, None] if s["known_lens"] is not None else torch.zeros_like(lens)
    seen = s["seen_lens"][:, None, None]
    positions = torch.where(at < known, s["positions"].long(), at + seen - lens)
    # first to go is last in this order: past the length, then by weight, the safe ones in front
    rank = torch.where((positions < c["sinks"]) | (positions >= seen - c["recent"]),
                       torch.full_like(w, math.inf), w)
    rank = torch.where(at < lens, rank, torch.full_like(w, -math.inf))
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    left = lens.clamp(max=c["budget"]).long()
    keep = torch.zeros_like(order, dtype=torch.bool).scatter_(2, order, at < left)
    hole, mover = ~keep & (at < left), keep & (at >= left)
    # the n-th kept token past the budget goes to the n-th gap
    count = mover.sum(dim=2, keepdim=True)
    to = torch.sort(~hole, dim=2, stable=True).indices
    frm = torch.sort(~mover, dim=2, stable=True).indices
    pair, head, nth = torch.nonzero(at < count, as_tuple=True)
    to, frm = to[pair, head, nth], frm[pair, head, nth]
    slots = s["tables"].long()
    src = slots[pair, frm // block] * block + frm % block
    dst = slots[pair, to // block] * block + to % block
    for cache in (s["k_cache"], s["v_cache"]):
        rows = cache.view(-1, hkv, d)
        rows[dst, head] = rows[src, head]
    for old, out in ((w, s["weights_out"]), (positions.int(), s["positions_out"])):
        out.copy_(torch.where(at < left, old, out))
        out[pair, head, to] = old[pair, head, frm]
    s["new_lens"].copy_(left.view(-1))
    return _written(s, c, new_lens=s["new_lens"], weights=s["weights_out"], positions=s["positions_out"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "decode": _exact_decode, "prefill": _exact_prefill,
            "evict": _exact_evict}[case["op"]](s, case)


def _numbers(cache, fp8):
    return (cache.view(torch.float8_e4m3fn) if fp8 else cache).double()


def _exact_rope(s, c):
    r = c["rotary"]
    turn = torch.polar(torch.tensor(s["factor"], dtype=torch.float64, device=s["q"].device).expand(len(s["positions"]), r // 2),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))

    def turned(x):
        x = x.double()
        y = x.clone()
        real, imag = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(x[:, :, real], x[:, :, imag]) * turn[:, None, :]
        y[:, :, real], y[:, :, imag] = z.real, z.imag
        return y

    caches = {}
    for name, new, scale in (("k_cache", turned(s["k"]), s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        y = _numbers(s[name], c["fp8"])
        flat = y.view(-1, c["kv_heads"], c["head_dim"])
        if c["fp8"]:
            new = (new / scale).clamp(-_E4M3_MAX, _E4M3_MAX)
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat[s["slots"][live]] = new[live]
        caches[name] = y
    return dict(caches, q=turned(s["q"]))


def _exact_sequence(cache, s, c, b, scale):
    """[Hkv][L][D] of sequence b in 64 bits."""
    n = int(s["lens"][b])
    blocks = s["tables"][b, :-(-n // c["block"])].long()
    return (_numbers(cache[blocks], c.get("fp8")).flatten(0, 1)[:n] * scale).transpose(0, 1)


def _exact_decode(s, c):
    g = c["heads"] // c["kv_heads"]
    ks, vs = (s["k_scale"], s["v_scale"]) if c["fp8"] else (1.0, 1.0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    weights = s["weights_out"].double()
    for b in range(c["seqs"]):
        n = int(s["lens"][b])
        if n == 0:
            continue
        k, v = _exact_sequence(s["k_cache"], s, c, b, ks), _exact_sequence(s["v_cache"], s, c, b, vs)
        q = s["q"][b].double().view(c["kv_heads"], g, -1)
        p = torch.softmax(torch.einsum("hgd,hld->hgl", q, k) * s["scale"], dim=2)
        out[b] = torch.einsum("hgl,hld->hgd", p, v).reshape(c["heads"], -1)
        weights[b, :, :n] = p.sum(dim=1)
        weights[b, :, :n - 1] += s["weights"][b, :, :n - 1].double()
    return {"out": out, "weights": weights}


def _exact_prefill(s, c):
    g = c["heads"] // c["kv_heads"]
    weights = s["weights_out"].double()
    start = s["query_start"].tolist()
    for b in range(c["seqs"]):
        n, new = int(s["lens"][b]), start[b + 1] - start[b]
        if n == 0:
            continue
        counted = min(new, c["window"]) if c["window"] else new
        k = _exact_sequence(s["k_cache"], s, c, b, 1.0)
        q = s["q"][start[b + 1] - counted:start[b + 1]].double()
        hidden = torch.ones((counted, n), dtype=torch.bool, device=q.device).triu(n - counted + 1)
        sums = torch.zeros((c["kv_heads"], n), dtype=torch.float64, device=q.device)
        for h in range(c["heads"]):
            scores = torch.einsum("td,ld->tl", q[:, h], k[h // g]) * s["scale"]
            sums[h // g] += torch.softmax(scores.masked_fill(hidden, -math.inf), dim=1).sum(dim=0)
        sums[:, :n - new] += s["weights"][b, :, :n - new].double()
        weights[b, :, :n] = sums
    return {"weights": weights}


def _exact_evict(s, c):
    """Nothing is computed here but copies: the same places, found one list at a time."""
    if c["seqs"] * c["kv_heads"] * s["weights"].shape[2] > 4_000_000:
        return None
    block, fp8 = c["block"], c["fp8"]
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    weights, positions = s["weights_out"].cpu().clone(), s["positions_out"].cpu().clone()
    w, known_at, tables = s["weights"].cpu(), s["positions"].cpu(), s["tables"].cpu().long()
    lens, seen = s["lens"].tolist(), s["seen_lens"].tolist()
    known = s["known_lens"].tolist() if s["known_lens"] is not None else [0] * c["seqs"]
    moves = []
    for b in range(c["seqs"]):
        n, left = lens[b], min(lens[b], c["budget"])
        for h in range(c["kv_heads"]):
            place = known_at[b, h, :known[b]].tolist() + list(range(known[b] + seen[b] - n, seen[b]))
            value = w[b, h, :n].tolist()
            order = sorted(range(n), key=lambda i: (
                -math.inf if place[i] < c["sinks"] or place[i] >= seen[b] - c["recent"] else -value[i], i))
            kept = set(order[:left])
            gaps = [i for i in range(left) if i not in kept]
            movers = [i for i in range(left, n) if i in kept]
            line = list(range(left))
            for to, frm in zip(gaps, movers):
                line[to] = frm
                moves.append((b, h, frm, to))
            weights[b, h, :left] = torch.tensor([value[i] for i in line])
            positions[b, h, :left] = torch.tensor([place[i] for i in line], dtype=torch.int32)
    if moves:
        m = torch.tensor(moves)
        src = (tables[m[:, 0], m[:, 2] // block] * block + m[:, 2] % block).to(k.device)
        dst = (tables[m[:, 0], m[:, 3] // block] * block + m[:, 3] % block).to(k.device)
        head = m[:, 1].to(k.device)
        for cache in (k, v):
            rows = cache.view(-1, c["kv_heads"], c["head_dim"])
            rows[dst, head] = rows[src, head].clone()
    left = torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32)
    return {"k_cache": _numbers(k, fp8), "v_cache": _numbers(v, fp8), "weights": weights.double(),
            "positions": positions, "new_lens": left}
