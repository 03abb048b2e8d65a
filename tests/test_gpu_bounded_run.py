"""The bounded-cache operators as a serving loop uses them: prompts are turned
and cached, attended to and weighed, cut to the budget; then tokens are
decoded one by one, each turned with its own position, cached, attended to and
weighed, with a cut whenever the trigger is passed.  After every step each
operator is compared with its definition on the inputs it had, and at the end
every cached key must be the turned key of the token whose position its entry
carries."""
import numpy as np
import pytest
import torch

from bounded_util import Batch, decode_reference, evict_reference, prefill_reference, same_bits, within
from paged_kv_cache_226_gb300 import build, lib
from paged_kv_cache_226_gb300 import inputs as pin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    lib.load()
    d = torch.device("cuda:0")
    lib.read_device_errors(d)
    return d


def snapshot(k, v, tables, lens, hq, bs, q=None):
    """The device state as a Batch of the references."""
    x = Batch.__new__(Batch)
    x.k, x.v, x.tables, x.lens = k.cpu(), v.cpu(), tables.cpu(), lens.cpu()
    x.hq, x.hkv, x.d, x.bs, x.dtype, x.fp8 = hq, k.shape[2], k.shape[3], bs, k.dtype, False
    x.k_scale = x.v_scale = None
    x.width, x.tokens = tables.shape[1], tables.shape[1] * bs
    x.q, x.scale = (q.cpu() if q is not None else None), k.shape[3] ** -0.5
    return x


@pytest.mark.parametrize("dtype,hq,hkv,d,window", [(torch.float16, 8, 2, 64, 0), (torch.bfloat16, 12, 3, 128, 16)])
def test_serving_loop(dev, dtype, hq, hkv, d, window):
    bs, budget, trigger, sinks, recent = 16, 48, 56, 2, 12
    prompts = [150, 40, 97]
    B, steps, width = len(prompts), 24, 12
    g = torch.Generator().manual_seed(hq)
    pool = pin.BlockPool(64, bs, order=np.random.default_rng(3).permutation(64))
    alloc = pin.PagedKVAllocator(pool)
    inv, factor = lib.rope_frequencies(d, 10000.0, "yarn", 4.0, 64)
    inv = inv.to(dev)
    kc = torch.randn(64, bs, hkv, d, generator=g).to(dtype).to(dev)
    vc = torch.randn(64, bs, hkv, d, generator=g).to(dtype).to(dev)
    turned = [{} for _ in range(B)]                  # position -> turned key [Hkv][D]
    values = [{} for _ in range(B)]

    def new_tokens(counts, first):
        """Allocates and caches `counts` new tokens per sequence at positions from `first`."""
        T = sum(counts)
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(dtype).to(dev)
        q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
        pos = torch.cat([torch.arange(f, f + c) for f, c in zip(first, counts)])
        slots = torch.tensor([alloc.append_token(b) for b, c in enumerate(counts) for _ in range(c)])
        q = lib.rope_and_cache(q, k, v, pos.to(dev), slots.to(dev), inv, kc, vc, factor=factor)
        torch.cuda.synchronize(dev)
        flat_k, flat_v = kc.cpu().view(-1, hkv, d), vc.cpu().view(-1, hkv, d)
        at = 0
        for b, c in enumerate(counts):
            for i in range(c):
                turned[b][first[b] + i] = flat_k[slots[at]].clone()
                values[b][first[b] + i] = flat_v[slots[at]].clone()
                at += 1
        return q

    def tables():
        return torch.from_numpy(alloc.table_array(range(B), width)).to(dev)

    for b in range(B):
        alloc.add_sequence(b)
    weights = torch.zeros(B, hkv, width * bs, device=dev)
    positions = torch.zeros(B, hkv, width * bs, dtype=torch.int32, device=dev)
    q = new_tokens(prompts, [0] * B)
    tb = tables()
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    seen = lens.clone()
    start = torch.tensor([0, *prompts]).cumsum(0).to(torch.int32).to(dev)
    out = lib.prefill(q, kc, vc, tb, lens, start, d ** -0.5, max(prompts))
    lib.prefill_weights(q, kc, tb, lens, start, d ** -0.5, max(prompts), max(prompts), window=window,
                        weights=weights)
    torch.cuda.synchronize(dev)
    x = snapshot(kc, vc, tb, lens, hq, bs)
    ww, wb = prefill_reference(x, q.cpu(), prompts, window)
    within(weights, ww, wb, "prompt weights")
    assert bool(torch.isfinite(out).all())
    known = None

    def cut():
        nonlocal lens, known
        before = snapshot(kc, vc, tb, lens, hq, bs)
        want = evict_reference(before, weights.cpu(), positions.cpu(), seen.cpu(),
                               known.cpu() if known is not None else None, budget, trigger, sinks, recent)
        new, _, _ = lib.evict(kc, vc, tb, lens, seen, budget, weights, positions, known_lens=known,
                              trigger=trigger, sinks=sinks, recent=recent)
        torch.cuda.synchronize(dev)
        assert same_bits(kc, want[0]) and same_bits(vc, want[1]) and new.cpu().tolist() == want[4].tolist()
        live = (torch.arange(width * bs) < want[4][:, None, None]).expand(weights.shape)
        assert same_bits(weights.cpu()[live], want[2][live]) and same_bits(positions.cpu()[live], want[3][live])
        lens, known = new, new.clone()
        for b in range(B):
            alloc.truncate(b, int(new[b]))

    cut()
    cuts = 0
    for step in range(steps):
        q = new_tokens([1] * B, [int(s) for s in seen])
        tb, lens, seen = tables(), lens + 1, seen + 1
        before = weights.cpu().clone()
        out, _ = lib.decode_weights(q, kc, vc, tb, lens, d ** -0.5, trigger + 1, weights=weights)
        torch.cuda.synchronize(dev)
        x = snapshot(kc, vc, tb, lens, hq, bs, q)
        at = torch.arange(width * bs)
        clean = torch.where(at < lens.cpu()[:, None, None], before, torch.zeros_like(before))
        want, ww, ob, wb = decode_reference(x, clean)
        within(out, want, ob, f"step {step} out")
        got = torch.where(at < lens.cpu()[:, None, None], weights.cpu(), torch.zeros_like(before))
        within(got, ww, wb, f"step {step} weights")
        if int(lens.max()) > trigger:
            cuts += 1
        cut()
    assert cuts >= 2 and int(lens.max()) <= trigger
    # every cached entry is the token its position names, each position once per head
    flat_k, flat_v, pos, tb = kc.cpu().view(-1, hkv, d), vc.cpu().view(-1, hkv, d), positions.cpu(), tb.cpu()
    for b in range(B):
        n = int(lens[b])
        for h in range(hkv):
            here = pos[b, h, :n].tolist()
            assert len(set(here)) == n and max(here) == int(seen[b]) - 1
            assert set(range(sinks)) <= set(here) and set(range(int(seen[b]) - recent, int(seen[b]))) <= set(here)
            for i, t in enumerate(here):
                slot = int(tb[b, i // bs]) * bs + i % bs
                assert torch.equal(flat_k[slot, h], turned[b][t][h]) and torch.equal(flat_v[slot, h], values[b][t][h])
    assert pool.num_free == 64 - sum(max(1, -(-int(n) // bs)) for n in lens)
    assert lib.read_device_errors(dev) == 0


def _batch_on(dev, x, blocks=None, shift=0):
    """x's tensors on the device; with ``blocks`` in a pool of that many, x's blocks `shift` further on."""
    def pool(t):
        if blocks is None:
            return t.to(dev)
        big = torch.zeros((blocks, *t.shape[1:]), dtype=t.dtype, device=dev)
        big[shift:shift + t.shape[0]] = t.to(dev)
        return big
    return dict(k=pool(x.k), v=pool(x.v), tables=(x.tables + shift).to(dev), lens=x.lens.to(dev), q=x.q.to(dev))


def test_pool_offsets_past_32_bits(dev):
    """The operators on blocks at the far end of a pool of 2.3 G elements (byte
    offsets past 2^32, element offsets past 2^31) give what they give on the
    same blocks in a small pool, bit for bit."""
    hq, hkv, d, bs, far = 8, 8, 128, 16, 140_000
    x = Batch([700, 33, 300], hq, hkv, d, bs, torch.bfloat16, seed=31, stale=False, slack_width=0)
    small, big = _batch_on(dev, x), _batch_on(dev, x, far + x.k.shape[0], far)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(9, 24 * d, generator=g).to(torch.bfloat16).to(dev)
    q, k, v = (t.view(9, -1, d) for t in qkv.split([8 * d, 8 * d, 8 * d], dim=1))
    pos = torch.arange(9, device=dev) + 1000
    slots = torch.randperm(x.k.shape[0] * bs, generator=g)[:9].to(dev)
    inv = lib.rope_frequencies(d)[0].to(dev)
    w = x.state().nan_to_num(0.0).to(dev)
    start = torch.tensor([0, 40, 73, 100], dtype=torch.int32, device=dev)
    qc = torch.randn(100, hq, d, generator=g).to(torch.bfloat16).to(dev)
    got = []
    for m, first in ((small, 0), (big, far * bs)):
        turned = lib.rope_and_cache(q, k, v, pos, slots + first, inv, m["k"], m["v"])
        out, wd = lib.decode_weights(m["q"], m["k"], m["v"], m["tables"], m["lens"], x.scale, 700,
                                     weights=w, weights_out=torch.zeros_like(w))
        wp = lib.prefill_weights(qc, m["k"], m["tables"], m["lens"], start, x.scale, 40, 700, weights=w,
                                 weights_out=torch.zeros_like(w))
        new, we, pe = lib.evict(m["k"], m["v"], m["tables"], m["lens"], m["lens"], 200, w,
                                torch.zeros(w.shape, dtype=torch.int32, device=dev), sinks=2, recent=30,
                                weights_out=torch.zeros_like(w),
                                positions_out=torch.zeros(w.shape, dtype=torch.int32, device=dev))
        n = x.k.shape[0]
        lo = first // bs
        got.append((turned, out, wd, wp, new, we, pe, m["k"][lo:lo + n].clone(), m["v"][lo:lo + n].clone()))
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    for a, b in zip(*got):
        assert same_bits(a, b)
    assert int(big["k"][:far].count_nonzero()) == 0 and int(big["v"][:far].count_nonzero()) == 0


def test_a_step_in_one_graph(dev):
    """Write, attend, weigh and cut, captured once and replayed on new
    contents, equal the same calls made eagerly."""
    hq, hkv, d, bs, B = 8, 2, 64, 16, 4
    g = torch.Generator().manual_seed(77)
    x = Batch([70, 33, 64, 1], hq, hkv, d, bs, torch.float16, seed=77, stale=False, slack_width=1)
    width = x.tokens
    inv = lib.rope_frequencies(d)[0].to(dev)
    s = _batch_on(dev, x)
    s.update(qkv=torch.zeros(B, (hq + 2 * hkv) * d, dtype=torch.float16, device=dev),
             pos=torch.zeros(B, dtype=torch.int64, device=dev), slots=torch.zeros(B, dtype=torch.int64, device=dev),
             seen=x.lens.to(dev), known=torch.zeros(B, dtype=torch.int32, device=dev),
             w=torch.zeros(B, hkv, width, device=dev), p=torch.zeros(B, hkv, width, dtype=torch.int32, device=dev),
             turned=torch.zeros(B, hq, d, dtype=torch.float16, device=dev), out=torch.zeros(B, hq, d, dtype=torch.float16, device=dev),
             new=torch.zeros(B, dtype=torch.int32, device=dev))

    def step(m):
        q, k, v = (t.view(B, -1, d) for t in m["qkv"].split([hq * d, hkv * d, hkv * d], dim=1))
        lib.rope_and_cache(q, k, v, m["pos"], m["slots"], inv, m["k"], m["v"], q_out=m["turned"])
        lib.decode_weights(m["turned"], m["k"], m["v"], m["tables"], m["lens"], d ** -0.5, width,
                           weights=m["w"], out=m["out"])
        lib.evict(m["k"], m["v"], m["tables"], m["lens"], m["seen"], 32, m["w"], m["p"], known_lens=m["known"],
                  trigger=64, sinks=1, recent=8, new_lens=m["new"])

    def fill(m, seed):
        g.manual_seed(seed)
        lens = torch.randint(1, width + 1, (B,), generator=g).to(torch.int32)
        lens = torch.minimum(lens, x.lens + 15 - (x.lens - 1) % 16)          # within the blocks held
        m["k"].copy_(x.k), m["v"].copy_(x.v), m["lens"].copy_(lens), m["seen"].copy_(lens + 5)
        m["qkv"].copy_(torch.randn(m["qkv"].shape, generator=g))
        m["pos"].copy_(lens.long() + 4)
        at = (lens - 1).long()
        m["slots"].copy_(x.tables[torch.arange(B), at // bs].long() * bs + at % bs)
        m["known"].copy_((lens - 3).clamp(min=0))
        m["w"].copy_(torch.rand(m["w"].shape, generator=g)), m["p"].copy_(torch.arange(width).expand(m["p"].shape))

    fill(s, 1)
    step(s)                                              # set-up outside the capture
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    e = {n: t.clone() for n, t in s.items()}
    for seed in (2, 3, 4):
        fill(s, seed), fill(e, seed)
        graph.replay()
        step(e)
        torch.cuda.synchronize(dev)
        live = torch.arange(width, device=dev) < e["new"][:, None, None]
        for n in ("k", "v", "turned", "out", "new"):
            assert same_bits(s[n], e[n]), n
        for n in ("w", "p"):
            assert same_bits(torch.where(live, s[n], 0 * s[n]), torch.where(live, e[n], 0 * e[n])), n
    assert lib.read_device_errors(dev) == 0


def test_prefill_weights_on_two_streams(dev):
    """Two persistent launches at once, each with its own workspace."""
    xs = [Batch([900, 77], 8, 2, 128, 16, torch.float16, seed=s) for s in (41, 42)]
    qs = [torch.randn(400, 8, 128, generator=x.gen).to(torch.float16) for x in xs]
    start = torch.tensor([0, 323, 400], dtype=torch.int32, device=dev)
    on = [_batch_on(dev, x) for x in xs]
    qd = [q.to(dev) for q in qs]
    torch.cuda.synchronize(dev)
    streams = [torch.cuda.Stream(dev) for _ in xs]
    got = []
    for _ in range(3):
        got = []
        for x, m, q, s in zip(xs, on, qd, streams):
            with torch.cuda.stream(s):
                got.append(lib.prefill_weights(q, m["k"], m["tables"], m["lens"], start, x.scale, 323, 900))
    torch.cuda.synchronize(dev)
    for x, q, w in zip(xs, qs, got):
        ww, wb = prefill_reference(x, q, [323, 77])
        within(w, ww, wb, "weights")
    assert lib.read_device_errors(dev) == 0


def calls_of(dev, seed):
    """One call of each operator on a small batch, with every array given."""
    x = Batch([40, 33], 4, 2, 64, 16, torch.float16, seed=seed, stale=False)
    k, v, tables, lens = x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev)
    q = x.q.to(dev)
    new = q[:, :2].contiguous()
    i64 = torch.tensor([3, 20], device=dev)
    w, p = torch.zeros(2, 2, x.tokens, device=dev), torch.zeros(2, 2, x.tokens, dtype=torch.int32, device=dev)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    inv = lib.rope_frequencies(64)[0].to(dev)
    return {
        "rope": (lib.rope_and_cache, dict(q=q, k=new, v=new, positions=i64, slot_mapping=i64, inv_freq=inv,
                                          k_cache=k, v_cache=v, q_out=torch.empty_like(q))),
        "decode": (lib.decode_weights, dict(q=q, k_cache=k, v_cache=v, block_tables=tables, context_lens=lens,
                                            scale=x.scale, max_context_len=40, weights=w,
                                            weights_out=torch.zeros_like(w), out=torch.empty_like(q),
                                            workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))),
        "prefill": (lib.prefill_weights, dict(q=q, k_cache=k, block_tables=tables, context_lens=lens,
                                              query_start=start, scale=x.scale, max_query_len=1,
                                              max_context_len=40, weights=w, weights_out=torch.zeros_like(w),
                                              workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))),
        "evict": (lib.evict, dict(k_cache=k, v_cache=v, block_tables=tables, context_lens=lens, seen_lens=lens,
                                  budget=32, weights=w, positions=p, known_lens=torch.zeros_like(lens),
                                  weights_out=torch.zeros_like(w), positions_out=torch.zeros_like(p),
                                  new_lens=torch.empty_like(lens),
                                  workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))),
    }


@pytest.mark.parametrize("name,gives", [("rope", ["q_out"]), ("decode", ["out", "weights_out"]),
                                        ("prefill", ["weights_out"]),
                                        ("evict", ["new_lens", "weights_out", "positions_out"])])
def test_binding_returns_and_references(dev, name, gives):
    """The given outputs come back as they are; neither a call, nor one that
    makes its outputs, nor a refused one keeps or drops a reference or memory;
    what is not an int32 or a number is refused."""
    import gc
    import sys
    fn, args = calls_of(dev, seed=70)[name]
    got = fn(**args)
    got = got if isinstance(got, tuple) else (got,)
    assert len(got) == len(gives) and all(a is args[g] for a, g in zip(got, gives))
    del got
    fresh = {k: v for k, v in args.items() if k not in (*gives, "workspace")}
    made = fn(**fresh)
    made = made if isinstance(made, tuple) else (made,)
    for a, g in zip(made, gives):
        assert a.shape == args[g].shape and a.dtype == args[g].dtype and a.device == args[g].device
    del made
    scalar = {"rope": "factor", "decode": "max_context_len", "prefill": "window", "evict": "budget"}[name]
    bad = [{scalar: "x"}, {"k_cache": args["k_cache"].float()}, {"v_cache" if name != "prefill" else "q": None}]
    if name != "rope":
        bad += [{scalar: 1 << 40}, {scalar: 1.5}, {"workspace": torch.empty(64, dtype=torch.uint8)},
                {"workspace": torch.empty(1 << 20, dtype=torch.uint8, device=dev)[::2]}]
    def everything():
        fn(**args)
        fn(**fresh)
        for b in bad:
            with pytest.raises((TypeError, ValueError)):
                fn(**{**args, **b})
    for _ in range(3):
        everything()
    gc.collect()
    held = {k: sys.getrefcount(v) for k, v in args.items()}
    memory = torch.cuda.memory_allocated(dev)
    for _ in range(50):
        everything()
    gc.collect()
    assert {k: sys.getrefcount(v) for k, v in args.items()} == held
    assert torch.cuda.memory_allocated(dev) == memory
    assert lib.read_device_errors(dev) == 0


def test_calls_from_threads(dev):
    """The operators called from four threads, each on a stream of its own,
    give what one thread gets."""
    import threading
    def outcome(seed):
        made = []
        s = torch.cuda.Stream(dev)
        with torch.cuda.stream(s):
            sets = calls_of(dev, seed)
            for _ in range(20):
                for name in ("decode", "prefill"):
                    fn, args = sets[name]
                    got = fn(**{k: v for k, v in args.items() if k not in ("out", "weights_out", "weights", "workspace")})
                    made.append(tuple(got) if isinstance(got, tuple) else (got,))
            fn, args = sets["evict"]
            got = fn(**args)
            made.append(tuple(t.clone() for t in got[:1]) + (args["k_cache"].clone(),))
        s.synchronize()
        return [tuple(t.cpu() for t in m) for m in made]
    want = {seed: outcome(seed) for seed in range(80, 84)}
    got = {}
    threads = [threading.Thread(target=lambda i=seed: got.__setitem__(i, outcome(i))) for seed in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for seed in want:
        for a, b in zip(want[seed], got[seed]):
            assert all(same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fp8", [False, True])
def test_step_plan_behind_the_rotary_write(dev, fp8):
    """A decode step of turned keys: rope_and_cache and a weights plan without
    new keys, called and replayed in one graph, attend to the turned keys and
    leave them in the cache."""
    hq, hkv, d, bs = 8, 2, 128, 16
    x = Batch([300, 17, 64], hq, hkv, d, bs, torch.float16, seed=53, fp8=fp8, stale=False)
    qkv = torch.randn(3, (hq + 2 * hkv) * d, generator=x.gen).to(torch.float16).to(dev)
    q, k, v = (t.view(3, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    at = (x.lens - 1).long()
    slots = (x.tables[torch.arange(3), at // bs].long() * bs + at % bs).to(dev)
    pos, inv = (at + 1000).to(dev), lib.rope_frequencies(d)[0].to(dev)
    start = x.state().nan_to_num(0.0).to(dev)
    kc, vc, tables, lens = x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev)
    kr, vr = kc.clone(), vc.clone()
    turned = lib.rope_and_cache(q, k, v, pos, slots, inv, kr, vr, **x.scales())
    want = lib.decode_weights(turned, kr, vr, tables, lens, x.scale, 300, weights=start.clone(), **x.scales())
    w, tq = start.clone(), torch.empty_like(turned)
    plan = lib.StepPlan(tq, None, None, None, kc, vc, tables, lens, x.scale, 300, mode="weights", weights=w,
                        **x.scales())

    def turn():
        lib.rope_and_cache(q, k, v, pos, slots, inv, kc, vc, q_out=tq, **x.scales())

    turn()
    assert same_bits(plan(), want[0]) and same_bits(w, want[1]) and same_bits(kc, kr) and same_bits(vc, vr)
    plan.capture_graph(before=turn)
    kc.copy_(x.k), vc.copy_(x.v), w.copy_(start)
    assert same_bits(plan.replay(), want[0]) and same_bits(w, want[1]) and same_bits(kc, kr) and same_bits(vc, vr)
    args = (tq, k.contiguous(), v.contiguous(), slots, kc, vc, tables, lens, x.scale, 300)
    for bad in ((1,), (3,), (1, 2)):                     # all three or none
        with pytest.raises((ValueError, TypeError)):
            lib.StepPlan(*[None if i in bad else a for i, a in enumerate(args)], mode="weights", weights=w, **x.scales())
    with pytest.raises(ValueError):
        lib.StepPlan(*[None if i in (1, 2, 3) else a for i, a in enumerate(args)], mode="fused", **x.scales())
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
