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
