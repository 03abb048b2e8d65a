"""The operators of speculative decoding as a serving loop uses them: prompts
are cached, then every step drafts a tree per sequence, caches and attends to it
in each layer, accepts a path and commits it in all layers at once.  Every
operator is compared with its definition on the inputs it had, and at the end
the caches must hold the accepted tokens in order.  Besides: the step in one
graph, pools past 32 bits, threads, and waits that run out."""
import threading

import numpy as np
import pytest
import torch

from bounded_util import Batch, same_bits, within
from paged_kv_cache_226_gb300 import build, lib
from paged_kv_cache_226_gb300 import inputs as pin
from test_gpu_bounded_run import _batch_on
from test_gpu_bounded_wait_timeout import test_lib, timed_out_then_right  # noqa: F401
from tree_util import accept_reference, commit_reference, lines, random_parents, starts, tree_reference

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


def snapshot(k, v, tables, lens, hq, bs, dtype, scales):
    """The device state as a Batch of the references."""
    x = Batch.__new__(Batch)
    x.k, x.v, x.tables, x.lens = k.cpu(), v.cpu(), tables.cpu(), lens.cpu()
    x.hq, x.hkv, x.d, x.bs, x.dtype = hq, k.shape[2], k.shape[3], bs, dtype
    x.fp8 = k.dtype == torch.uint8
    x.k_scale, x.v_scale = scales.get("k_scale"), scales.get("v_scale")
    x.width, x.tokens = tables.shape[1], tables.shape[1] * bs
    x.scale = k.shape[3] ** -0.5
    return x


@pytest.mark.parametrize("dtype,hq,hkv,d,fp8", [(torch.float16, 6, 2, 64, False), (torch.bfloat16, 8, 2, 128, False),
                                                (torch.float16, 16, 2, 128, True)])
def test_serving_loop(dev, dtype, hq, hkv, d, fp8):
    layers, bs, width, steps = 3, 16, 16, 5
    prompts, sizes = [150, 9, 0, 97], [12, 26, 7, 1]
    B = len(prompts)
    g = torch.Generator().manual_seed(hq)
    pool = pin.BlockPool(80, bs, order=np.random.default_rng(3).permutation(80))
    alloc = pin.PagedKVAllocator(pool)
    inv = lib.rope_frequencies(d, 10000.0)[0].to(dev)
    axes = (torch.arange(d // 2) % 2).to(torch.int32).to(dev)
    weights = [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype).to(dev) for _ in range(2)]
    scales = dict(k_scale=0.03, v_scale=0.02) if fp8 else {}
    make = (lambda: torch.randint(0, 120, (80, bs, hkv, d), generator=g, dtype=torch.uint8).to(dev)) if fp8 else \
        (lambda: torch.randn(80, bs, hkv, d, generator=g).to(dtype).to(dev))
    ks, vs = [make() for _ in range(layers)], [make() for _ in range(layers)]
    held = [[] for _ in range(B)]                    # of each sequence: (K row, V row) per layer of every token

    def rows(slots):
        return [(k.view(-1, hkv, d)[slots].cpu(), v.view(-1, hkv, d)[slots].cpu()) for k, v in zip(ks, vs)]

    def cache(counts, depths, first):
        """New tokens of every layer; returns their turned q, per layer, and their slots."""
        T = sum(counts)
        slots = torch.tensor([alloc.append_token(b) for b, c in enumerate(counts) for _ in range(c)]).to(dev)
        pos = torch.cat([torch.tensor([f + x for x in depths[b]], dtype=torch.int64) for b, f in enumerate(first)])
        pos = torch.stack([pos, pos // 2]).to(dev)
        qs = []
        for k, v in zip(ks, vs):
            qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(dtype).to(dev)
            q, kn, vn = (t.view(T, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
            qs.append(lib.norm_rope_and_cache(q, kn, vn, pos, slots, inv, k, v, *weights, axes=axes, **scales))
        return qs, slots

    for b in range(B):
        alloc.add_sequence(b)
    _, slots = cache(prompts, [list(range(n)) for n in prompts], [0] * B)
    at = 0
    for b, n in enumerate(prompts):
        per_layer = rows(slots[at:at + n])
        held[b] = [[(kk[i], vv[i]) for kk, vv in per_layer] for i in range(n)]
        at += n
    lens = torch.tensor(prompts, dtype=torch.int32)
    for step in range(steps):
        nodes = [max(1, s - step) if (b + step) % 4 else s for b, s in enumerate(sizes)]
        parents = random_parents(nodes, g)
        depths, at = [], 0
        for c in nodes:
            depths.append([len(x) - 1 for x in lines(parents[at:at + c].tolist())])
            at += c
        qs, slots = cache(nodes, depths, lens.tolist())
        full = (lens + torch.tensor(nodes, dtype=torch.int32)).to(dev)
        tables = torch.from_numpy(alloc.table_array(range(B), width)).to(dev)
        start, par = starts(nodes).to(dev), parents.to(dev)
        for k, v, q in zip(ks, vs, qs):
            out = lib.tree_attention(q, k, v, tables, full, start, par, d ** -0.5, max(nodes), int(full.max()), **scales)
            torch.cuda.synchronize(dev)
            want, bound = tree_reference(snapshot(k, v, tables, full, hq, bs, dtype, scales), q.cpu(), nodes, parents)
            within(out, want, bound, f"step {step}")
        target = torch.randint(0, 3, (sum(nodes),), generator=g)
        draft = torch.randint(0, 3, (sum(nodes),), generator=g)
        path, n, following = lib.accept_tree(draft.to(dev), target.to(dev), par, start, max(nodes))
        for a, w in zip((path, n, following), accept_reference(draft, target, parents, nodes, max(nodes))):
            assert same_bits(a, w)
        per_layer = rows(slots)
        pools = [t.cpu() for t in (*ks, *vs)]
        wanted, new = commit_reference(pools, tables.cpu(), full.cpu(), nodes, path.cpu(), n.cpu(), bs)
        got = lib.commit_path(ks, vs, tables, full, start, path, n)
        assert same_bits(got, new)
        for a, w in zip((*ks, *vs), wanted):
            assert same_bits(a, w)
        at = 0
        for b, c in enumerate(nodes):
            held[b] += [[(kk[at + i], vv[at + i]) for kk, vv in per_layer] for i in path[b, :int(n[b])].tolist()]
            alloc.truncate(b, int(new[b]))
            at += c
        lens = new
    assert lib.read_device_errors(dev) == 0
    tables = torch.from_numpy(alloc.table_array(range(B), width))
    for b in range(B):
        assert len(held[b]) == int(lens[b]) > prompts[b]
        for i, per_layer in enumerate(held[b]):
            slot = int(tables[b, i // bs]), i % bs
            for (kk, vv), k, v in zip(per_layer, ks, vs):
                assert same_bits(k[slot], kk) and same_bits(v[slot], vv), f"token {i} of sequence {b}"


def test_a_step_in_one_graph(dev):
    """Write, attention, acceptance and commit captured once and replayed on other trees."""
    nodes, lens, hq, hkv, d, bs = [9, 16], [300, 800], 8, 2, 128, 16
    x = Batch(lens, hq, hkv, d, bs, torch.bfloat16, seed=41, stale=False)
    T = sum(nodes)
    inv = lib.rope_frequencies(d)[0].to(dev)
    m = dict(q=torch.zeros(T, hq, d, dtype=x.dtype), k=torch.zeros(T, hkv, d, dtype=x.dtype),
             v=torch.zeros(T, hkv, d, dtype=x.dtype), pos=torch.zeros(T, dtype=torch.int64),
             slots=torch.zeros(T, dtype=torch.int64), parents=torch.zeros(T, dtype=torch.int32),
             draft=torch.zeros(T, dtype=torch.int64), target=torch.zeros(T, dtype=torch.int64),
             tables=x.tables, lens=x.lens, start=starts(nodes), kc=x.k, vc=x.v)
    m = {k: v.to(dev) for k, v in m.items()}

    def step():
        q = lib.norm_rope_and_cache(m["q"], m["k"], m["v"], m["pos"], m["slots"], inv, m["kc"], m["vc"])
        out = lib.tree_attention(q, m["kc"], m["vc"], m["tables"], m["lens"], m["start"], m["parents"], x.scale, 16, 900)
        path, n, following = lib.accept_tree(m["draft"], m["target"], m["parents"], m["start"], 16)
        return q, out, path, n, following, lib.commit_path(m["kc"], m["vc"], m["tables"], m["lens"], m["start"], path, n)

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        parents = random_parents(nodes, g)
        at = 0
        pos, slots = [], []
        for b, c in enumerate(nodes):
            base = lens[b] - c
            pos += [base + len(l) - 1 for l in lines(parents[at:at + c].tolist())]
            slots += [int(x.tables[b, (base + i) // bs]) * bs + (base + i) % bs for i in range(c)]
            at += c
        for name, t in dict(q=torch.randn(T, hq, d, generator=g), k=torch.randn(T, hkv, d, generator=g),
                            v=torch.randn(T, hkv, d, generator=g), pos=torch.tensor(pos), slots=torch.tensor(slots),
                            parents=parents, draft=torch.randint(0, 2, (T,), generator=g),
                            target=torch.randint(0, 2, (T,), generator=g), kc=x.k, vc=x.v).items():
            m[name].copy_(t)

    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        fill(1)
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(2, 6):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize(dev)
        got = [t.clone() for t in (*kept, m["kc"], m["vc"])]
        fill(seed)
        want = (*step(), m["kc"], m["vc"])
        torch.cuda.synchronize(dev)
        for a, b in zip(got, want):
            assert same_bits(a, b)
        assert int(got[3].max()) > 0
    assert lib.read_device_errors(dev) == 0


def test_pool_offsets_past_32_bits(dev):
    """Blocks at the far end of a pool of 2.3 G elements give what they give in a small one."""
    hq, hkv, d, bs, far = 16, 8, 128, 16, 140_000
    nodes = [30, 33, 12]
    x = Batch([700, 33, 300], hq, hkv, d, bs, torch.bfloat16, seed=32, stale=False, slack_width=0)
    small, big = _batch_on(dev, x), _batch_on(dev, x, far + x.k.shape[0], far)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(9, h, d, generator=g).to(torch.bfloat16).to(dev) for h in (hq, hkv, hkv))
    pos, slots = torch.arange(9, device=dev) + 1000, torch.randperm(x.k.shape[0] * bs, generator=g)[:9].to(dev)
    inv = lib.rope_frequencies(d)[0].to(dev)
    parents, start = random_parents(nodes, g).to(dev), starts(nodes).to(dev)
    qt = torch.randn(sum(nodes), hq, d, generator=g).to(torch.bfloat16).to(dev)
    path = torch.tensor([[0, 3, 9, 29], [0, 1, 32, -1], [5, 7, 8, 11]], dtype=torch.int32, device=dev)
    n = torch.tensor([4, 3, 4], dtype=torch.int32, device=dev)
    got = []
    for m, first in ((small, 0), (big, far * bs)):
        turned = lib.norm_rope_and_cache(q, k, v, pos, slots + first, inv, m["k"], m["v"])
        out = lib.tree_attention(qt, m["k"], m["v"], m["tables"], m["lens"], start, parents, x.scale, 33, 700)
        new = lib.commit_path(m["k"], m["v"], m["tables"], m["lens"], start, path, n)
        lo = first // bs
        got.append((turned, out, new, m["k"][lo:lo + x.k.shape[0]].clone(), m["v"][lo:lo + x.k.shape[0]].clone()))
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    for a, b in zip(*got):
        assert same_bits(a, b)
    assert int(big["k"][:far].count_nonzero()) == 0 and int(big["v"][:far].count_nonzero()) == 0


def test_calls_from_threads(dev):
    """Four threads, each on a stream of its own, get what one gets."""
    def outcome(seed):
        s = torch.cuda.Stream(dev)
        with torch.cuda.stream(s):
            nodes, lens = [16, 5, 20], [400 + seed, 60, 1500]
            x = Batch(lens, 8, 2, 128, 16, torch.float16, seed=seed, stale=False)
            parents = random_parents(nodes, x.gen)
            q = torch.randn(41, 8, 128, generator=x.gen).to(x.dtype).to(dev)
            k, v, tables, ln = (t.to(dev) for t in (x.k, x.v, x.tables, x.lens))
            start, par = starts(nodes).to(dev), parents.to(dev)
            draft, target = (torch.randint(0, 2, (41,), generator=x.gen).to(dev) for _ in range(2))
            made = []
            for _ in range(20):
                made.append(lib.tree_attention(q, k, v, tables, ln, start, par, x.scale, 20, 1900))
                path, n, following = lib.accept_tree(draft, target, par, start, 20)
                made += [path, n, following]
            made += [lib.commit_path(k, v, tables, ln, start, path, n), k, v]
        s.synchronize()
        return [t.cpu() for t in made]
    want = {seed: outcome(seed) for seed in range(90, 94)}
    got = {}
    threads = [threading.Thread(target=lambda i=seed: got.__setitem__(i, outcome(i))) for seed in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for seed in want:
        assert all(same_bits(a, b) for a, b in zip(want[seed], got[seed]))
    assert lib.read_device_errors(dev) == 0


def test_attention_behind_writers_of_its_inputs(dev):
    """Lengths, starts and parents that the kernel before writes are those the call reads,
    also where its second launch runs ahead of the first."""
    nodes, lens = [16] * 24, [600 + 50 * i for i in range(24)]
    x = Batch(lens, 8, 2, 128, 16, torch.float16, seed=51, stale=False)
    q = torch.randn(sum(nodes), 8, 128, generator=x.gen).to(x.dtype).to(dev)
    k, v, tables = (t.to(dev) for t in (x.k, x.v, x.tables))
    sets = []
    for i in range(3):
        c = [n - 5 * i for n in nodes]
        sets.append([t.to(dev) for t in (x.lens - 64 * i, starts(c), torch.cat([random_parents(c, x.gen), torch.zeros(sum(nodes) - sum(c), dtype=torch.int32)]))])
    held = [t.clone() for t in sets[0]]
    want = [lib.tree_attention(q, k, v, tables, *s, x.scale, 16, 1800) for s in sets]
    torch.cuda.synchronize(dev)
    for turn in range(30):
        i = turn % 3
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        got = lib.tree_attention(q, k, v, tables, *held, x.scale, 16, 1800)
        rows = int(sets[i][1][-1])
        assert same_bits(got[:rows], want[i][:rows]), turn
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("lens,nodes,hq,d,fp8,faults", [
    ([900, 700], [40, 30], 8, 128, False, [(0, 0), (3, 1), (5, 2)]),       # ranges, joined by the second launch
    ([3000, 2500], [64, 60], 16, 128, False, [(0, 3), (7, 6)]),            # two query tiles a CTA, two sides
    ([200, 150], [9, 30], 8, 128, False, [(0, 0), (1, 1)]),                # whole pairs
    ([900, 700], [16, 30], 8, 64, False, [(0, 1), (2, 2)]),
    ([2000, 700], [16, 30], 8, 128, True, [(0, 0), (1, 3), (4, 6)])])
def test_waits_that_run_out(test_lib, monkeypatch, lens, nodes, hq, d, fp8, faults):  # noqa: F811
    dev = torch.device("cuda:0")
    x = Batch(lens, hq, 2, d, 16, torch.float16, seed=6, fp8=fp8, stale=False)
    q = torch.randn(sum(nodes), hq, d, generator=x.gen).to(x.dtype)
    parents = random_parents(nodes, x.gen)
    want, bound = tree_reference(x, q, nodes, parents)
    out = torch.zeros(q.shape, dtype=x.dtype, device=dev)
    args = [t.to(dev) for t in (q, x.k, x.v, x.tables, x.lens, starts(nodes), parents)]

    def call():
        out.zero_()
        lib.tree_attention(*args, x.scale, max(nodes), max(lens), out=out, **x.scales())

    timed_out_then_right(test_lib, monkeypatch, faults, call, lambda: within(out, want, bound, "out"))
