"""GPU parity of pa_evict against the cut made token by token: everything is
a copy, so everything is equal bit for bit."""
import numpy as np
import pytest
import torch

from bounded_util import Batch, evict_reference, same_bits
from paged_kv_cache_226_gb300 import build, lib

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    lib.load()
    d = torch.device("cuda:0")
    lib.read_device_errors(d)
    return d


def earlier_cut(x, known_back):
    """positions, known and seen lengths of a batch that has been cut before:
    all but the last known_back tokens hold scattered earlier positions."""
    g = x.gen
    seen = x.lens * 2 + 5
    known = (x.lens - known_back).clamp(min=0)
    positions = torch.full((x.num_seqs, x.hkv, x.tokens), -(2 ** 31), dtype=torch.int32)
    for b in range(x.num_seqs):
        for h in range(x.hkv):
            n = int(seen[b]) - (int(x.lens[b]) - int(known[b]))
            positions[b, h, :int(known[b])] = torch.randperm(max(n, 1), generator=g)[:int(known[b])].to(torch.int32)
    return positions, known.to(torch.int32), seen.to(torch.int32)


def run(dev, x, w, positions, known, seen, budget, trigger=None, sinks=0, recent=0, in_place=False):
    trig = budget if trigger is None else trigger
    want = evict_reference(x, w, positions, seen, known, budget, trig, sinks, recent)
    k, v = x.k.to(dev), x.v.to(dev)
    wd, pd = w.to(dev), positions.to(dev)
    outs = {} if in_place else dict(weights_out=torch.full_like(wd, -7.0), positions_out=torch.full_like(pd, -7))
    new, wo, po = lib.evict(k, v, x.tables.to(dev), x.lens.to(dev), seen.to(dev), budget, wd, pd,
                            known_lens=known.to(dev) if known is not None else None, trigger=trigger,
                            sinks=sinks, recent=recent, **outs)
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    assert new.cpu().tolist() == want[4].tolist()
    live = (torch.arange(x.tokens) < want[4][:, None, None]).expand(w.shape)
    assert same_bits(po.cpu()[live], want[3][live]), "positions"
    assert same_bits(wo.cpu()[live], want[2][live]), "weights"
    if not in_place:
        assert bool((wo.cpu()[~live] == -7).all()) and bool((po.cpu()[~live] == -7).all())
        assert same_bits(wd, w) and same_bits(pd, positions), "inputs were changed"
    assert same_bits(k, want[0]) and same_bits(v, want[1]), "caches"


LENS = [0, 1, 15, 40, 64, 65, 66, 127, 300, 1500]


@pytest.mark.parametrize("dtype,hkv,d,bs,fp8", [(F16, 2, 64, 16, False), (BF16, 3, 128, 32, False),
                                               (F16, 1, 128, 16, True)])
@pytest.mark.parametrize("budget,sinks,recent", [(64, 4, 16), (64, 0, 0), (64, 0, 64), (64, 64, 0), (1, 0, 1),
                                                 (1, 0, 0), (1000, 4, 100), (5000, 4, 100), (37, 3, 5)])
def test_evict_prompts(dev, dtype, hkv, d, bs, fp8, budget, sinks, recent):
    x = Batch(LENS, hkv, hkv, d, bs, dtype, seed=budget + d, fp8=fp8)
    positions = torch.full((x.num_seqs, hkv, x.tokens), -(2 ** 31), dtype=torch.int32)
    run(dev, x, x.state(), positions, None, x.lens.clone(), budget, sinks=sinks, recent=recent)


@pytest.mark.parametrize("budget,back,in_place", [(64, 1, True), (64, 16, False), (300, 40, True), (7, 300, False)])
def test_evict_after_an_earlier_cut(dev, budget, back, in_place):
    x = Batch(LENS, 2, 2, 128, 16, BF16, seed=budget)
    positions, known, seen = earlier_cut(x, back)
    run(dev, x, x.state(), positions, known, seen, budget, sinks=2, recent=min(5, budget - 2), in_place=in_place)


def test_trigger(dev):
    x = Batch(LENS, 2, 2, 64, 16, F16, seed=3)
    positions, known, seen = earlier_cut(x, 3)
    run(dev, x, x.state(), positions, known, seen, 40, trigger=100, sinks=1, recent=8)


@pytest.mark.parametrize("kind", ["equal", "zeros", "signs", "inf_nan", "close", "negative"])
def test_ties_and_special_weights(dev, kind):
    x = Batch([700, 65, 2000], 2, 2, 64, 16, F16, seed=4)
    g = torch.Generator().manual_seed(9)
    shape = (3, 2, x.tokens)
    w = {"equal": torch.ones(shape), "zeros": torch.zeros(shape),
         "signs": torch.where(torch.rand(shape, generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0)),
         "inf_nan": torch.tensor([float("inf"), float("-inf"), float("nan"), -float("nan"), 1.0, 3.4e38, 1e-45])[
             torch.randint(0, 7, shape, generator=g)],
         "close": 1 + torch.randint(0, 50, shape, generator=g) * 2.0 ** -23,
         "negative": -torch.rand(shape, generator=g)}[kind].float()
    positions = torch.zeros(shape, dtype=torch.int32)
    run(dev, x, w, positions, None, x.lens.clone(), 64, sinks=3, recent=7)


def test_long_contexts(dev):
    x = Batch([40000, 17, 60001], 1, 1, 64, 16, F16, seed=5)
    positions = torch.zeros(3, 1, x.tokens, dtype=torch.int32)
    run(dev, x, x.state(), positions, None, x.lens.clone(), 30000, sinks=4, recent=1000)
    run(dev, x, x.state(), positions, None, x.lens.clone(), 512, sinks=4, recent=128)
    # known positions and few moves on the same tables
    positions, known, seen = earlier_cut(x, 20)
    run(dev, x, x.state(), positions, known, seen, 39990, sinks=4, recent=128)


@pytest.mark.parametrize("n,budget", [(2048, 1024), (2049, 2048), (8192, 100), (8193, 8192), (16385, 8000),
                                      (70000, 69000), (140001, 1000)])
def test_slices_of_every_cluster_size(dev, n, budget):
    """Contexts around the sizes at which the threads, the cluster and the
    passes over a slice change; equal weights put ties across the slices."""
    x = Batch([n, n // 2 + 1], 1, 1, 64, 16, F16, seed=n, stale=False, slack_width=0)
    w = torch.floor(torch.rand(2, 1, x.tokens, generator=x.gen) * 5)
    positions = torch.zeros(2, 1, x.tokens, dtype=torch.int32)
    run(dev, x, w, positions, None, x.lens.clone(), budget, sinks=2, recent=60)


@pytest.mark.parametrize("seqs,hkv,fp8,budget", [(29, 4, False, 64), (57, 2, False, 1500), (57, 2, True, 2000),
                                                 (28, 4, False, 1500)])
def test_full_grids_move_by_themselves(dev, seqs, hkv, fp8, budget):
    """Enough rows to fill the GPU (and just too few): each CTA makes all of
    its moves, up to and past one round of its threads."""
    lens = [2049 + (i * 977) % 2900 for i in range(seqs - 4)] + [0, 1, budget, budget + 1]
    x = Batch(lens, hkv, hkv, 128 if fp8 else 64, 16, F16, seed=seqs + budget, fp8=fp8, stale=False)
    positions = torch.zeros(seqs, hkv, x.tokens, dtype=torch.int32)
    w = x.state().nan_to_num(0.25)
    w *= torch.linspace(0.01, 1.0, x.tokens)             # the heavy ones at the end: many moves
    run(dev, x, w, positions, None, x.lens.clone(), budget, sinks=4, recent=40)
    positions, known, seen = earlier_cut(x, 20)
    run(dev, x, w, positions, known, seen, budget, sinks=4, recent=40, in_place=True)


def test_bad_tables_and_lengths_are_bounded(dev):
    """Moves through a block id outside the pool are left out and reported;
    a length past the table is clamped."""
    x = Batch([64], 1, 1, 64, 16, F16, seed=6, stale=False, slack_width=0)
    w = torch.arange(64).float().view(1, 1, 64)             # the last 16 stay
    tables = x.tables.clone()
    tables[0, 3] = x.k.shape[0]
    k, v = x.k.to(dev), x.v.to(dev)
    zero = torch.zeros(1, 1, 64, dtype=torch.int32, device=dev)
    lens = torch.tensor([64], dtype=torch.int32, device=dev)
    new, wo, po = lib.evict(k, v, tables.to(dev), lens, lens, 16, w.to(dev), zero)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    assert same_bits(k, x.k) and same_bits(v, x.v)
    assert wo[0, 0, :16].tolist() == list(range(48, 64)) and po[0, 0, :16].tolist() == list(range(48, 64))
    big = torch.tensor([1000], dtype=torch.int32, device=dev)
    new, _, _ = lib.evict(k, v, x.tables.to(dev), big, big, 16, w.to(dev), zero.clone())
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT and new.tolist() == [16]


def test_inconsistent_positions_stay_in_bounds(dev):
    """More protected tokens than the budget (positions that no run produces):
    the lowest indices stay."""
    x = Batch([100], 1, 1, 64, 16, F16, seed=7, stale=False)
    positions = torch.zeros(1, 1, x.tokens, dtype=torch.int32)
    known = torch.tensor([10 ** 9], dtype=torch.int32)
    run(dev, x, x.state(), positions, known, x.lens.clone(), 30, sinks=4, recent=2)


def test_graph_and_streams(dev):
    x = Batch([300, 90, 64], 2, 2, 64, 16, F16, seed=8)
    w = x.state()
    positions = torch.zeros(3, 2, x.tokens, dtype=torch.int32)
    d = dict(k_cache=x.k.to(dev), v_cache=x.v.to(dev), block_tables=x.tables.to(dev),
             context_lens=x.lens.to(dev), seen_lens=x.lens.to(dev), budget=64, weights=w.to(dev),
             positions=positions.to(dev), sinks=2, recent=9, weights_out=torch.zeros(w.shape, device=dev),
             positions_out=torch.zeros_like(positions, device=dev),
             new_lens=torch.zeros(3, dtype=torch.int32, device=dev))
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(s):
        lib.evict(**d)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.evict(**d)
    y = Batch([200, 64, 130], 2, 2, 64, 16, F16, seed=8)     # same pool, other lengths
    lens = torch.tensor([200, 64, 30], dtype=torch.int32)
    x.lens = lens
    w2 = y.state().nan_to_num(1.5)[:, :, :w.shape[2]]
    w2 = torch.cat((w2, torch.ones(3, 2, w.shape[2] - w2.shape[2])), 2) if w2.shape[2] < w.shape[2] else w2
    d["k_cache"].copy_(x.k), d["v_cache"].copy_(x.v), d["weights"].copy_(w2)
    d["context_lens"].copy_(lens), d["seen_lens"].copy_(lens)
    g.replay()
    torch.cuda.synchronize(dev)
    want = evict_reference(x, w2, positions, lens, None, 64, 64, 2, 9)
    assert same_bits(d["k_cache"], want[0]) and same_bits(d["v_cache"], want[1])
    assert d["new_lens"].tolist() == want[4].tolist()
    live = (torch.arange(x.tokens) < want[4][:, None, None]).expand(w.shape)
    assert same_bits(d["weights_out"].cpu()[live], want[2][live])
    assert same_bits(d["positions_out"].cpu()[live], want[3][live])


def test_refusals(dev):
    x = Batch([64], 1, 1, 64, 16, F16, seed=6, stale=False)
    lens = x.lens.to(dev)
    w = torch.zeros(1, 1, x.tokens, device=dev)
    d = dict(k_cache=x.k.to(dev), v_cache=x.v.to(dev), block_tables=x.tables.to(dev), context_lens=lens,
             seen_lens=lens, budget=16, weights=w, positions=w.int())
    for bad in (dict(weights=w.double()), dict(positions=w), dict(weights=w[..., :8].contiguous()),
                dict(known_lens=lens.long()), dict(new_lens=lens[:0]), dict(positions=w.int()[..., :-1].contiguous())):
        with pytest.raises((ValueError, TypeError)):
            lib.evict(**{**d, **bad})
    for bad in (dict(budget=0), dict(sinks=9, recent=8), dict(trigger=15), dict(sinks=-1), dict(recent=-1),
                dict(new_lens=lens), dict(workspace=torch.zeros(16, dtype=torch.uint8, device=dev))):
        with pytest.raises(lib.PaError):
            lib.evict(**{**d, **bad})
