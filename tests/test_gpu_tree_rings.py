"""Tree attention over E4M3 caches, whose codes pass through rings that several
warps keep in step: pairs that one slot takes alone beside pairs that both take
in turn or share, again and again, bit for bit, and against the definition
(tree_util.py)."""
import pytest
import torch

from bounded_util import Batch, same_bits, within
from paged_kv_cache_226_gb300 import build, lib
from tree_util import random_parents, starts, tree_reference

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


def call_args(dev, x, nodes, parents, q):
    return [q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev),
            parents.to(dev), x.scale, max(nodes), int(x.lens.max())]


# ranges of long pairs, of one query tile and of two, and of pairs of one alone;
# pairs of one to eight tiles, dealt whole, several of them a lane, of one query
# tile and of one or two; ranges of pairs of up to 32 tiles; the same with pairs
# of two query tiles among those of one
RINGS = [
    ([9001, 4000, 7003], [8, 30, 4], 8, 1),
    ([1500 + (431 * i) % 1500 for i in range(24)], [1 + (5 * i) % 14 for i in range(24)], 16, 4),
    ([1 + (83 * i) % 500 for i in range(90)], [1 + (5 * i) % 9 for i in range(90)], 8, 8),
    ([60 + (97 * i) % 450 for i in range(60)], [1 + (23 * i) % 60 for i in range(60)], 16, 4),
    ([20 + (431 * i) % 2000 for i in range(40)], [1 + (7 * i) % 16 for i in range(40)], 8, 2),
    ([60 + (431 * i) % 1500 for i in range(24)], [1 + (11 * i) % 60 for i in range(24)], 16, 4),
    ([130 + (29 * i) % 90 for i in range(120)], [128 - i % 60 for i in range(120)], 2, 2)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(RINGS)))
def test_e4m3_repeats_bit_for_bit(dev, case, dtype):
    lens, nodes, hq, hkv = RINGS[case]
    nodes = [min(c, n) for c, n in zip(nodes, lens)]
    x = Batch(lens, hq, hkv, 128, 16, dtype, seed=60 + case, fp8=True)
    parents = random_parents(nodes, x.gen)
    q = torch.randn(sum(nodes), hq, 128, generator=x.gen).to(dtype)
    want, bound = tree_reference(x, q, nodes, parents)
    args = call_args(dev, x, nodes, parents, q)
    first = lib.tree_attention(*args, **x.scales())
    within(first, want, bound, "out")
    for _ in range(200):
        assert same_bits(lib.tree_attention(*args, **x.scales()), first)
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", [2, 3, 4, 6])
def test_e4m3_values_that_are_not_finite_stay_with_their_lines(dev, case, dtype):
    """Every tree's second node and the pool behind the contexts hold NaN: only the
    rows whose line it is on show it."""
    lens, nodes, hq, hkv = RINGS[case]
    nodes = [min(c, n) for c, n in zip(nodes, lens)]
    x = Batch(lens, hq, hkv, 128, 16, dtype, seed=70 + case, fp8=True)
    parents = random_parents(nodes, x.gen)
    at = 0
    for c in nodes:                                  # every third node below the second, the others not
        for i in range(2, c):
            parents[at + i] = 1 if i % 3 == 0 else 0
        at += c
    q = torch.randn(sum(nodes), hq, 128, generator=x.gen).to(dtype)
    want, bound = tree_reference(x, q, nodes, parents)
    seen = torch.zeros(sum(nodes), dtype=torch.bool)
    at = 0
    for b, (n, c) in enumerate(zip(lens, nodes)):
        if c > 1:
            where = n - c + 1
            x.v[int(x.tables[b, where // 16]), where % 16] = 0x7f
            seen[at + 1] = True
            seen[at + 3:at + c:3] = True
        at += c
    args = call_args(dev, x, nodes, parents, q)
    for _ in range(20):
        got = lib.tree_attention(*args, **x.scales()).cpu()
        within(got[~seen], want[~seen], bound[~seen], "rows that do not see it")
        assert bool(got[seen].isnan().all())
    assert lib.read_device_errors(dev) == 0
