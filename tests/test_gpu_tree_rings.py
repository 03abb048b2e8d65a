"""Tree attention over E4M3 caches, whose codes pass through rings that several
warps keep in step: again and again, bit for bit, and against the definition
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


# ranges of long pairs, of one query tile and of two, and of pairs of one alone
RINGS = [
    ([9001, 4000, 7003], [8, 30, 4], 8, 1),
    ([1500 + (431 * i) % 1500 for i in range(24)], [1 + (5 * i) % 14 for i in range(24)], 16, 4)]


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
