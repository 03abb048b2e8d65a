"""What the operators of speculative decoding do with trees, lengths and arguments
at and past the bounds that their contracts name."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nodes,most", [([12, 3], 5), ([40, 64], 33), ([140, 128], 128), ([9, 200], 128), ([7, 2], 1)])
def test_nodes_of_a_tree_cut_off_are_right(dev, nodes, most, fp8):
    """The first nodes of a tree with more than max_query_len of them stay where they are."""
    lens = [nodes[0] + 300, nodes[1]]
    x = Batch(lens, 8, 2, 128, 16, torch.bfloat16, seed=most, fp8=fp8)
    parents = random_parents(nodes, x.gen)
    q = torch.randn(sum(nodes), 8, 128, generator=x.gen).to(x.dtype)
    want, bound = tree_reference(x, q, nodes, parents)
    out = torch.full(q.shape, 3.0, dtype=x.dtype, device=dev)
    lib.tree_attention(q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev),
                       parents.to(dev), x.scale, most, max(lens), out=out, **x.scales())
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    at = 0
    for c in nodes:
        kept = min(c, most)
        within(out[at:at + kept], want[at:at + kept], bound[at:at + kept], "kept nodes")
        assert bool((out[at + kept:at + c] == 3.0).all()), "rows of nodes cut off"
        at += c
