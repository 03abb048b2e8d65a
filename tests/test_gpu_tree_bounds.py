"""What the operators of speculative decoding do with trees, lengths and arguments
at and past the bounds that their contracts name."""
import pytest
import torch

from bounded_util import Batch, same_bits, within
from paged_kv_cache_226_gb300 import build, lib
from tree_util import commit_reference, random_parents, starts, tree_reference

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


def commit_args(dev, x, nodes, path, n):
    return [x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev), path.to(dev), n.to(dev)]


def test_commit_without_a_place_for_the_tree_moves_nothing(dev):
    """A length past the table or below 0, and more nodes than tokens: which rows are
    the tree's is not known."""
    x = Batch([40, 40, 40, 40], 2, 2, 64, 16, torch.float16, seed=5, stale=False)
    path = torch.tensor([[0, 2, 5], [0, 2, 5], [0, 2, 5], [1, 3, 4]], dtype=torch.int32)
    n = torch.full((4,), 3, dtype=torch.int32)
    most = x.width * 16
    for lens, nodes, want in (([most + 1, -1, 40, 40], [6, 6, 6, 6], [most, 0, 37, 37]),
                              ([40, 40, 5, 40], [6, 41, 6, 40], [37, 40, 5, 3])):
        x.lens = torch.tensor(lens, dtype=torch.int32)
        good = [b for b in range(4) if want[b] == lens[b] - nodes[b] + 3]
        (wk, wv), new = commit_reference([x.k, x.v], x.tables[good], x.lens[good], [nodes[b] for b in good], path[good],
                                         n[good], 16)
        k, v = x.k.to(dev), x.v.to(dev)
        got = lib.commit_path(k, v, *commit_args(dev, x, nodes, path, n))
        assert got.tolist() == want and new.tolist() == [want[b] for b in good]
        assert same_bits(k, wk) and same_bits(v, wv)
        assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    x.lens = torch.tensor([40, 40, 40, 40], dtype=torch.int32)
    start = torch.tensor([0, 6, 3, 9, 15], dtype=torch.int32)           # the second has -3 nodes
    k, v = x.k.to(dev), x.v.to(dev)
    got = lib.commit_path(k, v, x.tables.to(dev), x.lens.to(dev), start.to(dev), path.to(dev), n.to(dev))
    assert got.tolist() == [37, 40, 37, 37] and lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT


def test_commit_of_a_tree_with_too_many_nodes(dev):
    """Acceptance and attention take its first 128; so does the commit, and all three say so."""
    nodes = [140, 9]
    x = Batch([200, 30], 2, 2, 64, 16, torch.float16, seed=6, stale=False)
    parents = random_parents(nodes, x.gen, chain=True)
    token = torch.arange(149) + 1                                        # every node follows the one before
    path, n, following = lib.accept_tree(token.to(dev), (token + 1).to(dev), parents.to(dev), starts(nodes).to(dev), 128)
    assert n.tolist() == [128, 9] and following.tolist() == [129, 150]
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    path = path.cpu()
    path[0, 1:4], n = torch.tensor([5, 90, 127], dtype=torch.int32), torch.tensor([4, 9], dtype=torch.int32)
    (wk, wv), new = commit_reference([x.k, x.v], x.tables, x.lens, nodes, path, n, 16)
    k, v = x.k.to(dev), x.v.to(dev)
    got = lib.commit_path(k, v, *commit_args(dev, x, nodes, path, n))
    assert same_bits(got, new) and same_bits(k, wk) and same_bits(v, wv)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    path[0, 3] = 128                                                     # cut off: it is no node of the tree
    k, v = x.k.to(dev), x.v.to(dev)
    got = lib.commit_path(k, v, *commit_args(dev, x, nodes, path, n))
    assert got.tolist() == [200, 30] and same_bits(k, x.k) and same_bits(v, x.v)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT | lib.PA_DEVERR_BAD_INDEX
