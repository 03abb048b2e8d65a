"""Tree attention of long contexts that one CTA walks from end to end: what the
sums lose must not grow with the context.  References in 64 bits, on the GPU."""
import pytest
import torch

from bounded_util import E4M3, half_step
from paged_kv_cache_226_gb300 import build, lib

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


@pytest.mark.parametrize("dtype,fp8,d", [(torch.float16, False, 128), (torch.bfloat16, False, 128),
                                         (torch.float16, False, 64), (torch.float16, True, 128),
                                         (torch.bfloat16, True, 128)])
@pytest.mark.parametrize("nodes", [8, 32])           # 64 rows, both slots in turn; 256, each tile for both
@pytest.mark.parametrize("n", [8200, 16390, 1 << 18])
def test_sums_of_long_contexts(dev, dtype, fp8, d, nodes, n):
    """A pair for each SM, all over the same n tokens, whose V has one sign: a sum
    that is cut off toward zero loses as much with every tile.

    The bound: out's own rounding; of sum p |v| 2^-20 (2 + A) for the scores (A =
    log2(e) scale max sum_d |q_d K_d|), 2^-15 (bf16) or 2^-22 (fp16) for p's two
    parts and 2^-31 n for fp16's range; and for the sums 2^-23 for each of the
    8 x 128 additions that tensor memory holds at a time, 2^-24 for each of the
    runs that follow one another, of which there are n / 8192 or half as many."""
    seqs, group = 152, 8
    g = torch.Generator().manual_seed(n + nodes)
    blocks = -(-n // 16)
    k = torch.randn(blocks, 16, 1, d, generator=g)
    v = 1 + 0.1 * torch.randn(blocks, 16, 1, d, generator=g)
    scales = dict(k_scale=2.0 ** -5, v_scale=2.0 ** -6) if fp8 else {}
    if fp8:
        k, v = ((x / s).clamp(-448, 448).to(E4M3) for x, s in zip((k, v), scales.values()))
        k64, v64 = (x.to(dev).double().view(-1, d)[:n] * s for x, s in zip((k, v), scales.values()))
        k, v = (x.view(torch.uint8).to(dev) for x in (k, v))
    else:
        k, v = (x.to(dtype).to(dev) for x in (k, v))
        k64, v64 = (x.double().view(-1, d)[:n] for x in (k, v))
    q = (torch.randn(seqs * nodes, group, d, generator=g) * 0.3).to(dtype).to(dev)
    parents = torch.cat([torch.tensor([-1] + [0] * (nodes - 1), dtype=torch.int32)] * seqs).to(dev)
    tables = torch.arange(blocks, dtype=torch.int32, device=dev).repeat(seqs, 1)
    lens = torch.full((seqs,), n, dtype=torch.int32, device=dev)
    start = torch.arange(seqs + 1, dtype=torch.int32, device=dev) * nodes
    scale = 1 / 8
    out = lib.tree_attention(q, k, v, tables, lens, start, parents, scale, nodes, n, **scales)
    seen = torch.ones(nodes, n, dtype=torch.bool, device=dev)
    seen[:, n - nodes:] = torch.eye(nodes, dtype=torch.bool, device=dev)
    seen[:, n - nodes] = True                        # node 0
    for b in (0, 75, 151):
        x = q.view(seqs, nodes, group, d)[b].double()
        s = (x @ k64.T * scale).masked_fill(~seen[:, None, :], -float("inf"))
        p = torch.softmax(s, -1)
        want, sums = p @ v64, p @ v64.abs()
        a = float((x.abs() @ k64.abs().T).max()) * scale * 1.4427
        parts = 2.0 ** -15 if dtype == torch.bfloat16 else 2.0 ** -22 + 2.0 ** -31 * n
        bound = half_step(dtype) * want.abs() + \
            (2.0 ** -20 * (2 + a) + parts + 2.0 ** -23 * 8 * 128 + 2.0 ** -24 * (n / 8192 + 1)) * sums
        err = (out.view(seqs, nodes, group, d)[b].double() - want).abs()
        assert bool((err <= bound).all()), f"sequence {b}: {float((err - bound).max())} over the bound"
    assert lib.read_device_errors(dev) == 0
