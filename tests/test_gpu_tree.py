"""GPU parity of the operators of speculative decoding against their
definitions in 64 bits (tree_util.py; the rotary write's bound:
test_gpu_rope.py)."""
import numpy as np
import pytest
import torch

from bounded_util import E4M3, Batch, half_step, same_bits, within
from paged_kv_cache_226_gb300 import build, lib
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


# ---- norm, rotary positions and cache write -----------------------------------

def normed(x, weight, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.double()


def turned(x, positions, axes, inv_freq, interleaved, factor):
    """(value, |x| + |y| of each element's pair); positions [A][T]."""
    r = 2 * len(inv_freq)
    a = (positions.double()[axes.long()].T * inv_freq.double())[:, None, :]
    cos, sin = torch.cos(a) * factor, torch.sin(a) * factor
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, size = x.clone(), x.abs()
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    size[..., i] = size[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, size


def check_norm(dev, T, hq, hkv, d, bs, dtype, rotary, axes=1, interleaved=False, fp8=False, weights=True, eps=1e-6,
               padding=0, factor=1.0, in_place=False, no_q=False, far=5000):
    """A normalised value is off by 2^-21 (the squares' sum of up to 128 terms in
    eight chains, rsqrt and two products: 16 roundings of 2^-25 in the root, 2 +
    2 of 2^-24), a turned one by that and 2^-21 f of the pair's |x| + |y|."""
    g = torch.Generator().manual_seed(T + d + rotary)
    size = torch.exp(2 * torch.randn(T, hq + 2 * hkv, 1, generator=g))
    m = (torch.randn(T, hq + 2 * hkv, d, generator=g) * size).to(dtype).view(T, -1)
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if padding:
        slots[T - padding:] = -1
    pool = (lambda: torch.randint(0, 255, (nb, bs, hkv, d), generator=g, dtype=torch.uint8)) if fp8 else \
        (lambda: torch.randn(nb, bs, hkv, d, generator=g).to(dtype))
    kc0, vc0 = pool(), pool()
    qw, kw = ((1 + torch.randn(d, generator=g)).to(dtype) for _ in range(2)) if weights else (None, None)
    inv, pairs = (lib.rope_frequencies(rotary)[0], rotary // 2) if rotary else (torch.zeros(0), 0)
    pos = torch.randint(-3, far, (axes, T), generator=g)
    ax = torch.randint(0, axes, (pairs,), generator=g).to(torch.int32)
    qkv, kc, vc = m.to(dev), kc0.to(dev), vc0.to(dev)
    q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    q0, k0, v0 = (t.view(T, -1, d) for t in m.split([hq * d, hkv * d, hkv * d], dim=1))
    sc = dict(k_scale=0.04, v_scale=0.03) if fp8 else {}
    out = lib.norm_rope_and_cache(
        None if no_q else q, k, v, (pos if axes > 1 else pos[0]).to(dev), slots.to(dev), inv.to(dev), kc, vc,
        q_weight=None if qw is None else qw.to(dev), k_weight=None if kw is None else kw.to(dev), eps=eps,
        axes=ax.to(dev) if axes > 1 else None, q_out=q if in_place else None, interleaved=interleaved,
        factor=factor, **sc)
    torch.cuda.synchronize(dev)
    f32, e32 = float(np.float32(factor)), float(np.float32(eps))

    def rounded(want, size):
        return half_step(dtype) * want.abs() + 2.0 ** -21 * (want.abs() + 2 * max(1.0, f32) * size) + \
            (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)

    if no_q:
        assert out is None
    else:
        want, size = turned(normed(q0, qw, e32), pos, ax, inv, interleaved, f32)
        within(out, want, rounded(want, size), "q")
    assert same_bits(qkv[:, hq * d:], m[:, hq * d:]), "k and v are inputs"
    live = torch.nonzero(slots >= 0)[:, 0]
    at = slots[live]
    want, size = turned(normed(k0, kw, e32), pos, ax, inv, interleaved, f32)
    want, size = want[live], size[live]
    got_k, got_v = kc.cpu().view(-1, hkv, d), vc.cpu().view(-1, hkv, d)
    if fp8:
        s32 = float(np.float32(0.04))
        bound = (want / s32).abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -20 * max(1.0, f32) * size / s32 + 2.0 ** -10
        within(got_k[at].view(E4M3), (want / s32).clamp(-448, 448), bound, "k codes")
        vv = (v0[live].float() / np.float32(0.03)).clamp(-448, 448).to(E4M3).view(torch.uint8)
        assert same_bits(got_v[at], vv), "v codes"
    else:
        within(got_k[at], want, rounded(want, size), "k")
        assert same_bits(got_v[at], v0[live]), "v"
    untouched = torch.ones(got_k.shape[0], dtype=torch.bool)
    untouched[at] = False
    assert same_bits(got_k[untouched], kc0.view(-1, hkv, d)[untouched])
    assert same_bits(got_v[untouched], vc0.view(-1, hkv, d)[untouched])
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,bs,dtype,rotary,axes", [
    (1, 8, 2, 64, 16, torch.float16, 64, 1), (1, 32, 8, 128, 16, torch.bfloat16, 128, 3),
    (37, 6, 2, 128, 32, torch.float16, 128, 2), (130, 5, 1, 64, 16, torch.bfloat16, 32, 3),
    (9, 16, 16, 128, 16, torch.float16, 48, 8), (200, 64, 8, 128, 16, torch.bfloat16, 96, 1),
    (3, 7, 7, 64, 32, torch.float16, 16, 4), (1500, 3, 1, 128, 16, torch.bfloat16, 128, 3),
    (2001, 2, 2, 64, 16, torch.float16, 64, 2), (5, 4, 2, 128, 16, torch.float16, 0, 1)])
def test_norm_shapes(dev, T, hq, hkv, d, bs, dtype, rotary, axes, interleaved):
    check_norm(dev, T, hq, hkv, d, bs, dtype, rotary, axes, interleaved)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,rotary,axes,padding", [(1, 8, 2, 128, 1, 0), (77, 12, 4, 64, 3, 5), (33, 3, 1, 16, 2, 33),
                                                          (1601, 3, 1, 128, 2, 7)])
def test_norm_e4m3(dev, T, hq, hkv, rotary, axes, padding, interleaved, dtype):
    check_norm(dev, T, hq, hkv, 128, 16, dtype, rotary, axes, interleaved, fp8=True, padding=padding)


@pytest.mark.parametrize("kw", [dict(weights=False), dict(eps=0.5), dict(in_place=True, factor=1.3), dict(no_q=True),
                                dict(far=1 << 20, axes=3), dict(padding=4)])
def test_norm_choices(dev, kw):
    check_norm(dev, 21, 8, 2, 128, 16, torch.bfloat16, 128, **kw)
    check_norm(dev, 21, 9, 3, 64, 16, torch.float16, 48, **kw)


def test_norm_of_zero_rows_and_large_values(dev):
    """eps holds a row of zeros at zero; fp16's largest values and bf16's up to 2^60
    do not overflow their squares' sum."""
    for dtype, big in ((torch.float16, 65504.0), (torch.bfloat16, 2.0 ** 60)):
        x = torch.zeros(3, 2, 64, dtype=dtype, device=dev)
        x[1] = big
        x[2, 0, 5] = big
        kc, vc = (torch.zeros(1, 16, 2, 64, dtype=dtype, device=dev) for _ in range(2))
        q = lib.norm_rope_and_cache(x, x, x, torch.arange(3, device=dev), torch.arange(3, device=dev),
                                    torch.zeros(32, device=dev), kc, vc)
        want = torch.zeros(3, 2, 64)
        want[1], want[2, 0, 5] = 1.0, 8.0
        assert torch.allclose(q.float().cpu(), want, rtol=2.0 ** -8) and same_bits(q, kc[0, :3])


def test_norm_bad_axes_and_slots(dev):
    x = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(1)).half().to(dev)
    pos = torch.tensor([[1, 2, 3, 4], [9, 9, 9, 9]], device=dev)
    inv = lib.rope_frequencies(64)[0].to(dev)
    ax = torch.zeros(32, dtype=torch.int32)
    good = ax.clone()
    ax[3], ax[7] = 2, -1
    kc, vc = (torch.zeros(1, 16, 2, 64, dtype=torch.float16, device=dev) for _ in range(2))
    slots = torch.tensor([0, 1, 99, -2], device=dev)
    a = lib.norm_rope_and_cache(x, x, x, pos, slots, inv, kc, vc, axes=ax.to(dev))
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_INDEX | lib.PA_DEVERR_BAD_SLOT
    b = lib.norm_rope_and_cache(x, x, x, pos, slots.clamp(max=1), inv, kc.clone(), vc.clone(), axes=good.to(dev))
    assert same_bits(a, b) and lib.read_device_errors(dev) == 0


def test_norm_refusals(dev):
    x = torch.zeros(4, 2, 64, dtype=torch.float16, device=dev)
    kc, vc = (torch.zeros(1, 16, 2, 64, dtype=torch.float16, device=dev) for _ in range(2))
    at = torch.arange(4, device=dev)
    inv, w = torch.ones(32, device=dev), torch.ones(64, dtype=torch.float16, device=dev)
    ax = torch.zeros(32, dtype=torch.int32, device=dev)
    base = dict(q=x, k=x, v=x, positions=at, slot_mapping=at, inv_freq=inv, k_cache=kc, v_cache=vc)
    for err, kw in ((TypeError, dict(q_weight=w.float())), (ValueError, dict(k_weight=w[:32])),
                    (ValueError, dict(q_weight=torch.ones(128, dtype=torch.float16, device=dev)[::2])),
                    (ValueError, dict(axes=ax)), (ValueError, dict(positions=at[None])),
                    (ValueError, dict(positions=torch.stack([at, at]), axes=ax[:5])),
                    (TypeError, dict(positions=torch.stack([at, at]), axes=ax.long())),
                    (TypeError, dict(positions=at.int())), (ValueError, dict(positions=at[:3])),
                    (ValueError, dict(positions=torch.stack([at[:3], at[:3]]), axes=ax)),
                    (lib.PaError, dict(positions=torch.stack([at] * 9), axes=ax)), (lib.PaError, dict(eps=-1.0)),
                    (lib.PaError, dict(inv_freq=torch.ones(4, device=dev))), (ValueError, dict(k_scale=1.0, v_scale=1.0))):
        with pytest.raises(err):
            lib.norm_rope_and_cache(**{**base, **kw})
    assert lib.read_device_errors(dev) == 0


# ---- attention of the trees ------------------------------------------------------

def check_tree(dev, lens, nodes, hq, hkv, d, bs, dtype, fp8=False, chain=False, seed=0, behind=0, sharp=1.0,
               parents=None):
    x = Batch(lens, hq, hkv, d, bs, dtype, seed=seed, fp8=fp8)
    q = (torch.randn(sum(nodes) + behind, hq, d, generator=x.gen) * sharp).to(dtype)
    if parents is None:
        parents = random_parents(nodes, x.gen, chain)
    full = torch.cat([parents, torch.full((behind,), 7, dtype=torch.int32)])
    want, bound = tree_reference(x, q, nodes, parents)
    out = torch.full(q.shape, 3.0, dtype=dtype, device=dev)
    got = lib.tree_attention(q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev),
                             starts(nodes).to(dev), None if chain else full.to(dev), x.scale,
                             max([1, *nodes]), max([1, *lens]), out=out, **x.scales())
    torch.cuda.synchronize(dev)
    assert got is out and lib.read_device_errors(dev) == 0
    n = sum(nodes)
    within(got[:n], want[:n], bound[:n], "out")
    assert bool((got[n:] == 3.0).all()), "rows behind the last sequence are left alone"


SHAPES = [
    ([1], [1], 1, 1, 64, 16), ([7], [7], 8, 2, 128, 16), ([129], [3], 6, 2, 64, 32),
    ([40, 0, 17, 1, 300], [5, 0, 17, 1, 2], 8, 8, 128, 16), ([128, 127, 129, 256], [16, 16, 16, 16], 4, 1, 128, 16),
    ([260, 131], [128, 101], 5, 1, 128, 32), ([140, 500], [40, 33], 14, 2, 64, 16), ([300, 290], [64, 60], 16, 2, 128, 16),
    ([700], [1], 3, 1, 128, 16), ([1000, 64, 10], [9, 64, 0], 6, 1, 128, 16)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,nodes,hq,hkv,d,bs", SHAPES)
def test_tree_shapes(dev, lens, nodes, hq, hkv, d, bs, dtype):
    check_tree(dev, lens, nodes, hq, hkv, d, bs, dtype, seed=len(lens) + hq, behind=3)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,nodes,hq,hkv,d,bs", [s for s in SHAPES if s[4] == 128])
def test_tree_e4m3(dev, lens, nodes, hq, hkv, d, bs, dtype):
    check_tree(dev, lens, nodes, hq, hkv, d, bs, dtype, fp8=True, seed=len(lens) + hq, behind=1)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (128, True)])
def test_tree_groups(dev, group, d, fp8):
    check_tree(dev, [200, 75, 330], [20, 33, 70], 2 * group, 2, d, 16, torch.bfloat16, fp8=fp8, seed=group)


@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 64, 65, 127, 128])
def test_tree_lines(dev, nodes):
    """Lines of drafted tokens, as a missing `parents` says, are causal chunks."""
    check_tree(dev, [nodes, nodes + 100], [nodes, nodes], 8, 2, 128, 16, torch.float16, chain=True, seed=nodes)


@pytest.mark.parametrize("base", [0, 1, 60, 100, 126, 127, 128, 129, 200])
def test_tree_across_key_tiles(dev, base):
    """Trees that begin and end on either side of a boundary of 128 keys, roots among the nodes."""
    nodes = 70
    g = torch.Generator().manual_seed(base)
    parents = random_parents([nodes], g)
    parents[5], parents[40] = -1, -9
    check_tree(dev, [base + nodes], [nodes], 4, 2, 128, 16, torch.bfloat16, seed=base, parents=parents)
    check_tree(dev, [base + nodes], [nodes], 4, 2, 64, 32, torch.float16, seed=base, parents=parents)


@pytest.mark.parametrize("dtype,fp8", [(torch.float16, False), (torch.bfloat16, False), (torch.float16, True),
                                       (torch.bfloat16, True)])
def test_tree_long(dev, dtype, fp8):
    check_tree(dev, [9000, 5003], [12, 40], 8, 2, 128, 16, dtype, fp8=fp8, seed=2)


@pytest.mark.parametrize("lens,nodes,hq,hkv,d,fp8", [
    ([6000], [9], 32, 32, 64, False),                      # KV heads of several lanes, joined pair by pair
    ([3001, 0, 2400], [30, 0, 17], 32, 16, 128, False),
    ([5000], [128], 16, 2, 128, False),                    # four CTAs side by side, 152 / 8 ranges
    ([4100], [100], 7, 1, 128, True),
    ([700 + 13 * i for i in range(16)], [1 + 3 * i for i in range(16)], 16, 8, 128, True),
    ([600 + 41 * i for i in range(9)], [5] * 9, 20, 5, 64, False)])
def test_tree_ranges_that_meet_in_pairs(dev, lens, nodes, hq, hkv, d, fp8):
    check_tree(dev, lens, nodes, hq, hkv, d, 16, torch.bfloat16, fp8=fp8, seed=hkv, behind=2)


@pytest.mark.parametrize("seqs,hq,hkv,d,longest", [(16, 8, 8, 64, 1024), (16, 8, 8, 64, 1025), (10, 8, 8, 128, 1000),
                                                   (9, 8, 8, 128, 1000), (20, 16, 8, 64, 1000), (8, 16, 2, 128, 700)])
def test_tree_lanes_with_a_pair_each(dev, seqs, hq, hkv, d, longest):
    """As many pairs as there are lanes, some fewer and some more, of up to 16 key tiles and one more."""
    lens = [longest - 97 * i % 600 for i in range(seqs)]
    nodes = [1 + 11 * i % 60 for i in range(seqs)]
    check_tree(dev, lens, nodes, hq, hkv, d, 16, torch.float16, seed=seqs)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_shared_and_repeated_blocks(dev, fp8):
    """Sequences with the same context, and a context that has one block over and over."""
    x = Batch([900, 900, 900], 8, 2, 128, 16, torch.bfloat16, seed=3, fp8=fp8, stale=False)
    nodes = [20, 33, 8]
    shared = (900 - max(nodes)) // 16
    x.tables[1, :shared] = x.tables[0, :shared]
    x.tables[2, :shared] = x.tables[0, 0]
    q = torch.randn(sum(nodes), 8, 128, generator=x.gen).to(torch.bfloat16)
    parents = random_parents(nodes, x.gen)
    want, bound = tree_reference(x, q, nodes, parents)
    got = lib.tree_attention(q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev),
                             parents.to(dev), x.scale, 33, 900, **x.scales())
    within(got, want, bound, "out")
    assert lib.read_device_errors(dev) == 0


def test_tree_strangers_are_refused(dev):
    """Rows that are not dense, out over q, on the host, or of another shape."""
    x = Batch([40], 4, 2, 64, 16, torch.float16, seed=1, stale=False)
    room = torch.zeros(12, 4, 64, dtype=torch.float16, device=dev)
    args = [x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), starts([8]).to(dev), None, x.scale, 8, 40]
    for q, out in ((room[::2], None), (room[:8], room[2:10]), (room[2:10], room[:8]), (room[:8], room[:8]),
                   (room[:8], room[:8].cpu()), (room[:8], room[8:]), (room[:8].cpu(), None),
                   (room[:8].transpose(1, 2).contiguous().transpose(1, 2), None)):
        with pytest.raises((ValueError, lib.PaError)):
            lib.tree_attention(q, *args, out=out)
    assert bool((room == 0).all()) and lib.read_device_errors(dev) == 0


def test_tree_many_sequences(dev):
    """More sequences than a warp walks at a time, every other length, empty ones among them."""
    n = 75
    lens = [(37 * i) % 300 for i in range(n)]
    nodes = [min(x, (5 * i) % 19) for i, x in enumerate(lens)]
    check_tree(dev, lens, nodes, 6, 2, 64, 16, torch.float16, seed=4)
    check_tree(dev, lens, nodes, 8, 2, 128, 16, torch.bfloat16, seed=5, fp8=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tree_sharp_scores(dev, dtype, fp8):
    """Scores of some hundreds, whose maximum rises again and again along the context."""
    check_tree(dev, [900, 600], [30, 64], 8, 2, 128, 16, dtype, fp8=fp8, seed=6, sharp=30.0)


def same_tree_args(dev, x, nodes, parents, q):
    return [q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev),
            parents.to(dev), x.scale, max(nodes), int(x.lens.max())]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_tree_hidden_tokens_have_no_part(dev, value, fp8):
    """K and V of a node that are not finite show in the rows that see it, and in no other."""
    if fp8 and value == value:
        pytest.skip("E4M3 has no infinity")
    nodes, lens = [50, 20], [250, 20]
    x = Batch(lens, 8, 2, 128, 16, torch.bfloat16, seed=9, fp8=fp8)
    parents = random_parents(nodes, x.gen)
    q = torch.randn(70, 8, 128, generator=x.gen).to(x.dtype)
    want, bound = tree_reference(x, q, nodes, parents)
    for who, b, off in ((11, 0, 200), (3, 1, 0)):
        where = int(x.tables[b, (off + who) // 16]), (off + who) % 16
        for pool in (x.k, x.v):
            pool[where] = 0x7f if fp8 else value
    got = lib.tree_attention(*same_tree_args(dev, x, nodes, parents, q), **x.scales()).double().cpu()
    at = 0
    for who, c in ((11, 50), (3, 20)):
        for i, line in enumerate(lines(parents[at:at + c].tolist())):
            if who not in line:
                within(got[at + i], want[at + i], bound[at + i], f"node {i}")
            else:
                assert not bool(torch.isfinite(got[at + i]).all()), f"node {i} sees it"
        at += c
    assert lib.read_device_errors(dev) == 0


def test_tree_bad_inputs_are_bounded(dev):
    """Lengths, rows, blocks and parents that cannot be are clamped or set aside and reported."""
    nodes, lens = [6, 5], [40, 30]
    x = Batch(lens, 4, 2, 64, 16, torch.float16, seed=3, stale=False)
    parents = random_parents(nodes, x.gen)
    q = torch.randn(11, 4, 64, generator=x.gen).to(x.dtype)
    want, bound = tree_reference(x, q, nodes, parents)
    args = same_tree_args(dev, x, nodes, parents, q)

    def call(i, t):
        got = lib.tree_attention(*args[:i], t.to(dev), *args[i + 1:])
        torch.cuda.synchronize(dev)
        return got, lib.read_device_errors(dev)

    bad = parents.clone()
    bad[6 + 2], bad[6 + 3] = 2, 100                      # itself; a later one
    fixed = parents.clone()
    fixed[6 + 2] = fixed[6 + 3] = -1
    got, flags = call(6, bad)
    w2, b2 = tree_reference(x, q, nodes, fixed)
    within(got, w2, b2, "as roots")
    assert flags == lib.PA_DEVERR_BAD_INDEX
    for t in (torch.tensor([40, -5]), torch.tensor([40, 1 << 20])):
        got, flags = call(4, t.to(torch.int32))
        within(got[:6], want[:6], bound[:6], "the other sequence")
        assert flags == lib.PA_DEVERR_BAD_CONTEXT
    for t in (torch.tensor([0, 6, 5]), torch.tensor([0, 6, 12]), torch.tensor([0, 6, 1 << 30])):
        got, flags = call(5, t.to(torch.int32))
        within(got[:6], want[:6], bound[:6], "the other sequence")
        assert flags == lib.PA_DEVERR_BAD_CONTEXT
    tables = x.tables.clone()
    tables[1, 0], tables[1, 1] = -3, 10 ** 6
    got, flags = call(3, tables)
    within(got[:6], want[:6], bound[:6], "the other sequence")
    assert flags == lib.PA_DEVERR_BAD_CONTEXT
    # bounds of the call below what there is
    got = lib.tree_attention(*args[:8], 5, 40)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    got = lib.tree_attention(*args[:8], 6, 35)
    within(got[6:], want[6:], bound[6:], "the shorter sequence")
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    within(lib.tree_attention(*args), want, bound, "afterwards")
    assert lib.read_device_errors(dev) == 0


def test_tree_no_nodes(dev):
    x = Batch([40, 0], 4, 2, 64, 16, torch.float16, seed=3)
    for T in (0, 4):
        q = torch.randn(T, 4, 64, generator=x.gen).to(x.dtype)
        out = torch.full(q.shape, 2.0, dtype=x.dtype, device=dev)
        lib.tree_attention(q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev),
                           starts([0, 0]).to(dev), torch.zeros(T, dtype=torch.int32, device=dev), 1.0, 8, 40, out=out)
        assert bool((out == 2.0).all())
    assert lib.read_device_errors(dev) == 0


def test_tree_refusals(dev):
    nodes = [6, 5]
    x = Batch([40, 30], 4, 2, 64, 16, torch.float16, seed=3)
    parents = random_parents(nodes, x.gen)
    q = torch.randn(11, 4, 64, generator=x.gen).to(x.dtype)
    args = same_tree_args(dev, x, nodes, parents, q)
    for err, i, bad in ((TypeError, 0, args[0].float()), (TypeError, 0, args[0].bfloat16()), (ValueError, 0, args[0][:, :, :32]),
                        (ValueError, 0, args[0].transpose(0, 1)), (ValueError, 5, args[5][:2]), (TypeError, 5, args[5].long()),
                        (ValueError, 6, args[6][:5]), (TypeError, 6, args[6].long()), (TypeError, 4, args[4].long()),
                        (ValueError, 4, args[4][:1]), (ValueError, 6, args[6].cpu()), (lib.PaError, 7, 0.0),
                        (lib.PaError, 8, 129), (lib.PaError, 8, -1), (ValueError, 9, 1 << 31), (lib.PaError, 0, args[0][:, :3].contiguous())):
        with pytest.raises(err):
            lib.tree_attention(*args[:i], bad, *args[i + 1:])
    with pytest.raises(lib.PaError):
        lib.tree_attention(*args, out=args[0])
    with pytest.raises(ValueError):
        lib.tree_attention(*args, out=args[0][:5])
    with pytest.raises(lib.PaError):
        lib.tree_attention(*args, workspace=torch.empty(8, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        lib.tree_attention(*args, k_scale=1.0, v_scale=1.0)
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_graph_and_streams(dev, fp8):
    """Captured once, the call follows lengths, trees and rows; two streams have a workspace each."""
    nodes, lens = [16, 9, 16], [700, 300, 1200]
    x = Batch(lens, 8, 2, 128, 16, torch.float16, seed=12, fp8=fp8, stale=False)
    args = same_tree_args(dev, x, nodes, random_parents(nodes, x.gen), torch.randn(41, 8, 128, generator=x.gen).to(x.dtype))
    out = torch.zeros_like(args[0])
    lib.tree_attention(*args, out=out, **x.scales())
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.tree_attention(*args, out=out, **x.scales())
    for step in range(3):
        lens2 = [max(c, n - 211 * step) for n, c in zip(lens, nodes)]
        nodes2 = [c - 3 * step for c in nodes]
        x.lens = torch.tensor(lens2, dtype=torch.int32)
        parents = random_parents(nodes2, x.gen)
        q = torch.randn(41, 8, 128, generator=x.gen).to(x.dtype)
        args[0].copy_(q), args[4].copy_(x.lens), args[5].copy_(starts(nodes2))
        args[6][:len(parents)].copy_(parents)
        g.replay()
        torch.cuda.synchronize(dev)
        want, bound = tree_reference(x, q, nodes2, parents)
        n = sum(nodes2)
        within(out[:n], want[:n], bound[:n], f"replay {step}")
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in streams]
    torch.cuda.synchronize(dev)
    for _ in range(10):
        for st, o in zip(streams, outs):
            with torch.cuda.stream(st):
                lib.tree_attention(*args, out=o, **x.scales())
    torch.cuda.synchronize(dev)
    for o in outs:
        assert same_bits(o[:n], out[:n])
    assert lib.read_device_errors(dev) == 0


def test_tree_repeats_bit_for_bit(dev):
    nodes, lens = [40, 33, 64], [3000, 700, 5200]
    x = Batch(lens, 16, 2, 128, 16, torch.bfloat16, seed=13)
    args = same_tree_args(dev, x, nodes, random_parents(nodes, x.gen), torch.randn(137, 16, 128, generator=x.gen).to(x.dtype))
    first = lib.tree_attention(*args)
    for _ in range(20):
        assert same_bits(lib.tree_attention(*args), first)


# ---- acceptance and commit -------------------------------------------------------

def check_accept(dev, nodes, width, seed, agree=0.8, chain=False):
    g = torch.Generator().manual_seed(seed)
    n = sum(nodes)
    parents = random_parents(nodes, g, chain)
    target = torch.randint(0, 50, (n,), generator=g) + (1 << 40)
    draft = torch.randint(0, 50, (n,), generator=g) + (1 << 40)
    at = 0
    for c in nodes:
        for i in range(1, c):
            if float(torch.rand(1, generator=g)) < agree:
                draft[at + i] = target[at + int(parents[at + i])]
        at += c
    want = accept_reference(draft, target, parents, nodes, width)
    got = lib.accept_tree(draft.to(dev), target.to(dev), None if chain else parents.to(dev), starts(nodes).to(dev), width)
    for a, b, what in zip(got, want, ("path", "path_lens", "next")):
        assert same_bits(a, b), f"{what}: {a} {b}"
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("agree", [0.0, 0.5, 0.9, 1.0])
@pytest.mark.parametrize("nodes,width", [([1], 1), ([0, 1, 2, 0], 5), ([26], 26), ([128, 127, 65, 64, 33, 32, 31], 128),
                                         ([60] * 40, 64)])
def test_accept(dev, nodes, width, agree):
    check_accept(dev, nodes, width, seed=len(nodes) + width, agree=agree)
    check_accept(dev, nodes, width, seed=len(nodes) + width, agree=agree, chain=True)


def test_accept_bad_inputs_are_bounded(dev):
    t = torch.arange(6, device=dev)
    start = torch.tensor([0, 6], dtype=torch.int32, device=dev)
    parents = torch.tensor([-1, 0, 2, 1, 99, -1], dtype=torch.int32, device=dev)
    draft, target = torch.zeros_like(t), torch.zeros_like(t)
    path, n, nxt = lib.accept_tree(draft, target, parents, start, 6)
    assert path.tolist() == [[0, 1, 3, -1, -1, -1]] and n.tolist() == [3] and nxt.tolist() == [0]
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_INDEX
    parents = torch.arange(-1, 5, dtype=torch.int32, device=dev)
    for s, want in (([0, 7], 0), ([-1, 3], 0), ([4, 2], 0), ([0, 6], 4)):
        path, n, nxt = lib.accept_tree(draft, target, parents, torch.tensor(s, dtype=torch.int32, device=dev), 4)
        assert n.tolist() == [want] and path.tolist() == [[0, 1, 2, 3] if want else [-1] * 4], s
        assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT, s
    with pytest.raises(lib.PaError):
        lib.accept_tree(draft, target, parents, start, 129)
    with pytest.raises(lib.PaError):
        lib.accept_tree(draft, target, parents, start, 0)
    for err, a in ((TypeError, (draft.int(), target, parents, start)), (ValueError, (draft, target[:3], parents, start)),
                   (TypeError, (draft, target, parents.long(), start)), (ValueError, (draft, target, parents[::2], start)),
                   (ValueError, (draft, target, parents, start[:0]))):
        with pytest.raises(err):
            lib.accept_tree(*a, 6)


def paths(nodes, lengths, width, g):
    path = torch.full((len(nodes), width), -1, dtype=torch.int32)
    for b, (c, n) in enumerate(zip(nodes, lengths)):
        path[b, :n] = torch.randperm(c, generator=g)[:n].sort().values
    return path


@pytest.mark.parametrize("dtype,fp8,d,hkv,bs", [(torch.float16, False, 64, 1, 16), (torch.bfloat16, False, 128, 8, 32),
                                                (torch.float16, True, 128, 3, 16)])
@pytest.mark.parametrize("layers", [1, 3, 65])
def test_commit(dev, dtype, fp8, d, hkv, bs, layers):
    nodes = [7, 1, 0, 128, 26, 40, 16]
    lens = [100, 1, 20, 128, 300, 47, 16]
    lengths = [3, 1, 0, 128, 26, 20, 0]
    x = Batch(lens, hkv, hkv, d, bs, dtype, seed=layers, fp8=fp8, stale=False)
    path = paths(nodes, lengths, 128, x.gen)
    shape = x.k.shape
    pools = [torch.randint(0, 256, shape, generator=x.gen, dtype=torch.uint8) if fp8 else
             torch.randn(shape, generator=x.gen).to(dtype) for _ in range(2 * layers)]
    n = torch.tensor(lengths, dtype=torch.int32)
    want, new = commit_reference(pools, x.tables, x.lens, nodes, path, n, bs)
    got = [p.to(dev) for p in pools]
    ks, vs = (got[0], got[1]) if layers == 1 else (got[:layers], got[layers:])
    r = lib.commit_path(ks, vs, x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev), path.to(dev), n.to(dev))
    assert same_bits(r, new)
    for i, (a, b) in enumerate(zip(got, want)):
        assert same_bits(a, b), f"cache {i}"
    assert lib.read_device_errors(dev) == 0


def test_commit_bad_paths_are_left_alone(dev):
    nodes, lens = [6, 6, 6, 6, 6, 6], [30, 30, 30, 30, 30, 30]
    x = Batch(lens, 2, 2, 64, 16, torch.float16, seed=1, stale=False)
    path = torch.tensor([[0, 2, 5, -1], [0, 2, 2, -1], [3, 1, -1, -1], [0, 6, -1, -1], [-1, 2, -1, -1], [0, 1, 2, 3]],
                        dtype=torch.int32)
    n = torch.tensor([3, 3, 2, 2, 2, 5], dtype=torch.int32)          # the last is longer than its row
    good = torch.tensor([3, 0, 0, 0, 0, 0], dtype=torch.int32)
    (wk, wv), _ = commit_reference([x.k, x.v], x.tables, x.lens, nodes, path, good, 16)
    k, v = x.k.to(dev), x.v.to(dev)
    args = [x.tables.to(dev), x.lens.to(dev), starts(nodes).to(dev), path.to(dev)]
    r = lib.commit_path(k, v, *args, n.to(dev))
    assert r.tolist() == [27, 30, 30, 30, 30, 30] and same_bits(k, wk) and same_bits(v, wv)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_INDEX
    r = lib.commit_path(k, v, *args, torch.tensor([-1, 7, 1 << 30, 0, 0, 0], dtype=torch.int32, device=dev))
    assert r.tolist() == [30, 30, 30, 24, 24, 24] and same_bits(k, wk)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_INDEX
    tables = x.tables.clone()
    tables[0] = 10 ** 6
    r = lib.commit_path(k, v, tables.to(dev), *args[1:], good.to(dev))
    assert r.tolist() == [27, 24, 24, 24, 24, 24] and same_bits(k, wk)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    for t in ([-4] * 6, [1 << 20] * 6):
        lib.commit_path(k, v, args[0], torch.tensor(t, dtype=torch.int32, device=dev), *args[2:], 0 * good.to(dev))
        assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    assert same_bits(k, wk) and same_bits(v, wv)
    with pytest.raises(lib.PaError):
        lib.commit_path(k, k, *args, n.to(dev))
    with pytest.raises(lib.PaError):
        lib.commit_path([k, v], [v, k], *args, n.to(dev))
    with pytest.raises(lib.PaError):
        lib.commit_path(k, v, *args, n.to(dev), new_lens=args[1])
    with pytest.raises(ValueError):
        lib.commit_path([k, v], [v, k[:1]], *args, n.to(dev))
    with pytest.raises(TypeError):
        lib.commit_path(k, v, *args[:3], path.long().to(dev), n.to(dev))


def test_empty_batches(dev):
    """No sequences, or no tokens, in every call of the step."""
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float16, device=dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    start, tables = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(0, 3, dtype=torch.int32, device=dev)
    rows = torch.zeros(0, 4, 64, dtype=torch.float16, device=dev)
    out = lib.tree_attention(rows, kc, kc, tables, none, start, none, 0.1, 4, 48)
    assert out.shape == rows.shape
    path, lens, following = lib.accept_tree(none.long(), none.long(), none, start, 4)
    assert path.shape == (0, 4) and lens.shape == (0,) and following.shape == (0,)
    assert path.dtype == lens.dtype == torch.int32 and following.dtype == torch.int64
    assert lib.commit_path(kc, kc.clone(), tables, none, start, path, lens).shape == (0,)
    q = lib.norm_rope_and_cache(rows, rows[:, :2], rows[:, :2], none.long(), none.long(), torch.ones(32, device=dev), kc, kc)
    assert q.shape == rows.shape
    # sequences, but no nodes: nothing is accepted and nothing moves
    two = torch.tensor([0, 0, 0], dtype=torch.int32, device=dev)
    held, tables = torch.tensor([20, 0], dtype=torch.int32, device=dev), torch.zeros(2, 3, dtype=torch.int32, device=dev)
    path, lens, following = lib.accept_tree(none.long(), none.long(), None, two, 4)
    assert path.tolist() == [[-1] * 4] * 2 and lens.tolist() == [0, 0] and following.tolist() == [-1, -1]
    assert lib.commit_path(kc, kc.clone(), tables, held, two, path, lens).tolist() == [20, 0]
    assert lib.tree_attention(rows, kc, kc, tables, held, two, None, 0.1, 4, 48).shape == rows.shape
    assert bool((kc == 0).all()) and lib.read_device_errors(dev) == 0


def test_acceptance_results_are_ordinary_tensors(dev):
    """Three parts of one allocation: each can be written, kept and computed with by itself."""
    nodes = [5, 3]
    draft, target = torch.arange(8, device=dev), torch.arange(8, device=dev) + 1
    parents = torch.tensor([-1, 0, 1, 2, 3, -1, 0, 1], dtype=torch.int32, device=dev)
    path, lens, following = lib.accept_tree(draft, target, parents, starts(nodes).to(dev), 5)
    assert lens.tolist() == [5, 3] and following.tolist() == [5, 8]
    kept = following.clone()
    path.fill_(7)
    lens += 1
    assert following.tolist() == kept.tolist() and lens.tolist() == [6, 4] and path.sum().item() == 70
    w = torch.ones(2, device=dev, requires_grad=True)
    (w * lens).sum().backward()
    assert w.grad.tolist() == [6.0, 4.0]
    with torch.inference_mode():
        again, _, _ = lib.accept_tree(draft, target, parents, starts(nodes).to(dev), 5)
    assert again.tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, -1, -1]]
