"""Host side of the operators of speculative decoding: argument checks before
anything is enqueued, workspace sizes, what the binding refuses, and the plain
implementations that the GPU tests use.  CPU only."""
import ctypes

import pytest
import torch

import tree_util as tu
from paged_kv_cache_226_gb300 import build, lib

FAKE = ctypes.c_void_p(1 << 20)      # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 2)
BAD, UNSUPPORTED = lib.PA_ERR_INVALID_ARG, lib.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def pa():
    build.build()
    return lib.load()


def shape(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                max_blocks_per_seq=4, num_blocks=16, dtype=lib.PA_FP16, reserved=0)
    base.update(kw)
    return ctypes.byref(lib.PaShape(**base))


def norm(pa, shp=None, fp8=None, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, na=1, ax=None,
             slot=FAKE, inv=FAKE, rot=128, il=0, factor=1.0, out=FAKE, os=1024, kc=FAKE, vc=FAKE, T=3)
    a.update(kw)
    if fp8:
        return pa.pa_norm_rope_and_cache_fp8(*a.values(), *fp8, shp or shape(), None)
    return pa.pa_norm_rope_and_cache(*a.values(), shp or shape(), None)


def test_norm_checks(pa):
    for kw in (dict(k=None), dict(v=None), dict(pos=None), dict(slot=None), dict(inv=None), dict(kc=None),
               dict(out=None), dict(k=ODD), dict(qw=ODD), dict(kw=ODD), dict(ax=BYTE), dict(ks=255), dict(T=-1),
               dict(rot=144), dict(il=2), dict(factor=float("nan")), dict(eps=-1e-9), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(na=0), dict(na=9), dict(na=-1), dict(qs=1032)):
        assert norm(pa, **kw) == BAD, kw
    for kw in (dict(rot=8), dict(rot=120)):
        assert norm(pa, **kw) == UNSUPPORTED, kw
    assert norm(pa, shape(head_dim=96)) == UNSUPPORTED
    assert norm(pa, shape(head_dim=64), fp8=(1.0, 1.0), rot=64) == UNSUPPORTED
    assert norm(pa, fp8=(0.0, 1.0)) == BAD
    assert norm(pa, T=0, k=None, q=None, qw=None, kw=None) == lib.PA_OK


def tree(pa, shp=None, fp8=None, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, par=FAKE, scale=0.1, T=9, max_q=8, max_ctx=64,
             ws=FAKE, n=1 << 40, out=ctypes.c_void_p(2 << 20))
    a.update(kw)
    v = list(a.values())
    if fp8:
        return pa.pa_tree_attention_fp8(*v[:8], *fp8, *v[8:], shp or shape(), None)
    return pa.pa_tree_attention(*v, shp or shape(), None)


def test_tree_checks(pa):
    for kw in (dict(q=None), dict(q=ODD), dict(kc=None), dict(vc=None), dict(vc=ODD), dict(bt=None), dict(cl=None),
               dict(qs=None), dict(qs=BYTE), dict(par=BYTE), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(T=-1), dict(T=1 << 31), dict(max_q=-1),
               dict(max_ctx=-1), dict(out=None), dict(out=ODD), dict(out=FAKE), dict(ws=ODD)):
        assert tree(pa, **kw) == BAD, kw
    assert tree(pa, max_q=129) == UNSUPPORTED
    assert tree(pa, ws=None) == lib.PA_ERR_WORKSPACE
    n = pa.pa_tree_attention_workspace_size(shape(), 8, 64)
    assert n > 0 and tree(pa, n=n - 1) == lib.PA_ERR_WORKSPACE
    assert pa.pa_tree_attention_workspace_size(shape(), 129, 64) == 0
    assert pa.pa_tree_attention_workspace_size(shape(), -1, 64) == 0
    assert pa.pa_tree_attention_workspace_size(shape(), 8, -1) == 0
    assert pa.pa_tree_attention_workspace_size(shape(head_dim=96), 8, 64) == 0
    assert tree(pa, shape(num_q_heads=64, num_kv_heads=2)) == UNSUPPORTED
    assert tree(pa, shape(head_dim=64), fp8=(1.0, 1.0)) == UNSUPPORTED
    assert tree(pa, fp8=(1.0, -1.0)) == BAD and tree(pa, fp8=(float("nan"), 1.0)) == BAD
    assert tree(pa, shape(num_seqs=0), q=None, out=None, qs=None, ws=None) == lib.PA_OK
    assert tree(pa, T=0, q=None, out=None) == lib.PA_OK
    assert tree(pa, max_q=0) == lib.PA_OK and tree(pa, max_ctx=0) == lib.PA_OK


def test_tree_sizes_and_overlaps(pa):
    assert tree(pa, scale=3e38) == BAD and tree(pa, scale=1e30, fp8=(1e10, 1.0), shp=shape(head_dim=128)) == BAD
    row = 8 * 128 * 2
    for off in (16, row, 9 * row - 16):
        assert tree(pa, T=9, q=ctypes.c_void_p(1 << 20), out=ctypes.c_void_p((1 << 20) + off)) == BAD
        assert tree(pa, T=9, q=ctypes.c_void_p((1 << 20) + off), out=ctypes.c_void_p(1 << 20)) == BAD
    # one KV head and 2^30 tokens: 2^24 key tiles and the pair, 128 sequences of them are too many
    big = shape(num_seqs=128, num_q_heads=1, num_kv_heads=1, block_size=16, max_blocks_per_seq=1 << 26)
    n = pa.pa_tree_attention_workspace_size(big, 8, 1 << 30)
    assert n > 0 and tree(pa, big, n=n, max_ctx=1 << 30) == UNSUPPORTED


@pytest.mark.parametrize("heads,kv_heads,nodes", [(8, 8, 16), (64, 8, 64), (16, 2, 128), (32, 32, 8), (5, 5, 3)])
def test_tree_workspace_grows_with_the_batch(pa, heads, kv_heads, nodes):
    """What is enough for a batch is enough for fewer sequences or shorter contexts."""
    for blocks in (1, 8, 32, 33, 48, 64, 65, 500):
        sizes = [pa.pa_tree_attention_workspace_size(
            shape(num_seqs=n, num_q_heads=heads, num_kv_heads=kv_heads, block_size=16, max_blocks_per_seq=blocks),
            nodes, 16 * blocks) for n in range(40)]
        assert sizes == sorted(sizes) and sizes[0] >= 16
    for n in (1, 9, 16, 40):
        sizes = [pa.pa_tree_attention_workspace_size(
            shape(num_seqs=n, num_q_heads=heads, num_kv_heads=kv_heads, block_size=16, max_blocks_per_seq=500),
            nodes, longest) for longest in range(0, 8000, 61)]
        assert sizes == sorted(sizes)


def test_commit_refuses_caches_over_one_another(pa):
    size, at = 16 * 16 * 2 * 128 * 2, 1 << 24
    for off in (16, size - 16):
        assert commit(pa, ks=(at,), vs=(at + off,)) == BAD
        assert commit(pa, ks=(at + off, 1 << 26), vs=(1 << 27, at)) == BAD


def accept(pa, **kw):
    a = dict(draft=FAKE, target=FAKE, par=FAKE, qs=FAKE, B=2, T=9, max_q=8, path=FAKE, lens=FAKE, next=FAKE)
    a.update(kw)
    return pa.pa_accept_tree(*a.values(), None)


def test_accept_checks(pa):
    odd4 = ctypes.c_void_p((1 << 20) + 4)
    for kw in (dict(draft=None), dict(target=None), dict(qs=None), dict(path=None), dict(lens=None), dict(next=None),
               dict(B=-1), dict(T=-1), dict(T=1 << 31), dict(max_q=0), dict(max_q=-1), dict(draft=odd4),
               dict(target=odd4), dict(next=odd4), dict(par=BYTE), dict(qs=BYTE), dict(path=BYTE), dict(lens=BYTE)):
        assert accept(pa, **kw) == BAD, kw
    assert accept(pa, max_q=129) == UNSUPPORTED
    assert accept(pa, B=0, draft=None, qs=None, path=None) == lib.PA_OK


def commit(pa, shp=None, fn="pa_commit_path", ks=(1 << 20,), vs=(2 << 20,), **kw):
    arrays = [(ctypes.c_void_p * max(1, len(x)))(*x) for x in (ks, vs)]
    a = dict(k=arrays[0], v=arrays[1], layers=len(ks), bt=FAKE, cl=FAKE, qs=FAKE, path=FAKE, stride=8, lens=FAKE,
             new=ctypes.c_void_p(3 << 20))
    a.update(kw)
    return getattr(pa, fn)(*a.values(), shp or shape(), None)


def test_commit_checks(pa):
    for kw in (dict(k=None), dict(v=None), dict(bt=None), dict(cl=None), dict(qs=None), dict(path=None),
               dict(lens=None), dict(new=None), dict(new=FAKE), dict(new=BYTE), dict(path=BYTE), dict(stride=-1),
               dict(layers=0), dict(layers=-1), dict(ks=(0,)), dict(ks=((1 << 20) + 8,)), dict(vs=(1 << 20,)),
               dict(ks=(1 << 20, 5 << 20), vs=(2 << 20, 5 << 20)), dict(ks=(1 << 20, 1 << 20), vs=(2 << 20, 4 << 20))):
        assert commit(pa, **kw) == BAD, kw
    assert commit(pa, ks=tuple((i + 1) << 20 for i in range(1025)),
                  vs=tuple((i + 2000) << 20 for i in range(1025))) == UNSUPPORTED
    assert commit(pa, shape(head_dim=64), fn="pa_commit_path_fp8") == UNSUPPORTED
    assert commit(pa, shape(num_seqs=0), k=None, bt=None, new=None) == lib.PA_OK


def test_binding_refuses_before_the_gpu(pa):
    kv = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    t = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.ones(1, dtype=torch.int32)
    x = torch.zeros(1, 4, 64, dtype=torch.float16)
    calls = {
        lib.norm_rope_and_cache: dict(q=x, k=x[:, :2], v=x[:, :2], positions=lens.long(), slot_mapping=lens.long(),
                                      inv_freq=torch.ones(32), k_cache=kv, v_cache=kv),
        lib.tree_attention: dict(q=x, k_cache=kv, v_cache=kv, block_tables=t, context_lens=lens, query_start=lens,
                                 parents=None, scale=1.0, max_query_len=1, max_context_len=16),
    }
    for fn, args in calls.items():
        with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
            fn(**args)
        for odd in (None, 3, kv.numpy()):
            with pytest.raises(TypeError, match="k_cache must be a torch.Tensor"):
                fn(**{**args, "k_cache": odd})
        with pytest.raises(TypeError):
            fn()
    args = dict(k_caches=kv, v_caches=kv, block_tables=t, context_lens=lens, query_start=t[0], path=t, path_lens=lens)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        lib.commit_path(**args)
    with pytest.raises(TypeError, match="k_cache must be a torch.Tensor"):
        lib.commit_path(**{**args, "k_caches": [1], "v_caches": [kv]})
    with pytest.raises(ValueError, match="for every layer"):
        lib.commit_path(**{**args, "k_caches": [kv, kv], "v_caches": [kv]})
    with pytest.raises(ValueError, match="for every layer"):
        lib.commit_path(**{**args, "k_caches": [kv]})
    with pytest.raises(ValueError, match="not be empty"):
        lib.commit_path(**{**args, "k_caches": [], "v_caches": []})
    with pytest.raises(ValueError, match="draft_tokens must be a CUDA tensor"):
        lib.accept_tree(lens.long(), lens.long(), None, t[0], 4)
    with pytest.raises(TypeError, match="expected 14 arguments"):
        lib._load_native().tree_attention(kv)


def test_plain_acceptance_by_hand():
    """   0 -> 1 -> 3      and    2 -> 4 -> 5 below 0: the model wants the second branch
    up to 4, and both of the first."""
    parents = torch.tensor([-1, 0, 0, 1, 2, 4], dtype=torch.int32)
    draft = torch.tensor([7, 10, 11, 12, 13, 14])
    target = torch.tensor([11, 12, 13, 99, 50, 60])
    path, n, following = tu.accept_reference(draft, target, parents, [6], 6)
    assert path.tolist() == [[0, 2, 4, -1, -1, -1]] and n.tolist() == [3] and following.tolist() == [50]
    target[0] = 10
    path, n, following = tu.accept_reference(draft, target, parents, [6], 6)
    assert path.tolist() == [[0, 1, 3, -1, -1, -1]] and following.tolist() == [99]
    target[0] = 1
    assert tu.accept_reference(draft, target, parents, [6], 6)[1].tolist() == [1]


def test_plain_visibility_by_hand():
    seen = tu.visible([-1, 0, 0, 2], 6, 4)
    assert seen.int().tolist() == [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0], [1, 1, 1, 0, 1, 1]]


@pytest.mark.parametrize("scale,k_scale", [(1e-25, 1e-25), (1e-20, 1e-19), (1e-38, 0.1), (1e-45, 1.0), (-1e-20, 1.0),
                                           (1e30, 1e10), (float("nan"), 1.0)])
def test_scales_whose_product_leaves_fp32(pa, scale, k_scale):
    assert tree(pa, scale=scale, fp8=(k_scale, 1.0)) == BAD
    if k_scale == 1.0:
        assert tree(pa, scale=scale) == BAD


def test_the_smallest_scale(pa):
    """Accepted up to the workspace's check, which comes after the scales'."""
    assert tree(pa, scale=2e-38, ws=None) == lib.PA_ERR_WORKSPACE
    assert tree(pa, scale=2e-19, fp8=(1e-19, 1.0), ws=None) == lib.PA_ERR_WORKSPACE
    assert tree(pa, scale=2e-39, ws=None) == BAD


def test_outputs_over_inputs_are_refused(pa):
    """Entry points that would read what another CTA, or the launch before, has written."""
    at = 1 << 20
    pointers = dict(bt=at, cl=2 * at, qs=3 * at, path=4 * at, lens=5 * at)          # of 2 sequences, 4 blocks, 8 nodes
    for name, size in dict(bt=32, cl=8, qs=12, path=64, lens=8).items():
        for off in (-4, 0, size - 4):
            assert commit(pa, ks=(64 * at,), vs=(128 * at,), **{k: ctypes.c_void_p(v) for k, v in pointers.items()},
                          new=ctypes.c_void_p(pointers[name] + off)) == BAD, (name, off)
    pointers = dict(draft=at, target=2 * at, par=3 * at, qs=4 * at, path=5 * at, lens=6 * at, next=7 * at)
    sizes = dict(draft=72, target=72, par=36, qs=12, path=64, lens=8, next=16)      # of 9 nodes, 8 a path
    for out in ("path", "lens", "next"):
        for name, size in sizes.items():
            for off in (8 - sizes[out], 0, size // 8 * 8 - 8):
                if name == out:
                    continue
                args = {**pointers, out: pointers[name] + off}
                assert accept(pa, **{k: ctypes.c_void_p(v) for k, v in args.items()}) == BAD, (out, name, off)
