"""Host side of the bounded-cache operators: argument checks before anything
is enqueued, workspace sizes, rotary frequencies, and the allocator's
truncation.  CPU only."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bounded_util as bu
from paged_kv_cache_226_gb300 import build, lib
from paged_kv_cache_226_gb300 import inputs as pin

FAKE = ctypes.c_void_p(1 << 20)      # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def pa():
    build.build()
    return lib.load()


def shape(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                max_blocks_per_seq=4, num_blocks=16, dtype=lib.PA_FP16, reserved=0)
    base.update(kw)
    return ctypes.byref(lib.PaShape(**base))


def rope(pa, shp=None, fp8=None, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, slot=FAKE, inv=FAKE, rot=128,
             il=0, factor=1.0, out=FAKE, os=1024, kc=FAKE, vc=FAKE, T=3)
    a.update(kw)
    if fp8:
        return pa.pa_rope_and_cache_fp8(*a.values(), *fp8, shp or shape(), None)
    return pa.pa_rope_and_cache(*a.values(), shp or shape(), None)


def test_rope_checks(pa):
    bad, unsup = lib.PA_ERR_INVALID_ARG, lib.PA_ERR_UNSUPPORTED
    for kw in (dict(k=None), dict(v=None), dict(pos=None), dict(slot=None), dict(inv=None), dict(kc=None),
               dict(out=None), dict(k=ODD), dict(q=ODD), dict(out=ODD), dict(ks=255), dict(vs=264 + 4),
               dict(qs=1016), dict(os=1000), dict(qs=1032), dict(T=-1), dict(rot=-16), dict(rot=144),
               dict(il=2), dict(factor=float("nan")), dict(factor=float("inf")),
               dict(pos=ctypes.c_void_p((1 << 20) + 4))):
        assert rope(pa, **kw) == bad, kw
    for kw in (dict(rot=8), dict(rot=120)):
        assert rope(pa, **kw) == unsup, kw
    assert rope(pa, shape(head_dim=96)) == unsup
    assert rope(pa, shape(num_q_heads=0)) == bad
    assert rope(pa, shape(head_dim=64), fp8=(1.0, 1.0), rot=64) == unsup
    assert rope(pa, fp8=(0.0, 1.0)) == bad and rope(pa, fp8=(1.0, float("nan"))) == bad
    assert rope(pa, T=0, k=None, q=None) == lib.PA_OK
    assert pa.pa_rope_and_cache(FAKE, 1024, FAKE, 256, FAKE, 256, FAKE, FAKE, FAKE, 128, 0, 1.0, FAKE, 1024,
                                FAKE, FAKE, 3, None, None) == bad


def weights(pa, shp=None, fp8=None, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, scale=0.1, max_ctx=64, P=32, w=FAKE, wo=FAKE,
             stride=64, ws=FAKE, n=1 << 30, out=FAKE)
    a.update(kw)
    v = list(a.values())
    if fp8:
        return pa.pa_decode_weights_fp8(*v[:6], *fp8, *v[6:], shp or shape(), None)
    return pa.pa_decode_weights(*v, shp or shape(), None)


def test_decode_weights_checks(pa):
    bad = lib.PA_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(kc=ODD), dict(bt=None), dict(max_ctx=-1), dict(P=24), dict(P=0),
               dict(wo=None), dict(wo=ODD), dict(w=ODD), dict(stride=63), dict(out=None), dict(out=ODD),
               dict(ws=ODD)):
        assert weights(pa, **kw) == bad, kw
    assert weights(pa, ws=None) == lib.PA_ERR_WORKSPACE
    n = pa.pa_decode_weights_workspace_size(shape(), 64, 32)
    # 2 x 8 heads x 2 partitions: outputs, maxima, sums and 32 scores each
    assert n == 2 * 8 * 2 * (128 * 4) + 2 * 256 + 2 * 8 * 2 * 32 * 4
    assert weights(pa, n=n - 1) == lib.PA_ERR_WORKSPACE
    assert pa.pa_decode_weights_workspace_size(shape(), 64, 24) == 0
    assert weights(pa, shape(num_q_heads=64, num_kv_heads=2)) == lib.PA_ERR_UNSUPPORTED
    assert weights(pa, shape(head_dim=64), fp8=(1.0, 1.0)) == lib.PA_ERR_UNSUPPORTED
    assert weights(pa, fp8=(1.0, -1.0)) == bad
    assert weights(pa, max_ctx=2 ** 31 - 1, P=16) == lib.PA_ERR_UNSUPPORTED
    assert weights(pa, shape(num_seqs=0), q=None, out=None, wo=None, ws=None) == lib.PA_OK


def prefill(pa, shp=None, **kw):
    a = dict(q=FAKE, kc=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, scale=0.1, T=9, max_q=8, max_ctx=64, window=0,
             w=FAKE, wo=FAKE, stride=64, ws=FAKE, n=1 << 30)
    a.update(kw)
    return pa.pa_prefill_weights(*a.values(), shp or shape(), None)


def test_prefill_weights_checks(pa):
    bad = lib.PA_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(q=ODD), dict(kc=None), dict(qs=None), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(T=-1), dict(max_q=-1), dict(max_ctx=-1), dict(window=-1),
               dict(wo=None), dict(stride=10), dict(ws=ODD)):
        assert prefill(pa, **kw) == bad, kw
    assert prefill(pa, ws=None) == lib.PA_ERR_WORKSPACE
    n = pa.pa_prefill_weights_workspace_size(shape(), 8, 64, 0)
    assert n > 0 and prefill(pa, n=n - 1) == lib.PA_ERR_WORKSPACE
    assert pa.pa_prefill_weights_workspace_size(shape(), 4096, 64, 4) <= n
    assert pa.pa_prefill_weights_workspace_size(shape(), -1, 64, 0) == 0
    assert prefill(pa, shape(num_seqs=0), qs=None, ws=None) == lib.PA_OK


def evict(pa, shp=None, fn="pa_evict", **kw):
    a = dict(kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, seen=ctypes.c_void_p(2 << 20), known=ctypes.c_void_p(3 << 20),
             w=FAKE, p=FAKE, stride=64, budget=32, trigger=32, sinks=4, recent=8, wo=FAKE, po=FAKE,
             new=ctypes.c_void_p(4 << 20), ws=FAKE, n=1 << 30)
    a.update(kw)
    return getattr(pa, fn)(*a.values(), shp or shape(), None)


def test_evict_checks(pa):
    bad = lib.PA_ERR_INVALID_ARG
    for kw in (dict(kc=None), dict(vc=ODD), dict(seen=None), dict(w=None), dict(p=None), dict(wo=None),
               dict(po=None), dict(new=None), dict(stride=63), dict(budget=0), dict(trigger=31),
               dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
               dict(new=FAKE), dict(new=ctypes.c_void_p(2 << 20)), dict(new=ctypes.c_void_p(3 << 20)),
               dict(w=ODD), dict(ws=ODD)):
        assert evict(pa, **kw) == bad, kw
    assert evict(pa, ws=None) == lib.PA_ERR_WORKSPACE
    n = pa.pa_evict_workspace_size(shape(), 32)
    assert evict(pa, n=n - 1) == lib.PA_ERR_WORKSPACE
    assert evict(pa, shape(head_dim=64), fn="pa_evict_fp8") == lib.PA_ERR_UNSUPPORTED
    assert pa.pa_evict_workspace_size(shape(), 0) == 0
    assert evict(pa, shape(num_seqs=0), seen=None, new=None, ws=None) == lib.PA_OK


def test_rope_frequencies():
    inv, f = lib.rope_frequencies(64, 10000.0)
    assert f == 1.0 and inv.dtype == torch.float32 and inv.shape == (32,)
    assert np.allclose(inv.numpy(), 10000.0 ** (-2 * np.arange(32) / 64), rtol=2 ** -24)
    lin, _ = lib.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.allclose(lin, inv / 4, rtol=2 ** -23)
    ntk, _ = lib.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(inv[-1]) / 4, rel_tol=1e-6)
    for kind in ("bands", "yarn"):
        got, f = lib.rope_frequencies(128, 500000.0, kind, 8.0, original_len=8192, slow=1.0, fast=4.0)
        plain, _ = lib.rope_frequencies(128, 500000.0)
        ratio = plain / got
        turns = 8192 * plain / (2 * math.pi)
        assert torch.allclose(ratio[turns > 5], torch.ones(1)) and torch.allclose(ratio[turns < 0.8], torch.full((1,), 8.0))
        assert bool((ratio[1:] - ratio[:-1] >= -1e-5).all())
        assert math.isclose(f, 0.1 * math.log(8) + 1 if kind == "yarn" else 1.0)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=64, scaling="x"),
                dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="yarn", factor=2.0),
                dict(rotary_dim=64, scaling="bands", factor=2.0, original_len=10, slow=4.0, fast=1.0)):
        with pytest.raises(ValueError):
            lib.rope_frequencies(**bad)


def test_truncate():
    pool = pin.BlockPool(8, 16)
    a = pin.PagedKVAllocator(pool)
    a.add_sequence(0)
    a.extend(0, 100)
    table = list(a.page_tables[0])
    a.truncate(0, 33)
    assert a.page_tables[0] == table[:3] and a.token_counts[0] == 33 and pool.num_free == 5
    assert a.append_token(0) == table[2] * 16 + 1
    a.truncate(0, 32)
    assert a.page_tables[0] == table[:2]
    assert a.append_token(0) // 16 not in table[:2]       # a fresh block
    a.truncate(0, 0)
    assert len(a.page_tables[0]) == 1 and a.append_token(0) == table[0] * 16
    with pytest.raises(ValueError):
        a.truncate(0, 2)
    a.fork(0, 1)
    with pytest.raises(ValueError):
        a.truncate(1, 1)


def test_plain_eviction_by_hand():
    """The reference that the GPU tests use, on a cut small enough to follow."""
    x = bu.Batch([6], 1, 1, 64, 16, seed=1, stale=False)
    w = torch.zeros(1, 1, x.tokens)
    w[0, 0, :6] = torch.tensor([0.0, 5.0, 1.0, 1.0, 0.5, 3.0])
    pos = torch.zeros(1, 1, x.tokens, dtype=torch.int32)
    k, v, wo, po, new = bu.evict_reference(x, w, pos, x.lens, None, 4, 4, 1, 1)
    # safe: position 0 (first) and 5 (newest); then 5.0 and the first 1.0; token 5 fills gap 3
    assert new.tolist() == [4] and po[0, 0, :4].tolist() == [0, 1, 2, 5]
    assert wo[0, 0, :4].tolist() == [0.0, 5.0, 1.0, 3.0]
    blk = int(x.tables[0, 0])
    assert torch.equal(k[blk, 3], x.k[blk, 5]) and torch.equal(v[blk, 2], x.v[blk, 2])


def test_binding_refuses_before_the_gpu(pa):
    """What the Python calls say about arguments that cannot be used at all."""
    kv = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    t = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.ones(1, dtype=torch.int32)
    x = torch.zeros(1, 4, 64, dtype=torch.float16)
    w = torch.zeros(1, 2, 32)
    calls = {
        lib.rope_and_cache: dict(q=x, k=x[:, :2], v=x[:, :2], positions=lens.long(), slot_mapping=lens.long(),
                                 inv_freq=torch.ones(32), k_cache=kv, v_cache=kv),
        lib.decode_weights: dict(q=x, k_cache=kv, v_cache=kv, block_tables=t, context_lens=lens, scale=1.0,
                                 max_context_len=16),
        lib.prefill_weights: dict(q=x, k_cache=kv, block_tables=t, context_lens=lens, query_start=lens,
                                  scale=1.0, max_query_len=1, max_context_len=16),
        lib.evict: dict(k_cache=kv, v_cache=kv, block_tables=t, context_lens=lens, seen_lens=lens, budget=4,
                        weights=w, positions=w.int()),
    }
    for fn, args in calls.items():
        with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
            fn(**args)
        for odd in (None, 3, kv.numpy()):
            with pytest.raises(TypeError, match="k_cache must be a torch.Tensor"):
                fn(**{**args, "k_cache": odd})
        with pytest.raises(TypeError):
            fn()
    with pytest.raises(TypeError, match="expected 16 arguments"):
        lib._load_native().evict(kv)


def test_binding_is_built_for_this_torch(pa):
    assert build.native_up_to_date()


@pytest.mark.parametrize("rotary,base,original", [(128, 10000.0, 65536), (64, 10000.0, 65536), (128, 10000.0, 4096),
                                                  (96, 500000.0, 8192), (64, 500.0, 131072)])
def test_yarn_ramp(rotary, base, original):
    """The ramp runs from the pair that turns 32 times over the original length
    to the one that turns once, in whole pairs, also where that one lies past
    the last of the R/2 pairs (up to R - 1)."""
    factor = 8.0
    got, mult = lib.rope_frequencies(rotary, base, "yarn", factor, original_len=original)

    def pair(turns):
        return rotary * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))

    first, last = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rotary - 1)
    for i in range(rotary // 2):
        f = base ** (-2 * i / rotary)
        share = min(max((i - first) / (last - first), 0.0), 1.0)        # of the stretched frequency
        assert math.isclose(float(got[i]), f * (1 - share) + f / factor * share, rel_tol=2.0 ** -23), i
    assert mult == 0.1 * math.log(factor) + 1


def test_binding_calls_the_loaded_library(pa, monkeypatch):
    """What the four calls enqueue, and the error bits that they set, belong to
    the library that every other call uses."""
    native = lib._load_native()
    assert lib._bound is pa
    other = ctypes.CDLL(lib.LIB_PATH)                  # a handle of its own
    monkeypatch.setattr(lib, "_lib", other)
    with pytest.raises(TypeError):
        lib.evict(*[None] * 7, torch.zeros(1))
    assert lib._bound is other and lib._native is native
    monkeypatch.undo()
    with pytest.raises(TypeError):
        lib.prefill_weights(*[None] * 8)
    assert lib._bound is pa
    for bad in (0, "x", None):
        with pytest.raises((TypeError, ValueError)):
            native.bind(bad)
    with pytest.raises(ImportError, match="pa_rope_and_cache"):
        native.bind(ctypes.CDLL(None)._handle)
