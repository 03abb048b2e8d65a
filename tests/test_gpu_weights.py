"""GPU parity of pa_decode_weights and pa_prefill_weights against the
definition in 64 bits (bounds: bounded_util), with NaN in every cache slot and
state entry that no result may depend on."""
import numpy as np
import pytest
import torch

from bounded_util import Batch, decode_reference, half_step, prefill_reference, same_bits, within
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


def _past(x, w, filler):
    """Entries past each length must still hold the filler."""
    at = torch.arange(w.shape[2])
    past = (at >= x.lens[:, None, None]).expand(w.shape)
    assert bool((w.cpu()[past] == filler).all()), "an entry past the length was written"
    return torch.where(past, torch.zeros_like(w.cpu()), w.cpu())


def run_decode(dev, x, before, **kw):
    want, ww, ob, wb = decode_reference(x, before)
    after = torch.full((x.num_seqs, x.hkv, x.tokens), -7.0, device=dev)
    out, got = lib.decode_weights(x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev),
                                  x.lens.to(dev), x.scale, max([1, *x.lens.tolist()]),
                                  weights=before.to(dev) if before is not None else None,
                                  weights_out=after, **x.scales(), **kw)
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    within(out, want, ob, "out")
    within(_past(x, got, -7.0), ww, wb, "weights")


RAGGED = [1, 2, 15, 16, 17, 0, 33, 100, 257, 700]


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [
    (F16, 8, 2, 64, 16), (BF16, 32, 8, 128, 16), (F16, 8, 1, 128, 32), (BF16, 4, 4, 128, 16),
    (F16, 6, 2, 64, 32), (BF16, 10, 2, 128, 16), (F16, 14, 2, 128, 16), (BF16, 2, 1, 64, 16)])
@pytest.mark.parametrize("partition", [None, 32, 256])
def test_decode_weights(dev, dtype, hq, hkv, d, bs, partition):
    x = Batch(RAGGED, hq, hkv, d, bs, dtype, seed=hq + d)
    run_decode(dev, x, x.state(), partition_size=partition)
    if partition is None:
        run_decode(dev, x, None)


@pytest.mark.parametrize("dtype,hq,hkv,bs", [(F16, 8, 2, 16), (BF16, 8, 1, 32), (F16, 3, 1, 16), (BF16, 4, 4, 16)])
@pytest.mark.parametrize("partition", [None, 64])
def test_decode_weights_e4m3(dev, dtype, hq, hkv, bs, partition):
    x = Batch(RAGGED, hq, hkv, 128, bs, dtype, seed=hq, fp8=True)
    run_decode(dev, x, x.state(), partition_size=partition)


def test_decode_weights_long(dev):
    run_decode(dev, Batch([20000, 3], 4, 1, 128, 16, BF16, seed=4), None)
    run_decode(dev, Batch([9001], 8, 1, 128, 32, F16, seed=5, fp8=True), None)


def test_decode_weights_sharp_scores(dev):
    """One token takes nearly all the weight, the others underflow to zero."""
    x = Batch([600, 33], 4, 1, 128, 16, F16, seed=6)
    x.scale = 8.0
    run_decode(dev, x, None)


def test_decode_weights_in_place_and_defaults(dev):
    x = Batch([40, 1, 300], 4, 2, 64, 16, F16, seed=7)
    before = x.state()
    _, ww, _, wb = decode_reference(x, before)
    w = torch.where(torch.isnan(before), torch.full_like(before, -7.0), before).to(dev)
    args = (x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), x.scale, 300)
    out, got = lib.decode_weights(*args, weights=w)
    assert got.data_ptr() == w.data_ptr()
    within(_past(x, got, -7.0), ww, wb, "in place")
    out2, fresh = lib.decode_weights(*args)
    within(fresh, decode_reference(x)[1], decode_reference(x)[3], "from nothing")
    assert same_bits(out, out2)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("d,dtype,fp8", [(64, F16, False), (128, BF16, False), (128, F16, True)])
def test_decode_weights_one_launch(dev, group, d, dtype, fp8):
    """Contexts of one partition, or of up to four short ones cut evenly: the
    partitions are joined in the decode kernel itself."""
    for lens, partition in (([1, 0, 16, 17, 64, 63, 31, 2], 64), ([128, 3, 65, 0, 97, 113], 64),
                            ([256, 255, 193, 33, 1, 0, 16], 64), ([700, 0, 1, 1000, 513], 1008), ([90], 32)):
        x = Batch(lens, 2 * group, 2, d, 16, dtype, seed=group + len(lens), fp8=fp8)
        run_decode(dev, x, x.state(), partition_size=partition)
    run_decode(dev, x, None, partition_size=64)


def test_decode_weights_bound_below_a_length(dev):
    """Tokens past the partitions of max_context_len are not attended, in
    either form, and their entries stay."""
    x = Batch([400, 100, 192, 193], 8, 2, 128, 16, F16, seed=37, stale=False)
    args = (x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), x.scale, 192)
    got = []
    for partition in (64, 32, 192):
        w = torch.full((4, 2, x.tokens), -7.0, device=dev)
        out, _ = lib.decode_weights(*args, weights_out=w, partition_size=partition)
        assert bool((w[0, :, 192:] == -7.0).all()) and bool((w[3, :, 192:] == -7.0).all())
        got.append((out.float(), w))
    x.lens = x.lens.clamp(max=192)
    want, ww, ob, wb = decode_reference(x)
    for out, w in got:
        within(out, want, ob, "out")
        within(_past(x, w, -7.0), ww, wb, "weights")


def test_decode_weights_all_empty(dev):
    x = Batch([0, 0], 4, 2, 64, 16, F16, seed=8)
    run_decode(dev, x, None)


def test_decode_matches_decode_split(dev):
    """Beside the weights, the output is that of the split decode (up to P's
    row sums, taken before their rounding here)."""
    x = Batch([700, 60], 8, 2, 128, 16, BF16, seed=9, stale=False)
    args = (x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev), x.scale, 700)
    a = lib.paged_attention(*args, mode="split", partition_size=256)
    b, _ = lib.decode_weights(*args, partition_size=256)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -8 * float(a.float().abs().max()) * 1.01


def test_bad_tables_and_lengths_are_bounded(dev):
    """A block id outside the pool reads as zeros, a length past the table is
    clamped; both are reported."""
    x = Batch([64, 64], 2, 1, 64, 16, F16, seed=10, stale=False, slack_width=0)
    tables = x.tables.clone()
    tables[0, 1] = -1
    tables[1, 3] = x.k.shape[0]
    x.k[x.tables[0, 1].long()] = 0
    x.v[x.tables[0, 1].long()] = 0
    x.k[x.tables[1, 3].long()] = 0
    x.v[x.tables[1, 3].long()] = 0
    want, ww, ob, wb = decode_reference(x)
    lens = torch.tensor([64, 1000], dtype=torch.int32)
    out, got = lib.decode_weights(x.q.to(dev), x.k.to(dev), x.v.to(dev), tables.to(dev), lens.to(dev),
                                  x.scale, 64)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    within(out, want, ob, "out")
    within(got, ww, wb, "weights")


def test_decode_weights_two_streams_and_graph(dev):
    """Two calls at once with workspaces of their own, and a captured call
    replayed on changed contents."""
    x, y = (Batch([500, 77, 1], 8, 2, 128, 16, F16, seed=s) for s in (11, 12))
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for b, s in zip((x, y), streams):
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            got.append(lib.decode_weights(b.q.to(dev), b.k.to(dev), b.v.to(dev), b.tables.to(dev),
                                          b.lens.to(dev), b.scale, 500))
    torch.cuda.synchronize(dev)
    for b, (out, w) in zip((x, y), got):
        want, ww, ob, wb = decode_reference(b)
        within(out, want, ob, "out")
        within(w, ww, wb, "weights")
    d = dict(q=x.q.to(dev), k_cache=x.k.to(dev), v_cache=x.v.to(dev), block_tables=x.tables.to(dev),
             context_lens=x.lens.to(dev), scale=x.scale, max_context_len=500,
             weights_out=torch.zeros(3, 2, x.tokens, device=dev), out=torch.zeros_like(x.q, device=dev))
    lib.decode_weights(**d)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.decode_weights(**d)
    d["q"].copy_(y.q)
    d["context_lens"].copy_(torch.tensor([300, 77, 0]))
    d["weights_out"].zero_()
    g.replay()
    torch.cuda.synchronize(dev)
    x.q, x.lens = y.q, torch.tensor([300, 77, 0], dtype=torch.int32)
    want, ww, ob, wb = decode_reference(x)
    within(d["out"], want, ob, "replayed out")
    within(d["weights_out"], ww, wb, "replayed weights")


def run_prefill(dev, x, chunks, window, before, max_q=None):
    q = torch.randn(sum(chunks) + 3, x.hq, x.d, generator=x.gen).to(x.dtype)
    q[sum(chunks):] = float("nan")                      # rows behind the last sequence
    ww, wb = prefill_reference(x, q, chunks, window, before)
    start = torch.tensor([0, *chunks]).cumsum(0).to(torch.int32)
    after = torch.full((x.num_seqs, x.hkv, x.tokens), -7.0, device=dev)
    got = lib.prefill_weights(q.to(dev), x.k.to(dev), x.tables.to(dev), x.lens.to(dev), start.to(dev),
                              x.scale, max_q or max([1, *chunks]), max([1, *x.lens.tolist()]),
                              window=window, weights=before.to(dev) if before is not None else None,
                              weights_out=after)
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    within(_past(x, got, -7.0), ww, wb, "weights")


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [
    (F16, 8, 2, 64, 16), (BF16, 32, 8, 128, 16), (F16, 8, 1, 128, 32), (BF16, 4, 4, 128, 16),
    (F16, 6, 2, 64, 32), (BF16, 10, 2, 128, 16), (F16, 14, 2, 128, 16), (BF16, 6, 1, 64, 16)])
@pytest.mark.parametrize("window", [0, 1, 9])
def test_prefill_weights(dev, dtype, hq, hkv, d, bs, window):
    lens = [1, 15, 16, 17, 0, 33, 100, 257, 300, 40, 128, 129]
    chunks = [1, 15, 1, 17, 0, 16, 37, 257, 150, 0, 128, 128]
    x = Batch(lens, hq, hkv, d, bs, dtype, seed=hq + d + window)
    run_prefill(dev, x, chunks, window, x.state())


@pytest.mark.parametrize("hq,hkv,d,dtype,lens", [
    (4, 1, 128, BF16, [128]),                               # one CTA, one whole tile
    (4, 1, 128, F16, [256, 1, 129]),                        # two tiles a CTA
    (3, 1, 64, F16, [257, 0, 512]),                         # clusters of two, some CTAs without tiles
    (8, 2, 128, BF16, [1024, 1000, 17]),                    # of four
    (10, 2, 64, BF16, [1100, 40]),                          # of five
    (7, 1, 128, F16, [2048, 1921, 2000]),                   # of eight
    (16, 8, 64, F16, [4096]),                               # of eight, four tiles a CTA
    (8, 1, 128, BF16, [3970, 4096, 255]),
    (1, 1, 128, BF16, [4097, 130]),                         # too long: two passes
    (16, 16, 64, F16, [100, 300, 500, 512, 260, 31, 1, 0, 77]),   # 144 pairs: one CTA each
    (16, 8, 128, BF16, [129 + 7 * i for i in range(24)])])  # 192 pairs: two passes
@pytest.mark.parametrize("window", [1, 16])
def test_prefill_weights_one_launch_or_two(dev, hq, hkv, d, dtype, lens, window):
    """Windows over contexts at the bounds of the one-launch form's clusters."""
    x = Batch(lens, hq, hkv, d, 16, dtype, seed=hq + len(lens))
    run_prefill(dev, x, [min(n, 16 + 9 * (i % 3)) for i, n in enumerate(lens)], window, x.state())
    run_prefill(dev, x, [min(n, 5) for n in lens], 0, None)


def test_prefill_weights_one_launch_bad_block(dev):
    """A block id outside the pool is reported and reads as zeros."""
    x = Batch([700, 300], 4, 2, 128, 16, F16, seed=33, stale=False)
    tables = x.tables.clone()
    x.k[x.tables[0, 5].long()] = 0
    x.k[x.tables[1, 2].long()] = 0
    tables[0, 5], tables[1, 2] = x.k.shape[0] + 7, -3
    start = torch.tensor([0, 8, 16], dtype=torch.int32, device=dev)
    q = torch.randn(16, 4, 128, generator=x.gen).to(F16).to(dev)
    w = lib.prefill_weights(q, x.k.to(dev), tables.to(dev), x.lens.to(dev), start, x.scale, 8, 700)
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
    ww, wb = prefill_reference(x, q.cpu(), [8, 8], 0, None)
    within(w, ww, wb, "weights")


def test_prefill_weights_long(dev):
    x = Batch([3001, 700], 4, 1, 128, 16, BF16, seed=21)
    run_prefill(dev, x, [513, 700], 0, None)
    x = Batch([5000, 2000, 31], 8, 2, 128, 16, F16, seed=22)
    run_prefill(dev, x, [64, 300, 31], 32, x.state(), max_q=512)


def test_prefill_weights_sharp_scores(dev):
    x = Batch([400, 150], 8, 2, 128, 16, F16, seed=23)
    x.scale = 6.0
    run_prefill(dev, x, [200, 150], 0, None)


def test_prefill_weights_no_queries(dev):
    """No chunk at all: what was added up before is carried over."""
    x = Batch([30, 1], 4, 2, 64, 16, F16, seed=24)
    run_prefill(dev, x, [0, 0], 0, x.state())


def test_one_query_equals_decode(dev):
    x = Batch([300, 17, 1000], 8, 2, 128, 16, BF16, seed=25)
    start = torch.arange(4, dtype=torch.int32)
    a = lib.prefill_weights(x.q.to(dev), x.k.to(dev), x.tables.to(dev), x.lens.to(dev), start.to(dev),
                            x.scale, 1, 1000)
    _, ww, _, wb = decode_reference(x)
    within(a, ww, wb, "one query")


def test_prefill_weights_bad_bounds_are_reported(dev):
    """A chunk longer than its context, rows past q, a length past the bound."""
    x = Batch([20, 40], 2, 1, 64, 16, F16, seed=26, stale=False)
    q = torch.randn(30, 2, 64, generator=x.gen).to(F16)
    args = (q.to(dev), x.k.to(dev), x.tables.to(dev), x.lens.to(dev))
    for start, bound in (([0, 25, 26], 40), ([0, 5, 40], 40), ([0, 5, 10], 39)):
        w = lib.prefill_weights(*args, torch.tensor(start, dtype=torch.int32, device=dev), x.scale, 32, bound)
        assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_CONTEXT
        assert bool(torch.isfinite(w).all())


def test_refusals(dev):
    x = Batch([20, 40], 4, 2, 64, 16, F16, seed=27, stale=False)
    d = dict(q=x.q.to(dev), k_cache=x.k.to(dev), v_cache=x.v.to(dev), block_tables=x.tables.to(dev),
             context_lens=x.lens.to(dev), scale=x.scale, max_context_len=40)
    w = torch.zeros(2, 2, x.tokens, device=dev)
    for bad in (dict(weights=w.double()), dict(weights=w[:, :, :16].contiguous()), dict(weights=w[:1]),
                dict(weights=w, weights_out=torch.zeros(2, 2, x.tokens + 1, device=dev)),
                dict(k_scale=1.0, v_scale=1.0), dict(out=d["q"][:1]), dict(weights=w.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lib.decode_weights(**d, **bad)
    for bad, status in ((dict(partition_size=24), lib.PA_ERR_INVALID_ARG),
                        (dict(max_context_len=-1), lib.PA_ERR_INVALID_ARG),
                        (dict(workspace=torch.zeros(64, dtype=torch.uint8, device=dev)), lib.PA_ERR_WORKSPACE)):
        with pytest.raises(lib.PaError) as e:
            lib.decode_weights(**{**d, **bad})
        assert e.value.status == status
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    p = dict(q=d["q"], k_cache=d["k_cache"], block_tables=d["block_tables"], context_lens=d["context_lens"],
             query_start=start, scale=x.scale, max_query_len=1, max_context_len=40)
    for bad in (dict(query_start=start.long()), dict(q=d["q"].bfloat16()), dict(weights=w[:1]),
                dict(k_cache=torch.zeros(x.k.shape, dtype=torch.uint8, device=dev))):
        with pytest.raises((ValueError, TypeError)):
            lib.prefill_weights(**{**p, **bad})
    for bad in (dict(scale=0.0), dict(scale=float("inf")), dict(window=-1), dict(max_query_len=-1),
                dict(workspace=torch.zeros(1, dtype=torch.uint8, device=dev))):
        with pytest.raises(lib.PaError):
            lib.prefill_weights(**{**p, **bad})


@pytest.mark.parametrize("fp8", [False, True])
def test_step_plan(dev, fp8):
    """StepPlan's weights mode: the cache write and the weighing decode, called,
    and replayed as a graph on new contents, equal the calls one by one."""
    x = Batch([300, 17, 64], 8, 2, 128, 16, BF16, seed=51, fp8=fp8, stale=False)
    kn, vn = (torch.randn(3, 2, 128, generator=x.gen).to(BF16).to(dev) for _ in range(2))
    at = (x.lens - 1).long()
    slots = (x.tables[torch.arange(3), at // 16].long() * 16 + at % 16).to(dev)
    start = x.state().nan_to_num(0.0).to(dev)

    def one_by_one(q, weights):
        k, v = x.k.to(dev), x.v.to(dev)
        if fp8:
            lib.reshape_and_cache_fp8(kn, vn, slots, k, v, x.k_scale, x.v_scale)
        else:
            lib.reshape_and_cache(kn, vn, slots, k, v)
        out, w = lib.decode_weights(q, k, v, x.tables.to(dev), x.lens.to(dev), x.scale, 300, weights=weights.clone(),
                                    **x.scales())
        return out, w, k

    q, k, v, w = x.q.to(dev), x.k.to(dev), x.v.to(dev), start.clone()
    plan = lib.StepPlan(q, kn, vn, slots, k, v, x.tables.to(dev), x.lens.to(dev), x.scale, 300, mode="weights",
                        weights=w, **x.scales())
    want = one_by_one(q, start)
    assert same_bits(plan(), want[0]) and same_bits(w, want[1]) and same_bits(k, want[2])
    plan.capture_graph()
    q.copy_(torch.randn(q.shape, generator=x.gen))
    w.copy_(start)
    want = one_by_one(q, start)
    assert same_bits(plan.replay(), want[0]) and same_bits(plan.weights_out, want[1])
    with pytest.raises(ValueError):
        lib.StepPlan(q, kn, vn, slots, k, v, x.tables.to(dev), x.lens.to(dev), x.scale, 300, mode="weights", **x.scales())
    with pytest.raises(ValueError):
        lib.StepPlan(q, kn, vn, slots, k, v, x.tables.to(dev), x.lens.to(dev), x.scale, 300, weights=w, **x.scales())
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("hq,hkv,d,high", [(8, 2, 64, 250), (8, 2, 128, 900), (32, 8, 128, 3000)])
def test_captured_calls_follow_the_lengths(dev, hq, hkv, d, high):
    """Both operators captured once and replayed with other lengths, empty and
    full ones among them, against eager calls, bit for bit."""
    x = Batch([high] * 4, hq, hkv, d, 16, F16, seed=41, stale=False)
    q, k, v, tables = x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev)
    chunk = torch.randn(64, hq, d, generator=x.gen).to(F16).to(dev)
    start = torch.tensor([0, 16, 32, 48, 64], dtype=torch.int32, device=dev)
    lens = x.lens.to(dev)
    wd, wp = (torch.zeros(4, hkv, x.tokens, device=dev) for _ in range(2))
    out = torch.empty_like(q)

    def step(a, b, o):
        lib.decode_weights(q, k, v, tables, lens, x.scale, high, weights_out=a, out=o)
        lib.prefill_weights(chunk, k, tables, lens, start, x.scale, 16, high, weights_out=b)

    step(wd, wp, out)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(wd, wp, out)
    for now in ([high, 17, 16, 100], [16, high, 129, 128], [high] * 4, [33, 20, 16, 16]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        for t in (wd, wp):
            t.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize(dev)
        a, b, o = (torch.full_like(t, -7.0) for t in (wd, wp, out))
        step(a, b, o)
        torch.cuda.synchronize(dev)
        assert same_bits(wd, a) and same_bits(wp, b) and same_bits(out, o)
    del g
    assert lib.read_device_errors(dev) == 0


def _crafted(kind, k, v, group=4):
    """One sequence of tokens whose K has k[i] and whose V has v[i] in its first dim (zero elsewhere),
    read by queries that are one in that dim: out[0, :, 0] is sum p v."""
    dtype, fp8 = {"fp16": (F16, False), "bf16": (BF16, False), "e4m3": (F16, True)}[kind]
    x = Batch([len(k)], group, 1, 128, 16, dtype, seed=1, fp8=fp8, stale=False)
    x.k_scale, x.v_scale = (1.0, 1.0) if fp8 else (None, None)
    at = torch.arange(len(k))
    for cache, values in ((x.k, k), (x.v, v)):
        cache.zero_()
        row = torch.tensor(values, dtype=torch.float32)
        row = row.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else row.to(dtype)
        cache[x.tables[0, at // 16].long(), at % 16, 0, 0] = row
    x.q.zero_()
    x.q[:, :, 0] = 1
    return x


def _first_dim(dev, x, partition):
    out, _ = lib.decode_weights(x.q.to(dev), x.k.to(dev), x.v.to(dev), x.tables.to(dev), x.lens.to(dev),
                                x.scale, int(x.lens.max()), partition_size=partition, **x.scales())
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0
    return out[0, :, 0].double().cpu()


@pytest.mark.parametrize("partition", [16, 64, 1024])
@pytest.mark.parametrize("kind,high,low", [("e4m3", 0.0, 0.97 * 2.0 ** -12), ("fp16", 0.0, 0.97 * 2.0 ** -12),
                                           ("fp16", 2.0 ** -12, 0.9 * 2.0 ** -20), ("e4m3", 0.0, 0.9 * 2.0 ** -18),
                                           ("bf16", 2.0 ** -10, 0.97 * 2.0 ** -18)])
def test_decode_probabilities_hold_32_bits(dev, kind, high, low, partition):
    """Probabilities of 1/2 + high + low beside ones of 1, the values chosen so
    that all but `low` cancels: a P in fewer bits than the plain form's loses it.

    P carries at most 2^-21 of itself (the scale in log2 units 2^-23, the
    difference to a reference 2^7 below 2^-22, the exponential 2^-22.5), the
    parts of the split 2^-22 and the sums 2^-23 of their terms, which are 1 at
    most: 2^-20 in all."""
    p = 0.5 + high + low
    x = _crafted(kind, [0.0, -1.0, -1.0, 0.0] * 20, [-1.0, 1.0, 1.0, -2 * high] * 20)
    x.scale = float(np.float32(-np.log(p)))
    p = float(np.exp(-x.scale))
    want = (2 * p - 1 - 2 * high) / (2 + 2 * p)
    got = _first_dim(dev, x, partition)
    assert bool(((got - want).abs() <= half_step(x.dtype) * abs(want) + 2.0 ** -20 + (kind != "bf16") * 2.0 ** -25).all()), \
        (got.tolist(), want)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("n,partition", [(1000, 1008), (4000, 4096)])
def test_decode_small_probabilities_add_up(dev, kind, n, partition):
    """One heavy token of value 0 and n light ones of weight 2^-26 and value 1:
    the light ones' sum is the output.  Each may lose 2^-32 of the largest
    weight, and 2^-20 of itself; an fp16 output has steps of 2^-24."""
    x = _crafted(kind, [0.0] + [-1.0] * n, [0.0] + [1.0] * n)
    x.scale = float(np.float32(26 * np.log(2)))
    p = float(np.exp(-x.scale))
    want = n * p / (1 + n * p)
    got = _first_dim(dev, x, partition)
    bound = (half_step(x.dtype) + 2.0 ** -20) * want + n * 2.0 ** -32 + (kind != "bf16") * 2.0 ** -25
    assert bool(((got - want).abs() <= bound).all()), (got.tolist(), want, bound)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("apart", [False, True])
def test_step_plan_capture_makes_no_step(dev, fp8, apart):
    """A capture leaves the weights as they were, asked for or made by the
    first replay; each replay is exactly one step."""
    x = Batch([300, 17, 64], 8, 2, 128, 16, BF16, seed=52, fp8=fp8, stale=False)
    kn, vn = (torch.randn(3, 2, 128, generator=x.gen).to(BF16).to(dev) for _ in range(2))
    at = (x.lens - 1).long()
    slots = (x.tables[torch.arange(3), at // 16].long() * 16 + at % 16).to(dev)
    start = x.state().nan_to_num(0.0).to(dev)

    def plan():
        w = start.clone()
        out = torch.full_like(w, -7.0) if apart else None
        return w, lib.StepPlan(x.q.to(dev), kn, vn, slots, x.k.to(dev), x.v.to(dev), x.tables.to(dev),
                               x.lens.to(dev), x.scale, 300, mode="weights", weights=w, weights_out=out,
                               **x.scales())

    w, eager = plan()
    once = eager().clone(), eager.weights_out.clone()
    twice = eager().clone(), eager.weights_out.clone()
    for captured in (False, True):
        w, p = plan()
        if captured:
            p.capture_graph()
            p.capture_graph()
            assert same_bits(w, start) and (not apart or bool((p.weights_out == -7.0).all()))
        assert same_bits(p.replay(), once[0]) and same_bits(p.weights_out, once[1])
        assert same_bits(p.replay(), twice[0]) and same_bits(p.weights_out, twice[1])
        assert not apart or same_bits(w, start)
    torch.cuda.synchronize(dev)
    assert lib.read_device_errors(dev) == 0


# More sequences than a warp walks at a time: ragged, some empty, a whole group of 32 empty.
MANY = {33: [37 * i % 301 for i in range(33)], 70: [53 * i % 401 for i in range(70)],
        100: [0 if 32 <= i < 64 else 29 * i % 257 for i in range(100)],
        97: [0] * 32 + [41 * i % 200 for i in range(65)]}


@pytest.mark.parametrize("n", sorted(MANY))
@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 2, 64, F16), (8, 2, 128, BF16)])
def test_prefill_weights_many_sequences(dev, n, hq, hkv, d, dtype):
    """Whole chunks (several query tiles) and windows in two passes."""
    lens = MANY[n]
    x = Batch(lens, hq, hkv, d, 16, dtype, seed=n)
    run_prefill(dev, x, [min(m, 90 + 7 * (i % 3)) for i, m in enumerate(lens)], 0, x.state())
    lens = [m + 4200 * (i == n // 2) for i, m in enumerate(lens)]         # one too long for the one-launch form
    x = Batch(lens, hq, hkv, d, 16, dtype, seed=n + 1)
    run_prefill(dev, x, [min(m, 20 + i % 5) for i, m in enumerate(lens)], 9, x.state())
    run_prefill(dev, x, [min(m, i % 4) for i, m in enumerate(lens)], 0, None)


def test_window_behind_writers_of_its_inputs(dev):
    """The two passes of a window start early on K, Q, lengths and tables:
    what the kernels directly in front of the call wrote is what they read.
    Eight rounds on a stream without a synchronisation, every round on other
    contents, the writers copies and the cache write of a step."""
    hq, hkv, d, rounds = 8, 2, 128, 8
    xs = [Batch([5000 + 300 * (r % 3), 4100, 700 * (r % 2)], hq, hkv, d, 16, F16, seed=60 + r, stale=False,
                slack_width=60) for r in range(rounds)]
    blocks, width = max(x.k.shape[0] for x in xs), max(x.width for x in xs)
    chunks, qs = [32, 20, 0], []
    start = torch.tensor([0, 32, 52, 52], dtype=torch.int32, device=dev)
    for x in xs:
        x.k = torch.cat([x.k, torch.zeros(blocks - x.k.shape[0], 16, hkv, d, dtype=F16)])
        x.tables = torch.cat([x.tables.clamp(max=blocks - 1),
                              torch.zeros(3, width - x.width, dtype=torch.int32)], 1).contiguous()
        x.width, x.tokens = width, width * 16
        qs.append(torch.randn(52, hq, d, generator=x.gen).to(F16))
    on = [(x.k.to(dev), q.to(dev), x.tables.to(dev), x.lens.to(dev)) for x, q in zip(xs, qs)]
    last = [torch.tensor([int(x.tables[b, (int(n) - 1) // 16]) * 16 + (int(n) - 1) % 16 if n else -1
                          for b, n in enumerate(x.lens)], device=dev) for x in xs]
    k, q, tables, lens = (torch.zeros_like(t) for t in on[0])
    v = torch.zeros_like(k)
    new = [torch.randn(3, hkv, d, generator=x.gen).to(F16) for x in xs]
    newd = [t.to(dev) for t in new]
    got = [torch.zeros(3, hkv, width * 16, device=dev) for _ in xs]
    torch.cuda.synchronize(dev)
    for r in range(rounds):
        tables.copy_(on[r][2]), lens.copy_(on[r][3]), q.copy_(on[r][1]), k.copy_(on[r][0])
        lib.reshape_and_cache(newd[r], newd[r], last[r], k, v)            # the newest keys, just before
        lib.prefill_weights(q, k, tables, lens, start, xs[r].scale, 32, 5600, window=16, weights_out=got[r])
    torch.cuda.synchronize(dev)
    for x, qq, w, t in zip(xs, qs, got, new):
        for b, n in enumerate(x.lens.tolist()):
            if n:
                x.k[int(x.tables[b, (n - 1) // 16]), (n - 1) % 16] = t[b]
        ww, wb = prefill_reference(x, qq, chunks, 16)
        within(w, ww, wb, "weights")
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_decode_sums_do_not_drift(dev, kind):
    """8192 tokens of value 1, then the same keys again with value -1, in one
    partition: the sum climbs and comes back to zero.  Sums that are cut off
    toward zero lose on both ways, some 2^-25 of the sum at each of 512 tiles
    per warp, about 2^-17 of all the weight.  Rounded sums are off by sqrt(512)
    steps of 2^-25 at most, six times that for safety by 2^-18.5 of half the
    largest sum, which is half the weight of a warp's tiles: 2^-20.5."""
    n = 8192
    k = torch.randn(n, generator=torch.Generator().manual_seed(9)).tolist()
    x = _crafted(kind, k + k, [1.0] * n + [-1.0] * n)
    x.scale = 0.25
    got = _first_dim(dev, x, 2 * n)
    assert bool((got.abs() <= 2.0 ** -20.5).all()), got.tolist()
