"""Waits of the attention-weights kernels that run out: the kernels end and
report PA_DEVERR_WAIT_TIMEOUT, the context stays usable, and the next call on
the same arrays is right.  As in test_gpu_wait_timeout.py, a build with test
hooks (include/pa_test.h) withholds one CTA's tiles, so that no copy is in
flight, and its waits give up after a few milliseconds."""
import ctypes

import pytest
import torch

from bounded_util import Batch, decode_reference, prefill_reference, within
from paged_kv_cache_226_gb300 import build, lib

pytestmark = pytest.mark.gpu

SHORT_LIMIT_NS = 2_000_000          # 2 ms
PRODUCT_LIMIT_NS = 1_000_000_000    # the product build's one second


@pytest.fixture(scope="module")
def test_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L = lib.load(build.build(test_hooks=True))
    L.pa_test_set_wait_fault.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_ulonglong]
    L.pa_test_set_wait_fault.restype = ctypes.c_int
    return L


def timed_out_then_right(test_lib, monkeypatch, faults, call, check):
    dev = torch.device("cuda:0")
    build.build()
    monkeypatch.setattr(lib, "_lib", test_lib)
    lib.read_device_errors(dev)
    call()                                               # set-up, and the sizes are right
    check()
    assert lib.read_device_errors(dev) == 0
    try:
        for cta, tile in faults:
            assert test_lib.pa_test_set_wait_fault(cta, tile, SHORT_LIMIT_NS) == lib.PA_OK
            call()
            torch.cuda.synchronize(dev)                  # the kernels end: no hang
            flags = lib.read_device_errors(dev)
            assert flags == lib.PA_DEVERR_WAIT_TIMEOUT, f"CTA {cta}, tile {tile}: flags {flags}"
    finally:
        assert test_lib.pa_test_set_wait_fault(-1, 0, PRODUCT_LIMIT_NS) == lib.PA_OK
    call()
    torch.cuda.synchronize(dev)
    check()
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("lens,partition,fp8,faults", [
    ([500, 300, 700], 64, False, [(0, 0), (13, 2)]),     # decode, then the merge
    ([500, 300, 700], 64, True, [(0, 0), (13, 2)]),
    ([256, 200, 31], 64, False, [(0, 0), (7, 1)]),       # joined in a cluster
    ([900, 40], 1008, False, [(0, 3), (1, 2)])])         # one partition
def test_decode_weights(test_lib, monkeypatch, lens, partition, fp8, faults):
    dev = torch.device("cuda:0")
    x = Batch(lens, 8, 2, 128, 16, torch.float16, seed=3, fp8=fp8, stale=False)
    before = x.state().nan_to_num(0.0)
    want, ww, ob, wb = decode_reference(x, before)
    w, out = torch.zeros(before.shape, device=dev), torch.zeros(x.q.shape, dtype=x.dtype, device=dev)
    args = [t.to(dev) for t in (x.q, x.k, x.v, x.tables, x.lens)]

    def call():
        w.zero_()
        lib.decode_weights(*args, x.scale, max(lens), weights=before.to(dev), weights_out=w, out=out,
                           partition_size=partition, **x.scales())

    def check():
        within(out, want, ob, "out")
        within(w, ww, wb, "weights")

    timed_out_then_right(test_lib, monkeypatch, faults, call, check)


@pytest.mark.parametrize("lens,chunks,hq,window,faults", [
    ([900, 700], [400, 300], 8, 0, [(0, 0), (0, 4), (3, 1)]),             # whole chunks
    ([16000, 12000], [40, 40], 8, 16, [(0, 0), (1, 1), (151, 2)]),        # a window, two passes
    ([900, 700], [40, 40], 8, 16, [(0, 0), (1, 1), (5, 0)])])             # in one launch
def test_prefill_weights(test_lib, monkeypatch, lens, chunks, hq, window, faults):
    dev = torch.device("cuda:0")
    x = Batch(lens, hq, 2, 128, 16, torch.float16, seed=4, stale=False)
    q = torch.randn(sum(chunks), hq, 128, generator=x.gen).to(x.dtype)
    before = x.state().nan_to_num(0.0)
    ww, wb = prefill_reference(x, q, chunks, window, before)
    w = torch.zeros(before.shape, device=dev)
    start = torch.tensor([0, *chunks]).cumsum(0).to(torch.int32)
    args = [t.to(dev) for t in (q, x.k, x.tables, x.lens, start)]

    def call():
        w.zero_()
        lib.prefill_weights(*args, x.scale, max(chunks), max(lens), window=window, weights=before.to(dev),
                            weights_out=w)

    timed_out_then_right(test_lib, monkeypatch, faults, call, lambda: within(w, ww, wb, "weights"))
