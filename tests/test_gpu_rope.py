"""GPU parity of pa_rope_and_cache against the formula in 64 bits.

Bound: cos and sin are off by at most 2^-22 (the angle 2^-23, the function
2 steps of 2^-24), so a turned value by 2^-21 f (|x| + |y|) with its products
and sum, and by half a step of its type (2^-25 below fp16's normal range; of
E4M3 2^-4 relative, 2^-10 below its normal range)."""
import numpy as np
import pytest
import torch

from bounded_util import E4M3, half_step, same_bits, within
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


def turned(x, positions, inv_freq, interleaved, factor):
    """(value, |x| + |y| of each element's pair) in 64 bits."""
    x = x.double()
    r = 2 * len(inv_freq)
    a = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = torch.cos(a) * factor, torch.sin(a) * factor
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    size[..., i] = size[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, size


def rounded(want, size, factor, dtype):
    return half_step(dtype) * want.abs() + 2.0 ** -21 * abs(factor) * size + \
        (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134) * (size > 0)


def coded(want, size, factor, scale):
    """Bound of want / scale held as E4M3."""
    return (want / scale).abs() * (2.0 ** -4 + 2.0 ** -21) + 2.0 ** -21 * abs(factor) * size / scale + 2.0 ** -10


def make(T, hq, hkv, d, bs, dtype, seed, fp8=False, far=5000, padding=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(dtype)
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if padding:
        slots[T - padding:] = -1
    pool = (lambda: torch.randint(0, 255, (nb, bs, hkv, d), generator=g, dtype=torch.uint8)) if fp8 else \
        (lambda: torch.randn(nb, bs, hkv, d, generator=g).to(dtype))
    return dict(qkv=qkv, slots=slots, pos=torch.randint(0, far, (T,), generator=g), kc=pool(), vc=pool())


def check(dev, T, hq, hkv, d, bs, dtype, rotary, interleaved, seed=1, fp8=False, far=5000, padding=0,
          factor=1.0, inv_freq=None, in_place=False, no_q=False):
    m = make(T, hq, hkv, d, bs, dtype, seed, fp8, far, padding)
    inv = lib.rope_frequencies(rotary)[0] if inv_freq is None else inv_freq
    qkv = m["qkv"].to(dev)
    q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    q0, k0, v0 = (t.view(T, -1, d) for t in m["qkv"].split([hq * d, hkv * d, hkv * d], dim=1))
    kc, vc = m["kc"].to(dev), m["vc"].to(dev)
    sc = dict(k_scale=0.04, v_scale=0.03) if fp8 else {}
    out = lib.rope_and_cache(None if no_q else q, k, v, m["pos"].to(dev), m["slots"].to(dev), inv.to(dev),
                             kc, vc, q_out=q if in_place else None, interleaved=interleaved,
                             factor=factor, **sc)
    torch.cuda.synchronize(dev)
    f32 = float(np.float32(factor))
    if no_q:
        assert out is None
    else:
        want, size = turned(q0, m["pos"], inv, interleaved, f32)
        within(out, want, rounded(want, size, factor, dtype), "q")
        r = 2 * len(inv)
        assert same_bits(out[..., r:], q0[..., r:]), "dims past rotary_dim are copied"
    assert same_bits(qkv[:, hq * d:], m["qkv"][:, hq * d:]), "k and v are inputs"
    live = torch.nonzero(m["slots"] >= 0)[:, 0]
    at = m["slots"][live]
    want, size = turned(k0, m["pos"], inv, interleaved, f32)
    want, size = want[live], size[live]
    got_k, got_v = kc.cpu().view(-1, hkv, d), vc.cpu().view(-1, hkv, d)
    if fp8:
        within(got_k[at].view(E4M3), (want / np.float32(0.04)).clamp(-448, 448), coded(want, size, factor, 0.04), "k codes")
        vv = (v0[live].float() / np.float32(0.03)).clamp(-448, 448).to(E4M3).view(torch.uint8)
        assert same_bits(got_v[at], vv), "v codes"
    else:
        within(got_k[at], want, rounded(want, size, factor, dtype), "k")
        assert same_bits(got_v[at], v0[live]), "v"
    untouched = torch.ones(got_k.shape[0], dtype=torch.bool)
    untouched[at] = False
    assert same_bits(got_k[untouched], m["kc"].view(-1, hkv, d)[untouched])
    assert same_bits(got_v[untouched], m["vc"].view(-1, hkv, d)[untouched])
    assert lib.read_device_errors(dev) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,bs,dtype,rotary", [
    (1, 8, 2, 64, 16, torch.float16, 64), (1, 32, 8, 128, 16, torch.bfloat16, 128),
    (37, 6, 2, 128, 32, torch.float16, 128), (130, 5, 1, 64, 16, torch.bfloat16, 32),
    (9, 16, 16, 128, 16, torch.float16, 48), (200, 64, 8, 128, 16, torch.bfloat16, 96),
    (3, 7, 7, 64, 32, torch.float16, 16)])
def test_rope_shapes(dev, T, hq, hkv, d, bs, dtype, rotary, interleaved):
    check(dev, T, hq, hkv, d, bs, dtype, rotary, interleaved, seed=T + rotary)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,rotary,padding", [(1, 8, 2, 128, 0), (77, 12, 4, 64, 5), (33, 3, 1, 16, 33)])
def test_rope_e4m3(dev, T, hq, hkv, rotary, padding, interleaved, dtype):
    check(dev, T, hq, hkv, 128, 16, dtype, rotary, interleaved, fp8=True, padding=padding)


def test_far_and_negative_positions(dev):
    """Whole turns drop out exactly: a position of 2^40 or below zero is as
    exact as a near one (the reference takes the turns off in integers)."""
    T, d = 6, 64
    pos = torch.tensor([2 ** 40 + 12345, 2 ** 31 + 7, -1, -5000, 0, 2 ** 20 - 1])
    inv = torch.tensor([1.0, 0.25, 2.0 ** -20, 3.0, 0.0, -0.5, 100.5, 2.0 ** -7] * 4, dtype=torch.float32)
    x = torch.randn(T, 1, d, generator=torch.Generator().manual_seed(3)).to(torch.float16)
    kc = torch.zeros(1, 16, 1, d, dtype=torch.float16, device=dev)
    out = lib.rope_and_cache(x.to(dev), x.to(dev), x.to(dev), pos.to(dev),
                             torch.arange(T, device=dev), inv.to(dev), kc, kc.clone())
    # cos / sin of pos * inv with the whole turns taken off in exact rationals
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592, 10 ** 63)
    cos, sin = torch.zeros(T, len(inv), dtype=torch.float64), torch.zeros(T, len(inv), dtype=torch.float64)
    for t in range(T):
        for i in range(len(inv)):
            a = Fraction(int(pos[t])) * Fraction(float(inv[i]))
            a -= round(a / (2 * pi)) * 2 * pi
            cos[t, i], sin[t, i] = np.cos(float(a)), np.sin(float(a))
    xa, xb = x[..., :d // 2].double(), x[..., d // 2:].double()
    want = torch.cat((xa * cos[:, None] - xb * sin[:, None], xb * cos[:, None] + xa * sin[:, None]), -1)
    size = (xa.abs() + xb.abs()).repeat(1, 1, 2)
    # the turns per position are held to 2^-53 of themselves (and 2^-64): their error times the position
    size = size * (1 + 2.0 ** 21 * 2 * np.pi * (pos.abs().double()[:, None, None] * (2.0 ** -53 * inv.abs().double() + 2.0 ** -64))).repeat(1, 1, 2)
    within(out, want, rounded(want, size, 1.0, torch.float16), "far positions")


def test_factor_in_place_and_keys_only(dev):
    check(dev, 19, 8, 2, 128, 16, torch.bfloat16, 128, False, factor=1.2079)
    check(dev, 19, 8, 2, 128, 16, torch.float16, 64, True, in_place=True)
    check(dev, 19, 8, 2, 128, 16, torch.float16, 128, False, no_q=True)
    check(dev, 19, 8, 2, 64, 16, torch.float16, 64, False, inv_freq=lib.rope_frequencies(
        64, 500000.0, "yarn", 8.0, 4096)[0], factor=lib.rope_frequencies(64, 500000.0, "yarn", 8.0, 4096)[1], far=32768)
    check(dev, 19, 8, 2, 64, 16, torch.float16, 16, False, inv_freq=torch.zeros(0), far=9)   # nothing turns


def test_bad_slots_are_skipped_and_flagged(dev):
    m = make(4, 4, 2, 64, 16, torch.float16, 5)
    n = m["kc"].shape[0] * 16
    slots = torch.tensor([n, -3, 2 ** 40, 5])
    q, k, v = (t.view(4, -1, 64).contiguous().to(dev) for t in m["qkv"].split([256, 128, 128], dim=1))
    kc, vc = m["kc"].to(dev), m["vc"].to(dev)
    lib.rope_and_cache(q, k, v, m["pos"].to(dev), slots.to(dev), lib.rope_frequencies(64)[0].to(dev), kc, vc)
    assert lib.read_device_errors(dev) == lib.PA_DEVERR_BAD_SLOT
    changed = (vc.cpu() != m["vc"]).flatten(2).any(-1).flatten().nonzero().flatten().tolist()
    assert changed == [5]


def test_empty_and_refused(dev):
    e = torch.zeros(0, 4, 64, dtype=torch.float16, device=dev)
    kv = torch.zeros(0, 2, 64, dtype=torch.float16, device=dev)
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device=dev)
    i64 = torch.zeros(0, dtype=torch.int64, device=dev)
    inv = lib.rope_frequencies(64)[0].to(dev)
    assert lib.rope_and_cache(e, kv, kv, i64, i64, inv, kc, kc.clone()).shape == (0, 4, 64)
    x = torch.zeros(3, 4, 64, dtype=torch.float16, device=dev)
    y = torch.zeros(3, 2, 64, dtype=torch.float16, device=dev)
    p = torch.zeros(3, dtype=torch.int64, device=dev)
    args = dict(q=x, k=y, v=y, positions=p, slot_mapping=p, inv_freq=inv, k_cache=kc, v_cache=kc.clone())
    for bad in (dict(k=y.bfloat16()), dict(q=x.transpose(0, 1)), dict(q=x[:2]), dict(positions=p.int()),
                dict(inv_freq=inv.double()), dict(v=y[..., :32]), dict(k_scale=1.0, v_scale=1.0),
                dict(q_out=torch.zeros_like(x).bfloat16()), dict(v_cache=kc.bfloat16()),
                dict(q=None, q_out=x)):
        with pytest.raises((ValueError, TypeError)):
            lib.rope_and_cache(**{**args, **bad})
    for bad in (dict(inv_freq=inv[:12].contiguous()), dict(inv_freq=torch.zeros(40, device=dev)),
                dict(factor=float("nan"))):
        with pytest.raises(lib.PaError):
            lib.rope_and_cache(**{**args, **bad})


def test_side_stream(dev):
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(s):
        check(dev, 37, 8, 2, 128, 16, torch.float16, 128, False, seed=11)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,dtype,rotary,fp8,padding", [
    (1368, 8, 2, 64, torch.float16, 64, False, 0),          # the last count that goes one token to a CTA
    (1369, 8, 2, 64, torch.float16, 64, False, 0),          # two, and an odd one at the end
    (1370, 6, 3, 128, torch.bfloat16, 128, False, 5), (3001, 5, 1, 128, torch.float16, 96, False, 40),
    (1369, 4, 4, 128, torch.bfloat16, 128, True, 0), (3001, 8, 2, 128, torch.float16, 64, True, 7)])
def test_rope_packed_prompts(dev, T, hq, hkv, d, dtype, rotary, fp8, padding, interleaved):
    """More tokens than fit the GPU one to a CTA."""
    check(dev, T, hq, hkv, d, 16, dtype, rotary, interleaved, seed=T, fp8=fp8, padding=padding)
    check(dev, T, hq, hkv, d, 32, dtype, rotary, interleaved, seed=T + 1, fp8=fp8, padding=padding, in_place=True)
    check(dev, T, hq, hkv, d, 16, dtype, rotary, interleaved, seed=T + 2, fp8=fp8, padding=padding, no_q=True)
