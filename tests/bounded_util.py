"""Plain implementations in 64 bits of the bounded-cache operators (rotary
positions with the cache write, the attention weights of decode and prefill,
eviction), from their definitions, on CPU tensors; and the batches the tests
run them on."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    """Largest relative rounding error of a normal value of the type."""
    return torch.finfo(dtype).eps / 2


class Batch:
    """Sequences over a scattered pool, made on the CPU; ``.to(dev)`` gives the
    device copies.  Slots that hold no token are filled with NaN unless
    ``stale`` is False: no result may depend on them."""

    def __init__(self, lens, hq, hkv, d, bs, dtype=torch.float16, seed=0, fp8=False, stale=True,
                 extra_blocks=3, slack_width=1):
        g = torch.Generator().manual_seed(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.hq, self.hkv, self.d, self.bs, self.dtype, self.fp8 = hq, hkv, d, bs, dtype, fp8
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + extra_blocks
        order = torch.randperm(nb, generator=g).to(torch.int32)
        self.width = max(1, max(need, default=0) + slack_width)
        self.tables = torch.full((len(lens), self.width), nb + 7, dtype=torch.int32)  # unused: bad ids
        at = 0
        live = torch.zeros(nb, bs, dtype=torch.bool)
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            for j in range(n):
                live[order[at + j], :max(0, min(bs, lens[b] - j * bs))] = True
            at += n
        self.k_scale, self.v_scale = (0.15, 0.07) if fp8 else (None, None)

        def pool():
            x = torch.randn(nb, bs, hkv, d, generator=g)
            if fp8:
                x = (x * 8).clamp(-448, 448).to(E4M3).view(torch.uint8)
                return torch.where(live[:, :, None, None], x, torch.full_like(x, 0x7f)) if stale else x
            x = x.to(dtype)
            return torch.where(live[:, :, None, None], x, torch.full_like(x, float("nan"))) if stale else x

        self.k, self.v = pool(), pool()
        self.q = torch.randn(len(lens), hq, d, generator=g).to(dtype)
        self.scale = d ** -0.5
        self.gen = g
        self.tokens = self.width * bs

    @property
    def num_seqs(self):
        return len(self.lens)

    def state(self):
        """weights [B][Hkv][tokens]: heavy and light entries, ties at zero, NaN past the length."""
        w = torch.randn(self.num_seqs, self.hkv, self.tokens, generator=self.gen)
        w = torch.where(w < -1, torch.zeros_like(w), torch.exp(2 * w))
        at = torch.arange(self.tokens)
        return torch.where(at < self.lens[:, None, None], w, torch.full_like(w, float("nan")))

    def rows(self, cache, b, scale=None):
        """[L][Hkv][D] of sequence b in 64 bits."""
        n = int(self.lens[b])
        idx = torch.arange(n)
        blk = self.tables[b, idx // self.bs].long()
        x = cache[blk, idx % self.bs]
        return (x.view(E4M3) if self.fp8 else x).double() * \
            (float(np.float32(scale)) if self.fp8 else 1.0)

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale) if self.fp8 else {}


def decode_reference(x: Batch, weights=None):
    """(out, weights, bound of out, bound of weights) of one query per sequence.

    Bounds: a score carries an error of at most 2^-20 (2 + A) in log2 units,
    A = log2(e) scale max_i sum_d |q_d K_id| (fp32 accumulation of D products,
    the scale and the exponential), so a weight is off by that share; out by
    that share and by P's rounding (2^-14 for the pair of a 16-bit cache, half
    a step of fp16 for an E4M3 one) of sum p |v|, and by its own rounding."""
    out = torch.zeros(x.num_seqs, x.hq, x.d, dtype=torch.float64)
    ob = torch.zeros_like(out)
    w = torch.zeros(x.num_seqs, x.hkv, x.tokens, dtype=torch.float64)
    wb = torch.zeros_like(w)
    g = x.hq // x.hkv
    p_step = half_step(torch.float16) if x.fp8 else 2.0 ** -14
    for b in range(x.num_seqs):
        n = int(x.lens[b])
        if n == 0:
            continue
        k, v = x.rows(x.k, b, x.k_scale), x.rows(x.v, b, x.v_scale)
        for h in range(x.hq):
            q = x.q[b, h].double()
            s = (k[:, h // g] @ q) * x.scale
            a = float((k[:, h // g].abs() @ q.abs()).max()) * x.scale * 1.4427
            rel = 2.0 ** -20 * (2 + a)
            p = torch.softmax(s, 0)
            out[b, h] = p @ v[:, h // g]
            ob[b, h] = half_step(x.dtype) * out[b, h].abs() + \
                (rel + 1.01 * p_step) * (p @ v[:, h // g].abs()) + 2.0 ** -24
            w[b, h // g, :n] += p
            wb[b, h // g, :n] += rel * p + 1e-30
        if weights is not None:
            w[b, :, :n - 1] += weights[b, :, :n - 1].double()
            wb[b, :, :n - 1] += 2.0 ** -23 * weights[b, :, :n - 1].double().abs()
    return out, w, ob, wb


def prefill_reference(x: Batch, q, chunks, window=0, weights=None):
    """(weights, bound): the counted queries' softmax weights per token.  The
    bound is decode's, and half a step for each of the N additions."""
    w = torch.zeros(x.num_seqs, x.hkv, x.tokens, dtype=torch.float64)
    wb = torch.zeros_like(w)
    g = x.hq // x.hkv
    at = 0
    for b, c in enumerate(chunks):
        n = int(x.lens[b])
        k = x.rows(x.k, b)
        counted = min(c, window) if window else c
        for h in range(x.hq):
            qq = q[at + c - counted:at + c, h].double()
            s = (qq @ k[:, h // g].T) * x.scale
            hidden = torch.ones(counted, n, dtype=torch.bool).triu(n - counted + 1)
            p = torch.softmax(s.masked_fill(hidden, -float("inf")), 1)
            a = float((qq.abs() @ k[:, h // g].T.abs()).max()) * x.scale * 1.4427 if counted and n else 0.
            w[b, h // g, :n] += p.sum(0)
            wb[b, h // g, :n] += (2.0 ** -20 * (2 + a) + 2.0 ** -24 * counted * g) * p.sum(0) + 1e-30
        if weights is not None and n > c:
            w[b, :, :n - c] += weights[b, :, :n - c].double()
            wb[b, :, :n - c] += 2.0 ** -23 * weights[b, :, :n - c].double().abs()
        at += c
    return w, wb


def evict_reference(x: Batch, weights, positions, seen, known, budget, trigger, sinks, recent):
    """(k, v, weights, positions, new_lens) after the cut, token by token."""
    k, v = x.k.clone(), x.v.clone()
    wo, po = weights.clone(), positions.clone()
    new = x.lens.clone()
    for b in range(x.num_seqs):
        n = int(x.lens[b])
        kn = int(known[b]) if known is not None else 0
        left = budget if n > trigger else n
        new[b] = left
        for h in range(x.hkv):
            place = [int(positions[b, h, i]) if i < kn else i + int(seen[b]) - n for i in range(n)]
            wt = [float(weights[b, h, i]) for i in range(n)]

            def order(i):
                safe = place[i] < sinks or place[i] >= int(seen[b]) - recent
                nan = wt[i] != wt[i]
                return (0 if safe else 1, 0 if safe or not nan else 1, 0.0 if safe or nan else -wt[i], i)

            kept = set(sorted(range(n), key=order)[:left])
            gaps = [i for i in range(left) if i not in kept]
            movers = [i for i in range(left, n) if i in kept]
            assert len(gaps) == len(movers)
            src = list(range(left))
            for to, frm in zip(gaps, movers):
                src[to] = frm
                sb, db = int(x.tables[b, frm // x.bs]), int(x.tables[b, to // x.bs])
                k[db, to % x.bs, h] = x.k[sb, frm % x.bs, h]
                v[db, to % x.bs, h] = x.v[sb, frm % x.bs, h]
            if left:
                wo[b, h, :left] = weights[b, h, src]
                po[b, h, :left] = torch.tensor([place[i] for i in src], dtype=torch.int32)
    return k, v, wo, po, new


def within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, f"{what}: {got.shape} vs {want.shape}"
    err = (got - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(int((err - bound).nan_to_num(float("inf")).argmax()), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{float(got[i])!r} want {float(want[i])!r} bound {float(bound[i])!r}")


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return a.shape == b.shape and a.dtype == b.dtype and \
        torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8))
