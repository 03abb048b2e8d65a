"""Plain implementations in 64 bits of the operators of speculative decoding,
from their definitions, on CPU tensors."""
import torch

from bounded_util import Batch, half_step


def random_parents(nodes, g, chain=False):
    """int32 [sum(nodes)]: every node but the first below an earlier one."""
    out = []
    for c in nodes:
        for i in range(c):
            out.append(i - 1 if chain or i == 0 else int(torch.randint(0, i, (1,), generator=g)))
    return torch.tensor(out, dtype=torch.int32)


def lines(parents):
    """Each node's line: the nodes from its root to itself."""
    made = []
    for i, p in enumerate(parents):
        made.append((made[p] if 0 <= p < i else []) + [i])
    return made


def starts(nodes):
    return torch.tensor([0, *nodes]).cumsum(0).to(torch.int32)


def visible(parents, n, c):
    """[c][n]: what the c nodes at the end of n cached tokens see."""
    seen = torch.zeros(c, n, dtype=torch.bool)
    seen[:, :n - c] = True
    for i, line in enumerate(lines(parents)):
        seen[i, [n - c + j for j in line]] = True
    return seen


def tree_reference(x: Batch, q, nodes, parents):
    """(out, bound) of the batch's nodes, rows behind them zero.

    A score carries an error of at most 2^-20 (2 + A) in log2 units, A = log2(e)
    scale max_i sum_d |q_d K_id| (fp32 accumulation of D products, the scale and
    the exponential), so a weight is off by that share, and out by that share of
    sum p |v|, by p's two parts (the first leaves up to 2^-7 of it (bf16, cut off)
    or 2^-11 (fp16, rounded), the second is off by 2^-8 or 2^-11 of that: 2^-15
    or 2^-22; and 2^-31 of the largest weight, which is at most 1, for each of n
    tokens), by the sums (2^-23 of a partial
    sum for each step of 8 tokens or more, and for the joins), and by its own
    rounding."""
    out = torch.zeros(len(q), x.hq, x.d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    g, at = x.hq // x.hkv, 0
    parts = 2.0 ** -15 if x.dtype == torch.bfloat16 else 2.0 ** -22
    for b, c in enumerate(nodes):
        n = int(x.lens[b])
        if c == 0:
            continue
        k, v = x.rows(x.k, b, x.k_scale), x.rows(x.v, b, x.v_scale)
        seen = visible(parents[at:at + c].tolist(), n, c)
        used = seen.any(0)
        k, v, seen = k[used], v[used], seen[:, used]
        for h in range(x.hq):
            qq, kk, vv = q[at:at + c, h].double(), k[:, h // g], v[:, h // g]
            s = (qq @ kk.T * x.scale).masked_fill(~seen, -float("inf"))
            a = float((qq.abs() @ kk.T.abs()).max()) * x.scale * 1.4427
            p = torch.softmax(s, 1)
            out[at:at + c, h] = p @ vv
            m, tiles = len(kk), -(-len(kk) // 128)
            pt = torch.nn.functional.pad(p, (0, 128 * tiles - m)).view(c, tiles, 128).transpose(0, 1)
            vt = torch.nn.functional.pad(vv, (0, 0, 0, 128 * tiles - m)).view(tiles, 128, -1)
            partial = (pt @ vt).cumsum(0).abs().amax(0) + (pt @ vt.abs()).amax(0)
            bound[at:at + c, h] = half_step(x.dtype) * out[at:at + c, h].abs() + 2.0 ** -24 + \
                (2.0 ** -20 * (2 + a) + parts) * (p @ vv.abs()) + \
                2.0 ** -31 * m * vv.abs().amax() + 2.0 ** -23 * (m / 8 + 16) * partial
        at += c
    return out, bound


def accept_reference(draft, target, parents, nodes, width):
    paths, lengths, following, at = [], [], [], 0
    for c in nodes:
        best = []
        for line in lines(parents[at:at + c].tolist()):
            if line[0] == 0 and len(line) > len(best) and \
                    all(draft[at + j] == target[at + i] for i, j in zip(line, line[1:])):
                best = line
        paths.append(best + [-1] * (width - len(best)))
        lengths.append(len(best))
        following.append(int(target[at + best[-1]]) if best else -1)
        at += c
    return (torch.tensor(paths, dtype=torch.int32).view(len(nodes), width),
            torch.tensor(lengths, dtype=torch.int32), torch.tensor(following))


def commit_reference(caches, tables, lens, nodes, path, path_lens, bs):
    """The caches after the moves, one row at a time, and the new lengths."""
    caches = [c.clone() for c in caches]
    new = []
    for b, n in enumerate(lens.tolist()):
        base = n - nodes[b]
        for j in range(int(path_lens[b])):
            frm, to = base + int(path[b, j]), base + j
            for c in caches:
                c[int(tables[b, to // bs]), to % bs] = c[int(tables[b, frm // bs]), frm % bs]
        new.append(base + int(path_lens[b]))
    return caches, torch.tensor(new, dtype=torch.int32)
