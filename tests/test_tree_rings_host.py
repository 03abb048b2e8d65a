"""The waits of tree attention's ring of V tiles over an E4M3 cache, as a model:
converters, issuers and softmax warps (which clear elements of V that are not
finite) take turns in random orders, products end when they like, and a barrier
tells a waiter no more than a parity does.  CPU only; what the kernel does with
the stages is in csrc/tree_attention.cu."""
import random

import pytest

STAGES = 3


class Barrier:
    """Completes a phase with every `count` arrivals; a wait for phase i passes
    where the phase under way has another parity than i."""

    def __init__(self, count):
        self.count, self.left, self.over = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.over = self.count, self.over + 1

    def passes(self, phase):
        return self.over % 2 != phase % 2


class Wrong(AssertionError):
    pass


def pieces(rng, tiles):
    """Owners of each tile, a set of slots: pieces that both slots share, that
    they take in turn, or, where they are short, that one takes alone."""
    out, turn = [], 0
    while len(out) < tiles:
        kind, n = rng.choice(("share", "split", "split", "alone", "alone")), rng.randint(1, 7)
        if kind == "share":
            out += [{0, 1}] * n
        elif kind == "split" and n > 2:
            out += [{k & 1} for k in range(n)]
        else:
            out += [{turn}] * min(n, 2)
            turn ^= 1
    return out[:tiles]


def walk(owners, rng, barriers, slow, late=1.0, told=True):
    """One run.  barriers: STAGES, or twice as many, that say a stage is free.
    told: a softmax warp hears from its issuer that its tile is there; else it
    waits for its product before and asks the tile's own barrier."""
    n_tiles = len(owners)
    full = [Barrier(1) for _ in range(STAGES)]
    empty = [Barrier(2) for _ in range(barriers)]
    holds = [None] * STAGES                  # the tile whose codes were brought there
    reading = [set() for _ in range(STAGES)]     # slots that have yet to let go of it
    convert, issue = [0, 1], [0, 0]              # next tile of each converter, of each slot's issuer
    products = [[], []]                          # under way, oldest first
    own = [[n for n in range(n_tiles) if s in owners[n]] for s in (0, 1)]
    masked = [rng.random() < 0.5 for _ in range(n_tiles)]
    soft, ready, over = [0, 0], [0, 0], [0, 0]   # own tiles begun, handed over, multiplied
    there = [Barrier(1), Barrier(1)]             # the issuers' word that a masked tile has come
    heard, said = [0, 0], [None, None]
    met = {}                                     # slots that have come to a shared tile's barrier

    def free(n):
        """What the converter of tile n waits for."""
        if n < STAGES:
            return True
        if barriers == STAGES:
            return empty[n % STAGES].passes(n // STAGES - 1)
        return empty[(n + STAGES) % barriers].passes((n - STAGES) // barriers)

    def converter(w):
        n = convert[w]
        if n >= n_tiles or not free(n):
            return False
        st = n % STAGES
        if reading[st] or holds[st] not in (None, n - STAGES):
            raise Wrong(f"tile {n} over tile {holds[st]}, which {reading[st]} read")
        holds[st], reading[st] = n, {0, 1}
        full[st].arrive()
        convert[w] += 2
        return True

    def issuer(s):
        n = issue[s]
        st = n % STAGES
        if n >= n_tiles or not full[st].passes(n // STAGES):
            return False
        if holds[st] != n:
            raise Wrong(f"slot {s} takes tile {holds[st]} for {n}")
        if s in owners[n]:
            if masked[n] and s == min(owners[n]) and said[s] != n:
                there[s].arrive()
                said[s] = n
                return True
            if n not in own[s][:ready[s]]:
                return False
            products[s].append(n)
        else:
            reading[st].discard(s)
            empty[n % barriers].arrive()
        issue[s] += 1
        return True

    def product(s):
        if not products[s]:
            return False
        n = products[s].pop(0)
        over[s] += 1
        if holds[n % STAGES] != n:
            raise Wrong(f"products on tile {n} read tile {holds[n % STAGES]}")
        reading[n % STAGES].discard(s)
        empty[n % barriers].arrive()
        return True

    def softmax(s):
        t = soft[s]
        if ready[s] < t:                                           # at a shared tile's barrier
            if len(met[own[s][t - 1]]) < 2:
                return False
            ready[s] += 1
            return True
        if t >= len(own[s]) or over[s] < t - 1:                    # its scores follow the products of two before
            return False
        n = own[s][t]
        if masked[n] and s == min(owners[n]):
            if told:
                if not there[s].passes(heard[s]):
                    return False
                heard[s] += 1
            elif over[s] < t:
                return False
            if not full[n % STAGES].passes(n // STAGES):
                return False
            if holds[n % STAGES] != n:
                raise Wrong(f"slot {s} clears tile {holds[n % STAGES]} for {n}")
        soft[s] += 1
        if masked[n] and len(owners[n]) == 2:
            met.setdefault(n, set()).add(s)
        else:
            ready[s] += 1
        return True

    actors = [(softmax, 0), (softmax, 1), (converter, 0), (converter, 1), (issuer, 0), (issuer, 1), (product, 0), (product, 1)]
    weights = [1.0, 1.0, late, late, 1.0, 1.0, slow, slow]
    while any(products) or min(issue) < n_tiles:
        order = []
        left = list(zip(actors, weights))
        while left:
            i = rng.choices(range(len(left)), [w for _, w in left])[0]
            order.append(left.pop(i)[0])
        if not any(act(who) for act, who in order):
            raise Wrong("nobody can move")


def outcome(barriers, seeds, **how):
    wrong = []
    for seed in range(seeds):
        rng = random.Random(seed)
        try:
            walk(pieces(rng, 60), rng, barriers, rng.choice((0.02, 0.2, 1.0, 5.0)), rng.choice((0.02, 1.0)), **how)
        except Wrong as e:
            wrong.append(str(e))
    return wrong


def test_a_barrier_for_every_other_use_of_a_stage():
    assert outcome(2 * STAGES, 200) == []


def test_a_barrier_a_stage_is_not_enough():
    """The model sees it: a converter, which waits for every other use of a stage,
    takes the release before the last for the last."""
    assert outcome(STAGES, 200) != []


def test_a_tiles_own_barrier_is_not_enough():
    """A slot's last tile may be five back, two laps of the ring's three stages:
    the barrier's parity is then that of the tile before the last, or nobody's."""
    assert any("clears" in e for e in outcome(2 * STAGES, 200, told=False))
