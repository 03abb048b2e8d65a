"""The waits of tree attention's ring of V tiles over an E4M3 cache, as a model:
converters, issuers and softmax warps take turns in random orders, products end
when they like, and a barrier tells a waiter no more than a parity does.  CPU
only; what the kernel does with the stages is in csrc/tree_attention.cu."""
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


def walk(owners, rng, barriers, slow):
    """One run.  barriers: STAGES, or twice as many, that say a stage is free."""
    n_tiles = len(owners)
    full = [Barrier(1) for _ in range(STAGES)]
    empty = [Barrier(2) for _ in range(barriers)]
    holds = [None] * STAGES                  # the tile whose codes were brought there
    reading = [set() for _ in range(STAGES)]     # slots that have yet to let go of it
    convert, issue = [0, 1], [0, 0]              # next tile of each converter, of each slot's issuer
    products = [[], []]                          # under way, oldest first

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
        if holds[n % STAGES] != n:
            raise Wrong(f"products on tile {n} read tile {holds[n % STAGES]}")
        reading[n % STAGES].discard(s)
        empty[n % barriers].arrive()
        return True

    actors = [(converter, 0), (converter, 1), (issuer, 0), (issuer, 1), (product, 0), (product, 1)]
    weights = [1.0, 1.0, 1.0, 1.0, slow, slow]
    while any(products) or min(issue) < n_tiles:
        order = []
        left = list(zip(actors, weights))
        while left:
            i = rng.choices(range(len(left)), [w for _, w in left])[0]
            order.append(left.pop(i)[0])
        if not any(act(who) for act, who in order):
            raise Wrong("nobody can move")


def outcome(barriers, seeds):
    wrong = 0
    for seed in range(seeds):
        rng = random.Random(seed)
        try:
            walk(pieces(rng, 60), rng, barriers, slow=rng.choice((0.02, 0.2, 1.0, 5.0)))
        except Wrong:
            wrong += 1
    return wrong


def test_a_barrier_for_every_other_use_of_a_stage():
    assert outcome(2 * STAGES, 600) == 0


def test_a_barrier_a_stage_is_not_enough():
    """The model sees it: a converter, which waits for every other use of a stage,
    takes the release before the last for the last."""
    assert outcome(STAGES, 600) > 0
