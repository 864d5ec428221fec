"""A model of the 8-bit product's protocol, run over random interleavings: two CTAs' producers (each loads its
half of a stage; both halves count on the even CTA's full barrier), the MMA issuer of the pair, whose commits
arrive in order on the empty and accfull barriers of both CTAs, and both CTAs' output warps, which read one of
two accumulators and release it on the even CTA's accempty barrier. A wait on parity P returns once the
barrier's phase of that parity has completed. The model checks that no schedule deadlocks, that every step
multiplies its own operands, that no stage is overwritten before the MMAs that read it are done, that every
tile's output reads its own finished sums, and that no accumulator starts afresh while one of them still
reads it."""
import random

import pytest

from tests.test_k2_ring_protocol import Barrier

WARPS = 2  # output warps of a CTA (the kernel's eight arrive alike)


def run(ST, tiles, steps, seed, accempty_lag=2):
    rng = random.Random(seed)
    full = [Barrier(1) for _ in range(ST)]
    empty = [[Barrier(1) for _ in range(ST)] for _ in range(2)]
    accfull = [[Barrier(1) for _ in range(2)] for _ in range(2)]
    accempty = [Barrier(2 * WARPS) for _ in range(2)]
    held = [[None] * ST for _ in range(2)]  # step whose operands the CTA's stage holds
    free = [-1] * ST                        # last step whose MMAs on the stage have completed
    acc = [None, None]                      # (tile, finished) of each accumulator
    reading = [set(), set()]
    landing, commits = [], []               # loads land in any order, commits in theirs

    def producer(cta):
        for it in range(tiles * steps):
            s = it % ST
            if it >= ST:
                while not empty[cta][s].done(((it // ST) - 1) & 1):
                    yield
                assert free[s] >= it - ST
            if cta == 0:
                full[s].arrive(expect_tx=2)
            landing.append((cta, s, it))
            yield

    def mma():
        it = 0
        for n in range(tiles):
            b = n & 1
            if n >= accempty_lag:
                while not accempty[b].done(((n >> 1) - 1) & 1):
                    yield
            assert not reading[b], "accumulator started afresh while it is read"
            acc[b] = (n, False)
            for _ in range(steps):
                s = it % ST
                while not full[s].done((it // ST) & 1):
                    yield
                assert held[0][s] == it and held[1][s] == it
                commits.append(("stage", s, it))
                it += 1
                yield
            commits.append(("acc", b, n))
            yield

    def output(cta, warp):
        for n in range(tiles):
            b = n & 1
            while not accfull[cta][b].done((n >> 1) & 1):
                yield
            assert acc[b] == (n, True), (acc[b], n)
            reading[b].add((cta, warp))
            yield
            assert acc[b] == (n, True), "sums overwritten while they are read"
            reading[b].discard((cta, warp))
            accempty[b].arrive()
            yield

    agents = [producer(0), producer(1), mma()] + [output(c, w) for c in range(2) for w in range(WARPS)]
    live = list(range(len(agents)))
    n = 0
    while live or landing or commits:
        c = rng.choice(live + (["land"] if landing else []) + (["commit"] if commits else []))
        n += 1
        assert n < 300000, "no progress"
        if c == "land":
            cta, s, it = landing.pop(rng.randrange(len(landing)))
            held[cta][s] = it
            full[s].tx -= 1  # a half may land before the even CTA has announced the stage's bytes
            full[s]._check()
        elif c == "commit":
            kind, i, step = commits.pop(0)
            if kind == "stage":
                free[i] = step
                for cta in range(2):
                    empty[cta][i].arrive()
            else:
                acc[i] = (step, True)
                for cta in range(2):
                    accfull[cta][i].arrive()
        else:
            try:
                next(agents[c])
            except StopIteration:
                live.remove(c)


@pytest.mark.parametrize("tiles,steps", [(1, 1), (1, 12), (2, 3), (5, 1), (7, 4)])
@pytest.mark.parametrize("seed", range(12))
def test_random_interleavings(tiles, steps, seed):
    run(5, tiles, steps, seed)


def test_the_first_two_tiles_alone_start_without_a_release():
    # an issuer that waits for releases only from the fifth tile on overwrites sums that are still read
    failures = 0
    for seed in range(20):
        try:
            run(5, 7, 2, seed, accempty_lag=4)
        except AssertionError:
            failures += 1
    assert failures >= 15
