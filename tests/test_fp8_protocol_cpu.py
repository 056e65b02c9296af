"""The barrier protocol of the FP8 tensor-core kernels, checked on the CPU.

A model of the roles of one block (fp8_gemm_kernel) or of a pair of blocks
(fp8_pair_kernel) runs random interleavings:
  producer   per step: wait empty (reuse); issue the block's loads, which land
             later and count on the leading block's `full`, where the leader's
             producer also announces the bytes (the peer's may land first);
  MMA issuer (leading block) wait acc_empty (reuse) and full, issue; the MMAs
             run in order, later, and their commits arrive on `empty` and
             `acc_full` of every block;
  scales     (pair) two warps per block: wait sc_empty (reuse), write a group
             of four steps, arrive on sc_full;
  promotion  wait sc_full at a group's first step and acc_full, read the
             scales and the accumulator, arrive on sc_empty after a group's
             last step and on the leader's acc_empty.
An mbarrier wait on parity P succeeds when the number of completed phases c
has c % 2 != P; waiting for completion t is only correct while c is t or
t + 1. The model also tracks what every stage, accumulator and scale slot
holds, and fails when one is overwritten before its readers are done or read
before it is written. Negative controls drop one wait each and must fail."""
import random

import pytest

STAGES = {1: 6, 2: 4}   # single blocks (128-column tiles), pairs
BUFS = {1: 4, 2: 2}
PROMO = 8               # promotion warps per block
GROUPS = 2              # scale groups in shared memory (pairs)


class Hazard(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.tx, self.completed = count, 0, 0, 0

    def _step(self):
        if self.arrived == self.count and self.tx == 0:
            self.arrived, self.completed = 0, self.completed + 1

    def arrive(self, tx=0):
        self.arrived += 1
        self.tx += tx
        assert self.arrived <= self.count
        self._step()

    def land(self):
        self.tx -= 1
        self._step()


def run(blocks, tiles, steps, seed, drop=None):
    rnd = random.Random(seed)
    stages, bufs = STAGES[blocks], BUFS[blocks]
    total = tiles * steps
    full = [Bar(1) for _ in range(stages)]
    acc_empty = [Bar(PROMO * blocks) for _ in range(bufs)]
    empty = [[Bar(1) for _ in range(stages)] for _ in range(blocks)]
    acc_full = [[Bar(1) for _ in range(bufs)] for _ in range(blocks)]
    sc_full = [[Bar(2) for _ in range(GROUPS)] for _ in range(blocks)]
    sc_empty = [[Bar(PROMO) for _ in range(GROUPS)] for _ in range(blocks)]
    stage = [[-1] * stages for _ in range(blocks)]    # step whose operands it holds
    acc = [-1] * bufs                                 # step whose sums it holds
    acc_reads = [0] * total                           # promotion warps that have read step g's sums
    slot = [[[-1, -1] for _ in range(GROUPS)] for _ in range(blocks)]  # group written, by scale warp
    gpt = -(-steps // 4)                              # groups per tile
    grp_reads = [[0] * (tiles * gpt) for _ in range(blocks)]
    mma_done = [0]
    landing, mmas = [], []                            # loads in flight; MMAs issued, in order

    def wait(bar, t, name):
        while name != drop:
            if not t <= bar.completed <= t + 1:
                raise Hazard(f"{name}: waits for completion {t} with {bar.completed}")
            if bar.completed % 2 != t % 2:
                return
            yield

    def producer(b):
        for g in range(total):
            s = g % stages
            if g >= stages:
                yield from wait(empty[b][s], g // stages - 1, "empty")
            if b == 0:
                full[s].arrive(tx=blocks)
                yield
            landing.append((b, s, g))
            yield

    def issuer():
        for g in range(total):
            s, u = g % stages, g % bufs
            if g >= bufs:
                yield from wait(acc_empty[u], g // bufs - 1, "acc_empty")
            yield from wait(full[s], g // stages, "full")
            mmas.append((g, s, u))
            yield

    def scales(b, w):
        for q in range(tiles * gpt):
            s = q % GROUPS
            if q >= GROUPS:
                yield from wait(sc_empty[b][s], q // GROUPS - 1, "sc_empty")
                if grp_reads[b][q - GROUPS] != PROMO:
                    raise Hazard(f"scale group {q - GROUPS} overwritten while it is read")
            slot[b][s][w] = q
            yield
            sc_full[b][s].arrive()
            yield

    def promote(b):
        g = q = 0
        for _ in range(tiles):
            for kb in range(steps):
                u = g % bufs
                if blocks == 2:
                    if kb % 4 == 0:
                        yield from wait(sc_full[b][q % GROUPS], q // GROUPS, "sc_full")
                    if slot[b][q % GROUPS] != [q, q]:
                        raise Hazard(f"scales of group {q} read from slot {slot[b][q % GROUPS]}")
                yield from wait(acc_full[b][u], g // bufs, "acc_full")
                if acc[u] != g:
                    raise Hazard(f"sums of step {g} read, the accumulator holds {acc[u]}")
                yield
                if blocks == 2 and (kb % 4 == 3 or kb == steps - 1):
                    grp_reads[b][q] += 1
                    sc_empty[b][q % GROUPS].arrive()
                    q += 1
                acc_reads[g] += 1
                acc_empty[u].arrive()
                g += 1
                yield

    def async_units():
        kinds = [k for k, on in (("load", landing), ("mma", mmas)) if on]
        if not kinds:
            return False
        if rnd.choice(kinds) == "load":
            b, s, g = landing.pop(rnd.randrange(len(landing)))
            if g >= stages and mma_done[0] <= g - stages:
                raise Hazard(f"load of step {g} lands while step {g - stages} is still to be multiplied")
            stage[b][s] = g
            full[s].land()
        else:
            g, s, u = mmas.pop(0)
            if any(stage[b][s] != g for b in range(blocks)):
                raise Hazard(f"step {g} multiplies {[stage[b][s] for b in range(blocks)]}")
            if g >= bufs and acc_reads[g - bufs] != PROMO * blocks:
                raise Hazard(f"step {g} overwrites sums of step {g - bufs} still being read")
            acc[u] = g
            mma_done[0] = g + 1
            for b in range(blocks):
                empty[b][s].arrive()
                acc_full[b][u].arrive()
        return True

    roles = [issuer()] + [producer(b) for b in range(blocks)] + [promote(b) for b in range(blocks) for _ in range(PROMO)]
    if blocks == 2:
        roles += [scales(b, w) for b in range(2) for w in range(2)]
    # Some roles run often, some rarely, so that each gets far ahead or behind.
    weight = [rnd.choice([1, 1, 4, 20]) for _ in roles]
    idle = 0
    while roles:
        if rnd.random() < 0.3:
            idle = 0 if async_units() else idle
        i = rnd.choices(range(len(roles)), weight)[0]
        before = (len(landing), len(mmas), sum(acc_reads), mma_done[0])
        try:
            next(roles[i])
        except StopIteration:
            del roles[i], weight[i]
            idle = 0
            continue
        after = (len(landing), len(mmas), sum(acc_reads), mma_done[0])
        idle = 0 if before != after else idle + 1
        if idle > 200000:
            raise Hazard("no role can go on")
    while async_units():
        pass
    assert mma_done[0] == total and all(r == PROMO * blocks for r in acc_reads)


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("tiles,steps", [(1, 1), (1, 3), (2, 4), (3, 5), (2, 16), (5, 2)])
def test_no_hazard_and_no_deadlock(blocks, tiles, steps):
    for seed in range(12):
        run(blocks, tiles, steps, seed)


@pytest.mark.parametrize("blocks,drop", [(1, "empty"), (1, "acc_empty"), (1, "full"), (1, "acc_full"), (2, "empty"),
                                         (2, "acc_empty"), (2, "full"), (2, "acc_full"), (2, "sc_full"), (2, "sc_empty")])
def test_each_wait_is_needed(blocks, drop):
    failed = 0
    for seed in range(30):
        try:
            run(blocks, 3, 10, seed, drop)
        except AssertionError:
            failed += 1
    assert failed, f"dropping {drop} went unnoticed"
