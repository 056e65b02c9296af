"""The barrier protocol of moe_linear's tensor-core kernels, checked on the CPU.

A model of the roles of one block (linear_gemm_kernel) or of a pair of blocks
(linear_pair_kernel) runs random interleavings:
  producer   per stage of one or two steps: wait empty (reuse); issue the
             block's loads, which land later and count on the leading block's
             `full`, where the leader's producer also announces the bytes (the
             peer's may land first);
  MMA issuer (leading block) wait acc_empty at a segment's first stage (reuse)
             and full, issue; the MMAs run in order, later, and their commits
             arrive on `empty`, and after a segment's last stage on `acc_full`,
             of every block;
  epilogue   per segment: wait acc_full, read the accumulator, arrive on the
             leader's acc_empty. Pair, after a tile's last segment, in passes:
             wait until the store of the last pass has read the staging area,
             load the residual into it, wait res, put the results there, store
             them.
An mbarrier wait on parity P succeeds when the number of completed phases c
has c % 2 != P; waiting for completion t is only correct while c is t or
t + 1. The model tracks what every stage, accumulator and staging area holds,
and fails when one is overwritten before its readers are done or read before
it is written. Negative controls drop one wait each and must fail."""
import random

import pytest

STAGES = {1: 3, 2: 4}  # single blocks, pairs (of 128 columns)
PER_STAGE = 2          # steps of 64 columns that a stage holds
EPI = 8                # epilogue warps per block
PASSES = 2             # staging passes per tile


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


def run(blocks, tiles, steps, seg, seed, drop=None):
    rnd = random.Random(seed)
    stages = STAGES[blocks]
    # Stage g: whether it begins its segment, the segment's number, whether it ends it, its loads.
    plan, n_seg = [], 0
    for _ in range(tiles):
        for kb in range(0, steps, PER_STAGE):
            n = min(PER_STAGE, steps - kb)
            last = (kb + n) % seg == 0 or kb + n == steps
            plan.append((kb % seg == 0, n_seg, last, n))
            n_seg += last
    per_tile = n_seg // tiles
    total = len(plan)
    full = [Bar(1) for _ in range(stages)]
    acc_empty = [Bar(EPI * blocks) for _ in range(2)]
    empty = [[Bar(1) for _ in range(stages)] for _ in range(blocks)]
    acc_full = [[Bar(1) for _ in range(2)] for _ in range(blocks)]
    stage = [[{} for _ in range(stages)] for _ in range(blocks)]  # by step: whose operands it holds
    acc = [(-1, 0)] * 2                             # segment, complete
    reads = [0] * n_seg                             # epilogue warps that have read a segment
    mma_done = [0]
    landing, mmas, copies = [], [], []              # loads; MMAs issued, in order; staging copies in flight

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
                full[s].arrive(tx=blocks * plan[g][3])
                yield
            for i in range(plan[g][3]):
                landing.append((b, s, g, i))
                yield

    def issuer():
        for g, (first, u, _, _) in enumerate(plan):
            if first and u >= 2:
                yield from wait(acc_empty[u & 1], (u >> 1) - 1, "acc_empty")
            yield from wait(full[g % stages], g // stages, "full")
            mmas.append(g)
            yield

    def epilogue(b):
        res, area = Bar(1), {"what": None, "busy": 0}  # area: residual or results of a pass; stores still reading
        loads = 0
        for t in range(tiles):
            for q in range(per_tile):
                u = t * per_tile + q
                last = q == per_tile - 1
                for p in range(PASSES if last else 1):
                    key = (t, p)
                    if blocks == 2 and last:
                        while area["busy"] and drop != "store_read":
                            yield
                        res.arrive(tx=1)
                        copies.append(("load", area, key, res))
                        yield
                    if p == 0:
                        yield from wait(acc_full[b][u & 1], u >> 1, "acc_full")
                    if blocks == 2 and last:
                        yield from wait(res, loads, "res")
                        loads += 1
                        if area["what"] != ("residual", key):
                            raise Hazard(f"residual of {key} read, the staging area holds {area['what']}")
                    if acc[u & 1] != (u, True):
                        raise Hazard(f"sums of segment {u} read, the accumulator holds {acc[u & 1]}")
                    yield
                    if p == (PASSES - 1 if last else 0):
                        reads[u] += 1
                        acc_empty[u & 1].arrive()
                        yield
                    if blocks == 2 and last:
                        area["what"] = ("result", key)
                        area["busy"] += 1
                        copies.append(("store", area, key, None))
                        yield

    def async_units():
        kinds = [k for k, on in (("load", landing), ("mma", mmas), ("copy", copies)) if on]
        if not kinds:
            return False
        kind = rnd.choice(kinds)
        if kind == "load":
            b, s, g, i = landing.pop(rnd.randrange(len(landing)))
            if g >= stages and mma_done[0] <= g - stages:
                raise Hazard(f"load of stage {g} lands while stage {g - stages} is still to be multiplied")
            stage[b][s][i] = g
            full[s].land()
        elif kind == "mma":
            g = mmas.pop(0)
            first, u, last, n = plan[g]
            if any(stage[b][g % stages].get(i) != g for b in range(blocks) for i in range(n)):
                raise Hazard(f"stage {g} multiplies {[stage[b][g % stages] for b in range(blocks)]}")
            if first:
                if u >= 2 and reads[u - 2] != EPI * blocks:
                    raise Hazard(f"segment {u} overwrites sums of segment {u - 2} still being read")
            acc[u & 1] = (u, last)
            mma_done[0] = g + 1
            for b in range(blocks):
                empty[b][g % stages].arrive()
                if last:
                    acc_full[b][u & 1].arrive()
        else:
            what, area, key, res = copies.pop(rnd.randrange(len(copies)))
            if what == "load":
                if area["busy"]:
                    raise Hazard(f"residual of {key} lands while a store reads the staging area")
                area["what"] = ("residual", key)
                res.land()
            else:
                if area["what"] != ("result", key):
                    raise Hazard(f"store of {key} writes {area['what']}")
                area["busy"] -= 1
        return True

    roles = [issuer()] + [producer(b) for b in range(blocks)] + [epilogue(b) for b in range(blocks) for _ in range(EPI)]
    weight = [rnd.choice([1, 1, 4, 20]) for _ in roles]  # each gets far ahead or behind
    idle = 0
    while roles:
        if rnd.random() < 0.3:
            idle = 0 if async_units() else idle
        i = rnd.choices(range(len(roles)), weight)[0]
        before = (len(landing), len(mmas), len(copies), sum(reads), mma_done[0])
        try:
            next(roles[i])
        except StopIteration:
            del roles[i], weight[i]
            idle = 0
            continue
        after = (len(landing), len(mmas), len(copies), sum(reads), mma_done[0])
        idle = 0 if before != after else idle + 1
        if idle > 200000:
            raise Hazard("no role can go on")
    while async_units():
        pass
    assert mma_done[0] == total and all(r == EPI * blocks for r in reads)


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("tiles,steps,seg", [(1, 1, 8), (1, 3, 8), (3, 5, 6), (2, 16, 8), (2, 17, 8), (3, 9, 4), (5, 2, 8)])
def test_no_hazard_and_no_deadlock(blocks, tiles, steps, seg):
    for seed in range(8):
        run(blocks, tiles, steps, seg, seed)


@pytest.mark.parametrize("blocks,drop", [(1, "empty"), (1, "acc_empty"), (1, "full"), (1, "acc_full"), (2, "empty"),
                                         (2, "acc_empty"), (2, "full"), (2, "acc_full"), (2, "res"), (2, "store_read")])
def test_each_wait_is_needed(blocks, drop):
    failed = 0
    for seed in range(20):
        try:
            run(blocks, 4, 13, 4, seed, drop)
        except AssertionError:
            failed += 1
    assert failed, f"dropping {drop} went unnoticed"
