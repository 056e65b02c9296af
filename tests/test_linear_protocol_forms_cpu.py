"""The barrier protocol of moe_linear's tensor-core kernels in every pipeline form they are built in, and of a tile
whose K a cluster of blocks shares, checked on the CPU.

The forms run on the model of test_linear_protocol_cpu.py: stages, and steps of
64 columns per stage, as the kernels' geometry has them, read from the source.

Split tile (linear_gemm_kernel, splits > 1): each block of the cluster runs its
share of the tile's steps and, when its last accumulator is complete, writes its
partial tile over the memory of its stages. All meet at a cluster barrier; each
block then reads every block's partial tile, and a second barrier keeps a block
(and its shared memory) until all have read. The model fails when a partial tile
is written while loads or MMAs still use the stages, read before it is written,
or read from a block that has left. Negative controls drop the wait for the
accumulator or one of the barriers and must fail."""
import os
import random
import re

import pytest

from tests import test_linear_protocol_cpu as base
from tests._lib import ROOT

# (blocks of a tile, steps per stage, stages) by kernel: single blocks of 128 columns, of 32 and 64; pairs of 256, of 128.
FORMS = [(1, 2, 3), (1, 4, 2), (2, 1, 6), (2, 2, 4)]


def test_forms_are_the_kernels():
    with open(os.path.join(ROOT, "int4_routed_expert_moe_gb300", "csrc", "linear_gemm.cu")) as f:
        src = f.read()
    geo, pair = src[src.index("struct Geo"):src.index("struct Bars")], src[src.index("struct Pair"):src.index("mma_f16_pair")]
    found = []
    for text, blocks, wide in ((geo, 1, 128), (pair, 2, 256)):
        kb = re.search(rf"kb = NT == {wide} \? (\d+) : (\d+);", text).groups()
        st = re.search(rf"stages = NT == {wide} \? (\d+) : (\d+);", text).groups()
        found += [(blocks, int(k), int(s)) for k, s in zip(kb, st)]
    assert sorted(found) == sorted(FORMS)


def _form(monkeypatch, blocks, kb, stages):
    monkeypatch.setattr(base, "PER_STAGE", kb)
    monkeypatch.setattr(base, "STAGES", {blocks: stages})


@pytest.mark.parametrize("blocks,kb,stages", FORMS)
@pytest.mark.parametrize("tiles,steps,seg", [(1, 1, 8), (2, 7, 64), (3, 8, 8), (2, 17, 8), (3, 9, 4), (2, 70, 64)])
def test_no_hazard_and_no_deadlock(monkeypatch, blocks, kb, stages, tiles, steps, seg):
    _form(monkeypatch, blocks, kb, stages)
    for seed in range(6):
        base.run(blocks, tiles, steps, seg, seed)


WAITS = ["empty", "acc_empty", "full", "acc_full"]


@pytest.mark.parametrize("blocks,kb,stages,drop", [(*f, w) for f in FORMS
                                                   for w in WAITS + (["res", "store_read"] if f[0] == 2 else [])])
def test_each_wait_is_needed(monkeypatch, blocks, kb, stages, drop):
    _form(monkeypatch, blocks, kb, stages)
    failed = 0
    for seed in range(20):
        try:
            base.run(blocks, 4, 26, 4 if kb < 4 else 8, seed, drop)
        except AssertionError:
            failed += 1
    assert failed, f"dropping {drop} went unnoticed"


class ClusterBar:
    """barrier.cluster: every thread of every block arrives, then waits."""

    def __init__(self, members):
        self.members, self.arrived, self.phase = members, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.members:
            self.arrived, self.phase = 0, self.phase + 1


def split(ranks, steps, kb, stages, seg, seed, drop=None):
    rnd = random.Random(seed)
    epi = 4
    meet = ClusterBar(ranks * (epi + 2))
    blocks = []
    for r in range(ranks):
        k0, k1 = steps * r // ranks, steps * (r + 1) // ranks
        plan, e, u = [], 0, 0
        for k in range(k0, k1, kb):  # a stage: whether it begins its segment, the segment, whether it ends it, its loads
            n = min(kb, k1 - k)
            last = e + n >= seg or k + n >= k1
            plan.append((e == 0, u, last, n))
            e, u = (0, u + 1) if last else (e + n, u)
        blocks.append(dict(plan=plan, segs=u, full=[base.Bar(1) for _ in range(stages)], empty=[base.Bar(1) for _ in range(stages)],
                           acc_full=[base.Bar(1) for _ in range(2)], acc_empty=[base.Bar(epi) for _ in range(2)],
                           landing=[], mmas=[], landed=0, done=0, acc=[(-1, False)] * 2, reads=[0] * u,
                           partial=0, there=True))

    def wait(bar, t, name):
        while name != drop:
            if not t <= bar.completed <= t + 1:
                raise base.Hazard(f"{name}: waits for completion {t} with {bar.completed}")
            if bar.completed % 2 != t % 2:
                return
            yield

    def cluster(name):
        if name == drop:
            return
        mine = meet.phase
        meet.arrive()
        while meet.phase == mine:
            yield

    def producer(b):
        for g, (_, _, _, n) in enumerate(b["plan"]):
            s = g % stages
            if g >= stages:
                yield from wait(b["empty"][s], g // stages - 1, "empty")
            b["full"][s].arrive(tx=n)
            for _ in range(n):
                b["landing"].append(g)
                yield
        yield from cluster("written")
        yield from cluster("read")

    def issuer(b):
        for g, (first, u, _, _) in enumerate(b["plan"]):
            if first and u >= 2:
                yield from wait(b["acc_empty"][u & 1], (u >> 1) - 1, "acc_empty")
            yield from wait(b["full"][g % stages], g // stages, "full")
            b["mmas"].append(g)
            yield
        yield from cluster("written")
        yield from cluster("read")

    def epilogue(b, w):
        total = sum(p[3] for p in b["plan"])
        for u in range(b["segs"]):
            yield from wait(b["acc_full"][u & 1], u >> 1, "acc_full")
            if b["acc"][u & 1] != (u, True):
                raise base.Hazard(f"sums of segment {u} read, the accumulator holds {b['acc'][u & 1]}")
            yield
            b["reads"][u] += 1
            if u < b["segs"] - 1:
                b["acc_empty"][u & 1].arrive()
        if b["landed"] < total or b["done"] < len(b["plan"]):
            raise base.Hazard("a partial tile over stages still in use")
        b["partial"] += 1
        yield
        yield from cluster("written")
        for p in rnd.sample(range(ranks), ranks):
            if blocks[p]["partial"] < epi:
                raise base.Hazard(f"block {p}'s partial tile read before it is written")
            if not blocks[p]["there"]:
                raise base.Hazard(f"block {p} has left while its partial tile is read")
            yield
        yield from cluster("read")

    def async_units():
        b = rnd.choice(blocks)
        kinds = [k for k in ("landing", "mmas") if b[k]]
        if not kinds:
            return
        if rnd.choice(kinds) == "landing":
            g = b["landing"].pop(rnd.randrange(len(b["landing"])))
            b["landed"] += 1
            b["full"][g % stages].land()
        else:
            g = b["mmas"].pop(0)
            first, u, last, _ = b["plan"][g]
            if first and u >= 2 and b["reads"][u - 2] != epi:
                raise base.Hazard(f"segment {u} overwrites sums still being read")
            b["acc"][u & 1] = (u, last)
            b["done"] = g + 1
            b["empty"][g % stages].arrive()
            if last:
                b["acc_full"][u & 1].arrive()

    roles = [(r, f) for r, b in enumerate(blocks) for f in [producer(b), issuer(b)] + [epilogue(b, w) for w in range(epi)]]
    left = [epi + 2] * ranks
    weight = [rnd.choice([1, 1, 4, 20]) for _ in roles]
    for _ in range(2_000_000):
        if not roles:
            break
        for _ in range(ranks):
            if rnd.random() < 0.3:
                async_units()
        i = rnd.choices(range(len(roles)), weight)[0]
        try:
            next(roles[i][1])
        except StopIteration:
            left[roles[i][0]] -= 1
            if left[roles[i][0]] == 0:
                blocks[roles[i][0]]["there"] = False
            del roles[i], weight[i]
    if roles:
        raise base.Hazard("no role can go on")
    assert all(b["partial"] == epi for b in blocks)


SPLITS = [(2, 2, 8), (2, 9, 8), (4, 4, 8), (4, 37, 8), (8, 8, 8), (8, 70, 4), (8, 19, 64)]


@pytest.mark.parametrize("kb,stages", [(2, 3), (4, 2)])
@pytest.mark.parametrize("ranks,steps,seg", SPLITS)
def test_split_tile(ranks, steps, seg, kb, stages):
    for seed in range(3):
        split(ranks, steps, kb, stages, seg, seed)


@pytest.mark.parametrize("drop", ["acc_full", "written", "read"])
def test_each_barrier_of_a_split_tile_is_needed(drop):
    failed = 0
    for seed in range(20):
        try:
            split(4, 37, 2, 3, 8, seed, drop)
        except AssertionError:
            failed += 1
    assert failed, f"dropping {drop} went unnoticed"
