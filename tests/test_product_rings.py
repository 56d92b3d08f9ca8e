"""The 8-bit product's rings, as a model on the CPU: the weights' and rows' copies, the two sets of converting warps, the
MMA issuer and the epilogue meet at barriers that know a phase only by its parity.  A role that asks for a phase two
ahead is told that it is complete; whether one ever does depends on the rings' lengths.  The model lets copies land late
and in any order and checks that every role finds in a slot what it is to find there."""
import random

import pytest

SETS = 2


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def complete(self, parity):  # of the last phase with this parity
        return (self.phase & 1) != parity


class Ring:
    def __init__(self, slot=0):
        self.slot, self.parity = slot, 0

    def step(self, n, by=1):
        self.slot += by
        if self.slot >= n:
            self.slot, self.parity = self.slot - n, self.parity ^ 1


def run(w_stages, steps, halves, accs, parts, seed, late_share=0.1):
    """parts: reduction blocks (weight stages) of each part of a tile; a step takes `halves` halves of a stage."""
    rng = random.Random(seed)
    of_stage = 2 // halves  # steps of a weight stage
    bars = lambda n, count=1: [Barrier(count) for _ in range(n)]  # noqa: E731
    w_full, w_empty = bars(w_stages), bars(w_stages, of_stage)
    x_full, step_full, step_empty = bars(steps), bars(steps), bars(steps)
    acc_full, acc_empty = bars(accs), bars(accs)
    w, x, a = [None] * w_stages, [None] * steps, [None] * steps  # [number, readers done] in each slot
    copies, late, mmas = [], [], []

    def weights():
        ring, n = Ring(), 0
        for blocks in parts:
            for _ in range(blocks):
                while not w_empty[ring.slot].complete(ring.parity ^ 1):
                    yield False
                assert w[ring.slot] is None or w[ring.slot][1] == of_stage, "weights overwritten"
                w[ring.slot] = [n, 0]
                (late if rng.random() < late_share else copies).append(w_full[ring.slot])
                n += 1
                ring.step(w_stages)
                yield True

    def rows():
        ring, n = Ring(), 0
        for blocks in parts:
            for _ in range(of_stage * blocks):
                while not step_empty[ring.slot].complete(ring.parity ^ 1):
                    yield False
                assert x[ring.slot] is None or x[ring.slot][1] == 1, "rows overwritten"
                x[ring.slot] = [n, 0]
                copies.append(x_full[ring.slot])
                n += 1
                ring.step(steps)
                yield True

    def convert(which):
        stride, ahead, base = SETS // of_stage, which // of_stage, 0
        ring, step = Ring(), Ring(which)
        ring.step(w_stages, ahead)
        for blocks in parts:
            while ahead < blocks:
                while not w_full[ring.slot].complete(ring.parity):
                    yield False
                assert w[ring.slot][0] == base + ahead, "another stage's weights"
                w[ring.slot][1] += 1
                w_empty[ring.slot].arrive()
                yield True
                while not step_empty[step.slot].complete(step.parity ^ 1):
                    yield False
                n = (base + ahead) * of_stage + (which % 2 if of_stage == 2 else 0)
                assert a[step.slot] is None or a[step.slot][1] == 1, "operand overwritten"
                a[step.slot] = [n, 0]
                while not x_full[step.slot].complete(step.parity):
                    yield False
                assert x[step.slot][0] == n, "another step's rows"
                step_full[step.slot].arrive()
                yield True
                ahead += stride
                ring.step(w_stages, stride)
                step.step(steps, SETS)
            ahead -= blocks
            base += blocks

    def mma():
        step, acc, n = Ring(), Ring(), 0
        for blocks in parts:
            while not acc_empty[acc.slot].complete(acc.parity ^ 1):
                yield False
            for i in range(of_stage * blocks):
                while not step_full[step.slot].complete(step.parity):
                    yield False
                assert a[step.slot][0] == n and x[step.slot][0] == n, "another step's operands"
                mmas.append((step.slot, acc.slot if i == of_stage * blocks - 1 else None))
                n += 1
                step.step(steps)
                yield True
            acc.step(accs)

    def epilogue():
        acc = Ring()
        for _ in parts:
            while not acc_full[acc.slot].complete(acc.parity):
                yield False
            yield True
            acc_empty[acc.slot].arrive()
            acc.step(accs)

    live, idle = [weights(), rows(), convert(0), convert(1), mma(), epilogue()], 0
    while live:
        luck = rng.random()
        if copies and luck < 0.25:
            copies.pop(rng.randrange(len(copies))).arrive()
        elif mmas and luck < 0.5:
            slot, done = mmas.pop(0)
            a[slot][1] = x[slot][1] = 1
            step_empty[slot].arrive()
            if done is not None:
                acc_full[done].arrive()
        else:
            role = rng.choice(live)
            try:
                idle = 0 if next(role) else idle + 1
            except StopIteration:
                live.remove(role)
            if idle > 60 and not copies and not mmas:
                assert late, "every role waits"
                late.pop(0).arrive()
            else:
                continue
        idle = 0


def plan(rows, experts):
    """(weight stages, steps, halves of a step, accumulators) as the library launches a tile of so many rows."""
    halves, steps = (1, 5) if rows > 128 else (2, (512 - 2 * rows) // 64)
    readers = 2 if rows > 128 else 1
    fixed = 1024 + 96 + 16 * rows + readers * 4096 + 4 * (3 * experts + 1) + 8 * (2 * 12 + 3 * 15 + 2 * 2 + 1)
    stages = min(12, (227 * 1024 - fixed - steps * halves * rows * 128) // 16384)
    return stages - stages % (SETS * halves // 2), steps, halves, 1 if rows > 128 else 2


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("experts", [1, 128, 1024])
def test_every_role_finds_what_it_is_to_find(rows, experts):
    w_stages, steps, halves, accs = plan(rows, experts)
    assert w_stages >= 2
    for seed in range(12):
        rng = random.Random(seed)
        run(w_stages, steps, halves, accs, [rng.randint(1, 20) for _ in range(3)] + [32, 32], seed)


@pytest.mark.parametrize("w_stages,steps", [(7, 6), (5, 4)])
def test_the_model_sees_a_set_that_meets_another_slot_in_every_round(w_stages, steps):
    with pytest.raises(AssertionError, match="another stage's weights"):
        for seed in range(20):
            run(w_stages, steps, 2, 2, [32] * 4, seed)
