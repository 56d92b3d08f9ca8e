"""How the 8-bit product's converting warps hold a slot of weights, as a model on the CPU.  Each of the eight warps waits for
its weights, begins to read them, waits for its place in tensor memory, stores there, and only when the stores are done has
it read everything: then it gives the slot back, and one warp of the four of a step waits for the step's rows before it
reports the step.  A slot is so held across the wait for tensor memory, which the MMAs of earlier steps give back; the
model shows that this always ends, down to two slots, and that giving a slot back earlier is seen."""
import random

import pytest

from test_product_rings import SETS, Barrier, Ring, plan

WARPS = 4  # of a set: a quarter of the channels each


def run(w_stages, steps, halves, accs, parts, seed, early=False, late_share=0.1):
    """parts: reduction blocks (weight stages) of each part of a tile; a step takes `halves` halves of a stage.  early: a
    warp gives its slot back once its loads are issued."""
    rng = random.Random(seed)
    of_stage = 2 // halves  # steps of a weight stage
    bars = lambda n, count=1: [Barrier(count) for _ in range(n)]  # noqa: E731
    w_full, w_empty = bars(w_stages), bars(w_stages, WARPS * of_stage)
    x_full, step_full, step_empty = bars(steps), bars(steps, WARPS), bars(steps)
    acc_full, acc_empty = bars(accs), bars(accs)
    w = [[None, 0] for _ in range(w_stages)]           # the block in a slot, warps that have read all of theirs
    x = [[None, True] for _ in range(steps)]           # the step in a slot, whether its MMAs are done
    a = [[[None, True] for _ in range(steps)] for _ in range(WARPS)]
    accumulators = [True] * accs                       # read
    copies, late, mmas = [], [], []

    def weights():
        ring, n = Ring(), 0
        for blocks in parts:
            for _ in range(blocks):
                while not w_empty[ring.slot].complete(ring.parity ^ 1):
                    yield False
                assert w[ring.slot][0] is None or w[ring.slot][1] == WARPS * of_stage, "weights overwritten"
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
                assert x[ring.slot][1], "rows overwritten"
                x[ring.slot] = [n, False]
                (late if rng.random() < late_share else copies).append(x_full[ring.slot])
                n += 1
                ring.step(steps)
                yield True

    def convert(which, warp):
        stride, ahead, base = SETS // of_stage, which // of_stage, 0
        ring, step = Ring(), Ring(which)
        ring.step(w_stages, ahead)
        for blocks in parts:
            while ahead < blocks:
                while not w_full[ring.slot].complete(ring.parity):
                    yield False
                assert w[ring.slot][0] == base + ahead, "another block's weights"
                if early:
                    w_empty[ring.slot].arrive()
                yield True  # reading
                while not step_empty[step.slot].complete(step.parity ^ 1):
                    yield False
                n = (base + ahead) * of_stage + (which % 2 if of_stage == 2 else 0)
                assert a[warp][step.slot][1], "operand overwritten"
                a[warp][step.slot] = [n, False]
                yield True  # storing
                assert w[ring.slot][0] == base + ahead, "weights overwritten"
                w[ring.slot][1] += 1
                if not early:
                    w_empty[ring.slot].arrive()
                yield True
                while warp == 0 and not x_full[step.slot].complete(step.parity):
                    yield False
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
            assert accumulators[acc.slot], "accumulator overwritten"
            accumulators[acc.slot] = False
            for i in range(of_stage * blocks):
                while not step_full[step.slot].complete(step.parity):
                    yield False
                assert x[step.slot][0] == n and all(q[step.slot][0] == n for q in a), "another step's operands"
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
            accumulators[acc.slot] = True
            acc_empty[acc.slot].arrive()
            acc.step(accs)

    live = [weights(), rows(), mma(), epilogue()] + [convert(s, q) for s in range(SETS) for q in range(WARPS)]
    idle = 0
    while live:
        luck = rng.random()
        if copies and luck < 0.1:
            copies.pop(rng.randrange(len(copies))).arrive()
        elif mmas and luck < 0.2:
            slot, done = mmas.pop(0)
            x[slot][1] = True
            for q in a:
                q[slot][1] = True
            step_empty[slot].arrive()
            if done is not None:
                acc_full[done].arrive()
        else:
            role = rng.choice(live)
            try:
                idle = 0 if next(role) else idle + 1
            except StopIteration:
                live.remove(role)
            if idle > 150 and not copies and not mmas:
                assert late, "every role waits"
                late.pop(0).arrive()
            else:
                continue
        idle = 0


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("experts", [1, 1024])
def test_a_slot_held_across_the_wait_for_tensor_memory(rows, experts):
    w_stages, steps, halves, accs = plan(rows, experts)
    for seed in range(40):
        rng = random.Random(seed)
        run(w_stages, steps, halves, accs, [rng.randint(1, 20) for _ in range(4)] + [32, 32], seed)


def test_the_smallest_ring_is_among_them():
    assert plan(256, 1024)[0] == 2


@pytest.mark.parametrize("rows", [64, 256])
def test_a_slot_given_back_before_it_is_read_is_seen(rows):
    w_stages, steps, halves, accs = plan(rows, 1024)
    with pytest.raises(AssertionError, match="weights overwritten"):
        for seed in range(20):
            run(w_stages, steps, halves, accs, [32] * 3, seed, early=True, late_share=0.0)
