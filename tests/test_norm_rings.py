"""The barriers of the norm gradient for wide rows, as a model on the CPU: copies that bring rows into stages, sums that the
warps of a cluster send to each other, and waits that run out.  The model lets copies and sums land late and in any order
and lets waits run out at any time, and checks that no barrier gets an arrival that it does not count, that a thread finds in a
stage the row that it waited for, that nothing lands in a thread block that has ended, and that all come to an end."""
import random

import pytest

TENSORS = 4  # brought by a lane each of the first warps


class Barrier:
    """Counts arrivals and what copies still have to bring; waits know a phase only by its parity."""

    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phase = count, count, 0, 0

    def _end(self):
        if self.pending == 0 and self.bytes == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def arrive(self, expect=0):
        assert self.pending > 0, "an arrival beyond the barrier's count"
        self.bytes += expect
        self.pending -= 1
        self._end()

    def land(self):
        self.bytes -= 1
        self._end()

    def complete(self, parity):  # the last phase with this parity
        return (self.phase & 1) != parity


class Together:
    """A barrier of hardware over n warps."""

    def __init__(self, n):
        self.n, self.arrived, self.round = n, 0, 0

    def wait(self):
        here = self.round
        self.arrived += 1
        if self.arrived == self.n:
            self.arrived, self.round = 0, here + 1
        while self.round == here:
            yield


class Block:
    def __init__(self, stages, warps):
        self.bars = [Barrier(TENSORS) for _ in range(stages)]
        self.sent = [Barrier(1) for _ in range(2)]
        self.stage = [[None] * TENSORS for _ in range(stages)]
        self.sums = [{}, {}]
        self.brought, self.sends = [0] * TENSORS, [0] * warps
        self.abort = False
        self.sync, self.left = Together(warps), 0


def run(ranks, warps, stages, rows, seed, row_out, sums_out, late=0.3, stops=True):
    """row_out, sums_out: how often a look at a barrier is the last of its wait.  stops False: a thread whose wait has run out goes
    on as if it had not."""
    rng = random.Random(seed)
    cluster = ranks > 1
    blocks = [Block(stages, warps) for _ in range(ranks)]
    everyone = Together(ranks * warps)
    flying, errors = [], []

    def warp(r, w):
        me, state = blocks[r], dict(ok=True, source=w < TENSORS, lost=False, brought=0)

        def bring(stage):
            if not state["source"] or state["brought"] >= rows:
                return
            row = state["brought"]
            me.bars[stage].arrive(expect=1)
            flying.append((r, lambda: (me.stage[stage].__setitem__(w, row), me.bars[stage].land())))
            state["brought"] += 1

        def run_out(bar, parity, often, flag):
            while True:
                if rng.random() < often:
                    return True
                if bar.complete(parity):
                    return False
                if stops and flag():
                    return True
                yield

        def wait_row(stage, parity, row):
            if (yield from run_out(me.bars[stage], parity, row_out, lambda: me.abort)):
                errors.append("row")
                state["ok"] = False
                if stops:
                    state["source"] = False
                    for block in blocks:
                        block.abort = True
            elif state["ok"]:
                assert me.stage[stage] == [row] * TENSORS, "a stage without its row"

        def send(index):
            slot = index & 1
            if w == 0:
                me.sent[slot].arrive(expect=ranks * warps)
            for q in range(ranks):
                to = blocks[q]
                flying.append((q, lambda to=to: (to.sums[slot].__setitem__((r, w), index), to.sent[slot].land())))

        def row_sums(index):
            if not cluster:
                yield from me.sync.wait()
                return
            send(index)
            yield
            if (yield from run_out(me.sent[index & 1], (index >> 1) & 1, sums_out, lambda: me.abort)):
                errors.append("sums")
                if stops:
                    state["lost"], state["source"] = True, False
                    for block in blocks:
                        block.abort = True
            else:
                assert set(me.sums[index & 1].values()) == {index} and len(me.sums[index & 1]) == ranks * warps

        for i in range(stages):
            bring(i)
            yield
        yield from wait_row(0, 0, 0)
        yield from row_sums(0)
        k = stage = parity = 0
        while k < rows and not state["lost"]:
            read = stage
            stage += 1
            if stage == stages:
                stage, parity = 0, parity ^ 1
            if state["ok"] and stops:
                assert me.stage[read] == [k] * TENSORS, "a row overwritten before it was read"
            if k + 1 < rows:
                yield from wait_row(stage, parity, k + 1)
            yield
            yield from row_sums(k + 1)
            bring(read)
            k += 1
            yield
        if not stops:
            return
        yield from (everyone if cluster else me.sync).wait()
        if not me.abort:
            return
        if w < TENSORS:
            me.brought[w] = state["brought"]
        me.sends[w] = k + 1
        yield from (everyone if cluster else me.sync).wait()

        def drain(bar, parity):
            for _ in range(20000):
                if bar.complete(parity):
                    return
                yield
            raise AssertionError("a phase that never ends")

        most = max(me.brought)
        if w < TENSORS:
            for i in range(state["brought"], most):
                me.bars[i % stages].arrive()
                yield
        if w == 0:
            for i in range(max(0, most - stages), most):
                yield from drain(me.bars[i % stages], (i // stages) & 1)
        if cluster:
            most = max(max(block.sends) for block in blocks)
            assert k + 1 >= most - 1
            if k + 1 < most:
                send(k + 1)
                yield
            if w == 0:
                for i in range(max(0, most - 2), most):
                    yield from drain(me.sent[i & 1], (i >> 1) & 1)
            yield from everyone.wait()

    roles = [(r, warp(r, w)) for r in range(ranks) for w in range(warps)]
    looks = 0
    while roles:
        looks += 1
        assert looks < 200000, "no end"
        i = rng.randrange(len(roles))
        r, role = roles[i]
        try:
            next(role)
        except StopIteration:
            roles.pop(i)
            blocks[r].left += 1
            assert blocks[r].left < warps or not any(q == r for q, _ in flying), "a thread block ends with data on its way to it"
        while flying and rng.random() > late:
            q, land = flying.pop(rng.randrange(len(flying)))
            assert blocks[q].left < warps, "data lands in a thread block that has ended"
            land()
    assert not flying
    return errors


SHAPES = [(1, 9, 8, 30), (1, 5, 2, 12), (1, 4, 6, 3), (2, 5, 3, 17), (4, 4, 2, 9), (6, 4, 4, 6), (2, 4, 8, 1)]


@pytest.mark.parametrize("ranks,warps,stages,rows", SHAPES)
def test_rows_arrive_and_nothing_is_left_over(ranks, warps, stages, rows):
    for seed in range(6):
        for late in (0.1, 0.6, 0.9):
            assert run(ranks, warps, stages, rows, seed, 0.0, 0.0, late) == []


@pytest.mark.parametrize("ranks,warps,stages,rows", SHAPES)
@pytest.mark.parametrize("row_out,sums_out", [(1.0, 1.0), (1.0, 0.0), (0.02, 0.0), (0.002, 0.0), (0.0, 1.0), (0.0, 0.02),
                                              (0.0, 0.002), (0.01, 0.005)])
def test_waits_that_run_out(ranks, warps, stages, rows, row_out, sums_out):
    for seed in range(8):
        for late in (0.1, 0.6, 0.9):
            run(ranks, warps, stages, rows, seed, row_out, sums_out, late)


@pytest.mark.parametrize("ranks", [1, 2])
def test_the_model_sees_threads_that_go_on_after_a_wait(ranks):
    # without a stop a stage is asked for again while its last copy is on its way, or a block ends before its data is there
    for row_out in (1.0, 0.3):
        with pytest.raises(AssertionError):
            for seed in range(100):
                run(ranks, 4, 2, 9, seed, row_out, 0.0, late=0.9, stops=False)
