"""The 4-bit tile product's rings, as a model on the CPU: the weights' and rows' copies, the sets of converting warps, the MMA
issuer and the epilogue meet at barriers that know a phase only by its parity, and the tiles' descriptions lie in a ring
that the weights' warp runs ahead in.  The model lets copies land late and in any order and MMAs finish late, and checks that
every role finds in a slot what it is to find there, and that all of them come to an end."""
import random

import pytest


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
    def __init__(self, n, by=0):
        self.n, self.slot, self.parity = n, 0, 0
        if by:
            self.step(by)

    def step(self, by=1):
        self.slot += by
        if self.slot >= self.n:
            self.slot, self.parity = self.slot - self.n, self.parity ^ 1


FORMS = {  # as product_i4_tiles.cu has them
    "16 and 32 rows": dict(blocks=2, slots=3, sets=3, accs=2, relayed=True, x_stages=6, w_stages=9),
    "64 rows": dict(blocks=2, slots=3, sets=3, accs=2, relayed=False, x_stages=3, w_stages=6),
    "wide": dict(blocks=1, slots=2, sets=1, accs=1, relayed=True, x_stages=4, w_stages=2),
}
TILE_RING = 32


def run(tiles, row_blocks, seed, blocks, slots, sets, accs, relayed, x_stages, w_stages, late=0.2):
    rng = random.Random(seed)
    steps_of_pair = 2 // blocks
    pairs = (row_blocks + 1) // 2
    steps = row_blocks if blocks == 1 else pairs  # of a tile
    stride, mine = (sets, 1) if blocks == 2 else (1, 2 // sets)

    def bars(n, count=1):
        return [Barrier(count) for _ in range(n)]

    w_full, w_empty = bars(w_stages), bars(w_stages, 1 if blocks == 2 else sets)
    x_full, step_full, step_empty = bars(x_stages), bars(slots), bars(slots)
    x_empty = bars(x_stages) if relayed else step_empty
    acc_full, acc_empty = bars(accs), bars(accs)
    w, x, a, acc = [None] * w_stages, [None] * x_stages, [None] * slots, [None] * accs
    tile = [None] * TILE_RING
    flying = []      # copies: what lands when
    mmas = []        # issued, in order: what each commit tells
    done = []

    def weights():
        ring, n = Ring(w_stages), 0
        for k in range(tiles):
            tile[k % TILE_RING] = k
            for p in range(pairs):
                while not w_empty[ring.slot].complete(ring.parity ^ 1):
                    yield False
                slot, what = ring.slot, (k, p)
                flying.append(lambda slot=slot, what=what: (w.__setitem__(slot, what), w_full[slot].arrive()))
                n += 1
                ring.step()
                yield True

    def rows():
        ring = Ring(x_stages)
        for k in range(tiles):
            for b in range(steps):
                while not x_empty[ring.slot].complete(ring.parity ^ 1):
                    yield False
                slot, what = ring.slot, (k, b)
                flying.append(lambda slot=slot, what=what: (x.__setitem__(slot, what), x_full[slot].arrive()))
                ring.step()
                yield True

    def convert(which):
        ahead = which if blocks == 2 else 0
        wr, s, xr = Ring(w_stages, ahead), Ring(slots, which), Ring(x_stages, which)
        fresh = slots // sets
        for k in range(tiles):
            if k > 0 and ahead < pairs:
                while not w_full[wr.slot].complete(wr.parity):
                    yield False
                assert tile[k % TILE_RING] == k, "a tile's description overwritten"
            while ahead < pairs:
                while not w_full[wr.slot].complete(wr.parity):
                    yield False
                assert w[wr.slot] == (k, ahead), "weights not there, or overwritten"
                for i in range(min(mine, row_blocks - 2 * ahead)):
                    while not step_empty[s.slot].complete(s.parity ^ 1):
                        yield False
                    if fresh:
                        fresh -= 1
                    elif relayed:
                        x_empty[(xr.slot + slots) % x_stages].arrive()
                    assert a[s.slot] is None, "a step overwritten"
                    yield True
                    number = ahead * steps_of_pair + (i if blocks == 1 else 0)
                    a[s.slot] = (k, number)
                    if i == mine - 1 or 2 * ahead + 1 >= row_blocks:
                        w_empty[wr.slot].arrive()
                    while not x_full[xr.slot].complete(xr.parity):
                        yield False
                    assert x[xr.slot] == (k, number), "rows not there, or overwritten"
                    step_full[s.slot].arrive()
                    s.step(sets)
                    xr.step(sets)
                    yield True
                ahead += stride
                wr.step(stride)
            ahead -= pairs

    def issue():
        s, xr, ar = Ring(slots), Ring(x_stages), Ring(accs)
        for k in range(tiles):
            while not acc_empty[ar.slot].complete(ar.parity ^ 1):
                yield False
            assert acc[ar.slot] is None
            for b in range(steps):
                while not step_full[s.slot].complete(s.parity):
                    yield False
                if b == 0 and k > 0:
                    assert tile[k % TILE_RING] == k, "a tile's description overwritten"
                assert a[s.slot] == (k, b), "a step not there"
                assert x[xr.slot] == (k, b), "rows not there"
                slot, xslot, aslot, end = s.slot, xr.slot, ar.slot, b == steps - 1

                def finish(slot=slot, xslot=xslot, aslot=aslot, end=end, k=k, b=b):
                    assert x[xslot] == (k, b) and a[slot] == (k, b), "operands changed under the MMAs"
                    a[slot] = None
                    step_empty[slot].arrive()
                    if end:
                        acc[aslot] = k
                        acc_full[aslot].arrive()

                mmas.append(finish)
                xr.step()
                yield True
                s.step()
            ar.step()

    def epilogue():
        ar = Ring(accs)
        for k in range(tiles):
            while not acc_full[ar.slot].complete(ar.parity):
                yield False
            assert acc[ar.slot] == k
            yield True
            acc[ar.slot] = None
            acc_empty[ar.slot].arrive()
            done.append(k)
            ar.step()

    roles = [weights(), rows(), issue(), epilogue()] + [convert(i) for i in range(sets)]
    idle = 0
    while roles:
        moved = False
        for role in rng.sample(roles, len(roles)):
            if rng.random() < 0.3:
                continue
            try:
                moved |= next(role)
            except StopIteration:
                roles.remove(role)
                moved = True
        while flying and rng.random() > late:
            flying.pop(rng.randrange(len(flying)))()
            moved = True
        if mmas and rng.random() > late:
            mmas.pop(0)()
            moved = True
        idle = 0 if moved else idle + 1
        assert idle < 2000, "no role goes on"
    assert done == list(range(tiles))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("row_blocks", [1, 2, 3, 4, 5, 8, 13, 14, 31, 32])
def test_every_role_finds_its_data(form, row_blocks):
    for seed in range(6):
        for late in (0.05, 0.5, 0.9):
            run(1 + 300 // row_blocks, row_blocks, seed, late=late, **FORMS[form])


def test_the_model_sees_a_weight_ring_that_sets_do_not_share_evenly():
    # a set that meets other slots in every round can take an older copy for its own
    bad = dict(FORMS["16 and 32 rows"], slots=9, x_stages=18, w_stages=4)
    with pytest.raises(AssertionError):
        for seed in range(200):
            run(30, 14, seed, late=0.9, **bad)
