"""Host model of the expanded latent attention's shared slots: K and V blocks in eight slots of 16 KB, block g's chunks of K
as numbers 5 g .. 5 g + 2, the halves of its V as 5 g + 3 and 5 g + 4, number i in slot i % 8.  The loader and the two
tiles' issuers run under random interleavings, waits test only the parity of a phase, as the hardware does; no slot may be
overwritten before both tiles have read it, no wait may pass a phase early, and nothing may deadlock."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1


def run(pieces, seed, early_v=True, slow=None):
    """pieces: (blocks of tile 0, of tile 1).  early_v: as built, V waits for the K block whose slots it takes."""
    rnd = random.Random(seed)
    kc = [Bar(1) for _ in range(6)]
    v_full = [Bar(1) for _ in range(2)]
    k_empty, v_empty = [Bar(2) for _ in range(2)], [Bar(2) for _ in range(2)]
    turn, pv_ready = [Bar(1), Bar(1)], [0, 0]
    slots = [None] * 8
    total = sum(max(p) for p in pieces)

    def loader():
        for g in range(total):
            if g > 1:
                yield k_empty[g % 2], g // 2 - 1
            slots[5 * g % 8] = ("k", g, 0)
            kc[3 * (g % 2)].arrive()
            if g > 1:
                yield v_empty[g % 2], (g - 2) // 2
            for c in (1, 2):
                slots[(5 * g + c) % 8] = ("k", g, c)
                kc[3 * (g % 2) + c].arrive()
            if g > 1:
                yield v_empty[g % 2], g // 2 - 1
            if early_v and g > 0:
                yield k_empty[(g - 1) % 2], (g - 1) // 2
            for h in (0, 1):
                slots[(5 * g + 3 + h) % 8] = ("v", g, h)
            v_full[g % 2].arrive()

    def issuer(t):
        gk = gv = turns = 0
        for p in pieces:
            nb, n = max(p), p[t]
            for j in range(nb + 1):
                if j < nb and j >= n:
                    for c in range(3):
                        yield kc[3 * (gk % 2) + c], gk // 2
                if j > 0:
                    yield v_full[gv % 2], gv // 2
                yield turn[t], turns + (0 if t else -1)
                turns += 1
                if 0 < j <= n:
                    for h in (0, 1):
                        assert slots[(5 * gv + 3 + h) % 8] == ("v", gv, h), "V overwritten"
                if j > 0:
                    v_empty[gv % 2].arrive()
                    gv += 1
                if j < n:
                    for c in range(3):
                        yield kc[3 * (gk % 2) + c], gk // 2
                        assert slots[(5 * gk + c) % 8] == ("k", gk, c), "K overwritten"
                        yield None   # the products take a while
                        assert slots[(5 * gk + c) % 8] == ("k", gk, c), "K overwritten"
                turn[1 - t].arrive()
                if j < nb:
                    k_empty[gk % 2].arrive()
                    gk += 1

    roles = {"loader": loader(), "tile0": issuer(0), "tile1": issuer(1)}
    waiting = {r: None for r in roles}
    while roles:
        ready = []
        for r, w in waiting.items():
            if r not in roles:
                continue
            # phase w[1] is over: its parity is no longer the current one
            if w is None or (w[0].phase & 1) != (w[1] & 1):
                assert w is None or w[0].phase == w[1] + 1, f"{r} passed a phase early"
                ready.append(r)
        assert ready, "deadlock"
        r = rnd.choice([x for x in ready if x != slow] or ready) if rnd.random() < 0.95 else rnd.choice(ready)
        try:
            waiting[r] = next(roles[r])
        except StopIteration:
            del roles[r]


@pytest.mark.parametrize("slow", [None, "loader", "tile0", "tile1"])
@pytest.mark.parametrize("pieces", [[(1, 1)], [(5, 6)], [(1, 2), (3, 0), (9, 10), (1, 1), (1, 0), (4, 4)], [(12, 7), (2, 2)]])
def test_shared_slots(pieces, slow):
    for seed in range(60):
        run(pieces, seed, slow=slow)


def test_the_model_sees_a_missing_wait():
    with pytest.raises(AssertionError):
        for seed in range(60):
            run([(9, 10), (6, 6)], seed, early_v=False, slow="tile1")
