"""The hand-overs of k_tree_mma between its warps, as a model on the CPU: copying warps, the issuing thread, softmax warps and the
tensor core's queue run in random order over the barriers of ar_tree_mma.cuh, with their parities.  Every run ends, and no wait
returns before the phase that it is meant for (two phases with the same parity look alike to a barrier)."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than the phase takes"
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def test(self, parity):
        return (self.phase - 1) & 1 == parity


def run(NM, GROUPS, NS, QS, RS, TILES, items, seed, scaled=False, boxes=False):
    """items: (tiles, whether its last tiles are mixed).  RS > 0: 8-bit, copied to stages first.  boxes: a warp asks for tensor
    copies, and the copying warps help.  Returns what every stuck process waits for, or None."""
    r = random.Random(seed)
    tiles = [(i == 0, i == n - 1, mixed and i >= n - 2) for n, mixed in items for i in range(n)]
    n, warps, small = len(tiles), 4 * GROUPS, RS > 0
    split = GROUPS == 2 and NM == 1
    # fill f: keys of tile f / 2, or its values where f is odd; each has a ring of its own
    KS, VS = NS // 2, NS - NS // 2

    def slot(f):
        return KS + (f >> 1) % VS if f & 1 else (f >> 1) % KS

    def turn(f):
        return (f >> 1) // (VS if f & 1 else KS)

    def before(f):
        return f - 2 * (VS if f & 1 else KS)

    hands = 2 if small else 4        # warps that finish a fill
    kv_full, kv_empty = [Bar(hands if boxes else 1) for _ in range(NS)], [Bar(1) for _ in range(NS)]
    q_full, q_empty = [Bar(4) for _ in range(QS)], [Bar(1) for _ in range(QS)]
    B = 2   # score buffers
    s_full, p_ready, o_done = [Bar(1) for _ in range(B)], [Bar(4) for _ in range(B)], [Bar(1) for _ in range(GROUPS)]
    p_used = [Bar(1) for _ in range(B)]
    tile_full, tile_empty = [Bar(1) for _ in range(TILES)], [Bar(warps + 1 + (4 if boxes else 0)) for _ in range(TILES)]
    arrived, sent, raw_empty = [Bar(1) for _ in range(8)], [0, 0, 1, 1], [Bar(2) for _ in range(RS)]
    given = {}
    told, taken = Bar(4), Bar(4)
    queues, copies = [[], []], []    # products of each warp in order, with the barriers they complete; copies on their way
    holds = [None] * 4               # the step whose weights lie in a buffer
    content = [None] * NS     # the fill that lies in a slot: what the products must find
    used = set()
    state = {"o": [None, None]}   # who may touch a group's O: None, or "read" while the first group reads the second's

    POWERS = 4 if NM == 2 else 6   # items whose queries' powers of two are kept
    powers = [[None] * POWERS for _ in range(4)]

    def fill(w, item):
        """A warp's part of an item's queries: the powers of two at once."""
        powers[w][item % POWERS] = item
        copies.append(q_full[item % QS].arrive)

    def wait(bar, phase, what):
        """Of the phase with this number, by its parity, as the kernel does."""
        return bar, phase & 1, phase, what

    def ready(bar, phase):
        """A test that does not wait."""
        good = bar.test(phase & 1)
        assert good == (bar.phase == phase + 1), "a parity of another phase"
        return good

    def copy(w):
        """Keys (w 0 and 2) or values (1 and 3) of alternate tiles."""
        values, tile, done, filled = w & 1, w >> 1, w >> 1, 0
        uses = [0] * 8            # phases of `arrived` that were waited for (16-bit)
        begins = [t for t in range(n) if tiles[t][0]]
        arrival = (lambda t: (2 * t + values) % RS) if small else (lambda t: (t & 1) * 4 + (t >> 1 & 3))

        def give(f):
            content[slot(f)] = f
            kv_full[slot(f)].arrive()

        def free(f):
            x = before(f)
            if x >= 0 and not sent[(x & 1) + (x >> 1 & 1) * 2] > x >> 1:
                return False
            return ready(kv_empty[slot(f)], turn(f) - 1)

        while True:
            moved = False
            if small:
                f = 2 * done + values
                if done < tile and free(f) and ready(arrived[arrival(done)], f // RS):
                    done, moved = done + 2, True
                    give(f)
                    sent[w] = done
            else:
                while done < tile and not (values and tiles[done][2]):
                    done += 2
                if done < tile and ready(arrived[arrival(done)], uses[arrival(done)]):
                    uses[arrival(done)] += 1
                    give(2 * done + 1)
                    done, moved = done + 2, True
            if filled < len(begins) and ready(q_empty[filled % QS], filled // QS - 1):
                fill(w, filled)
                filled, moved = filled + 1, True
            if tile < n:
                f = 2 * tile + values
                room = (tile - done) // 2 < RS // 4 if small else free(f)
                if room and (values or ready(tile_empty[tile % TILES], tile // TILES - 1)):
                    if not values:
                        tile_full[tile % TILES].arrive()
                    needs = small or (values and tiles[tile][2])
                    copies.append(arrived[arrival(tile)].arrive if needs else lambda f=f: give(f))
                    tile, moved = tile + 2, True
                    if not small:
                        sent[w] = tile
            if not moved and tile >= n and done >= n and filled == len(begins):
                return
            yield None

    def ask(values):
        """The warps of tensor copies, of keys and of values."""
        def land(f):
            content[slot(f)] = f
            for _ in range(hands):
                kv_full[slot(f)].arrive()

        for t in range(n):
            if not values:
                yield wait(tile_empty[t % TILES], t // TILES - 1, f"room for tile {t}")
                tile_full[t % TILES].arrive()
            f = 2 * t + values
            if small:
                yield wait(raw_empty[f % RS], f // RS - 1, f"stage of fill {f}")
                copies.append(arrived[f % RS].arrive)
            else:
                yield wait(kv_empty[slot(f)], turn(f) - 1, f"slot of fill {f}")
                copies.append(arrived[t % 8].arrive if f & 1 and tiles[t][2] else lambda f=f: land(f))

    def help_out(w):
        begins, filled, uses = [t for t in range(n) if tiles[t][0]], 0, [0] * 8

        def until(bar, phase):
            """Fills queries' slots while it waits."""
            nonlocal filled
            while not ready(bar, phase):
                if filled < len(begins) and ready(q_empty[filled % QS], filled // QS - 1):
                    fill(w, filled)
                    filled += 1
                yield None

        def give(f):
            given[f] = given.get(f, 0) + 1
            if given[f] == hands:
                content[slot(f)] = f
            kv_full[slot(f)].arrive()

        for t in range(n):
            yield from until(tile_full[t % TILES], t // TILES)
            if small:
                f = 2 * t + (w >> 1)
                yield from until(arrived[f % RS], f // RS)
                yield from until(kv_empty[slot(f)], turn(f) - 1)
                give(f)
                raw_empty[f % RS].arrive()
            elif tiles[t][2]:
                yield from until(arrived[t % 8], uses[t % 8])
                uses[t % 8] += 1
                give(2 * t + 1)
            tile_empty[t % TILES].arrive()
        while filled < len(begins):
            if ready(q_empty[filled % QS], filled // QS - 1):
                fill(w, filled)
                filled += 1
            yield None

    S = NM   # steps of a tile
    group_of, phase_of = ((lambda u: u & 1), (lambda u: u >> 1)) if GROUPS == 2 else ((lambda u: 0), (lambda u: u))

    def scores():
        begun = 0
        for u in range(n * S):
            t = u // S
            if u % S == 0:
                yield wait(tile_full[t % TILES], t // TILES, f"tile {t}")
                if tiles[t][0]:
                    yield wait(q_full[begun % QS], begun // QS, f"queries of tile {t}")
                    begun += 1
                yield wait(kv_full[slot(2 * t)], turn(2 * t), f"keys of tile {t}")
            yield wait(p_used[u % B], u // B - 1, f"product {u - B}")
            assert holds[u % B] is None, "scores are written over weights that are still to be used"
            last = tiles[t][1] or t == n - 1
            queues[0].append((2 * t, None, [s_full[u % B]] +
                              ([kv_empty[slot(2 * t)]] + ([q_empty[(begun - 1) % QS]] if last else []) if u % S == S - 1 else [])))

    def values():
        for u in range(n * S):
            t = u // S
            f = 2 * t + 1
            if u % S == 0:
                yield wait(tile_full[t % TILES], t // TILES, f"tile {t}")
                tile_empty[t % TILES].arrive()
                yield wait(kv_full[slot(f)], turn(f), f"values of step {u}")
            yield wait(p_ready[u % B], u // B, f"weights {u}")
            queues[1].append((f, u, [o_done[group_of(u)], p_used[u % B]] + ([kv_empty[slot(f)]] if u % S == S - 1 else [])))

    def softmax(w):
        m, begun, joins, awaits, own = w // 4, 0, 0, False, -1
        for t in range(n):
            yield wait(tile_full[t % TILES], t // TILES, f"tile {t}")
            if tiles[t][0]:
                own = -1
                begun += 1
            for u in [S * t + (m if NM == 2 else 0)] if not split or t & 1 == m else []:
                yield wait(s_full[u % B], u // B, f"scores {u}")
                if scaled and own < 0:
                    assert powers[w % 4][(begun - 1) % POWERS] == begun - 1, "a row's power of two was written over"
                if own >= 0 and r.random() < 0.5:   # the reference moves
                    yield wait(o_done[m], phase_of(u) - 1, f"product before step {u}")
                if tiles[t][2]:
                    yield wait(kv_full[slot(2 * t + 1)], turn(2 * t + 1), f"values of tile {t}")
                bad = tiles[t][2] and r.random() < 0.5
                if (bad or tiles[t][1] or t == n - 1) and phase_of(u) > 0:
                    yield wait(o_done[m], phase_of(u) - 1, f"product before step {u}")
                if split and awaits:
                    yield wait(taken, joins - 1, f"the join before step {u}")
                    awaits = False
                if w % 4 == 0:
                    holds[u % B] = u
                p_ready[u % B].arrive()
                own = u
                if bad:
                    yield wait(o_done[m], phase_of(u), f"product of step {u}")
            if tiles[t][1] or t == n - 1:
                if own >= 0:
                    yield wait(o_done[m], phase_of(own), f"product of step {own}")
                if split and m == 1:
                    if awaits:
                        yield wait(taken, joins - 1, f"the join before tile {t}")
                    told.arrive()
                    joins, awaits = joins + 1, True
                elif split:
                    yield wait(told, joins, f"references at tile {t}")
                    joins += 1
                    state["o"][1] = (state["o"][1] or 0) + 1
                    yield None   # reading both
                    state["o"][1] -= 1
                    taken.arrive()
            tile_empty[t % TILES].arrive()

    running = {f"copy {w}": help_out(w) if boxes else copy(w) for w in range(4)}
    if boxes:
        running.update({"copy keys": ask(0), "copy values": ask(1)})
    running.update({"scores": scores(), "values": values()})
    running.update({f"softmax {w}": softmax(w) for w in range(warps)})
    waits, idle = dict.fromkeys(running), 0
    while running:
        can = [k for k in running if waits[k] is None or waits[k][0].test(waits[k][1])]
        for k in can:
            if waits[k] is not None:   # not before its phase, and not after the next one with its parity
                assert waits[k][0].phase == waits[k][2] + 1, (k, waits[k][3])
        choice = can + [q for q in (0, 1) if queues[q]] + (["memory"] * 2 if copies else [])
        idle = idle + 1 if all(isinstance(k, str) and k.startswith("copy") for k in choice) else 0
        if not choice or idle > 20000:   # copying warps never wait: they look for something to do
            return {k: waits[k] and waits[k][3] for k in running}
        k = r.choice(choice)
        if k in (0, 1):   # the tensor core: each warp's products in order, the two in any
            f, u, bars = queues[k].pop(0)
            assert content[slot(f)] == f, "a product reads another fill than its own"
            if u is not None:
                assert not state["o"][group_of(u)], "an O is written that is still read"
                assert holds[u % B] == u, "a product reads another step's weights"
                holds[u % B] = None
            used.add(f)
            for b in bars:
                b.arrive()
            continue
        if k == "memory":
            copies.pop(r.randrange(min(len(copies), 6)))()
            continue
        try:
            waits[k] = next(running[k])
        except StopIteration:
            del running[k]
    assert used == set(range(2 * n))
    return None


# NM, GROUPS, NS, QS, RS, TILES, scaled as TreeMmaShape has them
SHAPES = {"16 bit, 64, 128 rows": (1, 2, 10, 2, 0, 8), "16 bit, 64, 256 rows": (2, 2, 10, 1, 0, 8), "16 bit, 128, 128 rows": (1, 2, 6, 1, 0, 8),
          "16 bit, 128, 256 rows": (2, 2, 5, 1, 0, 8), "16 bit, 192": (1, 1, 7, 1, 0, 8), "16 bit, 256": (1, 1, 5, 1, 0, 8),
          "8 bit, 64, 128 rows": (1, 2, 8, 2, 8, 6, True), "8 bit, 64, 256 rows": (2, 2, 8, 1, 8, 6, True),
          "8 bit, 128, 128 rows": (1, 2, 4, 1, 4, 6, True), "8 bit, 128, 256 rows": (2, 2, 3, 1, 4, 6, True),
          "8 bit, 192": (1, 1, 5, 1, 4, 6, True), "8 bit, 256": (1, 1, 3, 1, 4, 6, True), "8 bit, 256, fp16 queries": (1, 1, 3, 1, 4, 8)}


@pytest.mark.parametrize("boxes", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_run_ends_and_every_wait_is_for_its_own_phase(shape, boxes):
    for seed in range(40):
        r = random.Random(seed)
        items = [(r.choice([1, 1, 2, 3, 5, 9]), r.random() < 0.7) for _ in range(r.randint(1, 8))]
        stuck = run(*SHAPES[shape][:6], items, seed, len(SHAPES[shape]) > 6, boxes)
        assert stuck is None, (items, stuck)
