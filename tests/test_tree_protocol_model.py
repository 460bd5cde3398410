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


def run(NM, NS, QS, LAG, TILES, items, seed, small=False, scaled=False):
    """items: (tiles, whether its last tiles are mixed).  Returns what every stuck process waits for, or None."""
    r = random.Random(seed)
    tiles = [(i == 0, i == n - 1, mixed and i >= n - 2) for n, mixed in items for i in range(n)]
    n, warps = len(tiles), 4 * NM
    kv_full, kv_empty = [Bar(4) for _ in range(NS)], [Bar(1) for _ in range(NS)]
    q_full, q_empty = [Bar(4) for _ in range(QS)], [Bar(1 + (warps if scaled else 0)) for _ in range(QS)]
    s_full, p_ready, o_done = [Bar(1), Bar(1)], [Bar(4), Bar(4)], [Bar(1) for _ in range(NM)]
    tile_full, tile_empty = [Bar(4) for _ in range(TILES)], [Bar(warps) for _ in range(TILES)]
    queue = []                # products in order, with the barriers they complete
    content = [None] * NS     # the fill that lies in a slot: what the products must find
    handed, used = {}, set()

    def wait(bar, phase, what):
        """Of the phase with this number, by its parity, as the kernel does."""
        return bar, phase & 1, phase, what

    def copy(w):
        wanted = filled = given = done = 0

        def hand_over():
            nonlocal filled, given, done
            f = done
            done += 1
            t, first = f >> 1, f & 1 == 0 and tiles[f >> 1][0]
            if first and filled == given:
                yield wait(q_empty[filled % QS], filled // QS - 1, f"late queries of tile {t}")
                yield wait(tile_full[t % TILES], t // TILES, f"description of tile {t}")
                filled += 1
            if small:
                yield wait(kv_empty[f % NS], f // NS - 1, f"slot of fill {f}")
            if first:
                q_full[given % QS].arrive()
                given += 1
            handed[f] = handed.get(f, 0) + 1
            if handed[f] == 4:
                content[f % NS] = f
            kv_full[f % NS].arrive()

        for t in range(n):
            yield wait(tile_empty[t % TILES], t // TILES - 1, f"room for tile {t}")
            tile_full[t % TILES].arrive()
            if tiles[t][0]:
                wanted += 1
                if filled + 1 == wanted and q_empty[filled % QS].test((filled // QS & 1) ^ 1):
                    filled += 1
            for f in (2 * t, 2 * t + 1):
                if not small:
                    yield wait(kv_empty[f % NS], f // NS - 1, f"slot of fill {f}")
                if f - done >= LAG:
                    yield from hand_over()
        while done < 2 * n:
            yield from hand_over()

    def issue():
        begun = 0

        def scores(u):
            nonlocal begun
            t, m = divmod(u, NM)
            if m == 0:
                yield wait(tile_full[t % TILES], t // TILES, f"tile {t}")
                if tiles[t][0]:
                    yield wait(q_full[begun % QS], begun // QS, f"queries of tile {t}")
                    begun += 1
                yield wait(kv_full[2 * t % NS], 2 * t // NS, f"keys of tile {t}")
            last = tiles[t][1] or t == n - 1
            queue.append(((2 * t,), [s_full[u & 1]] + ([kv_empty[2 * t % NS]] + ([q_empty[(begun - 1) % QS]] if last else []) if m == NM - 1 else [])))

        yield from scores(0)
        for u in range(n * NM):
            t, m = divmod(u, NM)
            f = 2 * t + 1
            if u + 1 < n * NM:
                if u > 0:
                    yield wait(o_done[(u - 1) % NM], (u - 1) // NM, f"product {u - 1}")
                yield from scores(u + 1)
            yield wait(p_ready[u & 1], u >> 1, f"weights {u}")
            if m == 0:
                yield wait(kv_full[f % NS], f // NS, f"values of tile {t}")
            queue.append(((f,), [o_done[m]] + ([kv_empty[f % NS]] if m == NM - 1 else [])))

    def softmax(w):
        m, begun = w // 4, 0
        for t in range(n):
            yield wait(tile_full[t % TILES], t // TILES, f"tile {t}")
            u = t * NM + m
            yield wait(s_full[u & 1], u >> 1, f"scores {u}")
            if tiles[t][0]:
                if scaled:
                    yield wait(q_full[begun % QS], begun // QS, f"factors of tile {t}")
                    q_empty[begun % QS].arrive()
                begun += 1
            elif r.random() < 0.5:   # the reference moves
                yield wait(o_done[m], t - 1, f"product before tile {t}")
            if tiles[t][2]:
                yield wait(kv_full[(2 * t + 1) % NS], (2 * t + 1) // NS, f"values of tile {t}")
            if t > 0:
                yield wait(o_done[m], t - 1, f"product before tile {t}")
            p_ready[u & 1].arrive()
            if tiles[t][1] or t == n - 1 or (tiles[t][2] and r.random() < 0.5):
                yield wait(o_done[m], t, f"product of tile {t}")
            tile_empty[t % TILES].arrive()

    running = {f"copy {w}": copy(w) for w in range(4)}
    running["issue"] = issue()
    running.update({f"softmax {w}": softmax(w) for w in range(warps)})
    waits = dict.fromkeys(running)
    while running:
        ready = [k for k in running if waits[k] is None or waits[k][0].test(waits[k][1])]
        for k in ready:
            if waits[k] is not None:   # not before its phase, and not after the next one with its parity
                assert waits[k][0].phase == waits[k][2] + 1, (k, waits[k][3])
        choice = ready + (["tensor core"] if queue else [])
        if not choice:
            return {k: waits[k][3] for k in running}
        k = r.choice(choice)
        if k == "tensor core":
            fills, bars = queue.pop(0)
            for f in fills:
                assert content[f % NS] == f, "a product reads another fill than its own"
                used.add(f)
            for b in bars:
                b.arrive()
            continue
        try:
            waits[k] = next(running[k])
        except StopIteration:
            del running[k]
    assert used == set(range(2 * n))
    return None


# NM, NS, QS, LAG, TILES, small, scaled as TreeMmaShape has them
SHAPES = {"16 bit, 64, 128 rows": (1, 8, 2, 6, 8), "16 bit, 64, 256 rows": (2, 8, 1, 6, 8), "16 bit, 128, 128 rows": (1, 5, 2, 3, 8),
          "16 bit, 128, 256 rows": (2, 5, 1, 3, 8), "16 bit, 192": (1, 7, 1, 5, 8), "16 bit, 256": (1, 5, 1, 3, 8),
          "8 bit, 64, 128 rows": (1, 8, 2, 7, 8, True, True), "8 bit, 64, 256 rows": (2, 8, 1, 7, 8, True, True),
          "8 bit, 128, 128 rows": (1, 3, 2, 3, 4, True, True), "8 bit, 128, 256 rows": (2, 3, 1, 3, 4, True, True),
          "8 bit, 192": (1, 5, 1, 3, 4, True, True), "8 bit, 256": (1, 3, 1, 3, 4, True, True), "8 bit, 256, fp16 queries": (1, 3, 1, 3, 8, True, False)}


@pytest.mark.parametrize("shape", SHAPES)
def test_every_run_ends_and_every_wait_is_for_its_own_phase(shape):
    NM, NS, QS, LAG, TILES, small, scaled = (SHAPES[shape] + (False, False))[:7]
    for seed in range(60):
        r = random.Random(seed)
        items = [(r.choice([1, 1, 2, 3, 5, 9]), r.random() < 0.7) for _ in range(r.randint(1, 8))]
        stuck = run(NM, NS, QS, LAG, TILES, items, seed, small, scaled)
        assert stuck is None, (items, stuck)
