"""What a block of k_tree_mma has under way when its waits run out, as a model on the CPU: the warps of tensor copies, the two that
issue products and the consumer of both, over a ring of slots, with a memory that may be late.  A warp that has done its part is not
the one whose wait runs out, so a block that lets only its stopped warps' copies and products land leaves with others under way, which
then come to memory that is no longer its own."""
import random

LIMIT, LAND = 60, 400   # rounds that a wait takes, and that a leaving block lets pass


def run(seed, rule):
    """Copies and products under way when the block has left, and whether it stopped.  rule: who waits before leaving, "own" (each
    warp that gave up, for what it has under way) or "block" (all, where one gave up)."""
    r = random.Random(seed)
    n, slots = r.randint(1, 8), r.choice([3, 5])
    late = r.random() < 0.7   # one copy comes only after the waits have run out
    landed, scored, weighted = set(), set(), set()
    under_way = []   # [owner, rounds left, what happens then]
    stop = False
    late_copy = (r.randrange(n), r.randrange(2))

    def start(owner, rounds, then):
        if not owner.startswith("copies"):   # a warp's products end in order
            rounds += max([x[1] for x in under_way if x[0] == owner], default=0)
        under_way.append([owner, rounds, then])

    def copies(values):
        for t in range(n):
            if t >= slots:
                yield (weighted if values else scored), t - slots
            rounds = LIMIT + r.randint(1, 100) if late and (t, values) == late_copy else r.randint(1, 9)
            start(f"copies {values}", rounds, lambda t=t: landed.add((t, values)))

    def scores():
        for t in range(n):
            yield landed, (t, 0)
            start("scores", r.randint(1, 5), lambda t=t: scored.add(t))

    def values():
        for t in range(n):
            yield landed, (t, 1)
            yield scored, t   # and its weights
            start("values", r.randint(1, 5), lambda t=t: weighted.add(t))

    def softmax():
        for t in range(n):
            yield scored, t
        yield weighted, n - 1

    warps = {"copies 0": copies(0), "copies 1": copies(1), "scores": scores(), "values": values(), "softmax": softmax()}
    waits = {k: None for k in warps}     # (set, element, rounds waited)
    leaving = {}                         # rounds that a warp still stays

    def step():
        for x in under_way:
            x[1] -= 1
        for x in [x for x in under_way if x[1] <= 0]:
            under_way.remove(x)
            x[2]()

    while warps or leaving:
        step()
        leaving = {k: v - 1 for k, v in leaving.items() if v > 1 and any(x[0] == k for x in under_way)}
        for k in list(warps):
            if waits[k] is not None:
                where, what, waited = waits[k]
                if what not in where:
                    if stop or waited >= LIMIT:
                        stop = True
                        del warps[k]
                        if rule == "own":
                            leaving[k] = LAND
                        continue
                    waits[k] = (where, what, waited + 1)
                    continue
            try:
                where, what = next(warps[k])
                waits[k] = (where, what, 0)
            except StopIteration:
                del warps[k]
    if rule == "block" and stop:
        for _ in range(LAND):
            step()
    return len(under_way), stop


def test_a_stopped_block_leaves_nothing_under_way():
    stops = 0
    for seed in range(2000):
        left, stop = run(seed, "block")
        assert left == 0, seed
        stops += stop
    assert 300 < stops < 2000   # both ends were seen


def test_warps_that_gave_up_are_not_the_only_ones_with_copies_under_way():
    """The rule that the kernel does not follow, which the model has to be able to tell apart."""
    assert any(run(seed, "own")[0] for seed in range(2000))
