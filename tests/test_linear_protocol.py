"""Model check of the barrier protocols of the 8-bit projections on tensor
cores (csrc/linear_few.cu, csrc/linear_tc.cu), run on the CPU.

The roles are played out as coroutines under random interleavings; copies land
in any order, products complete in the order of their issue.

  copies     a ring of `stages`: iteration it arms full[it % stages] after
             empty[it % stages] has completed for its previous use
  few        two or four widening sets take the iterations in turn, each into a
             slot of its own: wait full, read, arrive on empty; wait freed[set],
             write the slot, arrive on ready[set].  Products of iteration it wait
             for ready[it % sets], read the slot and complete freed[it % sets].
  tc         both sets take a half of every iteration: chunk q = 2 it + half goes
             to slot q % slots; the products of a chunk complete freed[slot],
             those of the second half empty as well (they read the stage's
             rows); a pair's two CTAs both widen, and ready counts both.

A wait names a completion by its parity alone, so it is only sound while the
barrier is at most one completion away; the model fails where it is further,
where a stage is refilled before it was read, or a slot rewritten before its
products read it."""
import random

import pytest


class Unsound(AssertionError):
    pass


class Barriers:
    def __init__(self):
        self.done, self.arrived = {}, {}

    def arrive(self, b, count):
        n = self.arrived.get(b, 0) + 1
        self.arrived[b] = n % count
        if n == count:
            self.done[b] = self.done.get(b, 0) + 1

    def passes(self, b, k):
        """The wait for completion number k (-1: the phase before the first)."""
        c = self.done.get(b, 0)
        if not k <= c <= k + 1 and not (k == -1 and c == 0):
            raise Unsound(f"{b}: waits for completion {k} with {c} done")
        return c == k + 1


def play(kind, total, stages, slots, ctas, seed):
    R, B = random.Random(seed), Barriers()
    landed, read, widened, used = {}, set(), {}, set()   # stage's iteration, (cta, it, set) read, slot's chunk, chunks multiplied
    flying, queue = [], []
    halves, sets = (1, slots) if kind == "few" else (2, 2)

    def copies(c):
        for it in range(total):
            s = it % stages
            while not B.passes(("empty", c, s), it // stages - 1):
                yield
            readers = [it % slots] if kind == "few" else [0, 1]
            if it >= stages and not all((c, it - stages, x) in read for x in readers):
                raise Unsound("a stage is refilled before its codes were read")
            if kind == "tc" and it >= stages and not all(2 * (it - stages) + h in used for h in (0, 1)):
                raise Unsound("a stage is refilled before its rows were multiplied")
            flying.append((c, s, it))
            yield

    def widen(c, x):
        uses = {}
        for it in range(x if kind == "few" else 0, total, slots if kind == "few" else 1):
            s = it % stages
            while not B.passes(("full", c, s), it // stages):
                yield
            if landed.get((c, s)) != it:
                raise Unsound("codes of another iteration")
            read.add((c, it, x))
            if kind == "few":
                B.arrive(("empty", c, s), 1)
            yield
            q = it if kind == "few" else 2 * it + x
            t = x if kind == "few" else q % slots
            k = uses.get(t, 0)
            uses[t] = k + 1
            while not B.passes(("freed", c, t), k - 1):
                yield
            if (c, t) in widened and widened[c, t] not in used:
                raise Unsound("a slot is rewritten before its products")
            widened[c, t] = q
            yield
            B.arrive(("ready", t), ctas)

    def products():
        for q in range(total * halves):
            t = q % slots
            while not B.passes(("ready", t), q // slots):
                yield
            if any(widened.get((c, t)) != q for c in range(ctas)):
                raise Unsound("products of another chunk")
            queue.append((q, t))
            yield

    def world():
        while True:
            if flying and R.random() < 0.5:
                c, s, it = flying.pop(R.randrange(len(flying)))
                landed[c, s] = it
                B.arrive(("full", c, s), 1)
            if queue and R.random() < 0.5:
                q, t = queue.pop(0)
                used.add(q)
                for c in range(ctas):
                    B.arrive(("freed", c, t), 1)
                    if kind == "tc" and q % 2:
                        B.arrive(("empty", c, q // 2 % stages), 1)
            yield

    roles = [products()] + [copies(c) for c in range(ctas)] + [widen(c, x) for c in range(ctas) for x in range(sets)]
    w = world()
    for _ in range(200000):
        if not roles and not queue:
            assert len(used) == total * halves
            return
        next(w)
        if roles:
            i = R.randrange(len(roles))
            try:
                next(roles[i])
            except StopIteration:
                roles.pop(i)
    raise Unsound("no progress")


@pytest.mark.parametrize("stages,sets", [(2, 2), (4, 2), (6, 2), (4, 4), (8, 4)])
@pytest.mark.parametrize("total", [1, 2, 3, 7, 20])
def test_batch_kernel(stages, sets, total):
    for seed in range(60):
        play("few", total, stages, sets, 1, seed)


@pytest.mark.parametrize("stages,slots", [(4, 4), (5, 4), (7, 8), (12, 8), (1, 4)])
@pytest.mark.parametrize("total", [1, 2, 5, 20])
def test_tile_kernel(stages, slots, total):
    for seed in range(25):
        play("tc", total, stages, slots, 2, seed)


def test_an_odd_ring_is_unsound_for_sets_that_take_turns():
    """With three stages a set meets a stage whose earlier use was the other
    set's, and takes an early look at it for a completion of its own."""
    with pytest.raises(Unsound):
        for seed in range(2000):
            play("few", 12, 3, 2, 1, seed)


@pytest.mark.parametrize("split", range(1, 9))
def test_shares_of_a_clusters_tiles(split):
    """linear_few.cu: blocks of a cluster share the stages of T tiles.  Each stage
    is one block's; a block has at most four tiles (as many accumulators), and at
    most one that it shares in each of its two buffers."""
    R = random.Random(split)
    for _ in range(400):
        tiles, clusters, kb = R.randint(1, 700), R.randint(1, 152 // split), R.randint(1, 512)
        clusters = min(clusters, tiles)
        T = -(-tiles // clusters)
        touched = 1 if T == 1 else T if split == 1 else -(-T // split) + 1
        if touched > 4 or -(-T * kb // split) < 6:
            continue
        for c in {0, clusters // 2, clusters - 1}:
            t = tiles * (c + 1) // clusters - tiles * c // clusters
            lo = [t * kb * p // split for p in range(split + 1)]
            assert t >= 1 and lo[0] == 0 and lo[-1] == t * kb
            for a, b in zip(lo, lo[1:]):
                assert a < b
                mine = range(a // kb, (b - 1) // kb + 1)
                assert len(mine) <= 4
                shared = [i for i in mine if not (a <= i * kb and (i + 1) * kb <= b)]
                assert sum(a < i * kb for i in shared) <= 1 and sum(a >= i * kb for i in shared) <= 1
