"""CPU model of the barriers of the products' kernel (csrc/fsdp_gemm.cuh): its
protocol, not its arithmetic.

Two blocks: each has a producer that copies its half of a step into a stage of
the ring, the first has the warp that issues the tensor cores' work, and each has
takers of the sums. Copies land and the tensor cores' work ends some time after
it was issued, the latter in order. Every wait may run out; a role whose wait ran
out stops. Over random schedules the model checks that no work reads a stage
whose copies have not landed or is overwritten while it reads, that sums are
taken once they are whole and before the next are added, and that nothing is on
its way to or from a block's shared memory when all roles have ended, whichever
wait ran out. What a wait for one's own copies or work waits for does come."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = 0
        self.phases = 0

    def arrive(self, expect=0):
        self.pending -= 1
        self.land(-expect)

    def land(self, n):
        self.bytes -= n
        if self.pending == 0 and self.bytes == 0:
            self.phases += 1
            self.pending = self.count

    def test_wait(self, parity):
        return (self.phases & 1) != parity


class Pair:
    def __init__(self, stages, items, steps, seed, run_out, always_drain=True):
        self.rnd, self.run_out, self.always_drain = random.Random(seed), run_out, always_drain
        self.stages, self.items, self.steps = stages, items, steps
        self.full = [Barrier(1) for _ in range(stages)]
        self.empty = [[Barrier(1) for _ in range(stages)] for _ in range(2)]
        self.done = [[Barrier(1) for _ in range(2)] for _ in range(2)]
        self.taken = [Barrier(2) for _ in range(2)]
        self.drained = Barrier(1)
        self.copies, self.work = [], []
        self.held = [[None] * stages for _ in range(2)]  # the step whose rows a stage holds, once landed
        self.sums = [None, None]  # of a half: [item, steps added]
        self.out_of_time = 0

    def wait(self, barrier, parity):
        while not barrier.test_wait(parity):
            if self.rnd.random() < self.run_out:
                self.out_of_time += 1
                return False
            yield
        return True

    def wait_own(self, barrier, parity):
        """For what has been issued: it comes, or nothing is on its way any more."""
        while not barrier.test_wait(parity) and (self.copies or self.work):
            yield

    def producer(self, rank):
        n, ok = 0, True
        for item in range(self.items):
            for s in range(self.steps):
                stage, phase = n % self.stages, n // self.stages & 1
                ok = yield from self.wait(self.empty[rank][stage], phase ^ 1)
                if not ok:
                    break
                if rank == 0:
                    self.full[stage].arrive(expect=2)
                assert not any(k == "mma" and at == stage for k, at, *_ in self.work), "a stage is overwritten while it is read"
                self.held[rank][stage] = None
                self.copies.append((rank, stage, (item, s)))
                n += 1
                yield
            if not ok:
                break
        if ok and not self.always_drain:
            return
        # its copies arrive before it ends: seen on the first block's barriers, by the second that its stages were
        # read, or, where that does not come, in time
        last = range(n - 1, max(-1, n - 1 - self.stages), -1)
        if rank == 0:
            for j in last:
                yield from self.wait_own(self.full[j % self.stages], j // self.stages & 1)
            return
        for j in last:
            ok = ok and (yield from self.wait(self.empty[1][j % self.stages], j // self.stages & 1))
        while not ok and any(c[0] == rank for c in self.copies):
            yield

    def issuer(self):
        n, ok = 0, True
        for item in range(self.items):
            half = item & 1
            ok = yield from self.wait(self.taken[half], (item >> 1 & 1) ^ 1)
            if not ok:
                break
            for s in range(self.steps):
                stage = n % self.stages
                ok = yield from self.wait(self.full[stage], n // self.stages & 1)
                if not ok:
                    break
                self.work.append(("mma", stage, half, (item, s)))
                self.work.append(("commit", [self.empty[0][stage], self.empty[1][stage]]))
                n += 1
                yield
            if not ok:
                break
            self.work.append(("commit", [self.done[0][half], self.done[1][half]]))
        if not ok or self.always_drain:
            self.work.append(("commit", [self.drained]))
            yield from self.wait_own(self.drained, 0)

    def taker(self, rank):
        for item in range(self.items):
            half = item & 1
            if not (yield from self.wait(self.done[rank][half], item >> 1 & 1)):
                return
            assert self.sums[half] == [item, self.steps], "sums are taken that are not whole"
            yield
            assert self.sums[half] == [item, self.steps], "sums are overwritten while they are taken"
            self.taken[half].arrive()

    def land(self):
        rank, stage, step = self.copies.pop(self.rnd.randrange(len(self.copies)))
        self.held[rank][stage] = step
        self.full[stage].land(1)

    def finish_work(self):
        kind, *what = self.work.pop(0)
        if kind == "commit":
            for b in what[0]:
                b.arrive()
            return
        stage, half, (item, s) = what
        assert self.held[0][stage] == self.held[1][stage] == (item, s), "a stage is read that does not hold its step"
        if s == 0:
            self.sums[half] = [item, 0]
        assert self.sums[half] == [item, s]
        self.sums[half][1] += 1

    def run(self):
        roles = {"p0": self.producer(0), "p1": self.producer(1), "i": self.issuer(), "t0": self.taker(0), "t1": self.taker(1)}
        for _ in range(10 ** 6):
            if not roles:
                assert not self.copies and not self.work, f"on its way when the blocks end: {self.copies} {self.work}"
                return self.out_of_time
            hardware = (["land"] if self.copies else []) + (["work"] if self.work else [])
            a = self.rnd.choice(list(roles) + hardware)
            if a == "land":
                self.land()
            elif a == "work":
                self.finish_work()
            elif next(roles[a], StopIteration) is StopIteration:
                del roles[a]
        raise AssertionError("no progress")


@pytest.mark.parametrize("stages, items, steps", [(2, 1, 1), (2, 5, 3), (6, 1, 20), (6, 7, 4), (8, 3, 11), (8, 9, 1)])
def test_waits_that_hold(stages, items, steps):
    for seed in range(60):
        assert Pair(stages, items, steps, seed, 0.0).run() == 0


@pytest.mark.parametrize("stages, items, steps", [(2, 1, 1), (2, 5, 3), (6, 1, 20), (6, 7, 4), (8, 3, 11), (8, 9, 1)])
def test_nothing_is_on_its_way_at_the_end_whichever_wait_runs_out(stages, items, steps):
    ran_out = sum(Pair(stages, items, steps, seed, p).run() for seed in range(150) for p in (0.3, 0.03, 0.003))
    assert ran_out > 100


def test_work_is_left_over_where_only_a_role_that_gave_up_waits_for_its_own():
    # the sums' takers give up while the last steps are computed, and nobody else waits for those
    with pytest.raises(AssertionError, match="on its way"):
        for seed in range(400):
            Pair(6, 1, 20, seed, 0.01, always_drain=False).run()
