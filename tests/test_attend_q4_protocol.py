"""The barrier protocol of the tensor-core form of the attention over the 4-bit cache (attend_q4_tc.cu), checked by
randomized interleavings on the CPU.

Roles, as in the kernel: one thread walks the CTA's pieces and passes them on to the 19 other warps through two places; two
lanes of one warp bring the K codes and the V codes of each step (two blocks) into one buffer each; two warpgroups unpack
alternate steps -- K a step ahead of V -- into two operand stages each and write the step's key scales into a ring of four, and
load the two halves of Q at a piece's start; one thread for each half issues S = Q K^T of the next step behind O += P V of this
one; a warpgroup for each half turns S into P in place, rescales O, and takes turns with the other half.  A half without rows in a
piece releases the stages without using them; a piece without keys takes part in nothing.

The model asserts that every parity wait lands on its intended phase, that every read finds the piece, step, scales and codes
it expects and that these stay until it is over, that O accumulates in order and is at rest when it is rescaled and read, that
the turns alternate, and that nothing deadlocks; six planted protocol mistakes must each be caught.  It models the protocol, not
the arithmetic; the GPU tests cover the arithmetic.
"""
import random

import pytest

from tests._protocol import Bar, run_actors, wait_for, wait_released

STAGES, SCS, TOLD = 2, 4, 19


class TqSim:
    """``pieces``: (steps, whether the second half has rows) of each."""

    def __init__(self, pieces, rng, mistake=None):
        self.pieces, self.rng, self.mistake = pieces, rng, mistake
        self.scs = 2 if mistake == "two_scale_places" else SCS
        names = {f"wfull{i}": 1 for i in range(2)} | {f"wempty{i}": TOLD for i in range(2)} | {"qfull": 256}
        for c in "kv":
            names |= {f"c{c}full{ug}": 1 for ug in range(2)} | {f"c{c}empty": 128}
            names |= {f"{c}full{s}": 128 for s in range(STAGES)} | {f"{c}empty{s}": 2 for s in range(STAGES)}
        names |= {f"scfull{i}": 128 for i in range(SCS)}
        for h in range(2):
            names |= {f"sfull{h}": 1, f"pfull{h}": 128, f"done{h}": 1, f"turn{h}": 128}
        self.B = {n: Bar(n, c) for n, c in names.items()}
        self.place = [None, None]                    # pieces passed on
        self.lanes = [0, 0]                          # pieces that the copying lanes have finished
        self.codes = {"k": None, "v": None}          # step whose codes have arrived
        self.stage = {c: [[None] * 4 for _ in range(STAGES)] for c in "kv"}    # by the unpacking warps' quarters
        self.scales = [[None] * 4 for _ in range(SCS)]
        self.q = [[None] * 4 for _ in range(2)]      # piece whose Q a half holds
        self.s = [[None] * 4 for _ in range(2)]      # per half and lane quadrant: ("S" | "P", step)
        self.o = [None, None]                        # (piece, step) of the last product added
        self.pipe, self.issued, self.completed = [[], []], [0, 0], [0, 0]
        self.commits, self.loads = [], []
        self.passes = []                             # (half, step) in the order of the turns

    # -- the tensor pipe: each issuing thread's products in order, its commits behind them
    def commit(self, w, bar):
        self.commits.append((w, self.issued[w], bar))

    def flush_commits(self):
        due = [c for c in self.commits if c[1] <= self.completed[c[0]]]
        self.commits = [c for c in self.commits if c[1] > self.completed[c[0]]]
        for c in due:
            self.B[c[2]].arrive()

    def issue(self, w, *what):
        self.pipe[w].append(what)
        self.issued[w] += 1

    def pipe_step(self, probe=False):
        busy = [w for w in range(2) if self.pipe[w]]
        if probe or not busy:
            return bool(busy)
        w = self.rng.choice(busy)
        kind, k, n, first = self.pipe[w].pop(0)
        held = self.stage["k" if kind == "qk" else "v"][n % STAGES]
        assert held == [n] * 4, f"{kind}({n}) of half {w} read a stage holding {held}"
        if kind == "qk":
            assert self.q[w] == [k] * 4, f"step {n}: Q of piece {self.q[w]}, not {k}"
            for was in self.s[w]:
                assert was is None or (was[0] == "P" and self.o[w] is not None and self.o[w][1] >= was[1]), \
                    f"S({n}) of half {w} overwrote {was} before its use"
            self.s[w] = [("S", n)] * 4
        else:
            assert self.s[w] == [("P", n)] * 4, f"PV({n}) of half {w} read {self.s[w]}"
            assert first or self.o[w] == (k, n - 1), f"PV({n}) of half {w} after {self.o[w]}"
            self.o[w] = (k, n)
        self.completed[w] += 1
        return True

    def load_step(self, probe=False):
        if probe or not self.loads:
            return bool(self.loads)
        c, n, bar = self.loads.pop(self.rng.randrange(len(self.loads)))
        self.codes[c] = n
        self.B[bar].arrive()
        return True

    # -- actors
    def told(self, k):
        yield from wait_for(self.B[f"wfull{k & 1}"], k >> 1)
        got = self.place[k & 1]
        assert got == k, f"piece {got} in the place of piece {k}"
        self.B[f"wempty{k & 1}"].arrive()

    def walker(self):
        for k in range(len(self.pieces) + 1):        # the last says that there are no more
            yield from wait_released(self.B[f"wempty{k & 1}"], k >> 1)
            self.place[k & 1] = k
            self.B[f"wfull{k & 1}"].arrive()

    def copier(self, lane):
        """Lanes 0 and 1 of a warp: they hear of a piece together, and bring its steps each at its own pace."""
        c, n = "kv"[lane], 0
        for k, (steps, _) in enumerate(self.pieces):
            if lane == 0:
                yield from self.told(k)
                self.lanes[0] = k + 1                # lane 1 goes on with lane 0
            else:
                yield lambda k=k: self.lanes[0] > k
            for _ in range(steps):
                yield from wait_released(self.B[f"c{c}empty"], n)
                bar = f"c{c}full{0 if self.mistake == 'one_codes_barrier' else n & 1}"
                self.loads.append((c, n, bar))
                n += 1
            if lane == 1:
                self.lanes[1] = k + 1
            else:
                yield lambda k=k: self.lanes[1] > k
        if lane == 0:
            yield from self.told(len(self.pieces))
        if n > 0 and self.mistake != "one_codes_barrier":   # no copies in flight at the end
            yield from wait_for(self.B[f"c{c}full{(n - 1) & 1}"], (n - 1) >> 1)

    def issuer(self, w):
        n0 = piece = used = done = 0

        def qk(k, n):
            yield from wait_for(self.B[f"kfull{n % STAGES}"], n // STAGES)
            self.issue(w, "qk", k, n, False)
            self.commit(w, f"sfull{w}")
            self.commit(w, f"kempty{n % STAGES}")

        for k, (steps, both) in enumerate(self.pieces):
            yield from self.told(k)
            if steps == 0:
                continue
            n1, part = n0 + steps, w == 0 or both
            yield from wait_for(self.B["qfull"], piece)
            if part:
                yield from qk(k, n0)
                for n in range(n0, n1):
                    if self.mistake == "next_s_before_pv" and n + 1 < n1:
                        yield from qk(k, n + 1)
                    yield from wait_for(self.B[f"pfull{w}"], used + n - n0)
                    yield from wait_for(self.B[f"vfull{n % STAGES}"], n // STAGES)
                    self.issue(w, "pv", k, n, n == n0)
                    self.commit(w, f"vempty{n % STAGES}")
                    if self.mistake != "next_s_before_pv" and n + 1 < n1:
                        yield from qk(k, n + 1)
                self.commit(w, f"done{w}")
                yield from wait_for(self.B[f"done{w}"], done)
                used, done = used + steps, done + 1
            else:
                for n in range(n0, n1):
                    for c in "kv":
                        yield from wait_for(self.B[f"{c}full{n % STAGES}"], n // STAGES)
                        if self.mistake != "absent_half_keeps_stages":
                            self.B[f"{c}empty{n % STAGES}"].arrive()
            n0, piece = n1, piece + 1
        yield from self.told(len(self.pieces))

    def unpacker(self, ug, uw):
        def codes(c, n):
            assert self.codes[c] == n, f"{c} codes of step {self.codes[c]}, not {n}"

        def unpack_k(n):
            full = (self.B["ckfull0"], n) if self.mistake == "one_codes_barrier" else (self.B[f"ckfull{ug}"], n >> 1)
            yield from wait_for(*full)
            if self.mistake == "codes_released_before_read":
                self.B["ckempty"].arrive(32)
                yield lambda: True
            codes("k", n)
            yield lambda: True                       # read into registers
            codes("k", n)
            if self.mistake != "codes_released_before_read":
                self.B["ckempty"].arrive(32)
            yield from wait_released(self.B[f"kempty{n % STAGES}"], n // STAGES)
            self.scales[n % self.scs][uw] = n
            self.B[f"scfull{n % SCS}"].arrive(32)
            yield lambda: True
            self.stage["k"][n % STAGES][uw] = n
            self.B[f"kfull{n % STAGES}"].arrive(32)

        n, done = 0, [0, 0]
        for k, (steps, both) in enumerate(self.pieces):
            yield from self.told(k)
            if steps == 0:
                continue
            for h in range(2):
                if done[h] > 0 and self.mistake != "q_before_products_end":
                    yield from wait_for(self.B[f"done{h}"], done[h] - 1)
            done[0] += 1
            done[1] += both
            self.q[ug][uw] = k
            self.B["qfull"].arrive(32)
            n1, first = n + steps, n + ((n ^ ug) & 1)
            if first < n1:
                yield from unpack_k(first)
            for m in range(first, n1, 2):
                if m + 2 < n1:
                    yield from unpack_k(m + 2)
                full = (self.B["cvfull0"], m) if self.mistake == "one_codes_barrier" else (self.B[f"cvfull{ug}"], m >> 1)
                yield from wait_for(*full)
                codes("v", m)
                yield from wait_released(self.B[f"vempty{m % STAGES}"], m // STAGES)
                codes("v", m)
                self.B["cvempty"].arrive(32)
                yield lambda: True
                self.stage["v"][m % STAGES][uw] = m
                self.B[f"vfull{m % STAGES}"].arrive(32)
            n = n1
        yield from self.told(len(self.pieces))

    def softmax(self, half, wq):
        n0 = used = done = turn = 0
        for k, (steps, both) in enumerate(self.pieces):
            yield from self.told(k)
            if steps == 0:
                continue
            n1, part = n0 + steps, half == 0 or both
            for n in range(n0, n1) if part else ():
                yield from wait_for(self.B[f"sfull{half}"], used)
                yield from wait_for(self.B[f"scfull{n % SCS}"], n // SCS)
                assert self.s[half][wq] == ("S", n), f"step {n}: half {half} holds {self.s[half][wq]}"
                if both and (half == 1 or turn > 0):
                    yield from wait_for(self.B[f"turn{half ^ 1}"], turn if half == 1 else turn - 1)
                if both and wq == 0:
                    self.passes.append((half, n))
                for _ in range(2):                   # (a pass may be repeated)
                    assert self.scales[n % self.scs] == [n] * 4, f"step {n}: scales of {self.scales[n % self.scs]}"
                    yield lambda: True
                if both:
                    self.B[f"turn{half}"].arrive(32)
                    turn += 1
                yield lambda: True
                assert self.scales[n % self.scs] == [n] * 4, f"step {n}: scales of {self.scales[n % self.scs]} at the pass's end"
                assert self.s[half][wq] == ("S", n)
                self.s[half][wq] = ("P", n)
                if n > n0:
                    assert self.o[half] == (k, n - 1), f"step {n}: O rescaled after {self.o[half]}"
                    yield lambda: True
                    assert self.o[half] == (k, n - 1)
                self.B[f"pfull{half}"].arrive(32)
                used += 1
            if part:
                yield from wait_for(self.B[f"done{half}"], done)
                for _ in range(2):
                    assert self.o[half] == (k, n1 - 1), f"piece {k}: O of {self.o[half]} read"
                    yield lambda: True
                done += 1
            n0 = n1
        yield from self.told(len(self.pieces))

    def run(self):
        actors = [self.walker(), self.copier(0), self.copier(1), self.issuer(0), self.issuer(1)]
        actors += [self.unpacker(ug, uw) for ug in range(2) for uw in range(4)]
        actors += [self.softmax(h, wq) for h in range(2) for wq in range(4)]
        run_actors(actors, [self.pipe_step, self.load_step], self.rng, before_step=self.flush_commits)
        assert not any(self.pipe) and not self.loads and not self.commits
        want = []
        n = 0
        for steps, both in self.pieces:
            want += [(h, m) for m in range(n, n + steps) for h in range(2)] if both else []
            n += steps
        assert self.passes == want, "the halves' passes do not take turns"


def _pieces(rng):
    # long pieces, single steps, pieces without keys, halves that come and go
    return [(rng.choice((0, 1, 1, 2, 3, rng.randrange(1, 12))), rng.random() < 0.6) for _ in range(rng.randrange(1, 7))]


@pytest.mark.parametrize("seed", range(150))
def test_protocol_holds_under_random_schedules(seed):
    rng = random.Random(seed)
    TqSim(_pieces(rng), rng).run()


@pytest.mark.parametrize("pieces", [
    [(9, True), (1, False), (1, False), (1, False), (9, True)],       # a half skips odd and even numbers of steps
    [(0, True), (5, False), (0, False), (6, True), (0, True)],
    [(1, True)] * 8, [(2, False)] * 3 + [(3, True)] * 3, [(0, False)] * 5, [(30, True)], [(7, False), (8, True), (5, False), (11, True)],
])
def test_protocol_holds_for_chosen_pieces(pieces):
    for seed in range(12):
        TqSim(pieces, random.Random(seed)).run()


@pytest.mark.parametrize("mistake", ["two_scale_places", "q_before_products_end", "codes_released_before_read",
                                     "absent_half_keeps_stages", "next_s_before_pv", "one_codes_barrier"])
def test_planted_mistakes_are_caught(mistake):
    for seed in range(200):
        rng = random.Random(seed)
        try:
            TqSim([(6, True), (4, False), (7, True)], rng, mistake).run()
        except AssertionError:
            return
    pytest.fail(f"{mistake} was not caught")
