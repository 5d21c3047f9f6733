"""The barriers between the warps of gla_delta_fused (csrc/gla_delta_fused.cu) in a model on the CPU: every role's sequence
of waits, arrivals and gate slots, run in random orders in which some roles lag far behind. A wait is by parity, as in the
kernel: it passes while the barrier's current phase has the other parity, so a barrier that gets two phases ahead of a
waiting warp holds it up. The model counts a stall (no role can go on), a gate slot read with another chunk's gates, and a
slot overwritten before its readers are done.

Waits have a limit. The second part of the model holds a copy or the products up until every wait has run out: then the
roles leave their loops, no copy is issued any more, and the CTA does not end before what was issued has arrived.

Sizes as in the kernel: 3 stages of K and Q, 2 of V, 4 gate slots; 8 chain, 4 drain and 8 prep warps."""
import random

import pytest

NKQ, NV, NG = 3, 2, 4


class Stall(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, parity):
        return self.phase & 1 != parity


class Sim:
    """Roles are generators of operations; each step lets one of those that can go on do its next."""

    def __init__(self, n, out, rng, rule="slot", hold=None):
        self.n, self.out, self.rng, self.rule = n, out, rng, rule
        # what does not arrive any more from some step on ("loads" or "tensor"); whether the limit is over; the flag
        self.hold, self.late, self.flag = hold, False, False
        b = self.bars = {}
        for name, k, count in (("kq_full", NKQ, 1), ("kq_empty", NKQ, 1), ("v_full", NV, 1), ("v_empty", NV, 1),
                               ("s_ready", 2, 8), ("r_ready", 2, 8), ("u_ready", 2, 8), ("p_ready", 1, 8),
                               ("g_read", 1, 8 if out else 4), ("t_ready", 2, 8), ("ks_full", 1, 1), ("u_full", 1, 1),
                               ("d_full", 2, 1), ("o_full", 1, 1), ("g_full", 1, 1), ("fin", 1, 1), ("o_empty", 1, 4),
                               ("gt_ready", NG, 1), ("l_ready", 1, 4), ("d_free", 1, 1), ("gt_free", NG, 4 if out else 8)):
            for i in range(k):
                b[name, i] = Bar(count)
        self.slot, self.readers = [None] * NG, [0] * NG
        self.tensor, self.loads = [], []
        self.roles = {"tma": self.tma(), "gates": self.gates(), "products": self.products()}
        for w in range(8):
            self.roles["chain%d" % w] = self.chain()
            self.roles["prep%d" % w] = self.prep(w)
        for w in range(4):
            self.roles["drain%d" % w] = self.drain() if out else self.scores()

    # ------------------------------------------------------------ what a role may do
    def can(self, op, next_op):
        if op[0] in ("wait", "drain"):
            return self.bars[op[1], op[2]].passed(op[3]) or (op[0] == "wait" and self.late)
        if op[0] == "sync":
            return sum(o is not None and o[:3] == op[:3] for o in next_op.values()) == op[2]
        return True

    def do(self, op):
        if op[0] in ("wait", "drain"):
            ok = self.bars[op[1], op[2]].passed(op[3])
            self.flag |= not ok
            return ok
        if op[0] == "arrive":
            self.bars[op[1], op[2]].arrive()
        elif op[0] == "commit":            # arrives once every product before it is done
            self.tensor.append(op[1:])
        elif op[0] == "load":
            self.loads.append(op[1:])
        elif self.late:
            pass                           # (gates are of any chunk by then)
        elif op[0] == "write":
            assert self.readers[op[1]] == 0, "gates of chunk %s overwritten before they are read" % self.slot[op[1]]
            # chain, prep, drain (or the four warps of the scores)
            self.slot[op[1]], self.readers[op[1]] = op[2], 8 + 8 + 4
        elif op[0] == "read":
            assert self.slot[op[1]] == op[2], "gates of chunk %s read for chunk %d" % (self.slot[op[1]], op[2])
            self.readers[op[1]] -= len(op) > 3                  # (the role's last look at them)

    def run(self, most=200000):
        rng = self.rng
        weight = {r: rng.choice([1, 1, 1, 0.02]) for r in self.roles}
        weight["gates"] = rng.choice([1, 0.01, 0.001])
        next_op = {r: next(g, None) for r, g in self.roles.items()}
        held, hold_at = None, rng.randrange(3000) if self.hold else None
        for step in range(most):
            if step == hold_at:
                held = self.hold
            at = [r for r, op in next_op.items() if op is not None and self.can(op, next_op)]
            queues = [q for q in ("tensor", "loads") if q != held and getattr(self, q)]
            if not at and not queues:
                if all(op is None for op in next_op.values()):
                    assert not self.tensor and not self.loads, "the CTA ends with something in flight"
                    return
                if held and not self.late:
                    self.late = True       # every role waits: the limit passes
                    continue
                if held:
                    held = None            # what was held up arrives after all
                    continue
                raise Stall({r: op for r, op in next_op.items() if op is not None})
            pick = rng.choices(at + queues, [weight[r] for r in at] + [rng.choice([1, 0.1]) for _ in queues])[0]
            if pick == "tensor":
                self.bars[self.tensor.pop(0)].arrive()      # in order
            elif pick == "loads":
                self.bars[self.loads.pop(rng.randrange(len(self.loads)))].arrive()
            else:
                op = next_op[pick]
                if op[0] == "sync":
                    # all of the group are at the barrier: they go on together, with the same word
                    group = [r for r, o in next_op.items() if o is not None and o[:3] == op[:3]]
                    word = any(len(next_op[r]) > 3 and next_op[r][3] for r in group)
                    for r in group:
                        next_op[r] = self.step(r, word)
                    continue
                next_op[pick] = self.step(pick, self.do(op))
        raise Stall("no end")

    def step(self, role, answer):
        try:
            return self.roles[role].send(answer)
        except StopIteration:
            return None

    def chunks(self, look=True):
        """A role's loop over the chunks; it leaves at its look at the flag."""
        for m in range(self.n):
            if look and self.flag:
                return
            yield m

    # ------------------------------------------------------------ the roles
    def tma(self):
        kq = v = 0
        ok = True
        for m in self.chunks():
            if m >= NKQ:
                ok &= yield "wait", "kq_empty", m % NKQ, (m // NKQ - 1) & 1
            if ok:
                yield "load", "kq_full", m % NKQ
                kq += 1
            if m >= NV:
                ok &= yield "wait", "v_empty", m % NV, (m // NV - 1) & 1
            if ok:
                yield "load", "v_full", m % NV
                v += 1
        for m in range(max(0, kq - NKQ), kq):
            yield "drain", "kq_full", m % NKQ, (m // NKQ) & 1
        for m in range(max(0, v - NV), v):
            yield "drain", "v_full", m % NV, (m // NV) & 1

    def gates(self):
        for m in self.chunks(look=False):
            ok = True
            if self.rule == "slot":
                if m >= NG:
                    ok = yield "wait", "gt_free", m % NG, (m // NG - 1) & 1
            elif m >= NG - 1:              # by the parity of the increment of three chunks before
                ok = yield "wait", "d_full", 1, (m - NG + 1) & 1
            if not ok:
                return
            yield "write", m % NG, m
            yield "arrive", "gt_ready", m % NG

    def products(self):
        n, out = self.n, self.out

        def commit(*bars):
            for x in bars:
                yield "commit", *x

        def gram(m):
            yield "wait", "kq_full", m % NKQ, (m // NKQ) & 1
            yield from commit(("g_full", 0))

        yield from gram(0)
        if not out and n > 1:
            yield "wait", "g_read", 0, 0
            yield from gram(1)
        for m in self.chunks():
            ph = m & 1
            for part in range(2):
                yield "wait", "s_ready", part, ph
                if out and part == 0 and m == 0:
                    yield "wait", "g_read", 0, 0
            yield from commit(("ks_full", 0))
            if out and m + 1 < n:
                yield from gram(m + 1)
            yield "wait", "t_ready", m & 1, (m >> 1) & 1
            yield "wait", "v_full", m % NV, (m // NV) & 1
            yield from commit(("v_empty", m % NV))
            for part in range(2):
                yield "wait", "r_ready", part, ph
            yield from commit(("u_full", 0))
            if out and m > 0:
                yield "wait", "o_empty", 0, (m - 1) & 1
            if out and m + 1 < n:
                yield "wait", "g_read", 0, (m + 1) & 1
            for part in range(2):
                yield "wait", "u_ready", part, ph
            yield from commit(("d_full", 0), ("d_full", 1))
            if not out:
                yield from commit(("kq_empty", m % NKQ))
                if m + 2 < n:
                    yield "wait", "g_read", 0, (m + 1) & 1
                    yield from gram(m + 2)
            else:
                yield "wait", "p_ready", 0, ph
                yield from commit(("o_full", 0), ("kq_empty", m % NKQ))
        yield "commit", "fin", 0
        yield "drain", "fin", 0, 0

    def chain(self):
        for p in range(2):
            yield "arrive", "s_ready", p
        for m in self.chunks():
            ph = m & 1
            yield "wait", "t_ready", m & 1, (m >> 1) & 1
            yield "read", m % NG, m
            yield "wait", "ks_full", 0, ph
            yield "read", m % NG, m
            for p in range(2):
                yield "arrive", "r_ready", p
            yield "wait", "u_full", 0, ph
            yield "read", m % NG, m, "last"
            for p in range(2):
                yield "arrive", "u_ready", p
            if not self.out:
                yield "arrive", "gt_free", m % NG
            if self.out:
                yield "arrive", "p_ready", 0
            for p in range(2):
                yield "wait", "d_full", p, ph
                if m + 1 < self.n:
                    yield "arrive", "s_ready", p

    def drain(self):
        for m in self.chunks(look=False):
            yield "wait", "o_full", 0, m & 1
            if (yield "sync", "drain", 4, self.flag):
                return
            yield "read", m % NG, m, "last"
            yield "arrive", "o_empty", 0
            yield "arrive", "gt_free", m % NG
            yield "sync", "drained", 4

    def scores(self):
        for m in self.chunks():
            yield "wait", "gt_ready", m % NG, (m // NG) & 1
            yield "wait", "g_full", 0, m & 1
            if m > 0:
                yield "wait", "d_free", 0, (m - 1) & 1
            yield "read", m % NG, m, "last"
            yield "arrive", "g_read", 0
            yield "arrive", "l_ready", 0

    def prep(self, w):
        for m in self.chunks(look=False):
            if self.out:
                yield "wait", "gt_ready", m % NG, (m // NG) & 1
                yield "wait", "g_full", 0, m & 1
                yield "read", m % NG, m
                yield "arrive", "g_read", 0
                yield "sync", "prep", 8
            else:
                yield "wait", "l_ready", 0, m & 1
            yield "read", m % NG, m, "last"
            if (yield "sync", "inverse", 8, self.flag):
                return
            if not self.out and w == 0:
                yield "arrive", "d_free", 0
            for k in range(3):
                yield "sync", "inverse%d" % k, 8
            yield "arrive", "t_ready", m & 1


@pytest.mark.parametrize("out", [True, False])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 13])
def test_no_order_stalls(n, out):
    for seed in range(15):
        Sim(n, out, random.Random(1000 * n + seed)).run()


def test_a_wait_on_a_barrier_that_gets_ahead_stalls():
    """The rule that the slots' own barriers replaced: found to stall by the same runs."""
    stalled = 0
    for seed in range(100):
        try:
            Sim(13, True, random.Random(seed), rule="increment").run()
        except Stall:
            stalled += 1
    assert stalled > 0


@pytest.mark.parametrize("out", [True, False])
@pytest.mark.parametrize("hold", ["loads", "tensor"])
def test_giving_up_leaves_nothing_in_flight(hold, out):
    gave_up = 0
    for seed in range(40):
        sim = Sim(13, out, random.Random(seed), hold=hold)
        sim.run()
        gave_up += sim.late
    assert gave_up > 13


def test_a_drain_under_the_passed_limit_ends_too_early():
    """What the drains' own limits replaced: waits that the passed deadline ends at once."""
    class Former(Sim):
        def can(self, op, next_op):
            return super().can(("wait", *op[1:]) if op[0] == "drain" else op, next_op)

    early = 0
    for seed in range(30):
        try:
            Former(13, True, random.Random(seed), hold="loads").run()
        except AssertionError as e:
            early += "in flight" in str(e)
    assert early > 0
