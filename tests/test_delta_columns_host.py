"""The TMEM columns of the gated delta rule's chain kernels against the order of their accesses. No GPU needed.

The chain kernels' warps meet at barriers alone. Here every access to TMEM of one block over a few chunks is an event:
the product warp's products (they run in the order of their issue, after the waits before it), two warps of the chain
and two output warps (one per half of the tokens, of the same 32 state rows). Barriers order what came before their
arrivals before what follows their waits. Two accesses of common columns, one of them a write, must be ordered; products
among themselves are. The columns are read from the header that the kernels use.
"""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "mamba_ssd_selective_gb300", "csrc", "gated_delta_columns.h")
CHUNKS = 3


def columns(name):
    with open(HEADER) as f:
        body = re.search(r"namespace %s \{(.*?)\}" % name, f.read(), re.S).group(1)
    return {n: int(v) for n, v in re.findall(r"k(\w+) = (\d+)", body)}


class Order:
    """Events of a block's actors, the barriers between them, and the accesses that nothing orders."""

    def __init__(self):
        self.after, self.last, self.arrived, self.access = [], {}, {}, []

    def _event(self, *before):
        self.after.append(frozenset(b for b in before if b is not None))
        return len(self.after) - 1

    def _step(self, actor, *before):
        self.last[actor] = self._event(self.last.get(actor), *before)
        return self.last[actor]

    def wait(self, actor, bar):
        self._step(actor, *self.arrived[bar])

    def arrive(self, actor, bar):
        self.arrived.setdefault(bar, []).append(self._step(actor))

    def touch(self, actor, what, reads=(), writes=()):
        self._keep(self._step(actor), what, reads, writes, False)

    def product(self, what, reads, writes):
        """Issued now; done some time after the products before it."""
        self.last["pipe"] = self._event(self._step("mma"), self.last.get("pipe"))
        self._keep(self.last["pipe"], what, reads, writes, True)

    def commit(self, bar):
        self.arrived.setdefault(bar, []).append(self._event(self._step("mma"), self.last["pipe"]))

    def _keep(self, event, what, reads, writes, product):
        span = lambda cols: {c for a, n in cols for c in range(a, a + n)}  # noqa: E731
        self.access.append((event, what, span(reads), span(writes), product))

    def run(self, *actors):
        """Actors are generators that yield the barrier they wait for next and the arrivals it needs."""
        waits = {a: next(a) for a in actors}
        while waits:
            ready = [a for a, (bar, need) in waits.items() if len(self.arrived.get(bar, ())) >= need]
            assert ready, "every wait ends"
            for a in ready:
                waits[a] = next(a, None)
            waits = {a: w for a, w in waits.items() if w}

    def unordered(self):
        past = []
        for before in self.after:  # events only follow earlier ones
            past.append(set(before).union(*(past[b] for b in before)))
        bad = []
        for i, (e, what, r, w, p) in enumerate(self.access):
            for e2, what2, r2, w2, p2 in self.access[i + 1:]:
                if (w & (r2 | w2) or w2 & r) and not (p and p2) and e not in past[e2] and e2 not in past[e]:
                    bad.append((what, what2))
        return bad


def halves(base, half, k_last):
    """The operand columns of one half of a product's steps: steps half, half + 2, ... of eight columns each."""
    return [(base + 8 * k, 8) for k in range(half, k_last, 2)]


def state_operand(op, half):
    return [(op + 64 * (k >> 2) + 32 * pn + 8 * (k & 3), 8) for pn in range(2) for k in range(half, 8, 2)]


def put_state(op, st, c0):
    return [(op + c0 // 2, 8), (op + 64 + c0 // 2, 8), (st + c0, 16)]


def forward(c, heads):
    o = Order()

    def mma():
        for i in range(CHUNKS):
            if i:
                yield ("O_READ", i - 1), 2
                o.wait("mma", ("O_READ", i - 1))
            for h in range(2):
                yield ("S_FULL", h, i), 2
                o.wait("mma", ("S_FULL", h, i))
                o.product(f"[Q S0 | K S0] {i}", state_operand(c["Op"], h), [(c["QS"], 128)])
            o.commit(("A_DONE", i))
            for h in range(2):
                yield ("R_FULL", h, i), 2
                o.wait("mma", ("R_FULL", h, i))
                o.product(f"[w | M w] {i}", [x for f in range(heads) for x in halves(c["Op"] + 64 * f, h, 8)], [(c["W"], 128)])
            o.commit(("B_DONE", i))
            for h in range(2):
                yield ("U_FULL", h, i), 2
                o.wait("mma", ("U_FULL", h, i))
                o.product(f"S {i}", halves(c["Op"], h, 8), [(c["S"], 128)])
            o.commit(("C_DONE", i))

    def chain(ch):
        me = f"chain {ch}"
        for k in range(4):
            o.touch(me, "first state", (), put_state(c["Op"], c["S"], 64 * ch + 16 * k))
        for h in range(2):
            o.arrive(me, ("S_FULL", h, 0))
        for i in range(CHUNKS):
            yield ("A_DONE", i), 1
            o.wait(me, ("A_DONE", i))
            for h in range(2):
                o.touch(me, f"reads K S0 {i}.{h}", [(c["KS"] + 32 * ch + 16 * h, 16)])
                for f in range(heads):
                    o.touch(me, f"R {i}.{h}", (), [(c["Op"] + 64 * f + 16 * ch + 8 * h + lo, 8) for lo in (0, 32)])
                o.arrive(me, ("R_FULL", h, i))
            yield ("B_DONE", i), 1
            o.wait(me, ("B_DONE", i))
            for h in range(2):
                o.touch(me, f"reads w {i}.{h}", [(c["W"] + 32 * ch + 16 * h, 16)])
                o.touch(me, f"update {i}.{h}", (), [(c["Op"] + 16 * ch + 8 * h + lo, 8) for lo in (0, 32)])
                o.arrive(me, ("U_FULL", h, i))
            yield ("C_DONE", i), 1
            o.wait(me, ("C_DONE", i))
            for h in range(2):
                for c0 in (64 * ch + 16 * h, 64 * ch + 16 * h + 32):
                    o.touch(me, f"reads S {i}.{h}", [(c["S"] + c0, 16)])
                    o.touch(me, f"state {i + 1}.{h}", (), put_state(c["Op"], c["S"], c0))
                o.arrive(me, ("S_FULL", h, i + 1))

    def out(ch):
        me = f"out {ch}"
        for i in range(CHUNKS):
            yield ("B_DONE", i), 1
            o.wait(me, ("B_DONE", i))
            o.touch(me, f"reads w, Q S0, M w {i}", [(c[n] + 32 * ch, 32) for n in ("W", "QS", "MW")])
            o.arrive(me, ("O_READ", i))

    o.run(mma(), chain(0), chain(1), out(0), out(1))
    return o


def reverse(c, heads):
    o = Order()

    def mma():
        for i in range(CHUNKS):
            yield ("OP_FULL", i), 2
            o.wait("mma", ("OP_FULL", i))
            if i:
                yield ("D_READ", i - 1), 2
                o.wait("mma", ("D_READ", i - 1))
            o.product(f"dY (M T) {i}", [(c["Y"], 32 * heads)], [(c["D"], 64)])
            for h in range(2):
                yield ("E_FULL", h, i), 2
                o.wait("mma", ("E_FULL", h, i))
                o.product(f"X {i}", state_operand(c["Op"], h), [(c["X"], 64)])
            o.commit(("A_DONE", i))
            o.product(f"dY Q {i}", [(c["Ye"], 64)], [(c["E"], 128)])
            o.commit(("OP_EMPTY", i))
            for h in range(2):
                yield ("Z_FULL", h, i), 2
                o.wait("mma", ("Z_FULL", h, i))
                o.product(f"z T {i}", [x for f in range(heads) for x in halves(c["Op"] + 64 * f, h, 8)], [(c["D"], 64)])
            o.commit(("B_DONE", i))
            for h in range(2):
                yield ("R_FULL", h, i), 2
                o.wait("mma", ("R_FULL", h, i))
                o.product(f"dR K {i}", halves(c["Op"], h, 8), [(c["E"], 128)])
            o.commit(("C_DONE", i))

    def chain(ch):
        me = f"chain {ch}"
        for k in range(4):
            o.touch(me, "first E", (), put_state(c["Op"], c["E"], 64 * ch + 16 * k))
        for h in range(2):
            o.arrive(me, ("E_FULL", h, 0))
        for i in range(CHUNKS):
            yield ("A_DONE", i), 1
            o.wait(me, ("A_DONE", i))
            for h in range(2):
                o.touch(me, f"reads X {i}.{h}", [(c["X"] + 32 * ch + 16 * h, 16)])
                for f in range(heads):
                    o.touch(me, f"z {i}.{h}", (), [(c["Op"] + 64 * f + 16 * ch + 8 * h + lo, 8) for lo in (0, 32)])
                o.arrive(me, ("Z_FULL", h, i))
            yield ("B_DONE", i), 1
            o.wait(me, ("B_DONE", i))
            for h in range(2):
                o.touch(me, f"reads dR {i}.{h}", [(c["D"] + 32 * ch + 16 * h, 16)])
                o.touch(me, f"dR {i}.{h}", (), [(c["Op"] + 16 * ch + 8 * h + lo, 8) for lo in (0, 32)])
                o.arrive(me, ("R_FULL", h, i))
            yield ("C_DONE", i), 1
            o.wait(me, ("C_DONE", i))
            for h in range(2):
                for c0 in (64 * ch + 16 * h, 64 * ch + 16 * h + 32):
                    o.touch(me, f"reads E {i}.{h}", [(c["E"] + c0, 16)])
                    o.touch(me, f"E {i + 1}.{h}", (), put_state(c["Op"], c["E"], c0))
                o.arrive(me, ("E_FULL", h, i + 1))

    def out(ch):
        me = f"out {ch}"

        def put_dy(i):
            o.touch(me, f"dY {i}", (), [(c["Y"] + 16 * ch, 16)] + [(c["Ye"] + 16 * ch + lo, 16) for lo in (0, 32)])
            o.arrive(me, ("OP_FULL", i))

        if heads == 2:
            o.touch(me, "zeros", (), [(c["Y"] + 32 + 16 * ch, 16)])
        put_dy(0)
        for i in range(CHUNKS):
            if i + 1 < CHUNKS:
                yield ("OP_EMPTY", i), 1
                o.wait(me, ("OP_EMPTY", i))
                put_dy(i + 1)
            yield ("B_DONE", i), 1
            o.wait(me, ("B_DONE", i))
            o.touch(me, f"reads D {i}", [(c["D"] + 32 * ch, 32)])
            o.arrive(me, ("D_READ", i))

    o.run(mma(), chain(0), chain(1), out(0), out(1))
    return o


@pytest.mark.parametrize("heads", [1, 2])
def test_forward_chain_accesses_are_ordered(heads):
    assert forward(columns("col"), heads).unordered() == []


@pytest.mark.parametrize("heads", [1, 2])
def test_reverse_chain_accesses_are_ordered(heads):
    assert reverse(columns("rev_col"), heads).unordered() == []


def test_a_product_over_columns_still_read_is_seen():
    """w in the columns of K S0^T: its product's first half may overtake the reads of the second half."""
    bad = forward({**columns("col"), "W": 64, "MW": 128}, 1).unordered()
    assert ("reads K S0 0.1", "[w | M w] 0") in bad or ("[w | M w] 0", "reads K S0 0.1") in bad


@pytest.mark.parametrize("name,sizes", [("col", dict(QS=64, KS=64, W=64, MW=64, S=128, Op=128)),
                                        ("rev_col", dict(X=64, D=64, E=128, Op=128, Y=64, Ye=64))])
def test_columns_lie_within_a_block_and_apart(name, sizes):
    c = columns(name)
    assert set(c) == set(sizes)
    used = sorted((c[n], c[n] + sizes[n]) for n in c)
    assert used[0][0] >= 0 and used[-1][1] <= 512
    assert all(a[1] <= b[0] for a, b in zip(used, used[1:]))
