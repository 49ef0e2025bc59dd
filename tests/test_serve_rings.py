"""The rings of barriers in the kernels that read a cache, walked on the CPU.

A wait on an mbarrier names its phase by one bit.  It is right only if the phase before has ended for sure, and loads
land in any order.  Here the roles of each kernel (who waits on which stage for which round, who arrives, what a
product reads) run as coroutines on a small machine that holds one load back until nothing else can go on, for every
load in turn, or picks the next step at random.  Every wait says which round it means; one that passes in another
round, a product that reads a stage whose tile has not landed, or a load into a stage that is still read, is a fault.
"""

import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_long_pooled_b200", "csrc")


def _constants(name, *patterns):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    found = []
    for p in patterns:
        m = re.findall(p, text)
        assert len(m) == 1, (name, p, m)
        found.append(m[0])
    return found


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.phase = name, count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count


class Machine:
    def __init__(self, hold=None, seed=None):
        self.hold, self.rng = hold, None if seed is None else random.Random(seed)
        self.flying, self.loads = [], 0          # (number, what happens when it lands)
        self.queues = {}                         # issuer -> products in flight, retired in order
        self.roles, self.syncs = [], {}
        self.cells, self.readers = {}, {}        # what a buffer holds, products that still read it

    def bars(self, name, n, count):
        return [Barrier(f"{name}[{i}]", count) for i in range(n)]

    def put(self, cell, what):
        if self.readers.get(cell):
            raise Fault(f"{cell} is overwritten with {what} while it is read")
        self.cells[cell] = what

    def read(self, cell, what):
        if self.cells.get(cell) != what:
            raise Fault(f"{cell} holds {self.cells.get(cell)}, not {what}")

    def load(self, cell, what, bar):
        self.put(cell, None)

        def land():
            self.put(cell, what)
            bar.arrive()
        self.flying.append((self.loads, land))
        self.loads += 1

    def product(self, issuer, reads, writes, arrivals):
        """Reads and writes [(cell, content)]; its arrivals come when it, and all before it, are done."""
        for cell, what in reads:
            self.read(cell, what)
            self.readers[cell] = self.readers.get(cell, 0) + 1
        for cell, _ in writes:
            self.put(cell, None)

        def done():
            for cell, _ in reads:
                self.readers[cell] -= 1
            for cell, what in writes:
                self.put(cell, what)
            for b in arrivals:
                b.arrive()
        self.queues.setdefault(issuer, []).append(done)

    def _ready(self, role):
        op = role[1]
        if op is None:
            return True
        if op[0] == "wait":
            return (op[1].phase & 1) != (op[2] & 1)
        return self.syncs[op[1]][0] != op[3]

    def _step(self, role):
        op = role[1]
        if op is not None and op[0] == "wait" and op[1].phase != op[2] + 1:
            raise Fault(f"{op[1].name}: a wait for round {op[2]} passed in round {op[1].phase}")
        try:
            op = next(role[0])
        except StopIteration:
            self.roles.remove(role)
            return
        if op[0] == "sync":                      # (name, members): a barrier of whole warps
            s = self.syncs.setdefault(op[1], [0, 0])
            op = (op[0], op[1], op[2], s[0])
            s[1] += 1
            if s[1] == op[2]:
                s[0], s[1] = s[0] + 1, 0
        role[1] = op

    def _land(self, i):
        self.flying.pop(i)[1]()

    def run(self, roles):
        self.roles = [[r, None] for r in roles]
        while self.roles or self.flying or any(self.queues.values()):
            free = [i for i, (n, _) in enumerate(self.flying) if n != self.hold]
            if self.rng is None:                 # everything goes as far as it can, but for the load held back
                moved = False
                for role in list(self.roles):
                    while role in self.roles and self._ready(role):
                        self._step(role)
                        moved = True
                for q in self.queues.values():
                    while q:
                        q.pop(0)()
                        moved = True
                if free:
                    self._land(free[0])
                    moved = True
                if moved:
                    continue
                if not self.flying:
                    raise Fault("nothing can go on: " + ", ".join(str(r[1][1:3]) for r in self.roles))
                self._land(0)
                continue
            ways = [("r", r) for r in self.roles if self._ready(r)]
            ways += [("q", q) for q in self.queues.values() if q] + [("f", i) for i in range(len(self.flying))]
            if not ways:
                raise Fault("nothing can go on")
            kind, x = self.rng.choice(ways)
            if kind == "r":
                self._step(x)
            elif kind == "q":
                x.pop(0)()
            else:
                self._land(x)


# ------------------------------------------------------------------ tree_wide.cu

def wide(m, K, V, copies, e4, valid, pieces, warps=4):
    """pieces: (M tiles 1 or 2, key tiles) in the CTA's order."""
    k_full, k_empty = m.bars("k_full", K, 1), m.bars("k_empty", K, 2)
    v_full, v_empty = m.bars("v_full", V, 1), m.bars("v_empty", V, 1 if e4 else 2)
    v_ready, v_used = m.bars("v_ready", max(V, copies), 1), m.bars("v_used", copies, 2)
    q_ready, s_full = m.bars("q_ready", 2, 4), m.bars("s_full", 4, 1)
    p_full, pv_done = m.bars("p_full", 4, 4), m.bars("pv_done", 4, 1)
    mask_k, mask_v = {}, {}
    total = sum(n for _, n in pieces)

    def producer(ring, stages, full, empty, masks, slots):
        for it in range(total):
            st = it % stages
            if it >= stages:
                yield "wait", empty[st], it // stages - 1
            masks[it % slots] = it
            m.load((ring, st), it, full[st])

    def issuer(s):
        base = cs = nq = 0
        for i, (w, n) in enumerate(pieces):
            pair = w == 2
            ns = n if pair else (n + 1 - s) // 2
            if ns > 0:
                yield "wait", q_ready[s], nq
                nq += 1
            for j in range(ns + 1 if ns > 0 else 0):
                if j < ns:
                    it, c = base + (j if pair else 2 * j + s), cs + j
                    st, b = it % K, c & 1
                    yield "wait", k_full[st], it // K
                    if j > 1:
                        yield "wait", pv_done[2 * s + b], (c >> 1) - 1
                    q = [(("q", s if pair else 0, x), i) for x in range(4)]
                    m.product(s, [(("k", st), it)] + q, [(("s", s, b), ("scores", c))],
                              [s_full[2 * s + b], k_empty[st]] + ([] if pair else [k_empty[st]]))
                if j > 0:
                    it, c = base + (j - 1 if pair else 2 * (j - 1) + s), cs + j - 1
                    st, b = it % V, c & 1
                    vs = it % copies if e4 else st
                    yield "wait", v_ready[vs], it // copies if e4 else it // V
                    yield "wait", p_full[2 * s + b], c >> 1
                    used = v_used[vs] if e4 else v_empty[st]
                    m.product(s, [(("copy" if e4 else "v", vs), it), (("s", s, b), ("weights", c))], [],
                              [used] + ([] if pair else [used]) + [pv_done[2 * s + b]])
            cs += ns
            base += n

    def v_warp(w):
        for it in range(w, total, warps):
            st = it % V
            yield "wait", v_full[st], it // V
            m.read(("v", st), it)
            if mask_v[st] != it:
                raise Fault(f"the mask of stage {st} is tile {mask_v[st]}'s, not {it}'s")
            if e4:
                if it >= copies:
                    yield "wait", v_used[it % copies], it // copies - 1
                m.read(("v", st), it)
                m.put(("copy", it % copies), it)
                v_empty[st].arrive()
                v_ready[it % copies].arrive()
            else:
                v_ready[st].arrive()

    def softmax(s, warp):
        base = cs = 0
        for i, (w, n) in enumerate(pieces):
            pair = w == 2
            if pair or s == 0:
                m.put(("q", s if pair else 0, warp), i)
            if not pair:
                yield "sync", "streams", 8
            if n > (0 if pair else s):
                q_ready[s].arrive()
            done = 0
            for x in range(0 if pair else s, n, 1 if pair else 2):
                b = cs & 1
                yield "wait", s_full[2 * s + b], cs >> 1
                if mask_k[(base + x) % valid] != base + x:
                    raise Fault(f"the mask of K tile {base + x} is gone")
                if done and (cs + warp) % 3 == 0:        # (a warp whose maximum grew)
                    yield "wait", pv_done[2 * s + (b ^ 1)], (cs - 1) >> 1
                m.read(("s", s, b), ("scores", cs) if warp == 0 else m.cells[("s", s, b)])
                m.cells.setdefault(("n", s, cs), set()).add(warp)
                if len(m.cells[("n", s, cs)]) == 4:      # the last of the four warps lays down its weights
                    m.cells[("s", s, b)] = ("weights", cs)
                p_full[2 * s + b].arrive()
                cs, done = cs + 1, done + 1
            if done:
                yield "wait", pv_done[2 * s + ((cs - 1) & 1)], (cs - 1) >> 1
            base += n
            if not pair:
                for _ in range(3):                       # the sums, then the columns, of the second stream
                    yield "sync", "streams", 8

    m.run([producer("k", K, k_full, k_empty, mask_k, valid), producer("v", V, v_full, v_empty, mask_v, V), issuer(0), issuer(1)]
          + [v_warp(w) for w in range(warps)] + [softmax(s, w) for s in (0, 1) for w in range(4)])


# ------------------------------------------------------------------ decode.cu

def few(m, S, tiles):
    full, empty = m.bars("full", S, 2), m.bars("empty", S, 4)
    mask = {}

    def producer():
        for it in range(tiles):
            st = it % S
            if it >= S:
                yield "wait", empty[st], it // S - 1
            mask[st] = it
            m.load(("k", st), it, full[st])
            m.load(("v", st), it, full[st])

    def consumer():
        for it in range(tiles):
            st = it % S
            yield "wait", full[st], it // S
            m.read(("k", st), it)
            m.read(("v", st), it)
            if mask[st] != it:
                raise Fault(f"the mask of stage {st} is tile {mask[st]}'s")
            empty[st].arrive()

    m.run([producer()] + [consumer() for _ in range(4)])


# ------------------------------------------------------------------ key_mass.cu

def mass(m, S, valid, pieces):
    """pieces: (passes, first key tile, key tiles)."""
    k_full, k_empty = m.bars("k_full", S, 1), m.bars("k_empty", S, 1)
    q_full, l_full, q_empty = m.bars("q_full", 2, 1), m.bars("l_full", 2, 2), m.bars("q_empty", 2, 9)
    s_full, s_free = m.bars("s_full", 4, 1), m.bars("s_free", 4, 4)
    masks = {}
    order = [(i, p, t) for i, (passes, t0, n) in enumerate(pieces) for p in range(passes) for t in range(t0, t0 + n)]
    turns = [(i, p) for i, (passes, _, n) in enumerate(pieces) for p in range(passes) if n]

    def producer():
        for it in range(len(order)):
            st = it % S
            if it >= S:
                yield "wait", k_empty[st], it // S - 1
            masks[it % valid] = it
            m.load(("k", st), it, k_full[st])

    def issuer():
        it, uses = 0, [0, 0]
        for nq, (i, _) in enumerate(turns):
            qb = nq & 1
            yield "wait", q_full[qb], nq >> 1
            _, t0, n = pieces[i]
            for t in range(t0, t0 + n):
                st, use = it % S, uses[t & 1]
                uses[t & 1] += 1
                b = 2 * (t & 1) + (use & 1)
                yield "wait", k_full[st], it // S
                if use >= 2:
                    yield "wait", s_free[b], (use >> 1) - 1
                m.product(0, [(("k", st), it), (("q", qb), nq)], [(("s", b), it)], [s_full[b], k_empty[st]])
                it += 1
            m.product(0, [], [], [q_empty[qb]])

    def loader(warp):
        for nq in range(len(turns)):
            qb = nq & 1
            if nq >= 2:
                yield "wait", q_empty[qb], (nq >> 1) - 1
            if warp == 0:
                m.load(("q", qb), nq, q_full[qb])
            m.put(("lse", qb, warp), nq)
            l_full[qb].arrive()

    def weights(half):
        it = use = 0
        for nq, (i, _) in enumerate(turns):
            qb = nq & 1
            yield "wait", l_full[qb], nq >> 1
            m.read(("lse", qb, 0), nq)
            m.read(("lse", qb, 1), nq)
            _, t0, n = pieces[i]
            for t in range(t0 + ((t0 ^ half) & 1), t0 + n, 2):
                b = 2 * half + (use & 1)
                yield "wait", s_full[b], use >> 1
                m.read(("s", b), it + t - t0)
                if masks[(it + t - t0) % valid] != it + t - t0:
                    raise Fault(f"the mask of K tile {it + t - t0} is gone")
                m.read(("lse", qb, 0), nq)
                s_free[b].arrive()
                use += 1
            it += n
            q_empty[qb].arrive()

    m.run([producer(), issuer(), loader(0), loader(1)] + [weights(h) for h in (0, 1) for _ in range(4)])


# ------------------------------------------------------------------ the tests

def _walk(model, *args):
    """The model with each of its loads held back in turn, then in random orders."""
    first = Machine()
    model(first, *args)
    for hold in range(first.loads):
        model(Machine(hold=hold), *args)
    for seed in range(8):
        model(Machine(seed=seed), *args)


WIDE_PIECES = [
    [(1, 29)],                                            # parity over three rounds of the longest ring
    [(2, 27)],                                            # pair
    [(1, 3), (1, 5), (2, 4), (1, 1), (1, 8), (2, 1), (2, 0), (1, 7)],
    [(2, 5), (1, 1), (2, 3), (1, 2), (1, 11), (2, 7)],
]


def _wide_rings():
    ks, vs, copies, warps, valid = _constants(
        "tree_wide.cu", r"int K_STAGES = E4 \|\| D == 64 \? (\d+) : (\d+);", r"int V_STAGES = E4 \|\| D == 64 \? (\d+) : (\d+);",
        r"int COPIES = (\d+);", r"int V_WARPS = (\d+);", r"constexpr int VALID = (\d+);")
    assert int(warps) == 4
    return {"e4m3": (int(ks[0]), int(vs[0]), int(copies), True, int(valid)),
            "bf16 64": (int(ks[0]), int(vs[0]), int(copies), False, int(valid)),
            "bf16 128": (int(ks[1]), int(vs[1]), int(copies), False, int(valid))}


@pytest.mark.parametrize("instance", ["e4m3", "bf16 64", "bf16 128"])
@pytest.mark.parametrize("pieces", range(len(WIDE_PIECES)))
def test_wide_tree_rings(instance, pieces):
    _walk(wide, *_wide_rings()[instance], WIDE_PIECES[pieces])


@pytest.mark.parametrize("e4", [False, True])
@pytest.mark.parametrize("v_stages", [5, 6, 7])
def test_a_v_ring_that_is_no_multiple_of_its_warps_fails(e4, v_stages):
    with pytest.raises(Fault, match="v_full|v_ready|mask of stage|'v'"):
        _walk(wide, 6, v_stages, 4, e4, 16, WIDE_PIECES[0])


def test_an_odd_k_ring_fails_in_parity():
    with pytest.raises(Fault, match="k_full|'k'"):
        _walk(wide, 5, 8, 4, True, 16, WIDE_PIECES[0])


@pytest.mark.parametrize("stages", range(2, 9))
def test_decode_rings(stages):
    _walk(few, stages, 27)


def test_key_mass_rings():
    (long, short), valid = _constants("key_mass.cu", r"int STAGES = E4 \|\| D == 64 \? (\d+) : (\d+);",
                                      r"constexpr int VALID = (\d+);")
    for stages in (int(long), int(short)):
        for pieces in ([(1, 0, 27)], [(3, 5, 9)], [(2, 0, 1), (1, 3, 4), (4, 1, 3), (1, 0, 1), (2, 8, 7), (1, 0, 0), (1, 2, 2)]):
            _walk(mass, stages, int(valid), pieces)


def test_a_short_ring_of_masks_fails():
    with pytest.raises(Fault, match="mask of K tile"):
        _walk(mass, 8, 8, [(1, 0, 27)])
    with pytest.raises(Fault, match="mask of K tile"):
        _walk(wide, 6, 8, 4, True, 6, WIDE_PIECES[0])
