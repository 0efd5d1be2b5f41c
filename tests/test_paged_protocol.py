"""CPU model of the synchronisation protocol of the paged decode kernel, and of how it shares its tiles out.

The model runs the roles of ``decode_paged_kernel`` (csrc/fa_decode_paged.cu) as coroutines: the TMA producer, the
page scales and queries, the S products, the PV products, the softmax groups (``turns`` of them take the tiles in
turn), the epilogue, the TMA engine and the tensor pipe of each issuing warp.  A random scheduler with random speeds
interleaves them.  Every wait is a parity wait on the barrier as the kernel writes it: it passes whenever the
barrier's phase has the other parity, so that a wait that could be passed by an older or missed by a newer phase shows.
The model checks for deadlock, for barriers that get more arrivals than their count, and that nothing is read before
it is written or rewritten before it is read: K, V, P and page factors of a stage, S buffers, queries, O accumulators,
statistics.  Planted mistakes must be caught.

The partition test restates in plain Python how a CTA finds its share of the tiles, and checks that every tile has
one CTA and that the CTAs of a cut unit agree on who takes part.
"""
import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_55_b200", "csrc",
                        "fa_decode_paged.cu")).read()


def counts(split, turns, rows):
    """{barrier: arrivals} from the kernel's mbar_init calls."""
    env = {"S::kSplit": split, "S::kGroups": split * turns, "R": rows}
    out = {}
    for name, expr in re.findall(r"mbar_init\(&b->(\w+)(?:\[\w+\])?, ([^;]+)\);", SRC):
        for k, v in env.items():
            expr = re.sub(r"(?<![\w:])" + re.escape(k) + r"\b", str(v), expr)
        assert re.fullmatch(r"[\d\s+*/()]+", expr), expr
        out[name] = eval(expr)  # noqa: S307 -- digits and operators only
    return out


class Violation(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arrived, self.phase = name, count, 0, 0

    def arrive(self, n=1):
        self.arrived += n
        if self.arrived > self.count:
            raise Violation(f"{self.name}: more arrivals than its count")
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def passes(self, parity):
        return (self.phase & 1) != (parity & 1)


class Model:
    def __init__(self, pieces, ns, split, turns, rng, plant=None):
        self.pieces, self.ns, self.split, self.turns, self.rng, self.plant = pieces, ns, split, turns, rng, plant
        self.bufs = 2 * turns
        K = counts(split, turns, 8 * split)
        ring = {"kv_full", "kv_empty", "p_full"}
        many = {"q_full", "q_empty", "s_full", "s_free"}
        for n in ring | many | {"o_full", "o_free", "stats_full"}:
            size = ns if n in ring else self.bufs if n in many else 2
            setattr(self, n, [Bar(f"{n}[{i}]", K[n] + (n == "kv_full")) for i in range(size)])
        self.tile = [(it, j) for it, n in enumerate(pieces) for j in range(n)]
        self.n = len(self.tile)
        self.stage_kv, self.stage_pg, self.stage_p = [None] * ns, [None] * ns, [0] * ns
        self.s_buf, self.q_buf, self.ref = [None] * self.bufs, [None] * self.bufs, [None] * self.bufs
        self.s_read, self.p_done, self.pv_done, self.s_done = [0] * self.n, [0] * self.n, -1, -1
        self.q_users = [set() for _ in pieces]
        self.o = [[None] * turns for _ in range(2)]
        self.stats = [None, None]
        self.epi_done = -1
        self.tma, self.pipe_s, self.pipe_pv, self.speeds = [], [], [], {}

    def need(self, ok, what):
        if not ok:
            raise Violation(what)

    # ------------------------------------------------------------------ roles
    def producer(self):
        for t in range(self.n):
            s = t % self.ns
            if t >= self.ns:
                yield [(self.kv_empty[s], t // self.ns + 1)]
                self.need(self.pv_done >= t - self.ns and self.s_done >= t - self.ns, f"stage {s} refilled while tile {t - self.ns} is read")
            self.kv_full[s].arrive()                # with the bytes to come, a third arrival below
            self.tma.append((s, t))

    def scales(self):
        for t, (it, j) in enumerate(self.tile):
            if j == 0:
                qb = it % self.bufs
                if it >= self.bufs and self.plant != "no q_empty":
                    yield [(self.q_empty[qb], it // self.bufs + 1)]
                old = self.q_buf[qb]
                if old is not None:
                    self.need(self.q_users[old] >= self.users(old), f"queries of piece {old} overwritten")
                self.q_buf[qb] = self.ref[qb] = it
                self.q_full[qb].arrive()
            s = t % self.ns
            if t >= self.ns:
                yield [(self.kv_empty[s], t // self.ns + 1)]
                self.need(self.pv_done >= t - self.ns, f"page factors of stage {s} rewritten early")
            self.stage_pg[s] = t
            self.kv_full[s].arrive()

    def users(self, it):
        """Who reads a piece's queries or their factors: S of its tiles, and the groups that have one of them."""
        return {("S", g) for g, (i, _) in enumerate(self.tile) if i == it} | {("X", g, p) for g, (i, _) in enumerate(self.tile)
                                                                               if i == it for p in range(self.split)}

    def s_warp(self):
        for g, (it, j) in enumerate(self.tile):
            s, sb, qb = g % self.ns, g % self.bufs, it % self.bufs
            if j == 0:
                yield [(self.q_full[qb], it // self.bufs)]
            w = [(self.kv_full[s], g // self.ns)]
            if g >= self.bufs and self.plant != "no s_free":
                w.append((self.s_free[sb], g // self.bufs + 1))
            yield w
            self.pipe_s.append(("S", g))
            self.pipe_s.append(("commit", self.s_full[sb]))
            if j == self.pieces[it] - 1:
                self.pipe_s.append(("commit", self.q_empty[qb]))

    def pv_warp(self):
        for g, (it, j) in enumerate(self.tile):
            s, ob = g % self.ns, it & 1
            if j == 0 and it >= 2 and self.plant != "no o_free":
                yield [(self.o_free[ob], (it >> 1) + 1)]
            yield [(self.p_full[s], g // self.ns)]
            self.pipe_pv.append(("PV", g))
            self.pipe_pv.append(("commit", self.kv_empty[s]))
            if j == self.pieces[it] - 1:
                self.pipe_pv.append(("commit", self.o_full[ob]))

    def softmax(self, part, turn):
        g0 = 0
        for it, n in enumerate(self.pieces):
            qb, ob, began = it % self.bufs, it & 1, False
            for g in range(g0, g0 + n):
                if g % self.turns != turn:
                    continue
                sb, s = g % self.bufs, g % self.ns
                yield [(self.kv_full[s], g // self.ns), (self.q_full[qb], it // self.bufs), (self.s_full[sb], g // self.bufs)]
                self.need(self.s_buf[sb] == g, f"S buffer {sb} read for tile {g}, holds {self.s_buf[sb]}")
                self.need(self.stage_pg[s] == g and self.stage_kv[s] == g, f"stage {s} read for tile {g}")
                self.need(self.q_buf[qb] == it, f"query factors of piece {it} read")
                self.q_users[it].add(("X", g, part))
                self.s_read[g] += 1
                self.s_free[sb].arrive(4)
                if began and self.rng.random() < 0.3:      # rescale
                    last = g - self.turns
                    if self.plant != "no rescale wait":
                        yield [(self.kv_empty[last % self.ns], last // self.ns)]
                    self.need(self.pv_done >= last, f"O rescaled before PV {last}")
                began = True
                self.need(self.pv_done >= g - self.ns, f"P of stage {s} rewritten before PV {g - self.ns}")
                self.p_done[g] += 1
                self.p_full[s].arrive(4)
            g0 += n
            if it >= 2:
                yield [(self.o_free[ob], (it >> 1) + 1)]
            self.need(self.epi_done >= it - 2, f"statistics of piece {it - 2} overwritten")
            if part == 0 and (began or self.plant == "ref without a tile"):
                self.need(self.ref[qb] == it, f"2^r of piece {it} read, is {self.ref[qb]}")
                self.stats[ob] = it
            self.q_empty[qb].arrive(4)
            self.stats_full[ob].arrive(4)

    def epilogue(self):
        for it, n in enumerate(self.pieces):
            ob = it & 1
            yield [(self.stats_full[ob], it >> 1)]
            self.need(self.stats[ob] == it, f"statistics of piece {it} read, are {self.stats[ob]}")
            yield [(self.o_full[ob], it >> 1)]
            first = sum(self.pieces[:it])
            for t in {g % self.turns for g in range(first, first + n)}:
                self.need(self.o[ob][t] == (it, max(g for g in range(first, first + n) if g % self.turns == t)), f"O of piece {it}")
            self.epi_done = it
            self.o_free[ob].arrive(4)

    # -------------------------------------------------------------- execution
    def run_pipe(self, pipe):
        op, x = pipe.pop(0)
        if op == "commit":
            x.arrive()
        elif op == "S":
            sb, s, it = x % self.bufs, x % self.ns, self.tile[x][0]
            self.need(x < self.bufs or self.s_read[x - self.bufs] == self.split, f"S {x} overwrote a buffer in use")
            self.need(self.stage_kv[s] == x and self.q_buf[it % self.bufs] == it, f"operands of S {x}")
            self.s_buf[sb], self.s_done = x, x
            self.q_users[it].add(("S", x))
        else:
            it, j = self.tile[x]
            s, ob, t = x % self.ns, it & 1, x % self.turns
            self.need(self.p_done[x] == self.split and self.stage_kv[s] == x, f"operands of PV {x}")
            if j < self.turns:
                self.need(self.epi_done >= it - 2, f"PV {x} overwrote O of piece {it - 2}")
            else:
                self.need(self.o[ob][t] == (it, x - self.turns), f"PV {x} accumulates into {self.o[ob][t]}")
            self.o[ob][t], self.pv_done = (it, x), x

    def run(self):
        roles = {"producer": self.producer(), "scales": self.scales(), "s": self.s_warp(), "pv": self.pv_warp(), "epi": self.epilogue()}
        for p in range(self.split):
            for t in range(self.turns):
                roles[f"soft{p}{t}"] = self.softmax(p, t)
        state = {n: next(g, None) for n, g in roles.items()}
        speed = lambda c: self.speeds.setdefault(c, 10.0 ** self.rng.uniform(-3, 0))  # noqa: E731
        for _ in range(200000):
            ready = [n for n, w in state.items() if w is not None and all(b.passes(p) for b, p in w)]
            choices = ready + (["tma"] if self.tma else []) + (["ps"] if self.pipe_s else []) + (["ppv"] if self.pipe_pv else [])
            if not choices:
                left = [n for n, w in state.items() if w is not None]
                if left:
                    raise Violation(f"deadlock: {left}")
                return
            c = self.rng.choices(choices, [speed(x) for x in choices])[0]
            if c == "tma":
                s, t = self.tma.pop(self.rng.randrange(len(self.tma)))
                self.stage_kv[s] = t
                self.kv_full[s].arrive()
            elif c == "ps":
                self.run_pipe(self.pipe_s)
            elif c == "ppv":
                self.run_pipe(self.pipe_pv)
            else:
                state[c] = next(roles[c], None)
        raise Violation("step limit")


CASES = [[1], [1] * 9, [3], [2, 5, 1, 4, 2], [7, 1, 1, 1, 6, 2], [13]]


@pytest.mark.parametrize("split,turns,ns", [(1, 2, 5), (2, 2, 5), (2, 2, 4), (4, 1, 4), (4, 1, 3)])
@pytest.mark.parametrize("pieces", CASES)
def test_protocol_holds_under_random_interleavings(pieces, split, turns, ns):
    for seed in range(30):
        Model(pieces, ns, split, turns, random.Random(seed)).run()


@pytest.mark.parametrize("plant", ["no o_free", "no s_free", "no q_empty", "no rescale wait", "ref without a tile"])
def test_planted_mistakes_are_caught(plant):
    caught = 0
    for seed in range(300):
        try:
            Model([1, 2, 1, 1, 4, 1, 1, 9, 1, 1], 5, 1, 2, random.Random(seed), plant).run()
        except Violation:
            caught += 1
    assert caught > 0


def test_configurations_are_the_kernels():
    """The (split, turns, ring depth) combinations above are those that the kernel's shapes have."""
    assert "kSplit = R / 8;" in SRC and "kTurns = R == 32 ? 1 : 2;" in SRC and "kBufs = 2 * kTurns;" in SRC
    assert "kNS = R == 8 ? 5 : R == 16 ? (D == 128 ? 5 : 4) : (D == 128 ? 4 : 3);" in SRC


# ------------------------------------------------------------------------------------------------- partition
PIECE = int(re.search(r"constexpr int kPieceCost = (\d+);", SRC).group(1))


def shares(nts, units, ctas=148):
    """Per CTA the first tile of its share, that of the next, and how far into a unit's line it begins."""
    total = sum(n + PIECE for n in nts if n) * units
    per = -(-total // ctas)

    def first(x):
        line = tiles = 0
        for n in nts:
            if n == 0:
                continue
            if x < line + (n + PIECE) * units:
                unit, rest = divmod(x - line, n + PIECE)
                return tiles + unit * n + max(rest - PIECE, 0), rest
            line, tiles = line + (n + PIECE) * units, tiles + n * units
        return tiles, 0

    return per, [(first(c * per)[0], first((c + 1) * per)[0], first(c * per)[1]) for c in range(ctas)] if total else []


def cdiv0(a, b):
    """C's division, towards zero."""
    return abs(a) // b if a >= 0 else -(abs(a) // b)


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_has_one_cta_and_cut_units_agree(seed):
    rng = random.Random(seed)
    B, units = rng.choice([1, 2, 5, 40, 300]), rng.choice([1, 2, 3, 8, 16])
    nts = [rng.choice([0, 1, 1, 2, 3, 7, 50, rng.randint(1, 400)]) for _ in range(B)]
    tiles = [((i, u), j, n) for i, n in enumerate(nts) for u in range(units) for j in range(n)]
    per, ranges = shares(nts, units)
    at, owner = 0, {}
    for c, (a, b, _) in enumerate(ranges):
        assert a == at and b >= a
        at = b
        owner.update({t: c for t in range(a, b)})
    assert at == len(tiles) == len(owner)
    first = {k: owner[t] for t, (k, j, n) in reversed(list(enumerate(tiles)))}
    last = {k: owner[t] for t, (k, j, n) in enumerate(tiles)}
    for c, (a, b, rest) in enumerate(ranges):
        unit_at, t = -rest, a
        while t < b:                       # the epilogue's walk over this CTA's pieces
            key, j0, nt = tiles[t]
            n = min(nt - j0, b - t)
            to = unit_at + PIECE
            if n != nt:
                assert c - (cdiv0(per - 1 - to, per) if j0 > 0 else 0) == first[key]
                assert c + cdiv0(to + nt - 1, per) == last[key]
                assert j0 > 0 or first[key] == c
            if j0 + n == nt:
                unit_at += nt + PIECE
            t += n
