"""A model of the many-row kernel's synchronisation (csrc/attn_fwd_rows_kernel.cuh), run on the CPU.

As the column-split kernel's model (test_colsplit_protocol_model.py), with what is new in this kernel: a scheduler that
hands the units to the other roles through a ring of four, roles that walk it with two cursors (the first one up to two
blocks ahead, the second one giving units back), results that go to a slot instead of through the store warp, and the
E4M3 form's raw ring and converters.  Agents run in random interleavings under the mbarrier parity rule; every read is
checked to find what it expects, and planted mistakes must fail."""
import random

import pytest

from test_colsplit_protocol_model import Barrier, Deadlock

QUEUE = 4


def run_cta(units, rng, f8=False, prefix=False, stages=4, raw_stages=5, queue=QUEUE, mistake=None):
    """units: (blocks, to_slot) in order."""
    seq = [(u, w, j) for u, w in enumerate(units) for j in range(w[0])]
    bars = {}
    bufs = 1 if f8 else 2   # Q buffers
    n_take = 2 + 1 + 1 + (0 if prefix else 1) + (2 if f8 else 0)   # (each warpgroup as one)
    for i in range(queue):
        bars[f"u_full{i}"], bars[f"u_empty{i}"] = Barrier(f"u_full{i}", 1), Barrier(f"u_empty{i}", n_take)
    for i in range(2):
        for name in (f"q_full{i}", f"q_empty{i}", f"s_full{i}", f"p_full{i}0", f"p_full{i}1"):
            bars[name] = Barrier(name, 1)
        bars[f"o_staged{i}"] = Barrier(f"o_staged{i}", 2)
    for i in range(stages):
        bars[f"kv_full{i}"], bars[f"kv_empty{i}"] = Barrier(f"kv_full{i}", 1), Barrier(f"kv_empty{i}", 1)
    for i in range(raw_stages):
        bars[f"raw_full{i}"], bars[f"raw_empty{i}"] = Barrier(f"raw_full{i}", 1), Barrier(f"raw_empty{i}", 1)
    for name, count in (("pv_done", 1), ("o_full", 1), ("o_free", 2), ("drain", 1)):
        bars[name] = Barrier(name, count)
    ring = [None] * queue
    state = {"stage": [None] * stages, "busy": [0] * stages, "raw": [None] * raw_stages, "q": [None, None],
             "q_busy": [0, 0], "staged": [None, None], "s": [None, None], "p": [[None, None], [None, None]],
             "o": None, "o_read": set(), "pv": -1, "results": []}
    tensor_q, tma_q = [], []

    def W(name, parity, k):
        assert (k >= 0 and parity == (k & 1)) or (k == -1 and parity == 1), (name, parity, k)
        yield ("wait", name, k)

    def scheduler():
        for o, w in enumerate(list(units) + [None]):
            q = o % queue
            if o >= queue:
                yield from W(f"u_empty{q}", (o // queue - 1) & 1, o // queue - 1)
            ring[q] = (o, w)
            bars[f"u_full{q}"].arrive()

    class Cursor:
        """Units of the ring in order; `give`: the one left behind is given back."""

        def __init__(self, give):
            self.give, self.ord, self.valid, self.j = give, 0, False, 0

        def next(self):
            if self.valid and self.give:
                bars[f"u_empty{(self.ord - 1) % queue}"].arrive()
            q = self.ord % queue
            yield from W(f"u_full{q}", (self.ord // queue) & 1, self.ord // queue)
            assert ring[q][0] == self.ord, "a unit was overwritten before its last reader"
            self.w, self.valid, self.u = ring[q][1], ring[q][1] is not None, self.ord
            self.j = 0
            self.ord += 1

        def advance(self):
            self.j += 1
            if self.j >= self.w[0]:
                yield from self.next()

    first_gives = mistake == "first cursor gives back"

    class Ring:
        def __init__(self, n):
            self.n, self.stage, self.phase, self.uses = n, 0, 0, [0] * n

        def step(self):
            self.uses[self.stage] += 1
            self.stage += 1
            if self.stage == self.n:
                self.stage, self.phase = 0, self.phase ^ 1

    def ordered(sc, pc, first, second):
        """K(0), K(1), then V(g), K(g+2): the loop of the producer and of the converters."""
        yield from sc.next()
        yield from pc.next()
        i = 0
        while sc.valid or pc.valid:
            if i >= 2:
                if not pc.valid:
                    break
                yield from second(pc)
                yield from pc.advance()
            if sc.valid:
                yield from first(sc)
                yield from sc.advance()
            i += 1

    def producer():
        r = Ring(raw_stages if f8 else stages)
        kind_full, kind_empty = ("raw_full", "raw_empty") if f8 else ("kv_full", "kv_empty")
        q_par, q_uses = [1, 1], [0, 0]

        def load(kind, c):
            st = r.stage
            yield from W(f"{kind_empty}{st}", r.phase ^ 1, r.uses[st] - 1)
            assert f8 or state["busy"][st] == 0, "ring stage reloaded while an MMA still reads it"
            tma_q.append(("raw" if f8 else "kv", st, (kind, c.u, c.j)))
            r.step()

        def load_k(c):
            if c.j == 0:
                qb = c.u % bufs
                yield from W(f"q_empty{qb}", q_par[qb], q_uses[qb] - 1)
                q_par[qb] ^= 1
                q_uses[qb] += 1
                assert state["q_busy"][qb] == 0 and state["staged"][qb] is None, "Q buffer reloaded while in use"
                tma_q.append(("q", qb, c.u))
            yield from load("K", c)

        yield from ordered(Cursor(first_gives), Cursor(True), load_k, lambda c: load("V", c))

    def converter(group):
        """Warpgroup `group` of the converters: the tiles of its parity."""
        r, raw = Ring(stages), Ring(raw_stages)
        n = [0]

        def convert(kind, c):
            mine = n[0] & 1 == group
            n[0] += 1
            if mine:
                st, kv = raw.stage, r.stage
                yield from W(f"raw_full{st}", raw.phase, raw.uses[st])
                if mistake != "converters do not wait":
                    yield from W(f"kv_empty{kv}", r.phase ^ 1, r.uses[kv] - 1)
                tile = state["raw"][st]
                assert tile == (kind, c.u, c.j), f"converters expect {(kind, c.u, c.j)}, the raw stage holds {tile}"
                assert state["busy"][kv] == 0, "converted over a tile still being read"
                yield ("step",)
                assert state["raw"][st] == tile, "raw stage refilled while being read"
                state["stage"][kv] = tile
                bars[f"raw_empty{st}"].arrive()
                bars[f"kv_full{kv}"].arrive()
            raw.step()
            r.step()

        yield from ordered(Cursor(first_gives), Cursor(True), lambda c: convert("K", c), lambda c: convert("V", c))

    def mma():
        r = Ring(stages)
        q_par, q_uses, of_par, n_units, i = [0, 0], [0, 0], 1, 0, 0
        sc, pc = Cursor(first_gives), Cursor(True)
        yield from sc.next()
        yield from pc.next()
        while sc.valid or pc.valid:
            if i >= 2:
                g = i - 2
                b, ph = g & 1, (g >> 1) & 1
                if not pc.valid:
                    break
                st = r.stage
                yield from W(f"kv_full{st}", r.phase, r.uses[st])
                r.step()
                assert state["stage"][st] == ("V", pc.u, pc.j), f"PV({g}) reads {state['stage'][st]}"
                state["busy"][st] += 1
                if pc.j == 0:
                    yield from W("o_free", of_par, n_units - 1)
                    of_par ^= 1
                    n_units += 1
                for h in range(2):
                    yield from W(f"p_full{b}{h}", ph, g >> 1)
                    assert state["p"][b][h] == g
                    tensor_q.append(("PV", g, h, st, pc.u, pc.j, pc.w[0]))
                tensor_q.append(("commit", "pv_done"))
                tensor_q.append(("commit", f"kv_empty{st}"))
                if pc.j == pc.w[0] - 1:
                    tensor_q.append(("commit", "o_full"))
                yield from pc.advance()
            if sc.valid:
                qb = sc.u % bufs
                if sc.j == 0:
                    yield from W(f"q_full{qb}", q_par[qb], q_uses[qb])
                    q_par[qb] ^= 1
                    q_uses[qb] += 1
                st = r.stage
                yield from W(f"kv_full{st}", r.phase, r.uses[st])
                r.step()
                assert state["stage"][st] == ("K", sc.u, sc.j) and state["q"][qb] == sc.u
                state["busy"][st] += 1
                state["q_busy"][qb] += 1
                tensor_q.append(("S", i, st, qb))
                tensor_q.append(("commit", f"s_full{i & 1}"))
                tensor_q.append(("commit", f"kv_empty{st}"))
                if sc.j == sc.w[0] - 1 and (sc.w[1] or mistake == "Q given back twice"):
                    tensor_q.append(("commit", f"q_empty{qb}"))
                yield from sc.advance()
            i += 1
        tensor_q.append(("commit", "drain"))
        yield from W("drain", 0, 0)

    def softmax(h):
        g, o_par, u, order = 0, 0, 0, 0
        while True:
            q = order % queue
            yield from W(f"u_full{q}", (order // queue) & 1, order // queue)
            assert ring[q][0] == order
            w = ring[q][1]
            if w is None:
                yield ("agree", "end")
                return
            bars[f"u_empty{q}"].arrive()
            order += 1
            for j in range(w[0]):
                b = g & 1
                yield from W(f"s_full{b}", (g >> 1) & 1, g >> 1)
                assert state["s"][b] == g
                if j > 0 and rng.random() < 0.5:
                    yield from W("pv_done", (g - 1) & 1, g - 1)
                    assert state["pv"] >= g - 1
                state["p"][b][h] = g
                bars[f"p_full{b}{h}"].arrive()
                g += 1
            yield from W("o_full", o_par, u)
            o_par ^= 1
            yield ("agree", u)
            assert state["o"] == (u, "done")
            state["o_read"].add(h)
            bars["o_free"].arrive()
            qb = u & 1
            if not w[1]:
                assert state["q_busy"][qb] == 0 and state["q"][qb] == u and state["staged"][qb] in (None, u)
                state["staged"][qb] = u
                bars[f"o_staged{qb}"].arrive()
            elif h == 0:
                state["results"].append(u)
            u += 1

    def store():
        par, uses, c = [0, 0], [0, 0], Cursor(True)
        yield from c.next()
        while c.valid:
            if not c.w[1]:
                qb = c.u & 1
                yield from W(f"o_staged{qb}", par[qb], uses[qb])
                par[qb] ^= 1
                uses[qb] += 1
                assert state["staged"][qb] == c.u
                yield ("step",)
                state["staged"][qb] = None
                state["results"].append(c.u)
                bars[f"q_empty{qb}"].arrive()
            yield from c.next()

    agents = {"scheduler": scheduler(), "producer": producer(), "mma": mma(), "sm0": softmax(0), "sm1": softmax(1)}
    if not prefix:
        agents["store"] = store()
    if f8:
        agents["converter0"], agents["converter1"] = converter(0), converter(1)
    pending, done = {a: None for a in agents}, set()

    def tensor():
        op = tensor_q.pop(0)
        if op[0] == "S":
            _, g, st, qb = op
            state["s"][g & 1], state["p"][g & 1] = g, [None, None]
            state["busy"][st] -= 1
            state["q_busy"][qb] -= 1
        elif op[0] == "PV":
            _, g, h, st, u, j, n = op
            if j == 0 and h == 0:
                assert state["o"] is None or (state["o"][0] == u - 1 and state["o_read"] == {0, 1})
                state["o"], state["o_read"] = (u, "acc"), set()
            if h == 1:
                state["busy"][st] -= 1
                state["pv"] = g
                if j == n - 1:
                    state["o"] = (u, "done")
        else:
            bars[op[1]].arrive()

    def tma():
        kind, st, what = tma_q.pop(rng.randrange(len(tma_q)))
        state[{"q": "q", "kv": "stage", "raw": "raw"}[kind]][st] = what
        bars[f"{kind}_full{st}"].arrive()

    while len(done) < len(agents):
        for a, ev in pending.items():
            if ev is not None and ev[0] == "wait":
                assert bars[ev[1]].phase <= ev[2] + 1, f"{a} waits two phases behind {ev}"

        def ready(a):
            ev = pending[a]
            if ev is None or ev[0] == "step":
                return True
            if ev[0] == "wait":
                return bars[ev[1]].phase > ev[2]
            return pending["sm1" if a == "sm0" else "sm0"] == ev

        options = [a for a in agents if a not in done and ready(a)]
        options += ["tensor"] * bool(tensor_q) + ["tma"] * bool(tma_q)
        if not options:
            raise Deadlock(str({a: e for a, e in pending.items() if a not in done}))
        a = rng.choice(options)
        if a == "tensor":
            tensor()
        elif a == "tma":
            tma()
        else:
            if pending[a] is not None and pending[a][0] == "agree":
                pending["sm0"] = pending["sm1"] = None
            try:
                pending[a] = next(agents[a])
            except StopIteration:
                pending[a] = None
                done.add(a)
    assert not tensor_q and not tma_q
    assert sorted(state["results"]) == list(range(len(units))) and len(seq) == sum(w[0] for w in units)


def draw_units(rng, prefix):
    n = rng.choice([0, 1, 2, 5, 12])
    return [(rng.choice([1, 1, 1, 2, 3, 6]), prefix or i in (0, n - 1) and rng.random() < 0.5) for i in range(n)]


@pytest.mark.parametrize("form", ["cross", "prefix", "prefix e4m3"])
@pytest.mark.parametrize("stages", [3, 4, 6, 8])
def test_protocol_runs_without_deadlock_or_race(form, stages):
    for seed in range(60):
        rng = random.Random(seed)
        units = draw_units(rng, form != "cross")
        run_cta(units, rng, f8=form.endswith("e4m3"), prefix=form != "cross", stages=stages)


@pytest.mark.parametrize("mistake", ["first cursor gives back", "converters do not wait", "Q given back twice", "two in the ring"])
def test_planted_mistakes_fail(mistake):
    failed = 0
    for seed in range(60):
        rng = random.Random(seed)
        f8 = mistake == "converters do not wait"
        units = [(1, f8)] * 9 if mistake != "Q given back twice" else [(2, False)] * 6
        try:
            run_cta(units, rng, f8=f8, prefix=f8, queue=2 if mistake == "two in the ring" else QUEUE,
                    mistake=mistake, stages=3)
        except (AssertionError, Deadlock):
            failed += 1
    assert failed > 0, f"no interleaving noticed: {mistake}"
