"""A CPU model of the hand-offs of attend_tiles_kernel (kv_tiles.cu), the tensor-core attention over the paged cache.

Its roles are those of the forward kernel, replayed by test_fwd_sync_model.py, with these differences: no loads before
the roles begin; the relay zeroes V's rows past a sequence's end between a copy's landing and the issuer's use of it;
the epilogue writes its stage and reads it back itself. Softmax warps are modelled one by one, eight of them. The
roles run in the kernel's order under random interleavings of themselves, the copies and the tensor pipe, and

  * nobody waits forever, and no warp arrives twice in a phase of a barrier;
  * every MMA reads the Q, K, V and P it was meant to, V's last tile after its zeroing, and O is read before reuse;
  * no copy lands in a stage that an MMA or an epilogue still reads.

A second test loses a copy: the waits for it run out, the abort flag goes up, and every role has to leave in whatever
order the warps come to see it. The named barriers have no limit, so after an abort all their rounds are still
joined: the relay and the issuer go on, with whatever the stages hold, and the softmax warps wait for the issuer
whatever the flag says. What waits for copies or stages (both producers, the relay, the epilogues) follows the flag.

A change to the kernel's hand-offs has to be made here too; planted faults (softmax warps that follow the flag, a named
barrier between the tiles' epilogues, a release that does not wait, a grant that does not) must be caught.
"""
import random

import pytest

from test_fwd_sync_model import MBarrier, NamedBarrier, ProtocolError

NQ, WARPS = 2, 4  # tiles of an item, softmax warps of a tile


def run(items, KST, VST, seed, lose=None, early=None, join="mbarrier", softmax_follows=False, producers_stop=True,
        release_waits=True, grant_waits=True):
    """Play the segments of one CTA (key tiles of each). `lose`: the number of a copy that never lands;
    `early`: the step at which a wait runs out although nothing is lost (the device was taken away for seconds)."""
    rnd = random.Random(seed)
    mb, nb = {}, {}
    abort = [False]
    for q in range(NQ):
        for name in ("q", "qfree", "s", "o", "grant"):
            mb[name, q] = MBarrier((name, q))
    for s in range(KST):
        mb["kfull", s], mb["kempty", s] = MBarrier(("kfull", s)), MBarrier(("kempty", s))
    for s in range(VST):
        mb["vfull", s], mb["vempty", s] = MBarrier(("vfull", s)), MBarrier(("vempty", s))
    mb["join"] = MBarrier("join", NQ * WARPS)

    smem_q, smem_k, smem_v = [None] * NQ, [None] * KST, [None] * VST
    tmem_s = [[None] * WARPS for _ in range(NQ)]  # of each warp's 32 lanes
    tmem_o = [None] * NQ
    o_read = [0] * NQ
    copies, pipe, issued = [], [], [0]
    consumed, staged = {}, {}   # V tile -> MMAs that read it; item -> warps that read their stage back
    whole = lose is None and early is None  # checks of what is read hold until a wait runs out

    def check(ok, what):
        if whole and not ok:
            raise ProtocolError(what)

    def tma(fn):
        issued[0] += 1
        if issued[0] - 1 != lose:
            copies.append(fn)

    def commit(bar):
        pipe.append(mb[bar].arrive)

    def busy(s):
        c = smem_v[s]
        if c is None:
            return False
        return consumed.get(c[1], 0) < NQ if c[0] in ("V", "VZ") else staged.get(c[1], 0) < NQ * WARPS

    # a role yields ("m", barrier, parity) and gets whether the wait succeeded ("i": one that does not follow the abort
    # flag), or ("n", barrier, generation), or None
    def sync(key, who, threads, count):
        b = nb.setdefault(key, NamedBarrier(key))
        gen = b.arrive(who, threads, count)
        yield ("n", key, gen)

    def arrive(key, who, threads, count):
        nb.setdefault(key, NamedBarrier(key)).arrive(who, threads, count)

    tiles, g = [], 0
    for n in items:
        tiles.append(list(range(g, g + n)))
        g += n
    last_of = {t[-1] for t in tiles if t}  # an item's last tile may reach past the sequence: zeroed by the relay

    def load(kind, s, value):
        bar = mb[kind, s]
        bar.arrive_expect_tx(1)
        ring = {"q": smem_q, "kfull": smem_k, "vfull": smem_v}[kind]
        if kind == "vfull":
            check(not busy(s), f"V copy into a busy stage {smem_v[s]}")

        def land():
            if kind == "vfull":
                check(not busy(s), f"V copy landed in a busy stage {smem_v[s]}")
            ring[s] = value
            bar.complete_tx(1)
        tma(land)

    def stops():  # a producer that sees the flag copies no more: stages are then given back without having been filled
        return producers_stop and abort[0]

    def kq():
        g, j = 0, 0
        for k, n in enumerate(items):
            if n == 0:
                continue
            for t in range(n):
                if not (yield ("m", ("kempty", g % KST), ((g // KST) & 1) ^ 1)) or stops():
                    return
                load("kfull", g % KST, ("K", g))
                if t == 0:
                    for q in range(NQ):
                        if j > 0 and (not (yield ("m", ("qfree", q), (j - 1) & 1)) or stops()):
                            return
                        load("q", q, ("Q", k))
                g += 1
            j += 1

    def v():
        pos, seen, prev = 0, [0] * VST, None

        def released(p):
            s, u = p % VST, p // VST
            if seen[s] <= u:
                if not (yield ("m", ("vempty", s), u & 1)) or stops():
                    return False
                seen[s] = u + 1
            return True

        for k, n in enumerate(items):
            for t in range(n):
                if pos >= VST and not (yield from released(pos - VST)):
                    return
                load("vfull", pos % VST, ("V", tiles[k][t]))
                pos += 1
            if pos >= VST and not (yield from released(pos - VST)):
                return
            if grant_waits and prev is not None and not (yield from released(prev)):
                return
            check(not busy(pos % VST), f"a busy stage granted: {smem_v[pos % VST]}")
            for q in range(NQ):
                mb["grant", q].arrive()
            prev = pos
            pos += 1

    def issuer():
        g, pos = 0, 0
        for k, n in enumerate(items):
            if n == 0:
                pos += 1
                continue

            def qk(q, g, k=k):
                def f():
                    check(smem_q[q] == ("Q", k) and smem_k[g % KST] == ("K", g), f"S read {smem_q[q]}, {smem_k[g % KST]}")
                    tmem_s[q] = [("S", g)] * WARPS
                pipe.append(f)
                commit(("s", q))

            def pv(q, g, vs, t, k=k):
                def f():
                    check(tmem_s[q] == [("P", g)] * WARPS, f"P V read {tmem_s[q]}, wanted P {g}")
                    check(smem_v[vs] == (("VZ" if g in last_of else "V"), g), f"P V read {smem_v[vs]}, wanted V {g}")
                    check(t > 0 or tmem_o[q] is None or o_read[q] == WARPS, "P V wrote over an O not yet read")
                    tmem_o[q], o_read[q] = ("O", k, g), 0
                    consumed[g] = consumed.get(g, 0) + 1
                pipe.append(f)

            for q in range(NQ):
                yield from sync("relay", "issuer", 32, 64)
                qk(q, g)
                if n == 1:
                    commit(("qfree", q))
            commit(("kempty", g % KST))
            for t in range(n):
                more = t + 1 < n
                yield from sync("relay", "issuer", 32, 64)
                for q in range(NQ):
                    yield from sync(("P", q), "issuer", 32, 160)
                    pv(q, g, pos % VST, t)
                    if more:
                        qk(q, g + 1)
                        if t + 2 == n:
                            commit(("qfree", q))
                    else:
                        commit(("o", q))
                commit(("vempty", pos % VST))
                if more:
                    commit(("kempty", (g + 1) % KST))
                g += 1
                pos += 1
            pos += 1

    def relay():
        ok, g, j, pos, loads = True, 0, 0, 0, [0] * VST
        for k, n in enumerate(items):
            if n == 0:
                pos += 1
                continue
            for q in range(NQ):
                if ok:
                    ok = yield ("m", ("q", q), j & 1)
                    if ok and q == 0:
                        ok = yield ("m", ("kfull", g % KST), (g // KST) & 1)
                yield from sync("relay", "relay", 32, 64)
            for t in range(n):
                s = pos % VST
                if ok:
                    ok = yield ("m", ("vfull", s), loads[s] & 1)
                    if ok and t + 1 < n:
                        ok = yield ("m", ("kfull", (g + 1) % KST), ((g + 1) // KST) & 1)
                loads[s] += 1
                if ok and g in last_of:
                    yield None
                    check(smem_v[s] == ("V", g), f"zeroed rows of {smem_v[s]}, wanted V {g}")
                    smem_v[s] = ("VZ", g)
                yield from sync("relay", "relay", 32, 64)
                g += 1
                pos += 1
            pos += 1
            j += 1

    def softmax(q, w):
        me = f"softmax {q} {w}"
        ok, g, j, pos, pending = True, 0, 0, 0, None
        issuers = "m" if softmax_follows else "i"

        def release():
            nonlocal ok
            good = True
            if join == "named":
                yield from sync("join", me, 32, 32 * NQ * WARPS)
            elif w > 0:
                return
            elif release_waits:
                good = ok = ok and (yield ("m", "join", pending[1] & 1))
            if w == 0 and good:
                mb["vempty", pending[0]].arrive()

        for k, n in enumerate(items):
            for t in range(n):
                if ok or not softmax_follows:
                    got = yield (issuers, ("s", q), g & 1)
                    ok = ok and got
                if ok or not softmax_follows:
                    check(tmem_s[q][w] == ("S", g), f"softmax read {tmem_s[q][w]}, wanted S {g}")
                    yield None
                    tmem_s[q][w] = ("P", g)
                    arrive(("P", q), me, 32, 160)
                else:
                    yield from sync(("P", q), me, 32, 160)
                if pending:
                    yield from release()
                    pending = None
                g += 1
                pos += 1
            if n > 0:
                if ok or not softmax_follows:
                    got = yield (issuers, ("o", q), j & 1)
                    ok = ok and got
                j += 1
            if pending:
                yield from release()
                pending = None
            if ok:
                ok = yield ("m", ("grant", q), k & 1)
            if ok:
                check(n == 0 or tmem_o[q] == ("O", k, g - 1), f"epilogue read {tmem_o[q]}")
                s = pos % VST
                check(smem_v[s] == ("STAGE", k) or not busy(s), f"staging in a busy stage {smem_v[s]}")
                smem_v[s] = ("STAGE", k)
                yield None
                check(smem_v[s] == ("STAGE", k), f"a stage written over: {smem_v[s]}")
                staged[k] = staged.get(k, 0) + 1
                if n > 0:
                    o_read[q] += 1
            if join == "mbarrier":
                if ok:
                    mb["join"].arrive()
            elif q < NQ - 1:
                if ok:
                    arrive("join", me, 32, 32 * NQ * WARPS)
                else:
                    yield from sync("join", me, 32, 32 * NQ * WARPS)
            if q == NQ - 1:
                pending = (pos % VST, k)
            pos += 1
        if pending:
            yield from release()

    roles = {"kq": kq(), "v": v(), "issuer": issuer(), "relay": relay()}
    roles.update({f"softmax {q} {w}": softmax(q, w) for q in range(NQ) for w in range(WARPS)})
    waiting = {r: None for r in roles}

    def ready(r):
        x = waiting[r]
        if x is None:
            return True
        return mb[x[1]].passed(x[2]) if x[0] in "mi" else nb[x[1]].generation > x[2]

    for step in range(1_000_000):
        if early is not None and step >= early and any(x is not None and x[0] == "m" for x in waiting.values()):
            abort[0] = True
        if not roles:
            if whole:
                check(staged == {k: NQ * WARPS for k in range(len(items))}, "an item without its epilogue")
            return
        able = [r for r in roles if ready(r)]
        quits = [r for r in roles if abort[0] and waiting[r] is not None and waiting[r][0] == "m" and r not in able]
        choices = len(able) + len(quits) + (1 if copies else 0) + (1 if pipe else 0)
        if choices == 0:
            if lose is None or abort[0]:
                raise ProtocolError(f"deadlock: {sorted(roles)} wait forever")
            abort[0] = True  # the limit of a wait: nothing else moves any more
            continue
        c = rnd.randrange(choices)
        if c < len(able) + len(quits):
            r = (able + quits)[c]
            try:
                waiting[r] = roles[r].send(None if waiting[r] is None else c < len(able))
            except StopIteration:
                del roles[r], waiting[r]
        elif copies and c == len(able) + len(quits):
            copies.pop(rnd.randrange(len(copies)))()
        else:
            pipe.pop(0)()
    raise ProtocolError("no progress")


CONFIGS = [(2, 3), (3, 3)]  # K and V stages at D = 128, D = 64


def segments(rnd):
    return [rnd.choice([0, 0, 1, 1, 2, 2, 3, 4, 5, 8]) for _ in range(rnd.randint(1, 8))]


@pytest.mark.parametrize("cfg", CONFIGS)
def test_the_hand_offs_hold(cfg):
    rnd = random.Random(5 + sum(cfg))
    for _ in range(500):
        run(segments(rnd), *cfg, seed=rnd.randrange(10 ** 9))


def copies_of(items):
    return sum(2 * n + NQ * (n > 0) for n in items)


@pytest.mark.parametrize("cfg", CONFIGS)
def test_every_role_leaves_when_a_copy_is_lost(cfg):
    rnd = random.Random(11 + sum(cfg))
    for _ in range(1500):
        items = segments(rnd)
        if copies_of(items):
            run(items, *cfg, seed=rnd.randrange(10 ** 9), lose=rnd.randrange(copies_of(items)))


@pytest.mark.parametrize("cfg", CONFIGS)
def test_every_role_leaves_when_a_wait_runs_out_early(cfg):
    rnd = random.Random(13 + sum(cfg))
    for _ in range(1500):
        items = segments(rnd)
        run(items, *cfg, seed=rnd.randrange(10 ** 9), early=rnd.randrange(20 + 60 * sum(items)))


def caught(trials, lose=False, **fault):
    rnd = random.Random(7)
    for _ in range(trials):
        items = segments(rnd)
        if lose and not copies_of(items):
            continue
        try:
            run(items, 2, 3, seed=rnd.randrange(10 ** 9), lose=rnd.randrange(copies_of(items)) if lose else None, **fault)
        except ProtocolError:
            return True
    return False


def test_softmax_warps_that_follow_the_abort_flag_are_caught():
    # a warp that has arrived for a round and then gives up would join the named barrier for the next round while its
    # neighbours have not joined this one: a generation completes without one of them, which then waits forever
    assert not caught(300, softmax_follows=True)
    assert caught(1000, lose=True, softmax_follows=True)


def test_producers_that_go_on_after_an_abort_are_caught():
    # (a copy into a stage whose last one never landed arrives on a barrier that is still open)
    assert caught(1000, lose=True, producers_stop=False)


def test_a_named_barrier_between_the_tiles_epilogues_is_caught():
    # the same between the tiles: one's warps could join it for the next item before the other's have for this one
    assert not caught(300, join="named")
    assert caught(3000, lose=True, join="named")


def test_a_release_that_does_not_wait_is_caught():
    assert caught(2000, release_waits=False)


def test_a_grant_that_does_not_wait_is_caught():
    assert caught(2000, grant_waits=False)
