"""A CPU model of the hand-offs of attend_tiles_kernel over a cache in 4 or 8 bits (kv_tiles.cu): those of bf16 pages, which
test_kv_tiles_sync_model.py replays, but that K and V come from eight warps that write them, an eighth of a tile each.

What is different, and modelled here: a tile's barrier, and an epilogue's grant, is arrived at by eight warps, each of which
waits for the stages by itself (none may be a phase behind another) and writes K and V in turn; two stages of V, one to
three of K; q has a producer of its own, whose copies are the only ones; a ring of eight tiles' powers of two, written
with K by every other warp (a quarter's) and read by the softmax; the issuer, the relay and the softmax warps are as they were. The roles run under random interleavings and

  * nobody waits forever, and no warp arrives twice in a phase of a barrier;
  * every MMA reads the Q, K, V and P it was meant to, no part of a tile is written while it may still be read, and the
    softmax reads the powers of two of its own tile;
  * with a copy of q lost, or a wait that runs out early, every role leaves.
"""
import random

import pytest

from test_fwd_sync_model import MBarrier, NamedBarrier, ProtocolError

NQ, WARPS, FILL, INFO = 2, 4, 8, 8  # tiles of an item, softmax warps of a tile, code warps, tiles whose info is kept


def run(items, KST, VST, seed, lose=None, early=None, grants=FILL):
    """`grants`: how many of V's warps have to grant an epilogue its stage."""
    rnd = random.Random(seed)
    mb, nb = {}, {}
    abort = [False]
    for q in range(NQ):
        for name in ("q", "qfree", "s", "o"):
            mb[name, q] = MBarrier((name, q))
        mb["grant", q] = MBarrier(("grant", q), grants)
    for s in range(KST):
        mb["kfull", s], mb["kempty", s] = MBarrier(("kfull", s), FILL), MBarrier(("kempty", s))
    for s in range(VST):
        mb["vfull", s], mb["vempty", s] = MBarrier(("vfull", s), FILL), MBarrier(("vempty", s))
    mb["join"] = MBarrier("join", NQ * WARPS)
    smem_q, smem_k, smem_v = [None] * NQ, [[None] * FILL for _ in range(KST)], [[None] * FILL for _ in range(VST)]
    info = [[None] * (FILL // 2) for _ in range(INFO)]
    tmem_s, tmem_o, o_read = [[None] * WARPS for _ in range(NQ)], [None] * NQ, [0] * NQ
    copies, pipe, issued = [], [], [0]
    k_read, v_read, staged = {}, {}, {}  # S of K tile g, P V of V tile g, epilogues of item k: how many are done
    whole = lose is None and early is None

    def check(ok, what):
        if whole and not ok:
            raise ProtocolError(what)

    def commit(bar):
        pipe.append(mb[bar].arrive)

    def v_busy(x):
        return x is not None and (v_read.get(x[1], 0) < NQ if x[0] == "V" else staged.get(x[1], 0) < NQ * WARPS)

    def sync(key, who, threads, count):
        b = nb.setdefault(key, NamedBarrier(key))
        gen = b.arrive(who, threads, count)
        yield ("n", key, gen)

    def arrive(key, who, threads, count):
        nb.setdefault(key, NamedBarrier(key)).arrive(who, threads, count)

    tiles, g0 = [], 0
    for n in items:
        tiles.append(list(range(g0, g0 + n)))
        g0 += n

    def q_producer():
        j = 0
        for k, n in enumerate(items):
            if n == 0:
                continue
            for q in range(NQ):
                if j > 0 and (not (yield ("m", ("qfree", q), (j - 1) & 1)) or abort[0]):
                    return
                bar = mb["q", q]
                bar.arrive_expect_tx(1)

                def land(q=q, k=k, bar=bar):
                    smem_q[q] = ("Q", k)
                    bar.complete_tx(1)
                issued[0] += 1
                if issued[0] - 1 != lose:
                    copies.append(land)
            j += 1

    def codes(w):
        g, pos, seen, prev = 0, 0, [0] * VST, None

        def released(p):
            s, u = p % VST, p // VST
            if seen[s] <= u:
                if not (yield ("m", ("vempty", s), u & 1)) or abort[0]:
                    return False
                seen[s] = u + 1
            return True

        for k, n in enumerate(items):
            for _ in range(n):
                s = g % KST
                if w % 2 == 0:
                    info[g % INFO][w // 2] = g
                if not (yield ("m", ("kempty", s), ((g // KST) & 1) ^ 1)) or abort[0]:
                    return
                was = smem_k[s][w]
                check(was is None or k_read.get(was, 0) == NQ, f"K {was} written over")
                yield None
                smem_k[s][w] = g
                yield None
                mb["kfull", s].arrive()
                if pos >= VST and not (yield from released(pos - VST)):
                    return
                check(not v_busy(smem_v[pos % VST][w]), f"V {smem_v[pos % VST][w]} written over")
                yield None
                smem_v[pos % VST][w] = ("V", g)
                yield None
                mb["vfull", pos % VST].arrive()
                g += 1
                pos += 1
            if pos >= VST and not (yield from released(pos - VST)):
                return
            if prev is not None and not (yield from released(prev)):
                return
            if w < grants:
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
                    check(smem_q[q] == ("Q", k) and smem_k[g % KST] == [g] * FILL, f"S read {smem_q[q]}, {smem_k[g % KST]}")
                    tmem_s[q] = [("S", g)] * WARPS
                    k_read[g] = k_read.get(g, 0) + 1
                pipe.append(f)
                commit(("s", q))

            def pv(q, g, vs, t, k=k):
                def f():
                    check(tmem_s[q] == [("P", g)] * WARPS, f"P V read {tmem_s[q]}, wanted P {g}")
                    check(smem_v[vs] == [("V", g)] * FILL, f"P V read {smem_v[vs]}, wanted V {g}")
                    check(t > 0 or tmem_o[q] is None or o_read[q] == WARPS, "P V wrote over an O not yet read")
                    tmem_o[q], o_read[q] = ("O", k, g), 0
                    v_read[g] = v_read.get(g, 0) + 1
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
        for n in items:
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
                yield from sync("relay", "relay", 32, 64)
                g += 1
                pos += 1
            pos += 1
            j += 1

    def softmax(q, w):
        me = f"softmax {q} {w}"
        ok, live, g, j, pos, pending = True, True, 0, 0, 0, None

        def release():
            nonlocal ok
            if ok:
                ok = yield ("m", "join", pending[1] & 1)
            if ok:
                mb["vempty", pending[0]].arrive()

        for k, n in enumerate(items):
            for t in range(n):
                if live:
                    live = yield ("i", ("s", q), g & 1)
                if live:
                    check(tmem_s[q][w] == ("S", g) and info[g % INFO] == [g] * (FILL // 2), f"softmax read {tmem_s[q][w]}, {info[g % INFO]}, wanted {g}")
                    yield None
                    check(info[g % INFO] == [g] * (FILL // 2), f"info of tile {g} written over")
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
                if live:
                    live = yield ("i", ("o", q), j & 1)
                j += 1
            if pending:
                yield from release()
                pending = None
            ok = ok and live
            if ok:
                ok = yield ("m", ("grant", q), k & 1)
            if ok:
                check(n == 0 or tmem_o[q] == ("O", k, g - 1), f"epilogue read {tmem_o[q]}")
                s = pos % VST
                for x in smem_v[s]:
                    check(x == ("STAGE", k) or not v_busy(x), f"staging in a busy stage {x}")
                smem_v[s] = [("STAGE", k)] * FILL
                yield None
                check(smem_v[s] == [("STAGE", k)] * FILL, f"a stage written over: {smem_v[s]}")
                staged[k] = staged.get(k, 0) + 1
                if n > 0:
                    o_read[q] += 1
                mb["join"].arrive()
            if q == NQ - 1 and w == 0:
                pending = (pos % VST, k)
            pos += 1
        if pending:
            yield from release()

    roles = {"q": q_producer(), "issuer": issuer(), "relay": relay()}
    roles.update({f"codes {w}": codes(w) for w in range(FILL)})
    roles.update({f"softmax {q} {w}": softmax(q, w) for q in range(NQ) for w in range(WARPS)})
    waiting = {r: None for r in roles}

    def ready(r):
        x = waiting[r]
        if x is None:
            return True
        return mb[x[1]].passed(x[2]) if x[0] in "mi" else nb[x[1]].generation > x[2]

    slow = rnd.choice([None, *roles])  # one role falls far behind the others now and then
    for step in range(1_000_000):
        if early is not None and step >= early and any(x is not None and x[0] == "m" for x in waiting.values()):
            abort[0] = True
        if not roles:
            if whole:
                check(staged == {k: NQ * WARPS for k in range(len(items))}, "an item without its epilogue")
            return
        able = [r for r in roles if ready(r)]
        if slow in able and len(able) > 1 and rnd.random() < 0.95:
            able.remove(slow)
        quits = [r for r in roles if abort[0] and waiting[r] is not None and waiting[r][0] == "m" and r not in able and not ready(r)]
        choices = len(able) + len(quits) + (1 if copies else 0) + (1 if pipe else 0)
        if choices == 0:
            if lose is None or abort[0]:
                raise ProtocolError(f"deadlock: {sorted(roles)} wait forever")
            abort[0] = True
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


CONFIGS = [(2, 2), (1, 2), (3, 2)]  # K and V stages: 4 bits and 8 bits at D = 128, 4 bits at D = 64 (8 bits: 2, 2)


def segments(rnd):
    return [rnd.choice([0, 0, 1, 1, 2, 2, 3, 4, 5, 8]) for _ in range(rnd.randint(1, 7))]


@pytest.mark.parametrize("cfg", CONFIGS)
def test_the_hand_offs_hold(cfg):
    rnd = random.Random(5 + sum(cfg))
    for _ in range(250):
        run(segments(rnd), *cfg, seed=rnd.randrange(10 ** 9))


@pytest.mark.parametrize("cfg", CONFIGS)
def test_every_role_leaves_when_a_copy_of_q_is_lost(cfg):
    rnd = random.Random(11 + sum(cfg))
    for _ in range(400):
        items = segments(rnd)
        n = NQ * sum(x > 0 for x in items)
        if n:
            run(items, *cfg, seed=rnd.randrange(10 ** 9), lose=rnd.randrange(n))


@pytest.mark.parametrize("cfg", CONFIGS)
def test_every_role_leaves_when_a_wait_runs_out_early(cfg):
    rnd = random.Random(13 + sum(cfg))
    for _ in range(400):
        items = segments(rnd)
        run(items, *cfg, seed=rnd.randrange(10 ** 9), early=rnd.randrange(40 + 90 * sum(items)))


def test_a_grant_by_one_warp_alone_is_caught():
    # (one of the warps may then fall a whole phase behind, and wait for one that is over)
    rnd = random.Random(7)
    for _ in range(3000):
        try:
            run(segments(rnd), 2, 2, seed=rnd.randrange(10 ** 9), grants=1)
        except ProtocolError:
            return
    raise AssertionError("not caught")
