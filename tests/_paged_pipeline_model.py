"""Host model of one CTA of the paged chunk kernel (test infrastructure only): the mbarrier
protocol of attn_paged.cu, played as `_pipeline_model.run_cta` plays attn_fwd.cu's, with what
differs: two producers share the K/V ring (K with the walk of the work, the descriptors and
Q; V), every role takes its pieces from a ring of four descriptors, and the softmax warps
meet twice more at the end of a piece whose tile is cut among CTAs."""
from __future__ import annotations

import random

from _pipeline_model import S_BUFS, SOFTMAX_WARPS, Barrier, ProtocolError, cfg, ring_pos_k, ring_pos_v

PIECES = 4
MUTATIONS = ("two_descriptors", "skip_kv_free_wait", "skip_q_free_wait", "skip_join_wait")


def run_cta(piece_blocks, parts, D=128, seed=0, rescale_rate=0.25, mutate=None, stall=0.85):
    """Play one CTA over pieces of the given key-block counts, `parts` saying which of them are parts of
    cut tiles; raises on a parity alias, a buffer hazard or a deadlock.  Returns the number of steps."""
    assert mutate is None or mutate in MUTATIONS
    rnd = random.Random(seed)
    QB, NS = cfg(D)
    bars = {}

    def B(name, count=1):
        if name not in bars:
            bars[name] = Barrier(name, count)
        return bars[name]

    for i in range(QB):
        B(("QF", i)), B(("QFREE", i))
    for i in range(S_BUFS):
        B(("SF", i)), B(("PF", i), SOFTMAX_WARPS), B(("PFREE", i))
    B("OFIN"), B("OFREE", SOFTMAX_WARPS), B("DRAIN", 2), B("PART", SOFTMAX_WARPS), B("JOIN")
    slots = 2 if mutate == "two_descriptors" else PIECES
    for i in range(slots):
        B(("PIECE", i))
    at = {r: 0 for r in ["v_producer", "s_issuer", "pv_issuer"] + [f"softmax{w}" for w in range(SOFTMAX_WARPS)]}
    n_pieces = len(piece_blocks)
    joining = {"last": None}

    def take(role, u):      # wait for descriptor u (the one after the last says that there is no more)
        at[role] = u
        return wait(B(("PIECE", u % slots)), (u // slots) & 1, u // slots)
    for s in range(NS):
        B(("KVF", s)), B(("KVFREE", s))

    events = []
    now = [0.0]
    pipe_end = [0.0]            # the tensor pipe completes MMAs in issue order
    last_mma = {"S": 0.0, "PV": 0.0}
    st = {"S": [None] * S_BUFS, "O": None, "O_issued": None, "stage": [None] * NS, "Q": [None] * QB}
    reads, writes = {}, {}

    def later(dt, fn):
        events.append((now[0] + dt, rnd.random(), fn))

    def mma(who, fn):
        t = max(now[0], pipe_end[0]) + rnd.uniform(0.2, 1.0)
        pipe_end[0] = last_mma[who] = t
        events.append((t, rnd.random(), fn))

    def commit(who, bar):
        events.append((max(now[0], last_mma[who]) + 1e-6, rnd.random(), bar.arrive))

    def wait(bar, parity, phase):
        if parity != (phase & 1):
            raise ProtocolError(f"{bar.name}: parity {parity} does not name phase {phase}")
        if bar.done < phase:
            raise ProtocolError(f"{bar.name}: wait for phase {phase} starts while phase {bar.done} is open")
        return ("wait", bar, phase)

    def load(s, rd, key):
        if st["stage"][s] is not None and st["stage"][s][2] != "free":
            raise ProtocolError(f"ring stage {s} overwritten while {st['stage'][s][:2]} is in use")
        B(("KVF", s)).expect_tx(1)
        st["stage"][s] = key + ("loading",)

        def land():
            st["stage"][s] = key + ("full",)
            B(("KVF", s)).complete_tx(1)
        later(rnd.uniform(0.5, 3.0), land)

    def k_producer():
        item0 = 0
        for u in range(n_pieces + 1):
            qb = u % QB
            if u >= QB and mutate != "skip_q_free_wait":
                yield wait(B(("QFREE", qb)), (u // QB - 1) & 1, u // QB - 1)
            for role, v in at.items():
                if v <= u - slots:
                    raise ProtocolError(f"descriptor {u} overwrites {u - slots}, which {role} still reads")
            B(("PIECE", u % slots)).arrive()
            if u == n_pieces:
                return
            if st["Q"][qb] is not None and st["Q"][qb][1] != "free":
                raise ProtocolError(f"Q buffer {qb} reloaded while piece {st['Q'][qb][0]} still uses it")
            B(("QF", qb)).expect_tx(1)
            st["Q"][qb] = (u, "loading")

            def land_q(qb=qb, u=u):
                st["Q"][qb] = (u, "full")
                B(("QF", qb)).complete_tx(1)
            later(rnd.uniform(0.5, 3.0), land_q)
            for j in range(piece_blocks[u]):
                item = item0 + ring_pos_k(j)
                if item >= NS and mutate != "skip_kv_free_wait":
                    yield wait(B(("KVFREE", item % NS)), (item // NS - 1) & 1, item // NS - 1)
                load(item % NS, item // NS, (u, ("K", j)))
                yield ("step",)
            item0 += 2 * piece_blocks[u]

    def v_producer():
        item0 = 0
        for u in range(n_pieces + 1):
            yield take("v_producer", u)
            if u == n_pieces:
                at["v_producer"] = u + PIECES
                return
            n = piece_blocks[u]
            for j in range(n):
                item = item0 + ring_pos_v(j, n)
                if item >= NS and mutate != "skip_kv_free_wait":
                    yield wait(B(("KVFREE", item % NS)), (item // NS - 1) & 1, item // NS - 1)
                load(item % NS, item // NS, (u, ("V", j)))
                yield ("step",)
            item0 += 2 * n

    def s_issuer():
        g, item0, sb, sph = 0, 0, 0, 0
        for u, n in enumerate(piece_blocks):
            yield take("s_issuer", u)
            qb = u % QB
            yield wait(B(("QF", qb)), (u // QB) & 1, u // QB)
            if st["Q"][qb] != (u, "full"):
                raise ProtocolError(f"S MMA of piece {u} reads Q buffer holding {st['Q'][qb]}")
            if u > 0:
                yield wait(B("OFIN"), (u - 1) & 1, u - 1)
            for j in range(n):
                gs = g + j
                if gs >= S_BUFS and mutate != "skip_buffer_wait":
                    yield wait(B(("PFREE", sb)), sph ^ 1, gs // S_BUFS - 1)
                it = item0 + ring_pos_k(j)
                s = it % NS
                yield wait(B(("KVF", s)), (it // NS) & 1, it // NS)
                if st["stage"][s] != (u, ("K", j), "full"):
                    raise ProtocolError(f"S({u},{j}) reads stage {s} holding {st['stage'][s]}")
                if st["S"][sb] is not None and st["S"][sb][1] != "consumed":
                    raise ProtocolError(f"S({u},{j}) overwrites buffer {sb} holding {st['S'][sb]}")
                st["S"][sb] = ((u, j), "computing")

                def s_done(sb=sb, key=(u, j), s=s):
                    st["S"][sb] = (key, "full")
                    st["stage"][s] = st["stage"][s][:2] + ("free",)
                mma("S", s_done)
                commit("S", B(("SF", sb)))
                commit("S", B(("KVFREE", s)))
                if j == n - 1:
                    def q_free(qb=qb, u=u):
                        st["Q"][qb] = (u, "free")
                    mma("S", q_free)
                    commit("S", B(("QFREE", qb)))
                sb += 1
                if sb == S_BUFS:
                    sb, sph = 0, sph ^ 1
                yield ("step",)
            g += n
            item0 += 2 * n
        yield take("s_issuer", n_pieces)
        at["s_issuer"] = n_pieces + PIECES
        commit("S", B("DRAIN"))
        yield wait(B("DRAIN"), 0, 0)

    def pv_issuer():
        g, item0, pb, pph = 0, 0, 0, 0
        for u, n in enumerate(piece_blocks):
            yield take("pv_issuer", u)
            for j in range(n):
                yield wait(B(("PF", pb)), pph, (g + j) // S_BUFS)
                if j == 0 and u > 0:
                    yield wait(B("OFREE"), (u - 1) & 1, u - 1)
                    if st["O"] != (u - 1, "read"):
                        raise ProtocolError(f"PV({u},0) overwrites O holding {st['O']}")
                it = item0 + ring_pos_v(j, n)
                s = it % NS
                yield wait(B(("KVF", s)), (it // NS) & 1, it // NS)
                if st["stage"][s] != (u, ("V", j), "full"):
                    raise ProtocolError(f"PV({u},{j}) reads stage {s} holding {st['stage'][s]}")
                if st["S"][pb] != ((u, j), "P"):
                    raise ProtocolError(f"PV({u},{j}) reads buffer {pb} holding {st['S'][pb]}")
                if j > 0 and st["O_issued"] != (u, j - 1):
                    raise ProtocolError(f"PV({u},{j}) issued after PV{st['O_issued']}")
                st["O_issued"] = (u, j)

                def pv_done(key=(u, j), pb=pb, s=s):
                    st["S"][pb] = (key, "consumed")
                    st["stage"][s] = st["stage"][s][:2] + ("free",)
                    st["O"] = (key[0], key[1], "done")
                mma("PV", pv_done)
                commit("PV", B(("PFREE", pb)))
                commit("PV", B(("KVFREE", s)))
                if j == n - 1:
                    commit("PV", B("OFIN"))
                pb += 1
                if pb == S_BUFS:
                    pb, pph = 0, pph ^ 1
                yield ("step",)
            g += n
            item0 += 2 * n
        yield take("pv_issuer", n_pieces)
        at["pv_issuer"] = n_pieces + PIECES
        commit("PV", B("DRAIN"))
        yield wait(B("DRAIN"), 0, 0)

    def softmax(w):
        g, sb, sph, pb, pph, n_parts = 0, 0, 0, S_BUFS - 1, 1, 0
        for u, n in enumerate(piece_blocks):
            yield take(f"softmax{w}", u)
            for j in range(n):
                yield wait(B(("SF", sb)), sph, g // S_BUFS)
                if st["S"][sb] not in (((u, j), "full"), ((u, j), "read")):
                    raise ProtocolError(f"softmax warp {w} reads buffer {sb} holding {st['S'][sb]} at ({u},{j})")
                reads[(sb, g)] = reads.get((sb, g), 0) + 1
                if reads[(sb, g)] == SOFTMAX_WARPS:
                    st["S"][sb] = ((u, j), "read")
                yield ("step",)
                if j > 0 and rnd.random() < rescale_rate:
                    yield wait(B(("PFREE", pb)), pph, (g - 1) // S_BUFS)
                    if st["O"] != (u, j - 1, "done"):
                        raise ProtocolError(f"O rescale at ({u},{j}) sees O state {st['O']}")
                # this warp's rows of P(g) go over the scores it has read
                writes[(sb, g)] = writes.get((sb, g), 0) + 1
                if writes[(sb, g)] == SOFTMAX_WARPS:
                    if reads.get((sb, g), 0) != SOFTMAX_WARPS:
                        raise ProtocolError("P written before every warp read its scores")
                    st["S"][sb] = ((u, j), "P")
                B(("PF", sb)).arrive()
                g += 1
                pb, pph = sb, sph
                sb += 1
                if sb == S_BUFS:
                    sb, sph = 0, sph ^ 1
                yield ("step",)
            yield wait(B("OFIN"), u & 1, u)
            if st["O"] != (u, n - 1, "done"):
                raise ProtocolError(f"epilogue of piece {u} reads O state {st['O']}")
            reads[("O", u)] = reads.get(("O", u), 0) + 1
            if reads[("O", u)] == SOFTMAX_WARPS:
                st["O"] = (u, "read")
            B("OFREE").arrive()
            yield ("step",)
            if parts[u]:
                B("PART").arrive()
                if w == 0:
                    yield wait(B("PART"), n_parts & 1, n_parts)
                    joining["last"] = u
                    B("JOIN").arrive()
                if mutate != "skip_join_wait":
                    yield wait(B("JOIN"), n_parts & 1, n_parts)
                if joining["last"] != u:
                    raise ProtocolError(f"softmax warp {w} reads who joins piece {u}: {joining['last']}")
                n_parts += 1
                yield ("step",)
        yield take(f"softmax{w}", n_pieces)
        at[f"softmax{w}"] = n_pieces + PIECES

    roles = {"k_producer": k_producer(), "v_producer": v_producer(), "s_issuer": s_issuer(), "pv_issuer": pv_issuer()}
    for w in range(SOFTMAX_WARPS):
        roles[f"softmax{w}"] = softmax(w)
    blocked = {r: None for r in roles}
    p_stall = {r: rnd.uniform(0.0, stall) for r in roles}
    alive = set(roles)
    steps = 0
    while alive:
        steps += 1
        progressed = False
        order = sorted(alive)
        rnd.shuffle(order)
        for r in order:
            if rnd.random() < p_stall[r]:
                progressed = True
                continue
            bw = blocked[r]
            if bw is not None:
                _, bar, k = bw
                if bar.done <= k:
                    continue
                if bar.done != k + 1:
                    raise ProtocolError(f"{r} waits for phase {k} of {bar.name}, {bar.done} have completed")
                blocked[r] = None
            try:
                ev = next(roles[r])
                progressed = True
                while ev[0] == "wait":
                    _, bar, k = ev
                    if bar.done > k:
                        if bar.done != k + 1:
                            raise ProtocolError(f"{r} waits for phase {k} of {bar.name}, {bar.done} have completed")
                        ev = next(roles[r])
                    else:
                        blocked[r] = ev
                        break
            except StopIteration:
                alive.discard(r)
        if events:
            events.sort(key=lambda e: (e[0], e[1]))
            for _ in range(rnd.randint(1, min(4, len(events)))):
                t, _, fn = events.pop(0)
                now[0] = max(now[0], t)
                fn()
            progressed = True
        if not progressed and alive:
            raise ProtocolError("deadlock: " + ", ".join(
                f"{r} on {blocked[r][1].name} phase {blocked[r][2]}" for r in sorted(alive) if blocked[r]))
    return steps
