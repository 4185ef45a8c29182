"""A model of the pool pre-fill kernel's synchronisation (prefill_pool_kernel), run over
random interleavings: one CTA works through a list of pieces (tiles, query tiles), each role
taking them in order from a ring that one warp fills.  Roles, barriers, counts and phase
arithmetic follow the kernel, one arrival per role; the checks are those of
tests/protocol_sim.py (no deadlock, every wait passes on the phase it means, every read
sees the version it expects).  Tensor memory as in the cache's pre-fill model, with a
piece's number in every version: S_t of the next piece may only overwrite P_t after the
last product has read it, O_t only after the softmax has read it out, Q only after the
piece's last S product."""
import pytest

from protocol_sim import Sim, wait

KQ, KST, RING = 2, 2, 4  # query tiles, K and V stages, pieces listed ahead


def cta(sim, pieces, q_waits=True, ring_waits=True, pv_before_next_s=True):
    """pieces: [(tiles, query tiles)].  The keyword arguments exist to plant mistakes."""
    for name in ["Q", "QEmpty"] + [f"{x}{s}" for x in ("KFull", "KEmpty", "VFull", "VEmpty") for s in range(KST)] + \
            [f"{x}{t}" for x in ("SFull", "PFull", "PRest", "OFull") for t in range(KQ)] + [f"Piece{i}" for i in range(RING)]:
        sim.bar(name)
    for i in range(RING):
        sim.bar(f"Free{i}", 3 + KQ)
    queue, done = [], set()

    def lister():
        for p, x in enumerate(pieces + [(0, 0)]):
            if p >= RING and ring_waits:
                yield wait(f"Free{p % RING}", p // RING - 1)
            sim.write(f"piece{p % RING}", (p, x))
            sim.arrive(f"Piece{p % RING}")
            yield None

    def take(p):
        """Reads piece p (after its wait)."""
        x = pieces[p] if p < len(pieces) else (0, 0)
        sim.read(f"piece{p % RING}", (p, x))
        return x

    def load(buf, version, bar):
        yield None
        sim.write(buf, version)
        sim.arrive(bar)

    def producer(is_k):
        name = "k" if is_k else "v"
        full, empty = ("KFull", "KEmpty") if is_k else ("VFull", "VEmpty")
        issued, p = 0, 0
        while True:
            yield wait(f"Piece{p % RING}", p // RING)
            nt, _ = take(p)
            if nt == 0:
                return
            if not is_k:
                if p > 0 and q_waits:
                    yield wait("QEmpty", p - 1)
                sim.spawn(load("q", ("Q", p), "Q"), f"tmaQ{p}")
            for j in range(nt):
                s = issued % KST
                if issued >= KST:
                    yield wait(f"{empty}{s}", issued // KST - 1)
                take(p)
                sim.spawn(load(f"{name}{s}", (name, p, j), f"{full}{s}"), f"tma{name}{p}.{j}")
                issued += 1
                yield None
            sim.arrive(f"Free{p % RING}")
            p += 1

    def engine():
        while True:
            if not queue:
                if "mma" in done:
                    return
                yield None
                continue
            queue.pop(0)()
            yield None

    def s_product(t, p, j, s):
        def op():
            sim.read("q", ("Q", p))
            sim.read(f"k{s}", ("k", p, j))
            sim.write(f"s{t}", ("S", p, j))
            sim.arrive(f"SFull{t}")
        return op

    def pv_product(t, p, j, s, part):
        def op():
            sim.read(f"s{t}", ("P", p, j))
            if part:
                sim.read(f"rest{t}", ("P", p, j))
                sim.read(f"v{s}", ("v", p, j))
                sim.write(f"o{t}", ("O", p, j))
                return
            sim.read(f"v{s}", ("v", p, j))
            if j > 0:
                sim.read(f"o{t}", ("O", p, j - 1))
            else:
                assert sim.buf.get(f"o{t}", ("read",))[-1] == "read", "O overwritten before it was read out"
            sim.write(f"o{t}", ("O", p, j, "first part"))
        return op

    def arrival(name):
        return lambda: sim.arrive(name)

    def mma_thread():
        k, v, pt, p = 0, 0, [0] * KQ, 0
        while True:
            yield wait(f"Piece{p % RING}", p // RING)
            nt, nq = take(p)
            sim.arrive(f"Free{p % RING}")
            if nt == 0:
                break
            yield wait("Q", p)
            yield wait(f"KFull{k % KST}", k // KST)
            for t in range(nq):
                queue.append(s_product(t, p, 0, k % KST))
            queue.append(arrival(f"KEmpty{k % KST}"))
            k += 1
            if nt == 1:
                queue.append(arrival("QEmpty"))
            for j in range(nt):
                for t in range(nq):
                    if t == 0:
                        yield wait(f"VFull{v % KST}", v // KST)
                        if j + 1 < nt:
                            yield wait(f"KFull{k % KST}", k // KST)
                    yield wait(f"PFull{t}", pt[t])
                    if pv_before_next_s:
                        queue.append(pv_product(t, p, j, v % KST, 0))
                    yield wait(f"PRest{t}", pt[t])
                    pt[t] += 1
                    pv = ([] if pv_before_next_s else [pv_product(t, p, j, v % KST, 0)]) + \
                        [pv_product(t, p, j, v % KST, 1)]
                    if t == nq - 1:
                        pv.append(arrival(f"VEmpty{v % KST}"))
                        v += 1
                    if j + 1 == nt:
                        queue.extend(pv + [arrival(f"OFull{t}")])
                        continue
                    nxt = [s_product(t, p, j + 1, k % KST)]
                    if t == nq - 1:
                        nxt.append(arrival(f"KEmpty{k % KST}"))
                        k += 1
                        if j + 2 == nt:
                            nxt.append(arrival("QEmpty"))
                    queue.extend(pv + nxt if pv_before_next_s else nxt + pv)
                    yield None
            p += 1
        done.add("mma")

    def softmax(t):
        tiles, outs, p = 0, 0, 0
        while True:
            yield wait(f"Piece{p % RING}", p // RING)
            nt, nq = take(p)
            if nt == 0:
                return
            if t >= nq:
                sim.arrive(f"Free{p % RING}")
                p += 1
                continue
            for j in range(nt):
                yield wait(f"SFull{t}", tiles)
                tiles += 1
                take(p)
                sim.read(f"s{t}", ("S", p, j))
                if j >= 1:
                    sim.read(f"o{t}", ("O", p, j - 1))
                    sim.write(f"o{t}", ("O", p, j - 1))
                sim.write(f"s{t}", ("P", p, j))  # the first keys' weights, then the others'
                sim.arrive(f"PFull{t}")
                yield None
                sim.write(f"rest{t}", ("P", p, j))
                sim.arrive(f"PRest{t}")
                yield None
            sim.arrive(f"Free{p % RING}")
            yield wait(f"OFull{t}", outs)
            outs += 1
            sim.read(f"o{t}", ("O", p, nt - 1))
            yield None
            sim.read(f"o{t}", ("O", p, nt - 1))
            sim.write(f"o{t}", ("O", p, "read"))
            p += 1

    for gen, name in ((lister(), "lister"), (producer(True), "k"), (producer(False), "v"), (mma_thread(), "mma_thread"),
                      (engine(), "mma")):
        sim.spawn(gen, name)
    for t in range(KQ):
        sim.spawn(softmax(t), f"softmax{t}")


LISTS = [[(1, 1)], [(1, 2), (1, 2)], [(3, 2), (1, 1), (2, 2)], [(2, 1), (4, 2), (1, 2), (1, 1), (3, 2), (2, 2)],
         [(1, 2)] * 9, [(1, 1), (1, 2)] * 5, [(7, 2), (6, 1), (2, 2)], []]


@pytest.mark.parametrize("pieces", LISTS, ids=str)
def test_protocol_random_interleavings(pieces):
    for seed in range(150):
        sim = Sim(seed)
        cta(sim, list(pieces))
        sim.run()


@pytest.mark.parametrize("mistake", ["q_waits", "ring_waits", "pv_before_next_s"])
def test_model_catches(mistake):
    caught = 0
    for seed in range(200):
        sim = Sim(seed)
        cta(sim, [(3, 2)] * 3 + [(1, 2)] * 6, **{mistake: False})
        try:
            sim.run()
        except AssertionError:
            caught += 1
    assert caught > 0
