"""The barriers of the tensor-core attention kernel, as a model on the CPU.

A role of the kernel (attention_tc.cu) is the list of its waits and arrivals, in program order.  An
mbarrier knows no more of a phase than its parity, so a wait for phase n is sound only if, whatever the
other warps' speed, phase n - 1 is complete when it begins (it would pass too early) and phase n + 1 is
not complete before it has passed (it would block for good).  More progress of the others never takes
away progress, so both are decided by the extremes: the others as far as they get without this warp, and
only as far as this warp needs them."""
import pytest


class Role:
    def __init__(self):
        self.ops = []

    def wait(self, bar, n):
        if n >= 0:  # (an empty ring's buffers: the phase before the first passes)
            self.ops.append(("wait", bar, n))

    def arrive(self, bar, n):
        self.ops.append(("arrive", bar, n))


def roles(segments, two, halves, fp8, NK, NV, NR=0, NS=0, reports=True, conv_of=lambda ik, NK: ik % NK, n_conv=8,
          stagger=4):
    """The roles of a CTA whose segments have the given numbers of key tiles.  two: two row tiles on the same
    keys; halves: turns of a tile; reports: an issuer without a tile in a segment arrives on o_full all the
    same and the softmax warps wait for it; conv_of: the converter that turns a key tile's scales."""
    r = {}

    def role(name):
        return r.setdefault(name, Role())

    def buffers(n):  # of a segment, in the order of their use
        if two:
            return [(bool(i & 1), i >> 1) for i in range(2 * n)]
        order = []
        for i in range(2 * n):
            if i == 2 * n - 1:
                order.append((True, n - 1))
            elif i < 2:
                order.append((False, i))
            else:
                order.append((i % 2 == 0, (i >> 1) - 1 if i % 2 == 0 else (i + 1) >> 1))
        return order

    it = 0
    for n in segments:  # producers
        for _ in range(n):
            k, v = role("keys"), role("values")
            k.wait(f"kempty{it % NK}", it // NK - 1)
            if fp8:
                k.arrive(f"xfull{it % NK}", it // NK)
            k.arrive(f"kfull{it % NK}", it // NK)
            ring, N = ("r", NR) if fp8 else ("v", NV)
            v.wait(f"{ring}empty{it % N}", it // N - 1)
            v.arrive(f"{ring}full{it % N}", it // N)
            it += 1
    if fp8:
        for cw in range(n_conv):
            c, ik, iv = role(f"converter{cw}"), 0, 0
            for n in segments:
                for v, _ in buffers(n):
                    if not v:
                        if conv_of(ik, NK) == cw:
                            c.wait(f"xfull{ik % NK}", ik // NK)
                            c.arrive(f"kfull{ik % NK}", ik // NK)
                        ik += 1
                    else:
                        c.wait(f"rfull{iv % NR}", iv // NR)
                        c.wait(f"vempty{iv % NV}", iv // NV - 1)
                        c.arrive(f"vfull{iv % NV}", iv // NV)
                        c.arrive(f"rempty{iv % NR}", iv // NR)
                        iv += 1
    step = 1 if two else 2
    for g in range(2):  # MMA issuers
        m, ik, iv, turns, scored, ends = role(f"issuer{g}"), 0, 0, 0, 0, 0
        for s, n in enumerate(segments):
            m.wait("q_full", s)
            if two and g == 1 and n >= stagger:
                m.wait("go", s)
            if reports and g >= n and not two:
                m.arrive(f"o_full{g}", ends)
                ends += 1
            for t in range(-step, n):
                now, more = t >= 0, t + step < n
                if not two and (t ^ g) & 1:
                    for v in (True, False):
                        if v and now:
                            m.wait(f"vfull{iv % NV}", iv // NV)
                            m.arrive(f"vempty{iv % NV}", iv // NV)
                            iv += 1
                        if not v and more:
                            m.wait(f"kfull{ik % NK}", ik // NK)
                            m.arrive(f"kempty{ik % NK}", ik // NK)
                            ik += 1
                    continue
                if now:
                    m.wait(f"vfull{iv % NV}", iv // NV)
                for half in range(halves):
                    if now:
                        m.wait(f"p_full{g}{half}", turns)
                        if halves > 1:
                            m.arrive(f"pv_done{g}", turns * halves + half)
                        if half == halves - 1:
                            m.arrive(f"vempty{iv % NV}", iv // NV)
                            if not more:
                                m.arrive(f"o_full{g}", ends)
                                ends += 1
                    if more:
                        if half == 0:
                            m.wait(f"kfull{ik % NK}", ik // NK)
                        m.arrive(f"s_full{g}{half}", scored)
                        if half == halves - 1:
                            m.arrive(f"kempty{ik % NK}", ik // NK)
                if now:
                    turns += 1
                    iv += 1
                if more:
                    ik += 1
                    scored += 1
    for g in range(2):  # softmax warps: the four of a stream, two of which are modelled
        for w in range(2):
            x, tiles, turn0, segs = role(f"softmax{g}{w}"), 0, 0, 0
            for s, n in enumerate(segments):
                x.arrive("q_full", s)
                turn = 0
                for t in range(0 if two else g, n, step):
                    for half in range(halves):
                        x.wait(f"s_full{g}{half}", tiles)
                        if halves > 1 and turn > 0:  # (a maximum that moves)
                            x.wait(f"pv_done{g}", turn0 + turn - 1)
                        if two and g == 0 and turn == 0:
                            x.arrive("go", s)
                        x.arrive(f"p_full{g}{half}", tiles)
                        turn += 1
                    tiles += 1
                turn0 += turn
                if reports or turn:
                    x.wait(f"o_full{g}", segs)
                    segs += 1
                meet = f"stream{g}" if two else "merge"  # hardware barriers
                x.arrive(meet, s)
                x.wait(meet, s)
    return r


def faults(r):
    """Waits that may pass too early, block for good, or never be served."""
    need = {}  # arrivals of each phase
    for name, role in r.items():
        for i, (what, bar, n) in enumerate(role.ops):
            if what == "arrive":
                need.setdefault((bar, n), []).append((name, i))
    found = []

    def complete(bar, pc):  # phases
        n = 0
        while (bar, n) in need and all(pc[name] > i for name, i in need[bar, n]):
            n += 1
        return n

    for victim, role in r.items():
        others = [x for x in r if x != victim]
        pc = dict.fromkeys(r, 0)
        for i, (what, bar, n) in enumerate(role.ops):
            pc[victim] = i
            if what == "arrive":
                continue
            moved = True
            while moved:  # the others as far as they get
                moved = False
                for x in others:
                    while pc[x] < len(r[x].ops):
                        w, b, k = r[x].ops[pc[x]]
                        if w == "wait" and complete(b, pc) <= k:
                            break
                        pc[x] += 1
                        moved = True
            done = complete(bar, pc)
            if done > n + 1:
                found.append((victim, bar, n, "missed"))
            if done <= n:
                found.append((victim, bar, n, "never served"))
                return found
    for victim, role in r.items():
        pc = dict.fromkeys(r, 0)

        def advance(name, to):  # no further than is needed
            while pc[name] < to:
                w, b, k = r[name].ops[pc[name]]
                if w == "wait":
                    for x, i in need[b, k]:
                        if x != name:
                            advance(x, i + 1)
                pc[name] += 1

        for i, (what, bar, n) in enumerate(role.ops):
            if what == "wait" and complete(bar, pc) < n:
                found.append((victim, bar, n, "early"))
            advance(victim, i + 1)
    return found


# key tiles of the segments of a CTA
SEGMENTS = [[1] * 9, [2] * 6, [1, 2, 1, 1, 3, 1, 1, 1, 2], [5, 1, 1, 1, 1, 1, 4], [3, 3, 1, 1], [9], [1, 1, 6, 2, 1, 7]]
# as in Cfg: (two, halves, fp8, NK, NV, NR); for heads of 64 every ring is twice as long
SHAPES = [(False, 1, False, 3, 3, 0), (False, 2, False, 3, 3, 0), (True, 2, False, 3, 2, 0),
          (False, 1, True, 3, 2, 4), (False, 2, True, 3, 2, 4), (True, 2, True, 3, 2, 2)]


@pytest.mark.parametrize("mul", [1, 2])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("segments", SEGMENTS, ids=str)
def test_every_wait_is_sound(shape, segments, mul):
    two, halves, fp8, *rings = shape
    assert faults(roles(segments, two, halves, fp8, *(mul * n for n in rings))) == []


@pytest.mark.parametrize("fp8", [False, True])
def test_the_model_sees_an_issuer_left_behind(fp8):
    """Segments of one tile: without a report of the second stream's issuer, the softmax warps and the
    first stream can begin two segments while it still waits for the queries of the one before."""
    found = faults(roles([1] * 9, False, 1, fp8, 3, 2 if fp8 else 3, 4 if fp8 else 0, reports=False))
    assert ("issuer1", "q_full", "missed") in {(v, b, w) for v, b, _, w in found}


def test_the_model_sees_a_phase_left_out():
    """A buffer's scales turned by another converter each time: one that left out a phase may take an
    older one for its own."""
    found = faults(roles([1] * 30, False, 1, True, 2, 3, 3, conv_of=lambda ik, NK: ik % 8))
    assert {(b[:5], w) for _, b, _, w in found} & {("xfull", "early"), ("xfull", "missed")}
