"""The barriers of the W4A8 tile kernel, followed through every order of events.

The kernel's warps hand operands on through mbarriers whose waits know a phase
by its parity alone: a wait for a phase that is two behind returns at once.
Here the copies, the unpacking groups, the MMA warps, the tensor cores and the
epilogue of one CTA are actors of a small model that holds the same barriers
with the same counts and the same waits in the same order (shapes and order are
read from the sources), and every interleaving of a few chunks is visited.  A
visit fails where a copy or a group writes over what is still to be read, where
a product reads anything but its own chunk, or where nobody can go on.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_26_b200", "csrc")


def shapes():
    """Each shape's layers, unpacking groups, ring stages, operand slots and TMEM
    buffers of a layer, as gptq_abi.cu and Cfg of w4a8_tiled.cuh define them."""
    text = open(os.path.join(CSRC, "gptq_abi.cu")).read()
    out = {}
    for name, args in re.findall(r"using (Small|Mid|Big) = w4a8t::Cfg<(.*)>;", text):
        for nl in (1, 2):
            v = []
            for a in args.split(","):
                pick = re.fullmatch(r"GATED \? (\d+) : (\d+)", a.strip())
                if pick:
                    v.append(int(pick[3 - nl]))
                elif a.strip() not in ("true", "false"):
                    v.append(eval(a.replace("/", "//"), {"NL": nl}))
            tn, uw, stages, slots = v[1], v[2], v[4], v[5]
            out[name, nl] = dict(nl=nl, ug=uw // 4, s=stages, slots=slots, nu=min(512 // tn, 8))
    assert len(out) == 6
    return out


def order(slots):
    """Which of its two barriers an MMA warp waits for first where a chunk is one run,
    with an even or odd number of slots."""
    text = open(os.path.join(CSRC, "w4a8_tiled.cuh")).read()
    text = text[text.index("- MMA warps\n"):text.index("- scale warp\n")]
    for line in text.splitlines():
        wait = re.search(r"W4T_\w*WAIT\w*\((tempty|afull)0", line)
        only = re.search(r"if constexpr \(AS % 2 (==|!=) 0\)", line)
        if wait and (not only or (only[1] == "==") == (slots % 2 == 0)):
            return wait[1]


class Wrong(Exception):
    pass


class Barrier:
    """A state of (phase, arrivals missing); its count comes with each arrival."""

    @staticmethod
    def arrive(state, count):
        phase, missing = state
        if missing is None:
            missing = count
        return (phase + 1, None) if missing == 1 else (phase, missing - 1)

    @staticmethod
    def passes(state, parity):
        return (state[0] & 1) != (parity & 1)


def visit(nl, ug, s, slots, nu, runs, first, chunks, parts=1):
    """Visits every interleaving; raises Wrong.  Every chunk's last run closes.  `parts`:
    warps of a group, each with its rows of a slot."""
    nb = nu // nl
    turns = nl == 2 or nu % (2 * runs) == 0
    stages = chunks // 2
    total = chunks * nl

    def chunk(k):
        return k // nl

    def unit(k, m):  # of the layer
        return chunk(k) * runs + m

    def buffer(k, m):
        return (k % nl) * nb + unit(k, m) % nb

    unpack = [[(op, k) for k in range(total) if k % ug == g // parts
               for op in ("full", "aempty", "write")] for g in range(ug * parts)]
    mma = []
    for w in range(2 if turns else 1):
        ops = []
        for k in range(total):
            if turns and k % 2 != w:
                continue
            if runs == 1 and first == "tempty":
                ops += [("tempty", k, 0), ("afull", k, 0), ("issue", k, 0)]
            else:
                ops.append(("afull", k, 0))
                for m in range(runs):
                    ops += [("tempty", k, m), ("issue", k, m)]
        mma.append(ops)
    mma_of = [[op for op in ops if op[0] == "issue"] for ops in mma]
    folds = [[(k, m) for k in range(total) for m in range(runs) if k % nl == l] for l in range(nl)]

    # names of the barriers, and how many arrivals complete a phase
    names = ([("full", i) for i in range(s)] + [("empty", i) for i in range(s)] +
             [("afull", i) for i in range(slots)] + [("aempty", i) for i in range(slots)] +
             [("tfull", i) for i in range(nu)] + [("tempty", i) for i in range(nu)])
    index = {b: i for i, b in enumerate(names)}
    count = {b: 1 for b in names}
    for i in range(slots):
        count["afull", i] = parts
    for i in range(s):
        count["empty", i] = 2 * nl * parts + (2 if turns else 1)

    def arrive(bars, name):
        i = index[name]
        bars[i] = Barrier.arrive(bars[i], count[name])

    # a state: copies issued; stages in flight; stage that each ring place holds;
    # each unpacking warp's place in its program; chunk that each slot's rows hold; each
    # MMA warp's place; its products done; product that each buffer holds; folds done
    # of each layer; barriers
    start = (0, (), (-1,) * s, (0,) * len(unpack), (-1,) * (slots * parts), (0,) * len(mma), (0,) * len(mma),
             (None,) * nu, (0,) * nl, ((0, None),) * len(names))

    def issued(w, place):
        return sum(op[0] == "issue" for op in mma[w][:place])

    issued_at = [[issued(w, i) for i in range(len(ops) + 1)] for w, ops in enumerate(mma)]

    def reading(state):
        """Products issued and not done."""
        return [mma_of[w][i] for w in range(len(mma))
                for i in range(state[6][w], issued_at[w][state[5][w]])]

    def moves(state):
        tma, flight, ring, ups, held, ms, done, bufs, fs, bars = state
        if tma < stages and Barrier.passes(bars[index["empty", tma % s]], (tma // s) & 1 ^ 1):
            if any(chunk(k) // 2 % s == tma % s for _, k, _ in reading(state)):
                raise Wrong("a copy over tokens that are being read")
            place = list(ring)
            place[tma % s] = -1
            yield (tma + 1, flight + (tma,), tuple(place), ups, held, ms, done, bufs, fs, bars)
        for j in flight:
            place, b = list(ring), list(bars)
            place[j % s] = j
            arrive(b, ("full", j % s))
            yield (tma, tuple(i for i in flight if i != j), tuple(place), ups, held, ms, done, bufs,
                   fs, tuple(b))
        for g in range(len(unpack)):
            if ups[g] == len(unpack[g]):
                continue
            op, k = unpack[g][ups[g]]
            j, slot = chunk(k) // 2, k % slots
            b, h = bars, held
            if op == "full":
                if not Barrier.passes(bars[index["full", j % s]], j // s):
                    continue
            elif op == "aempty":
                if not Barrier.passes(bars[index["aempty", slot]], (k // slots) ^ 1):
                    continue
            else:
                if ring[j % s] != j:
                    raise Wrong("words of another stage unpacked")
                if any(r % slots == slot for _, r, _ in reading(state)):
                    raise Wrong("a slot written while it is read")
                h, b = list(held), list(bars)
                h[slot * parts + g % parts] = k
                arrive(b, ("afull", slot))
                arrive(b, ("empty", j % s))
            at = list(ups)
            at[g] += 1
            yield (tma, flight, ring, tuple(at), tuple(h), ms, done, bufs, fs, tuple(b))
        for w in range(len(mma)):
            if ms[w] < len(mma[w]):
                op, k, m = mma[w][ms[w]]
                bf = bufs
                if op == "afull":
                    ok = Barrier.passes(bars[index["afull", k % slots]], k // slots)
                elif op == "tempty":
                    ok = Barrier.passes(bars[index["tempty", buffer(k, m)]], (unit(k, m) // nb) ^ 1)
                else:
                    rows = held[k % slots * parts:(k % slots + 1) * parts]
                    if rows != (k,) * parts or ring[chunk(k) // 2 % s] != chunk(k) // 2:
                        raise Wrong("a product of another chunk's operands")
                    before = unit(k, m) - nb
                    if before >= 0 and fs[k % nl] <= before:
                        raise Wrong("sums written over before they were folded")
                    bf, ok = list(bufs), True
                    bf[buffer(k, m)] = (k, m)
                if ok:
                    at = list(ms)
                    at[w] += 1
                    yield (tma, flight, ring, ups, held, tuple(at), done, tuple(bf), fs, bars)
            if done[w] < issued_at[w][ms[w]]:
                _, k, m = mma_of[w][done[w]]
                b, at = list(bars), list(done)
                at[w] += 1
                arrive(b, ("tfull", buffer(k, m)))
                if m == runs - 1:
                    arrive(b, ("aempty", k % slots))
                    c, l = chunk(k), k % nl
                    if (nl == 1 or c & 1) if turns else (c & 1 and l == nl - 1):
                        arrive(b, ("empty", c // 2 % s))
                yield (tma, flight, ring, ups, held, ms, tuple(at), bufs, fs, tuple(b))
        for l in range(nl):
            if fs[l] == len(folds[l]):
                continue
            k, m = folds[l][fs[l]]
            if Barrier.passes(bars[index["tfull", buffer(k, m)]], unit(k, m) // nb):
                if bufs[buffer(k, m)] != (k, m) or ("issue", k, m) in reading(state):
                    raise Wrong("sums of another run folded")
                b, at = list(bars), list(fs)
                at[l] += 1
                arrive(b, ("tempty", buffer(k, m)))
                yield (tma, flight, ring, ups, held, ms, done, bufs, tuple(at), tuple(b))

    seen, todo, ended = {start}, [start], 0
    while todo:
        state = todo.pop()
        stuck = True
        for new in moves(state):
            stuck = False
            if new not in seen:
                seen.add(new)
                todo.append(new)
        if stuck:
            if state[8] != tuple(len(f) for f in folds):
                raise Wrong("nobody can go on")
            ended += 1
    assert ended
    return len(seen)


@pytest.mark.parametrize("nl", [1, 2])
@pytest.mark.parametrize("name", ["Small", "Mid", "Big"])
@pytest.mark.parametrize("runs", [1, 2, 4])
def test_every_order_of_events(name, nl, runs):
    shape = shapes()[name, nl]
    # with one run a chunk every slot, stage and buffer comes round twice or more; more
    # runs and layers have more orders, and get as many chunks as seconds allow
    chunks = {(1, 1): 20, (1, 2): 10, (1, 4): 6, (2, 1): 8, (2, 2): 4, (2, 4): 2}[nl, runs]
    visit(**shape, runs=runs, first=order(shape["slots"]), chunks=chunks)


def test_warps_of_a_group_apart():
    """The shape whose slots change hands, with the warps of each unpacking group
    ahead of one another."""
    shape = shapes()["Big", 1]
    visit(**shape, runs=1, first=order(shape["slots"]), chunks=12, parts=2)


def test_the_model_finds_a_parity_two_phases_back():
    """Three operand slots between two MMA warps: a warp that waits for its slot
    first takes the fill before last for its own."""
    three = dict(nl=1, ug=2, s=2, slots=3, nu=2, runs=1, chunks=8)
    with pytest.raises(Wrong, match="another chunk's operands"):
        visit(**three, first="afull")
    visit(**three, first="tempty")


def test_the_model_finds_what_the_ring_orders():
    """With three slots it is the ring that keeps one unpacking group from taking
    the release before last for its own: three stages do, four do not."""
    three = dict(nl=1, ug=2, slots=3, nu=2, runs=1, chunks=12, first="tempty")
    visit(**three, s=3)
    with pytest.raises(Wrong):
        visit(**three, s=4)
