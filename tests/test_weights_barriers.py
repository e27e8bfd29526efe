"""The barriers of the accumulated weight's tensor-core kernel (csrc/attn_weights_tc.cu), in every order its warps can
run: each warp as the list of its waits, arrivals, stores and reads, each barrier with an mbarrier's rules (a phase
ends at its count of arrivals; a wait passes while the current phase's parity is not the one waited for).
A read of anything but what was stored for it, or a state that no warp can leave, is a fault."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_lightning_gb300", "csrc")


def constant(name):
    with open(os.path.join(CSRC, "attn_weights_tc.cu")) as f:
        return int(re.search(rf"constexpr int {name} = (\d+);", f.read()).group(1))


def explore(programs, counts):
    """None, or what goes wrong, over all interleavings.  counts: arrivals a phase takes, by barrier."""
    bars = sorted(counts)
    at = {b: i for i, b in enumerate(bars)}
    cells = sorted({op[1] for p in programs for op in p if op[0] in ("put", "read")})
    cell_at = {c: i for i, c in enumerate(cells)}
    first = (tuple(0 for _ in programs), tuple((0, 0) for _ in bars), tuple(None for _ in cells))
    seen, todo = {first}, [first]
    while todo:
        pcs, bs, cs = todo.pop()
        moved = False
        for w, p in enumerate(programs):
            if pcs[w] == len(p):
                continue
            kind, what, value = p[pcs[w]]
            nb, nc = bs, cs
            if kind == "wait":
                if (bs[at[what]][0] & 1) == value:
                    continue
            elif kind == "arrive":
                phase, n = bs[at[what]]
                new = (phase + 1, 0) if n + 1 == counts[what] else (phase, n + 1)
                nb = bs[:at[what]] + (new,) + bs[at[what] + 1:]
            elif kind == "put":
                nc = cs[:cell_at[what]] + (value,) + cs[cell_at[what] + 1:]
            elif cs[cell_at[what]] != value:
                return f"warp {w} reads {cs[cell_at[what]]} of {what} for {value}"
            moved = True
            state = (pcs[:w] + (pcs[w] + 1,) + pcs[w + 1:], nb, nc)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(pc < len(p) for pc, p in zip(pcs, programs)):
            return f"stuck at {pcs}"
    return None


def sums(buffers, barriers, chunks=6, warps=3):
    """The MMA warp and the weights warps over one query's chunks.  (Three of them: one reads, two do not.)"""
    counts = {("s_full", i): 1 for i in (0, 1)} | {("s_empty", i): warps for i in (0, 1)}
    counts |= {("red_full", i): warps for i in range(barriers)}
    mma = []
    for n in range(chunks):
        mma += [("wait", ("s_empty", n & 1), ((n >> 1) & 1) ^ 1), ("arrive", ("s_full", n & 1), None)]
    programs = [mma]
    for w in range(warps):
        p = []
        for n in range(chunks):
            p += [("wait", ("s_full", n & 1), (n >> 1) & 1), ("arrive", ("s_empty", n & 1), None),
                  ("put", ("red", n % buffers, w), n), ("arrive", ("red_full", n % barriers), None)]
            if w == 0:
                p.append(("wait", ("red_full", n % barriers), (n // barriers) & 1))
                p += [("read", ("red", n % buffers, v), n) for v in range(warps)]
        programs.append(p)
    return explore(programs, counts)


def test_two_barriers_for_four_buffers_can_be_overtaken():
    assert "reads" in sums(4, 2)


def test_sums_are_read_after_they_are_stored():
    n = constant("kSums")
    assert sums(n, n) is None


def queries(good, qchunks, waits, slots, chunks=1):
    """Queries one after another in a CTA, each a block of qchunks chunks of the ring and, where its sequence is good,
    `chunks` chunks of rows.  waits: on a refused query, the weights warps wait for the release of its block."""
    warps = 4
    counts = {("k_full", i): 1 for i in range(slots)} | {("k_empty", i): 1 for i in range(slots)}
    counts |= {("s_full", i): 1 for i in (0, 1)} | {("s_empty", i): warps for i in (0, 1)}
    counts["q_full", 0] = warps
    producer, mma, weigh = [], [], [[] for _ in range(warps)]
    use = n = 0  # chunks that went through the ring; chunks of rows
    for t, ok in enumerate(good):
        block = [(use + c) % slots for c in range(qchunks)]
        for c in range(qchunks + (chunks if ok else 0)):
            slot, turn = (use + c) % slots, (use + c) // slots
            producer += [("wait", ("k_empty", slot), (turn & 1) ^ 1), ("put", ("ring", slot), (t, c)),
                         ("arrive", ("k_full", slot), None)]
        mma.append(("wait", ("q_full", 0), t & 1))
        mma += [("arrive", ("k_empty", s), None) for s in block]
        for w, p in enumerate(weigh):
            c = w // 2  # heads 32 w ..: in the block's first or second chunk, or (few heads) in none
            if c < qchunks:
                p += [("wait", ("k_full", block[c]), ((use + c) // slots) & 1), ("read", ("ring", block[c]), (t, c))]
            p.append(("arrive", ("q_full", 0), None))
            if not ok and waits:
                p.append(("wait", ("k_empty", block[-1]), ((use + qchunks - 1) // slots) & 1))
        use += qchunks
        for _ in range(chunks if ok else 0):
            slot, turn = use % slots, use // slots
            mma += [("wait", ("s_empty", n & 1), ((n >> 1) & 1) ^ 1), ("wait", ("k_full", slot), turn & 1),
                    ("arrive", ("k_empty", slot), None), ("arrive", ("s_full", n & 1), None)]
            for p in weigh:
                p += [("wait", ("s_full", n & 1), (n >> 1) & 1), ("arrive", ("s_empty", n & 1), None)]
            use, n = use + 1, n + 1
    return explore([producer, mma] + weigh, counts)


@pytest.mark.parametrize("qchunks", [1, 2])
def test_refused_queries_can_be_overtaken_without_a_wait(qchunks):
    assert queries([False] * 4 + [True], qchunks, False, 3) is not None


@pytest.mark.parametrize("good", ["0000", "00010", "10010", "01011", "1111"])
@pytest.mark.parametrize("qchunks", [1, 2])
def test_refused_queries_keep_the_ring_in_order(good, qchunks):
    assert queries([g == "1" for g in good], qchunks, True, constant("kStages")) is None
