"""The order of the many-row attention kernel's roles (csrc/paged_attn_tc.cu),
as a model whose every interleaving is walked on the CPU.

A process is a role's barrier operations and accesses in program order, in steps
that happen at once. Barriers count as the hardware's: a wait for parity p passes
when the phase in progress has the other parity; an arrival that brings the
count to zero starts the next phase. Products run in the order in which they
were issued, at any time after that; a commit arrives when all before it are
done. A place being written holds nothing, from the wait before the write (the
earliest that it can begin) to the arrival after it (the latest that it can end).
Every read has to find the tile it is for.
"""
import pytest

K_EMPTY, K_FULL, V_EMPTY, V_FULL, S_FULL, P_READY = range(6)


def roles(n, v_waits):
    """Arrivals per phase, and the programs of 2 K warps, 2 V warps, the softmax and the issuing warp over n tiles.

    (One row tile and two operand warps of four: one more is one more that may be late.)
    """
    counts = {(K_EMPTY, 0): 1, (K_FULL, 0): 4, (V_EMPTY, 0): 1, (V_FULL, 0): 2, (S_FULL, 0): 1, (P_READY, 0): 1}
    counts.update({(b, 1): c for (b, _), c in counts.items()})

    def empty(b, j):  # also: the phase of two tiles before
        return ("wait", (b, j & 1), ((j >> 1) & 1) ^ 1)

    def full(b, j):
        return ("wait", (b, j & 1), (j >> 1) & 1)

    programs = []
    for w in range(2):  # K operand
        steps = []
        for j in range(n):
            steps += [[empty(K_EMPTY, j), ("begin", ("kx", w, j & 3)), ("begin", ("k", w, j & 1))],
                      [("end", ("kx", w, j & 3), j), ("end", ("k", w, j & 1), j), ("arrive", (K_FULL, j & 1))]]
        programs.append(steps)
    for w in range(2):  # V operand
        steps = []
        for j in range(n):
            steps += [([empty(K_FULL, j)] if v_waits else []) + [("begin", ("vx", w, j & 3))],
                      [("end", ("vx", w, j & 3), j), ("arrive", (K_FULL, j & 1))],
                      [empty(V_EMPTY, j), ("begin", ("v", w, j & 1))],
                      [("end", ("v", w, j & 1), j), ("arrive", (V_FULL, j & 1))]]
        programs.append(steps)
    steps = []
    for j in range(n):  # softmax of both halves
        for h in range(2):
            steps += [[("wait", (S_FULL, h), j & 1), ("begin", ("p", h))],
                      [("read", ("kx", h, j & 3), j), ("read", ("vx", h, j & 3), j), ("end", ("p", h), j), ("arrive", (P_READY, h))]]
    programs.append(steps)

    def s(h, j):  # S of half h of tile j
        return [("issue", ("read", ("k", h, j & 1), j)), ("issue", ("arrive", (S_FULL, h)))]

    steps = [[full(K_FULL, 0)] + s(0, 0) + s(1, 0) + [("issue", ("arrive", (K_EMPTY, 0)))]]
    for j in range(n):
        more = j + 1 < n
        steps += [[full(V_FULL, j)]] + ([[full(K_FULL, j + 1)]] if more else [])
        for h in range(2):
            step = [("wait", (P_READY, h), j & 1), ("issue", ("read", ("v", h, j & 1), j)), ("issue", ("read", ("p", h), j))]
            if h:
                step += [("issue", ("arrive", (V_EMPTY, j & 1)))]
            if more:
                step += s(h, j + 1) + ([("issue", ("arrive", (K_EMPTY, (j + 1) & 1)))] if h else [])
            steps.append(step)
    programs.append(steps)
    return counts, programs


def walk(n, v_waits):
    """Every reachable state; the first fault found, or None if every way through ends with all roles done."""
    counts, programs = roles(n, v_waits)
    bars = {b: i for i, b in enumerate(sorted(counts))}
    places = {x: i for i, x in enumerate(sorted({op[1] for p in programs for step in p for op in step if op[0] == "begin"}, key=str))}
    issue = len(programs) - 1
    queue = [op[1] for step in programs[issue] for op in step if op[0] == "issue"]  # what the tensor pipe does, in order
    issued = [0]
    for step in programs[issue]:
        issued.append(issued[-1] + sum(op[0] == "issue" for op in step))
    pipe = len(programs)

    def apply(step, phases, mem):
        """The state after a step, None where it has to wait, or the fault as a string."""
        for op in step:
            if op[0] == "wait":
                if phases[bars[op[1]]][0] & 1 == op[2]:
                    return None
            elif op[0] == "arrive":
                i = bars[op[1]]
                phase, left = phases[i]
                phases = phases[:i] + ((phase + 1, counts[op[1]]) if left == 1 else (phase, left - 1),) + phases[i + 1:]
            elif op[0] in ("begin", "end"):
                i = places[op[1]]
                mem = mem[:i] + (None if op[0] == "begin" else op[2],) + mem[i + 1:]
            elif op[0] == "read" and mem[places[op[1]]] != op[2]:
                return f"{op[1]} is read for tile {op[2]} while it holds {mem[places[op[1]]]}"
        return phases, mem

    first = ((0,) * (pipe + 1), tuple((0, counts[b]) for b in bars), (None,) * len(places))
    seen, todo = {first}, [first]
    while todo:
        at, phases, mem = todo.pop()
        stuck = True
        for i in range(pipe + 1):
            if i == pipe:
                if at[i] == issued[at[issue]]:
                    continue
                after = apply([queue[at[i]]], phases, mem)
            elif at[i] < len(programs[i]):
                after = apply(programs[i][at[i]], phases, mem)
            else:
                continue
            if after is None:
                continue
            if isinstance(after, str):
                return after
            stuck = False
            state = (at[:i] + (at[i] + 1,) + at[i + 1:], *after)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if stuck and any(k < len(p) for k, p in zip(at, programs)):
            return f"no role can go on: {at}"
    return None


@pytest.mark.parametrize("n", [1, 2, 3, 5])
def test_every_order_of_the_roles_reads_what_was_written(n):
    assert walk(n, v_waits=True) is None


def test_the_walk_finds_an_arrival_in_another_ones_place():
    """Without the V warps' wait, theirs for tile 2 completes the phase of a K warp that has not written tile 0."""
    assert walk(2, v_waits=False) is None
    fault = walk(3, v_waits=False)
    assert fault is not None and "('k', " in fault
