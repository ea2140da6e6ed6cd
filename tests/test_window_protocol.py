"""The barriers of the tcgen05 window attention forward (csrc/window_tc.cu) in a
model: row warps, the thread that issues the matrix instructions and the matrix
pipe, in every order in which their steps can happen.

Scores of tile t go to buffer t & 1 as soon as P(t - 2) V is done there; a warp
turns its rows of the buffer into probabilities and arrives; P(t) V is issued when
all warps of the tile have arrived.  A barrier is the number of its completed phases
and the arrivals of the present one; a wait by parity passes where the present
phase's parity differs."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "protein_structure_models_b200", "csrc",
                      "window_tc.cu")


def explore(barriers, tiles, warps):
    """(wrong reads, states without an end) with that many barriers for the warps' arrivals, used in turn."""
    def passes(phases, k):
        return (phases & 1) != (k & 1)

    def put(x, k, v):
        return x[:k] + (v,) + x[k + 1:]

    # rows' (tile, whether S was read), issuer's (tile, whether S(t + 1) was issued), issued operations,
    # completed phases of S and of P V, (phases, arrivals) of the rows' barriers, what each warp's rows of the buffers hold
    start = (((0, 0),) * warps, (0, 0), (("S", 0),), (0, 0), (0, 0), ((0, 0),) * barriers, ((None,) * warps,) * 2)
    seen, todo, wrong, stuck = {start}, [start], set(), set()
    while todo:
        state = todo.pop()
        row, (it, issued), pipe, s_full, pv_done, p_full, buf = state
        then = []
        if pipe:
            (op, t), rest, b = pipe[0], pipe[1:], pipe[0][1] & 1
            if op == "S":
                then.append((row, (it, issued), rest, put(s_full, b, s_full[b] + 1), pv_done, p_full, put(buf, b, (("S", t),) * warps)))
            else:
                wrong |= {("P V", t, x) for x in buf[b] if x != ("P", t)}
                then.append((row, (it, issued), rest, s_full, put(pv_done, b, pv_done[b] + 1), p_full, buf))
        if it < tiles and not issued:
            if it + 1 >= tiles:
                then.append((row, (it, 1), pipe, s_full, pv_done, p_full, buf))
            elif it == 0 or passes(pv_done[(it - 1) & 1], (it - 1) >> 1):
                then.append((row, (it, 1), pipe + (("S", it + 1),), s_full, pv_done, p_full, buf))
        elif it < tiles and passes(p_full[it % barriers][0], it // barriers):
            then.append((row, (it + 1, 0), pipe + (("V", it),), s_full, pv_done, p_full, buf))
        for w, (t, read) in enumerate(row):
            if t >= tiles:
                continue
            if not read:
                if passes(s_full[t & 1], t >> 1):
                    if buf[t & 1][w] != ("S", t):
                        wrong.add(("row", t, buf[t & 1][w]))
                    then.append((put(row, w, (t, 1)), (it, issued), pipe, s_full, pv_done, p_full, buf))
            else:
                phases, n = p_full[t % barriers]
                arrived = (phases + 1, 0) if n + 1 == warps else (phases, n + 1)
                then.append((put(row, w, (t + 1, 0)), (it, issued), pipe, s_full, pv_done, put(p_full, t % barriers, arrived),
                             put(buf, t & 1, put(buf[t & 1], w, ("P", t)))))
        if not then and (it < tiles or any(t < tiles for t, _ in row)):
            stuck.add(state)
        for x in then:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return wrong, stuck


@pytest.mark.parametrize("tiles,warps", [(1, 2), (2, 3), (7, 2), (5, 3), (5, 4)])
def test_the_barriers_of_the_source_suffice(tiles, warps):
    inits = re.findall(r"for \(int s = 0; s < (\d+); \+\+s\) \{[^}]*mbar_init\(&p_full\[s\], kFinish\)", open(SOURCE).read())
    barriers = int(inits[0]) if inits else 1
    assert explore(barriers, tiles, warps) == (set(), set())


def test_one_barrier_does_not():
    """A warp a tile ahead arrives for one that is behind: scores are read as probabilities, or a phase is missed for good."""
    wrong, stuck = explore(1, 5, 2)
    assert any(op == "P V" and x[0] == "S" for op, _, x in wrong) and stuck
