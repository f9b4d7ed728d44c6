"""The hand-overs of one stream of the attention over a 4-bit cache, searched
exhaustively: every order in which its roles can come to their barriers.

A model of csrc/attn_kv4.cuh, on the CPU, with two warps to a warpgroup.  The roles of a
stream, and what each does for its tiles 0, 1, 2, .. in order:
  products  issues S(0), then S(n + 1), O(n) in turn within a segment, O of the last at its
            end; they complete in that order, later
  K         waits until S(n - 1) is complete, writes K(n), arrives
  V         waits until O(n - 1) is complete, writes V(n), arrives (the gathered form has one
            warpgroup for both, K first)
  softmax   waits for S(n), votes, may scale O once O(n - 1) is complete, writes P(n), arrives;
            after a segment's last tile waits for its O and reads it
An mbarrier is its count of completed phases; a wait names a parity only, and passes
where the phase under way has the other one."""
import pytest

WARPS = 2


def search(segments, gathered, weights=2, own_end=True):
    """What goes wrong in any order.  `weights`: barriers for V and P, one per buffer of P
    as built; `own_end`: whether a segment's end has a barrier of its own, as built."""
    total, ends = sum(segments), []
    issue = []                                     # of the tensor core, in order
    for m in segments:
        first = sum(segments[:len(ends)])
        issue += [("S", first)]
        for n in range(first + 1, first + m):
            issue += [("S", n), ("O", n - 1)]
        issue += [("O", first + m - 1)]
        ends.append(first + m)
    softmax = []
    for n in range(total):
        softmax += [("see", n)] + ([("scale", n)] if n and n not in ends else []) + [("weigh", n)]
        softmax += [("read", n)] if n + 1 in ends else []
    place = {op: i for i, op in enumerate(softmax)}
    passed = lambda phases, parity: phases & 1 != parity & 1
    count = lambda done, op: sum(o == op for o, _ in issue[:done])

    # issued, complete; tiles of K's and V's warps; softmax warps' places; the barriers of V and
    # P and the one of K and S, as (arrivals, phases)
    start = (0, 0, (0,) * WARPS, (0,) * WARPS, (0,) * WARPS, ((0, 0),) * weights, (1, 0))
    seen, todo, wrong = {start}, [start], set()

    def arrive(bar, expected):
        return (0, bar[1] + 1) if bar[0] + 1 == expected else (bar[0] + 1, bar[1])

    def weighed(bars, n):
        i = n % weights
        return bars[:i] + (arrive(bars[i], 2 * WARPS),) + bars[i + 1:]

    while todo:
        issued, done, k, v, at, pv, qk = state = todo.pop()
        scores, outputs = count(done, "S"), count(done, "O")
        after = []
        if done < issued:
            after.append((issued, done + 1, k, v, at, pv, qk))
        if issued < len(issue):
            op, n = issue[issued]
            if op == "S" and passed(qk[1], n):
                if min(k) <= n or any(x <= place["see", n - 1] for x in at if n):
                    wrong.add("S asked for early")
                after.append((issued + 1, done, k, v, at, pv, qk))
            if op == "O" and passed(pv[n % weights][1], n // weights):
                if any(x <= place["weigh", n] for x in at):
                    wrong.add("P missing")
                if min(v) <= n:
                    wrong.add("V missing")
                if n in ends and any(x <= place["read", n - 1] for x in at):
                    wrong.add("O lost")
                after.append((issued + 1, done, k, v, at, pv, qk))
        for w in range(WARPS):
            up = lambda t: t[:w] + (t[w] + 1,) + t[w + 1:]
            n = k[w]
            if n < total and (not gathered or v[w] == n) and passed(scores, n - 1):
                if scores < n:
                    wrong.add("K overwritten")
                after.append((issued, done, up(k), v, at, pv, arrive(qk, WARPS + 1)))
            n = v[w]
            if n < total and (not gathered or k[w] == n + 1) and passed(outputs, n - 1):
                if outputs < n:
                    wrong.add("V overwritten")
                after.append((issued, done, k, up(v), at, weighed(pv, n), qk))
            if at[w] == len(softmax):
                continue
            op, n = softmax[at[w]]
            if op == "see":
                # A vote: every warp is at it, or has been.
                if passed(scores, n) and all(x >= at[w] for x in at):
                    bar = arrive(qk, WARPS + 1) if min(up(at)) > at[w] else qk    # S is free
                    after.append((issued, done, k, v, up(at), pv, bar))
            elif op == "scale":
                after.append((issued, done, k, v, up(at), pv, qk))               # or not
                if passed(outputs, n - 1) and outputs != n:
                    wrong.add("O scaled at the wrong time")
            elif op == "weigh":
                if outputs < n - 1:
                    wrong.add("P overwritten")
                after.append((issued, done, k, v, up(at), weighed(pv, n), qk))
            elif passed(sum(e <= outputs for e in ends), ends.index(n + 1)) if own_end else passed(outputs, n):
                if outputs < n + 1:
                    wrong.add("O read early")
                after.append((issued, done, k, v, up(at), pv, qk))
        if not after and (issued < len(issue) or min(at) < len(softmax)):
            wrong.add("deadlock")
        todo += [s for s in after if s not in seen]
        seen.update(after)
    return wrong


SEGMENTS = [[1], [2], [5], [1, 3, 2], [4, 1, 1, 3], [1, 1, 1, 1], [2, 2, 2]]


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("segments", SEGMENTS)
def test_every_order_of_the_hand_overs_is_sound(segments, gathered):
    assert search(segments, gathered) == set()


def test_the_search_finds_missing_waits():
    """One barrier for both buffers of weights lets the softmax stand in for V; without
    one of its own a segment's end is taken for that of the tile before."""
    assert {"V missing", "deadlock"} <= search([4, 3], False, weights=1)
    assert "O read early" in search([4, 3], False, own_end=False)
