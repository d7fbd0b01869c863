"""The hand-over of the activations' buffers in the few-token experts layer, replayed on the host in every order that
its waits allow (no GPU): coders fill a buffer, issuers and promotion read it, and all of them tell its turns apart by
the parity of two barriers."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_scaled_fp8_gb300", "csrc",
                      "moe_mlp.cu")
ISSUERS = 2


def counted_readers():
    """Promotion's warps and issuers that a buffer's refill waits for, as the kernel initialises its barrier."""
    text = open(SOURCE).read()
    names = {"kIssuers": int(re.search(r"kIssuers = (\d+);", text).group(1))}
    count = re.search(r"mbar_init\(hempty0 \+ 8 \* i, ([^)]+)\);", text).group(1)
    if count in (named := dict(re.findall(r"constexpr int (\w+) = ([^;]+);", text))):
        count = named[count]
    return 4, eval(count, {}, names) - 4


class Barrier:
    """(phases completed, arrivals in the running one) of a barrier of `count` arrivals."""

    def __init__(self, count):
        self.count = count

    def arrive(self, state):
        phases, arrived = state
        return (phases + 1, 0) if arrived + 1 == self.count else (phases, arrived + 1)


def passes(phases, awaited):
    """What a wait by parity answers for phase `awaited`, and whether it is right to."""
    answer = (phases - awaited) % 2 == 1
    assert not answer or phases > awaited, "a wait took an older phase for its own"
    return answer


def replay(buffers, experts, stages, first, product_bufs, promotion, issuers_counted):
    """Explores every order.  stages: of an expert; first: stages before the second part (their parity decides whose the
    next one is).  Returns the states in which nobody can go on although not all is done."""
    teams = 1 if buffers <= 2 else 3 if buffers < 6 else 6
    empty = Barrier(promotion + issuers_counted)
    # coder teams' next expert; issuers' (expert, stage, seen); promotion's (expert, stage, seen); full phases a buffer; empty
    # (phases, arrivals) a buffer; products issued, products released by each warp of promotion
    start = (tuple(range(teams)), ((0, 0, False),) * ISSUERS, ((0, 0, False),) * promotion, (0,) * buffers, ((0, 0),) * buffers,
             ())
    seen, todo, stuck = {start}, [start], []

    def put(t, i, v):
        return t[:i] + (v,) + t[i + 1:]

    def moves(state):
        coders, issuers, warps, full, empties, issued = state
        for i, r in enumerate(coders):  # fill expert r's buffer
            if r < experts and passes(empties[r % buffers][0], r // buffers - 1):
                yield (put(coders, i, r + teams), issuers, warps, put(full, r % buffers, full[r % buffers] + 1), empties, issued)
        for i, (r, j, saw) in enumerate(issuers):
            if r == experts:
                continue
            if not saw:
                if passes(full[r % buffers], r // buffers):
                    e = put(empties, r % buffers, empty.arrive(empties[r % buffers])) if issuers_counted else empties
                    yield (coders, put(issuers, i, (r, j, True)), warps, full, e, issued)
                continue
            n = r * stages + j
            nxt = (r, j + 1, True) if j + 1 < stages else (r + 1, 0, False)
            if (first + n) % ISSUERS != i:
                yield (coders, put(issuers, i, nxt), warps, full, empties, issued)
            elif all(w[0] * stages + w[1] > n - product_bufs for w in warps):  # its product buffer was released
                yield (coders, put(issuers, i, nxt), warps, full, empties, tuple(sorted(issued + (n,))))
        for i, (r, j, saw) in enumerate(warps):
            if r == experts:
                continue
            if not saw:
                if passes(full[r % buffers], r // buffers):
                    yield (coders, issuers, put(warps, i, (r, j, True)), full, empties, issued)
            elif r * stages + j in issued:
                if j + 1 < stages:
                    yield (coders, issuers, put(warps, i, (r, j + 1, True)), full, empties, issued)
                else:
                    e = put(empties, r % buffers, empty.arrive(empties[r % buffers]))
                    yield (coders, issuers, put(warps, i, (r + 1, 0, False)), full, e, issued)

    while todo:
        state = todo.pop()
        coders, issuers, warps, full, empties, issued = state
        low = min(w[0] * stages + w[1] for w in warps)  # (products that all of promotion has taken are forgotten)
        following = [s[:5] + (tuple(n for n in s[5] if n >= low),) for s in moves(state)]
        if not following and not (all(r >= experts for r in coders) and all(x[0] == experts for x in issuers + warps)):
            stuck.append(state)
        for s in following:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stuck


@pytest.mark.parametrize("buffers,stages", [(1, 1), (1, 2), (2, 1), (2, 3), (3, 1), (3, 2), (5, 1), (6, 1), (8, 1)])
@pytest.mark.parametrize("first", [0, 1])
def test_no_order_of_the_waits_ends_in_one_for_good(buffers, stages, first):
    promotion, issuers = counted_readers()
    assert promotion == 4 and issuers in (0, ISSUERS)
    experts = min(2 * buffers + 1, buffers + 4)
    # two warps of promotion stand for the four: a phase ends with the last of them either way
    assert not replay(buffers, experts, stages, first, 4, 1 if buffers > 3 else 2, issuers)


def test_the_replay_sees_a_reader_that_is_not_counted():
    """An expert of one stage is one issuer's: the other, held up, finds the next turn's parity."""
    assert replay(2, 5, 1, 0, 4, 2, 0) and not replay(2, 5, 1, 0, 4, 2, ISSUERS)
