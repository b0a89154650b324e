"""How blocks of one launch that wait for one another count arrivals (csrc/meet.h), under
every order that a random scheduler finds: the header's own rules, compiled for the host."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routed_relu_expert_gb300", "csrc")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("meet")
    src, lib = str(d / "meet.cpp"), str(d / "meet.so")
    with open(src, "w") as f:
        f.write('#include "meet.h"\nextern "C" {\nint word(int n) { return moe::meet_word(n); }\n'
                "int count(int n, int b) { return moe::meet_count(n, b); }\nint words() { return moe::kMeetWords; }\n"
                "int state(int seen, int n, int b) { return moe::meet_state(seen, n, b); }\n"
                "int gave_up() { return moe::kMeetGaveUp; }\n}\n")
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


class OneWord:
    """All arrivals in one word: what the rules must not be."""
    words = staticmethod(lambda: 1)
    word = staticmethod(lambda n: 0)
    count = staticmethod(lambda n, b: (n + 1) * b)


def program(meetings, ahead):
    """A block's steps: come to each meeting with its part of it done, wait for it, use what the others did.
    Ahead: it comes to the next one before it waits, as the waves of a long list do."""
    if not ahead:
        return [s for n in range(meetings) for s in (("come", n), ("wait", n), ("use", n))]
    return [("come", 0)] + [s for n in range(meetings) for s in (("come", n + 1), ("wait", n), ("use", n))]


def early(rules, blocks, meetings, ahead, seed):
    """Uses of a meeting before all blocks had come to it, over one random order of all steps."""
    rng = random.Random(seed)
    steps = program(meetings, ahead)
    met, came, at, found = [0] * rules.words(), [0] * blocks, [0] * blocks, 0
    # blocks of very different speeds, some of them asleep for a while
    speed = [rng.choice((1.0, 1.0, 0.3, 0.01)) for _ in range(blocks)]
    left = set(range(blocks))
    while left:
        moved = False
        for b in rng.sample(sorted(left), len(left)):
            if rng.random() > speed[b] and (moved or len(left) > 1):
                continue
            what, n = steps[at[b]]
            if what == "wait" and met[rules.word(n)] < rules.count(n, blocks):
                continue
            if what == "come":
                assert came[b] == n
                came[b] += 1
                met[rules.word(n)] += 1
            elif what == "use":
                found += min(came) <= n
            moved = True
            at[b] += 1
            if at[b] == len(steps):
                left.discard(b)
        if not moved:                                        # nobody but sleepers could: wake one, or all wait for ever
            ready = [b for b in left if steps[at[b]][0] != "wait"
                     or met[rules.word(steps[at[b]][1])] >= rules.count(steps[at[b]][1], blocks)]
            assert ready, "every block waits"
            speed[rng.choice(ready)] = 1.0
    return found


@pytest.mark.parametrize("blocks", [1, 2, 3, 20, 152])
@pytest.mark.parametrize("ahead", [False, True])
def test_nobody_passes_a_meeting_that_a_block_has_not_come_to(rules, blocks, ahead):
    for meetings in (1, 2, 3, 7, 25):
        for seed in range(40 if blocks < 20 else 4):
            assert early(rules, blocks, meetings, ahead, seed) == 0


def test_one_word_for_all_meetings_would_be_found():
    """A block that is one meeting ahead stands for one that has not come."""
    assert sum(early(OneWord, 2, 1, True, seed) for seed in range(40)) > 0
    assert sum(early(OneWord, 20, 5, True, seed) for seed in range(5)) > 0
    assert sum(early(OneWord, 20, 5, False, seed) for seed in range(5)) == 0     # (nobody ahead: one word is enough)


WAIT, MET, ENDED = range(3)


def outcomes(rules, blocks, meetings, seed, swap=True):
    """Of each block: what its waits came to, over one random order of steps in which waits may give up.  A block
    ends with its first wait that fails.  swap: a word is marked by compare-and-swap; else each block goes by
    the time alone."""
    rng = random.Random(seed)
    mark = rules.gave_up()
    met, got = [0] * rules.words(), [[] for _ in range(blocks)]
    came, seen = [False] * blocks, [None] * blocks           # at the meeting len(got[b]); what was read of its word
    left = set(range(blocks))
    for _ in range(400 * blocks * meetings):
        if not left:
            break
        b = rng.choice(sorted(left))
        n = len(got[b])
        w, state = rules.word(n), None
        if not came[b]:
            if rng.random() < 0.3:
                met[w] += 1
                came[b] = True
        elif seen[b] is None:                                # a look at the word
            state = rules.state(met[w], n, blocks)
            seen[b] = met[w] if state == WAIT else None
        elif rng.random() < 0.05:                            # it has taken too long
            if not swap:
                state = ENDED
            elif met[w] == seen[b]:
                met[w] |= mark
            seen[b] = None
        else:
            seen[b] = None
        if state in (MET, ENDED):
            got[b].append(state)
            came[b] = False
            if state == ENDED or len(got[b]) == meetings:
                left.discard(b)
    assert not left, "a block waits for ever"
    return got


@pytest.mark.parametrize("blocks", [2, 3, 20, 152])
def test_a_meeting_ends_in_one_way_for_all(rules, blocks):
    """A release either changes the table and the list in all of its blocks or in none."""
    ends = set()
    for seed in range(300 if blocks < 20 else 20 if blocks < 152 else 2):
        got = outcomes(rules, blocks, 3, seed)
        assert all(g == got[0] for g in got), seed
        ends.add(tuple(got[0]))
    assert len(ends) > 1 or blocks > 3                       # (some of them met three times, some gave up)


def test_waits_that_give_up_by_themselves_would_be_found(rules):
    assert any(any(g != got[0] for g in got) for got in (outcomes(rules, 3, 3, seed, swap=False) for seed in range(100)))


def test_the_mark_is_above_every_count(rules):
    for number, blocks in ((0, 1), (0, 152), (200_000, 152)):
        n = rules.count(number, blocks)
        assert 0 < n < rules.gave_up()
        assert [rules.state(x, number, blocks) for x in (n - 1, n, n + 1, (n - 1) | rules.gave_up(), n | rules.gave_up())] == [
            WAIT, MET, MET, ENDED, ENDED]
