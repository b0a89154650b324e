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
                "int count(int n, int b) { return moe::meet_count(n, b); }\nint words() { return moe::kMeetWords; }\n}\n")
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
