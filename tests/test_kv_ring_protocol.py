"""The cache attention's ring of records that two warps share (17 and more query columns), checked on the CPU.

Both warps of a group walk the same pages.  A page lies in stage u % stages; both release it there, and the first warp
refills a stage one page after its own last use of it.  Pages whose id is out of range are not copied: nothing but
the ring's "free" barriers then holds a warp back, and their phase parity cannot tell a phase from the next but one.  So
every warp waits until both have released the page before, not the refilling one alone.  The model replays that
with mbarrier parity semantics, copies that land at any time and warps at any relative speed."""
import os
import random
import re

import pytest

KV = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_q4_gb300", "csrc", "q4_kv.cu")
STAGES, MEMBERS = 6, 2


def replay(there, all_wait, rng, eager=None, max_steps=200000):
    """None, or what went wrong.  ``there[u]``: page u is copied; ``eager``: a member that runs whenever it can."""
    n = len(there)
    copied, landing = [0] * STAGES, []          # completed phases; pages on their way
    free, arrived = [0] * STAGES, [0] * STAGES
    landed, released = set(), [set() for _ in range(MEMBERS)]
    issued = [0]
    error = []

    def passed(done, parity):
        return (done & 1) != parity

    def issue(member):                           # (every member keeps the books, the first one copies)
        u = issued[0]
        if member == 0 and u < n:
            old = u - STAGES
            if old >= 0 and any(old not in r for r in released):
                error.append(f"stage {u % STAGES} refilled for page {u} before page {old} was released")
            if there[u]:
                landing.append(u)
            issued[0] += 1

    def walk(member):
        phases, filled = [0] * STAGES, min(n, STAGES)
        for u in range(n):
            s = u % STAGES
            if there[u]:
                while not passed(copied[s], phases[s]):
                    yield False
                phases[s] ^= 1
                if u not in landed:
                    error.append(f"member {member} read page {u} before it landed")
            yield True
            released[member].add(u)
            arrived[s] += 1
            if arrived[s] == MEMBERS:
                arrived[s] = 0
                free[s] += 1
            yield True
            b = u - 1
            if b >= 0:
                if (member == 0 or all_wait) and filled < n:
                    while not passed(free[b % STAGES], (b // STAGES) & 1):
                        yield False
                    if any(b not in r for r in released):
                        error.append(f"member {member} passed the wait for page {b} before it was released")
                if filled < n:
                    issue(member)
                    filled += 1

    for _ in range(min(n, STAGES)):
        issue(0)
    walks = {m: walk(m) for m in range(MEMBERS)}
    waiting = set()                              # members that have polled in vain since anything last happened
    for _ in range(max_steps):
        if error:
            return error[0]
        if not walks:
            return None
        if landing and (rng.random() < 0.5 or waiting == set(walks)):
            u = landing.pop(rng.randrange(len(landing)))
            landed.add(u)
            copied[u % STAGES] += 1
            waiting.clear()
            continue
        m = eager if eager in walks and rng.random() < 0.98 else rng.choice(sorted(walks))
        try:
            waiting = set() if next(walks[m]) else waiting | {m}
        except StopIteration:
            del walks[m]
            waiting = set()
        if walks and waiting == set(walks) and not landing:
            return "a warp waits for a phase that nothing completes"
    return "no end"


def tables():
    rng = random.Random(3)
    yield [True] * 50
    yield [False] * 60
    yield [False] * 40 + [True] * 3                     # freed leading pages
    yield [True] * 4 + [False] * 13 + [True]            # two rounds of the ring, then a page that only the first warp copies
    yield [True] + [False] * 37
    for n in (1, 2, 5, 6, 7, 13, 80):
        yield [rng.random() < 0.3 for _ in range(n)]
    runs = []
    while len(runs) < 300:
        runs += [False] * rng.randint(12, 40) + [True] * rng.randint(1, 4)
    yield runs


@pytest.mark.parametrize("there", tables(), ids=lambda t: f"{len(t)}-{sum(t)}")
@pytest.mark.parametrize("eager", [None, 0, 1])
def test_a_ring_whose_members_all_wait_is_safe(there, eager):
    rng = random.Random(len(there))
    for _ in range(10):
        assert replay(there, True, rng, eager) is None


def test_a_ring_whose_first_member_alone_waits_is_not():
    """The model is sharp enough to see it: a run of missing pages lets the other warp complete a phase too many."""
    rng = random.Random(1)
    bad = [replay([True] * 4 + [False] * 13 + [True] * 3 + [False] * 30 + [True], False, rng, 1) for _ in range(20)]
    assert any(bad)
    assert all(replay([True] * 60, False, rng, 1) is None for _ in range(5))    # (without missing pages it is held back by the copies)


def test_the_kernel_lets_every_member_wait():
    with open(KV) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    ring = text[text.index("q4_kv_attention_kernel(const KvParams p)"):text.index("kv_finish_state(st);\n    if (!ok)")]
    wait = re.search(r"if \(([^()]*)\) \{\s*ok = kv_wait\([^;]*\(b % kStages\) \+ 8,", ring)
    assert wait and wait.group(1).strip() == "next < u1", wait and wait.group(1)
