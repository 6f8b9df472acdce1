"""Host-side models, run under random interleavings, of the barrier protocols of
csrc/mx4_gemm.cu (the mx4 product on CTA pairs) and of the decoder groups of
csrc/tc_gemm.cu.

mx4_gemm_kernel, one step at a time, a ring of STAGES stages and SLOTS places for
scales in tensor memory:
- the producers of both CTAs wait for their own empty[s]; the even one arms full[s]
  with both CTAs' bytes; the copies of both count there and land in any order;
- the scale warp (even CTA) waits for full[s] and, from the SLOTS-th block on, for
  the empty[] of the block SLOTS back, copies the scales to slot n % SLOTS and
  commits sfull[s];
- the MMA warp waits for tempty, then per block for full[s] and sfull[s], issues and
  commits empty[s] of both CTAs; after a tile's last block it commits tfull of both;
- eight epilogue warps (four per CTA) wait for tfull and arrive on tempty.
Checked: every MMA reads its own block's operands and scales, no copy overwrites a
stage or a slot in use, every accumulator is complete when it is read and not
rewritten before, nothing deadlocks.  Commits of one warp arrive in issue order.
"""

import random

import pytest

from tests.test_tc_gemm_protocol_model import Bar

STAGES, SLOTS, EPI = 6, 5, 8


def drive(actors, landings, commit_queues, rng, what):
    waits, alive = [None] * len(actors), list(range(len(actors)))
    while alive or landings or any(commit_queues):
        ready = [("step", i) for i in alive if waits[i] is None or waits[i]()]
        ready += [("land", j) for j in range(len(landings))]
        ready += [("commit", q) for q, c in enumerate(commit_queues) if c]
        assert ready, f"deadlock: {what}"
        kind, i = rng.choice(ready)
        if kind == "land":
            landings.pop(i)()
        elif kind == "commit":
            commit_queues[i].pop(0)()
        else:
            try:
                waits[i] = next(actors[i])
            except StopIteration:
                alive.remove(i)


def run(ntiles, kblocks, seed, slot_wait=SLOTS, mma_waits_scales=True, tempty_count=EPI,
        odd_waits_empty=True):
    rng = random.Random(seed)
    full, sfull = [Bar(1) for _ in range(STAGES)], [Bar(1) for _ in range(STAGES)]
    empty = [[Bar(1) for _ in range(STAGES)] for _ in range(2)]
    tfull, tempty = [[Bar(1) for _ in range(2)] for _ in range(2)], [Bar(tempty_count) for _ in range(2)]
    held = [[None] * STAGES for _ in range(2)]   # block whose operands a CTA's stage holds
    slots = [None] * SLOTS                       # block whose scales a slot holds
    reading = set()                              # blocks whose MMAs have not completed
    dbuf, reads = [None] * 2, [0] * 2
    landings, mma_commits, scale_commits, consumed = [], [], [], []
    total = ntiles * kblocks

    def producer(cta):
        for n in range(total):
            s, ph = n % STAGES, (n // STAGES) & 1
            if cta == 0 or odd_waits_empty:
                yield lambda s=s, ph=ph: empty[cta][s].done(ph ^ 1)
            if cta == 0:
                # the odd CTA's bytes may already have been counted
                full[s].tx += 2
                full[s].arrive()

            def land(s=s, n=n):
                assert n - STAGES not in reading, "a copy overwrites a stage the MMAs still read"
                held[cta][s] = n
                full[s].tx -= 1
                full[s]._advance()
            landings.append(land)

    def scales():
        for n in range(total):
            s, ph = n % STAGES, (n // STAGES) & 1
            yield lambda s=s, ph=ph: full[s].done(ph)
            old = n - slot_wait
            if old >= 0:
                yield lambda old=old: empty[0][old % STAGES].done((old // STAGES) & 1)
            assert held[0][s] == held[1][s] == n
            assert n - SLOTS not in reading, "scales overwritten while the MMAs read them"
            slots[n % SLOTS] = n
            scale_commits.append(lambda s=s: sfull[s].arrive())

    def mma():
        n = 0
        for local in range(ntiles):
            buf = local & 1
            yield lambda buf=buf, local=local: tempty[buf].done(((local >> 1) & 1) ^ 1)
            if local >= 2:
                assert reads[buf] == EPI, "accumulator rewritten before the epilogues read it"
            dbuf[buf], reads[buf] = (local, False), 0
            for _ in range(kblocks):
                s, ph = n % STAGES, (n // STAGES) & 1
                yield lambda s=s, ph=ph: full[s].done(ph)
                if mma_waits_scales:
                    yield lambda s=s, ph=ph: sfull[s].done(ph)
                assert held[0][s] == held[1][s] == n and slots[n % SLOTS] == n, "operands or scales of another block"
                reading.add(n)
                consumed.append(n)

                def release(s=s, n=n):
                    reading.discard(n)
                    empty[0][s].arrive()
                    empty[1][s].arrive()
                mma_commits.append(release)
                n += 1

            def finish(buf=buf, local=local):
                dbuf[buf] = (local, True)
                for cta in range(2):
                    tfull[cta][buf].arrive()
            mma_commits.append(finish)

    def epilogue(cta):
        for local in range(ntiles):
            buf = local & 1
            yield lambda buf=buf, local=local: tfull[cta][buf].done((local >> 1) & 1)
            assert dbuf[buf] == (local, True)
            reads[buf] += 1
            tempty[buf].arrive()

    drive([producer(0), producer(1), scales(), mma()] + [epilogue(c) for c in (0, 1) for _ in range(4)],
          landings, [mma_commits, scale_commits], rng, f"{ntiles} tiles x {kblocks}")
    assert consumed == list(range(total))


def cases(n):
    rng = random.Random(11 * n)
    for seed in range(n):
        yield rng.randint(1, 5), rng.choice([1, 2, 3, 5, 6, 7, 16, 40]), seed


def test_pair_product_consumes_every_block_without_deadlock():
    for ntiles, kblocks, seed in cases(150):
        run(ntiles, kblocks, seed)


@pytest.mark.parametrize("mutation", [
    dict(slot_wait=SLOTS + 1),        # a slot rewritten one block early
    dict(mma_waits_scales=False),
    dict(tempty_count=4),             # one CTA's epilogue releases the accumulator
    dict(odd_waits_empty=False),
])
def test_the_pair_model_catches_a_broken_protocol(mutation):
    caught = False
    for ntiles, kblocks, seed in cases(150):
        try:
            run(ntiles, kblocks, seed, **mutation)
        except AssertionError:
            caught = True
            break
    assert caught


def test_drain_after_a_wait_that_gave_up():
    """The CTAs stop after different numbers of stages (both within one ring of what
    the MMAs have released).  The even CTA makes up for the bytes of stages that only
    one of them issued; when its waits are done no copy is in flight in either."""
    rng = random.Random(5)
    for _ in range(2000):
        done = rng.randint(0, 9)                       # blocks consumed by MMAs
        issued = [done + rng.randint(0, STAGES) for _ in range(2)]
        full = [Bar(1) for _ in range(STAGES)]
        flight = []

        def land(s):
            full[s].tx -= 1
            full[s]._advance()
        for n in range(max(issued)):                   # arming and issuing, in order
            s = n % STAGES
            if n < issued[0]:
                full[s].tx += 2
                full[s].arrive()
            for cta in range(2):
                if n < issued[cta]:
                    if n < done or rng.random() < 0.5:
                        land(s)
                    else:
                        flight.append(s)
        a, b = issued
        for n in range(b, a):                          # bytes that the odd CTA never sends
            land(n % STAGES)
        for n in range(a, b):                          # stages that the even CTA never armed
            full[n % STAGES].tx += 1
            full[n % STAGES].arrive()
        most = max(issued)
        pending = [n for n in range(max(0, most - STAGES), most)]
        while flight:
            waiting = [n for n in pending if not full[n % STAGES].done((n // STAGES) & 1)]
            assert waiting, "the waits are done while a copy is in flight"
            land(flight.pop(rng.randrange(len(flight))))
        assert all(full[n % STAGES].done((n // STAGES) & 1) for n in pending)


def run_groups(ntiles, kblocks, groups, seed, own_turn=True):
    """tc_gemm_kernel with `groups` decoder groups of four warps on alternate k blocks
    and a ring of four stages: a group waits only for the stages of its own blocks."""
    rng = random.Random(seed)
    S, total = 4, ntiles * kblocks
    full, empty, decd = ([Bar(c) for _ in range(S)] for c in (1, 1, 4))
    held, decoded, in_use = [None] * S, [[None] * 4 for _ in range(S)], [None] * S
    landings, commits, consumed = [], [], []

    def producer():
        for n in range(total):
            s, ph = n % S, (n // S) & 1
            yield lambda s=s, ph=ph: empty[s].done(ph ^ 1)
            full[s].arrive_expect_tx(1)

            def land(s=s, n=n):
                assert in_use[s] is None
                held[s] = n
                full[s].complete_tx(1)
            landings.append(land)

    def decoder(g, w):
        for n in range(total):
            if n % groups != (g if own_turn else 0):
                continue
            s, ph = n % S, (n // S) & 1
            yield lambda s=s, ph=ph: full[s].done(ph)
            assert held[s] == n and in_use[s] is None
            decoded[s][w] = n
            decd[s].arrive()

    def mma():
        for n in range(total):
            s, ph = n % S, (n // S) & 1
            yield lambda s=s, ph=ph: decd[s].done(ph)
            assert held[s] == n and all(d == n for d in decoded[s])
            in_use[s] = n
            consumed.append(n)

            def release(s=s):
                in_use[s] = None
                empty[s].arrive()
            commits.append(release)

    drive([producer(), mma()] + [decoder(g, w) for g in range(groups) for w in range(4)], landings, [commits],
          rng, f"{groups} groups")
    assert consumed == list(range(total))


@pytest.mark.parametrize("groups", [1, 2, 4])
def test_decoder_groups(groups):
    for ntiles, kblocks, seed in cases(80):
        run_groups(ntiles, kblocks, groups, seed)


def test_three_groups_on_four_stages_are_caught():
    """A group that waits for a stage whose earlier phases belong to others can take
    an older phase of the same parity for its own."""
    with pytest.raises(AssertionError):
        for ntiles, kblocks, seed in cases(80):
            run_groups(ntiles, kblocks, 3, seed)


def test_decoder_groups_that_share_a_block_are_caught():
    with pytest.raises(AssertionError):
        for ntiles, kblocks, seed in cases(20):
            run_groups(ntiles, kblocks, 2, seed, own_turn=False)
