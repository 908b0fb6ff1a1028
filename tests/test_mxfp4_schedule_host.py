"""A replay on the CPU of the MXFP4 GEMM loops' loads, waits, barriers and
reads (the ping-pong loop of full tiles and the ring of the tail tiles, as
csrc/gemm_mxfp4.hip issues them).  Per wave, memory operations complete in
issue order and a wait for at most n outstanding ones completes all but the
last n.  Checked: what a tick reads was waited for by the group that loaded it
at an earlier tick's end, and a stage is loaded only after the last read of
what it held.  Wrong waits and early loads, planted here, are caught."""
import pytest


class Bad(Exception):
    pass


def replay_pp(nk, wait_extra=1, scale_tick_shift=0, drop_wait=False):
    """The ping-pong loop over nk K-steps.  wait_extra: how many more operations than the 4 code
    loads may stay outstanding when the scales went out in the same tick."""
    H = 2 * nk
    queue = {0: [], 1: []}           # per group: outstanding operations, oldest first
    done = {}                        # item -> tick whose barrier publishes it
    last_read = {}                   # item -> last tick that reads it
    held = {}                        # stage -> item

    def issue(g, t, item, stage, n):
        if stage in held and last_read.get(held[stage], -99) >= t:
            raise Bad(f"{item} overwrites {held[stage]} at tick {t}")
        held[stage] = item
        queue[g] += [item] * n

    def wait(g, t, n):
        q = queue[g]
        keep = q[len(q) - n:] if n else []
        for item in q[:len(q) - n] if n else q:
            if item not in keep:
                done.setdefault(item, t)
        queue[g] = keep

    def codes(g, t, which, j):
        issue(g, t, (which, j), (which, j & 1), 4)

    def scales(g, t, c):
        which = "As" if g == 0 else "Bs"
        issue(g, t, (which, c), (which, c & 1), 1)

    # A halves: a0 by group 0, a1 by group 1; B halves: b1 by group 0, b0 by group 1
    mine = {0: ("a0", "b1"), 1: ("a1", "b0")}
    for g in (0, 1):
        scales(g, -9, 0)
        for w in mine[g]:
            codes(g, -9, w, 0)
        if nk > 1:
            for w in mine[g]:
                codes(g, -9, w, 1)
        wait(g, -1, 8 if nk > 1 else 0)

    def read(g, t, hs):
        j, c = hs >> 1, hs >> 2
        for item in ((f"a{g}", j), ("b0", j), ("b1", j), ("As", c), ("Bs", c)):
            if done.get(item, 1 << 30) >= t:
                raise Bad(f"group {g} reads {item} at tick {t}, published {done.get(item)}")
            if held[(item[0], item[1] & 1)] != item:
                raise Bad(f"group {g} reads {item} at tick {t}: overwritten")
            last_read[item] = t

    def loads(g, t):
        def sc(j):
            if (j + scale_tick_shift) % 2 == 0 and (j + scale_tick_shift) // 2 * 2 < nk:
                scales(g, t, (j + scale_tick_shift) // 2)
        if g == 0:
            if t & 3 == 1:
                j = (t + 7) >> 2
                if 2 <= j < nk:
                    sc(j)
                    codes(0, t, "a0", j)
            else:
                assert t & 3 == 3
                j = (t + 5) >> 2
                if 2 <= j < nk:
                    codes(0, t, "b1", j)
        elif t & 3 == 2:
            j = (t + 6) >> 2
            if 2 <= j < nk:
                sc(j)
                codes(1, t, "b0", j)
        else:
            assert t & 3 == 0
            j = (t + 4) >> 2
            if 2 <= j < nk:
                codes(1, t, "a1", j)

    def end(g, t):
        if drop_wait:
            return
        if t & 3 == 1:
            j = (t + 3) >> 2
            jn = j + 1 if g == 0 else j
            wait(g, t, 0 if jn < 2 or jn >= nk else (4 + wait_extra if g == 0 and jn % 2 == 0 else 4))
        elif t & 3 == 2 and g == 1:
            jn = ((t + 2) >> 2) + 1
            wait(g, t, 0 if jn < 2 or jn >= nk else (4 + wait_extra if jn % 2 == 0 else 4))

    read(0, 0, 0)
    multiplied = {0: 0, 1: 0}
    for t in range(2 * H):
        for g in (0, 1):
            if t % 2 == g:                       # compute tick of half K-step (t - g) / 2
                hs = (t - g) // 2
                multiplied[g] += 1
                if hs + 1 < H:
                    read(g, t, hs + 1)
            elif g == 1 and t == 0:
                loads(1, 0)
                read(1, 0, 0)
            else:
                loads(g, t)
        for g in (0, 1):
            end(g, t)
    assert multiplied == {0: H, 1: H}


def replay_ring(nk, ahead=2, stages=3, extra=1):
    queue, done, held, last_read = [], set(), {}, {}

    def issue(kt, at):
        if kt % 2 == 0:
            put(("s", kt // 2), ("s", kt // 2 % 2), 1, at)
        put(("k", kt), ("k", kt % stages), 5, at)

    def put(item, stage, n, at):
        if stage in held and last_read.get(held[stage], -9) >= at:
            raise Bad(f"{item} overwrites {held[stage]}")
        held[stage] = item
        queue.extend([item] * n)

    for j in range(ahead):
        issue(j, -1)
    for kt in range(nk):
        n = 5 + extra if kt % 2 else 5
        for item in queue[:len(queue) - n]:
            done.add(item)
        del queue[:len(queue) - n]
        issue(kt + ahead, kt)
        for item, stage in ((("k", kt), ("k", kt % stages)), (("s", kt // 2), ("s", kt // 2 % 2))):
            if item not in done or item in queue or held[stage] != item:
                raise Bad(f"reads {item} at {kt}")
            last_read[item] = kt


@pytest.mark.parametrize("nk", list(range(1, 41)))
def test_ping_pong_and_ring(nk):
    replay_pp(nk)
    replay_ring(nk)


def test_planted_mistakes_are_caught():
    for wrong in (dict(wait_extra=5), dict(scale_tick_shift=2), dict(drop_wait=True)):
        with pytest.raises(Bad):
            for nk in range(1, 20):
                replay_pp(nk, **wrong)
    for wrong in (dict(extra=6), dict(ahead=3)):
        with pytest.raises(Bad):
            for nk in range(1, 20):
                replay_ring(nk, **wrong)
