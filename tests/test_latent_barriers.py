"""The barrier protocol of the latent attention's backward blocks, searched exhaustively on the CPU.

A block's warps meet at barriers of which a waiter knows the phase's parity only. A wait therefore goes wrong in two
ways: it passes on the phase before the one that is meant (too early), or the phase that is meant and the next one are
both over when it looks, the parity is the old one again, and it waits for good. The roles below are those of a block
of dk and dv (``dkv_block`` in csrc/latent_bwd.cu) and of a block of dq, with two warps in place of eight; products
complete in the order of their issue, copies in any order, every role as fast or slow as it likes."""
import os

import pytest

WARPS = 2
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kimi_delta_attention_25_b200", "csrc")


class Block:
    """Roles as lists of (what, barrier, phase): wait for a phase, arrive, order a copy or a product that arrives."""

    def __init__(self):
        self.roles, self.count = [], {}

    def barrier(self, names, count=1):
        for n in names:
            self.count[n] = count

    def role(self, steps):
        self.roles.append([s if len(s) == 3 else (*s, 0) for s in steps])

    def search(self):
        """Visits every state; returns the first fault as text, or None."""
        names = sorted(self.count)
        at = {n: i for i, n in enumerate(names)}
        start = (tuple(0 for _ in self.roles), tuple((0, 0) for _ in names), (), ())
        seen, stack = {start}, [start]

        def arrive(bars, n):
            phase, got = bars[at[n]]
            got += 1
            if got == self.count[n]:
                phase, got = phase + 1, 0
            return bars[:at[n]] + ((phase, got),) + bars[at[n] + 1:]

        while stack:
            pcs, bars, copies, products = state = stack.pop()
            after = []
            for r, steps in enumerate(self.roles):
                if pcs[r] == len(steps):
                    continue
                what, bar, phase = steps[pcs[r]]
                moved = pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:]
                if what == "wait":
                    now = bars[at[bar]][0]
                    if (now ^ phase) & 1:                  # the parity differs from the running phase's: passed
                        if now <= phase:
                            return "role %d passes %s before its phase %d is over" % (r, bar, phase)
                        after.append((moved, bars, copies, products))
                elif what == "arrive":
                    after.append((moved, arrive(bars, bar), copies, products))
                elif what == "copy":
                    after.append((moved, bars, tuple(sorted(copies + (bar,))), products))
                else:
                    after.append((moved, bars, copies, products + (bar,)))
            for c in set(copies):
                rest = list(copies)
                rest.remove(c)
                after.append((pcs, arrive(bars, c), tuple(rest), products))
            if products:
                after.append((pcs, arrive(bars, products[0]), copies, products[1:]))
            if not after and any(pcs[r] < len(s) for r, s in enumerate(self.roles)):
                return "stuck: " + ", ".join("role %d at %s" % (r, s[pcs[r]]) for r, s in enumerate(self.roles) if pcs[r] < len(s))
            for s in after:
                if s not in seen:
                    seen.add(s)
                    stack.append(s)
        return None


def dkv_block(tiles, shared, own_barriers):
    """The block of dk and dv; ``own_barriers``: the statistics' buffers have a barrier each that says they are free."""
    b = Block()
    b.barrier(["res", "f1.0", "f1.1", "e1.0", "e1.1", "f2", "e2", "s", "p", "dr", "acc", "statf.0", "statf.1"])
    b.barrier(["pready", "ds", "pfree", "state.0", "state.1"], WARPS)
    n = range(tiles)
    loader, stat, warp = [("copy", "res")], [], []
    for j in n:
        x = j & 1
        if j >= 2:
            loader.append(("wait", "e1.%d" % x, (j >> 1) - 1))
        loader.append(("copy", "f1.%d" % x))
        if j >= 1:
            loader.append(("wait", "e2", j - 1))
        loader.append(("copy", "f2"))
        if j >= 2:
            stat.append(("wait", "state.%d" % x, (j >> 1) - 1) if own_barriers else ("wait", "ds", j - 2))
        stat.append(("arrive", "statf.%d" % x))
        warp += [("wait", "statf.%d" % x, j >> 1), ("wait", "s", j)]
        if j > 0:
            warp += ([("wait", "dr", j - 1)] if shared else []) + [("arrive", "pfree")]
        if j == tiles - 1:
            warp.append(("wait", "f2", j))
        warp += [("arrive", "pready"), ("wait", "p", j), ("arrive", "ds"), ("arrive", "state.%d" % x)]
    warp += ([("wait", "dr", tiles - 1)] if shared else []) + [("wait", "acc", tiles - 1)]
    scores = lambda j: [("wait", "f1.%d" % (j & 1), j >> 1), ("product", "s")]  # noqa: E731
    dp = lambda j: [("wait", "f2", j), ("product", "p")]  # noqa: E731
    mma = [("wait", "res", 0)] + scores(0) + dp(0)
    for j in n:
        more = j + 1 < tiles
        mma += [("wait", "pready", j), ("product", "e2")] + (scores(j + 1) if more else []) + [("wait", "ds", j)]
        mma += ([("product", "dr")] if shared else []) + [("product", "e1.%d" % (j & 1)), ("product", "acc")]
        if more:
            mma += [("wait", "pfree", j)] + dp(j + 1)
    b.role(loader)
    b.role(mma)
    b.role(stat)
    for _ in range(WARPS):
        b.role(warp)
    return b


def dq_block(tiles):
    """The block of dq, its rings of one tile of keys and one of values (the kernel's are longer)."""
    b = Block()
    b.barrier(["res", "f1", "e1", "f2", "e2", "s", "p", "acc"])
    b.barrier(["sfree", "pfree", "ds"], WARPS)
    loader, mma, accumulate, warp = [("copy", "res")], [("wait", "res", 0)], [], []
    for j in range(tiles):
        loader += ([("wait", "e1", j - 1)] if j else []) + [("copy", "f1")] + ([("wait", "e2", j - 1)] if j else []) + [("copy", "f2")]
        mma += ([("wait", "sfree", j - 1)] if j else []) + [("wait", "f1", j), ("product", "s")]
        mma += ([("wait", "pfree", j - 1)] if j else []) + [("wait", "f2", j), ("product", "e2"), ("product", "p")]
        accumulate += [("wait", "ds", j), ("product", "e1"), ("product", "acc")]
        warp += [("wait", "s", j), ("arrive", "sfree"), ("wait", "p", j), ("arrive", "pfree")]
        warp += ([("wait", "acc", j - 1)] if j else []) + [("arrive", "ds")]
    warp.append(("wait", "acc", tiles - 1))
    for steps in [loader, mma, accumulate] + [warp] * WARPS:
        b.role(steps)
    return b


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("tiles", [1, 2, 5])
def test_dk_and_dv_blocks_never_wait_for_a_phase_that_is_past(tiles, shared):
    with open(os.path.join(CSRC, "latent_bwd.cu")) as f:
        own = "wait(K_STATE + (j & 1), ((j >> 1) - 1) & 1)" in f.read()          # which of the two the kernel does
    assert dkv_block(tiles, shared, own).search() is None


def test_one_barrier_for_both_statistics_buffers_can_be_overtaken():
    """Why each buffer has its own: the warps finish a tile that the statistics' warp is yet to look for."""
    assert dkv_block(5, True, own_barriers=False).search().startswith("stuck")


@pytest.mark.parametrize("tiles", [1, 2, 4])
def test_dq_blocks_never_wait_for_a_phase_that_is_past(tiles):
    assert dq_block(tiles).search() is None


def test_no_wait_of_the_norms_runs_out_unnoticed():
    """The norm's calls have no status word, so a wait that gave up must show in the results: the outcome of every
    bounded wait is used (or dropped in so many words, where copies in flight are waited for after that)."""
    with open(os.path.join(CSRC, "rms_norm.cu")) as f:
        lines = [x.strip() for x in f if "mbar_wait(" in x]
    assert lines and not [x for x in lines if x.startswith(("mbar_wait(", "sm100::mbar_wait("))]
