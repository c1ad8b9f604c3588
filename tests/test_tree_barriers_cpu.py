"""A model of the tree attention's warps and their barriers, explored over every order
in which loads land, products finish and warps make a step.

An mbarrier counts phases; a wait names a parity, and passes while the last phase that
has ended has it.  A warp that looks too late finds the next phase ended, too, and waits
for one that may never come."""
import pytest

KST = 3


def stuck(first_wait, vst, tiles):
    """Whether an order exists in which the CTA stops before its last tile.

    first_wait: what V's first load waits for: "k0" (the barrier of K's first stage),
    "once" (a barrier that the MMA warp arrives at when it has seen K's first tile), or
    None.  State: K tiles issued and landed, QK issued and done, V tiles issued and landed,
    PV issued and done, tiles of weights made."""
    start = (0,) * 9

    def landings(landed, stage, stages):      # phases that a stage's barrier has ended
        return (landed - stage + stages - 1) // stages if landed > stage else 0

    def parity(ended, want):
        return ended % 2 != want % 2

    def steps(s):
        ki, kl, qi, qd, vi, vl, pi, pd, w = s
        # K's warp: the stage was freed by the product that read it
        if ki < tiles and (ki < KST or parity(landings(qd, ki % KST, KST), ki // KST - 1)):
            yield (ki + 1, kl, qi, qd, vi, vl, pi, pd, w)
        if kl < ki:
            yield (ki, kl + 1, qi, qd, vi, vl, pi, pd, w)
        # V's warp
        if vi < tiles:
            if vi >= vst:
                go = parity(landings(pd, vi % vst, vst), vi // vst - 1)
            elif vi == 0 and first_wait == "k0":
                go = parity(landings(kl, 0, KST), 0)
            elif vi == 0 and first_wait == "once":
                go = qi > 0
            else:
                go = True
            if go:
                yield (ki, kl, qi, qd, vi + 1, vl, pi, pd, w)
        if vl < vi:
            yield (ki, kl, qi, qd, vi, vl + 1, pi, pd, w)
        # the MMA warp: QK of tiles 0 and 1, then PV of tile j and QK of tile j + 2
        if qi < tiles and qi < pi + 2:
            if parity(landings(kl, qi % KST, KST), qi // KST):
                yield (ki, kl, qi + 1, qd, vi, vl, pi, pd, w)
        elif pi < tiles:
            if parity(landings(vl, pi % vst, vst), pi // vst) and \
                    parity(landings(w, pi % 2, 2), pi // 2):
                yield (ki, kl, qi, qd, vi, vl, pi + 1, pd, w)
        # products finish in the order in which they were issued; QK j + 2 after PV j
        if qd < qi and (qd < 2 or pd > qd - 2):
            yield (ki, kl, qi, qd + 1, vi, vl, pi, pd, w)
        if pd < pi and qd >= min(pd + 2, tiles):
            yield (ki, kl, qi, qd, vi, vl, pi, pd + 1, w)
        # the softmax warps
        if w < tiles and parity(landings(qd, w % 2, 2), w // 2):
            yield (ki, kl, qi, qd, vi, vl, pi, pd, w + 1)

    seen, todo = {start}, [start]
    while todo:
        s = todo.pop()
        after = list(steps(s))
        if not after and s[7] < tiles:
            return True
        for x in after:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return False


@pytest.mark.parametrize("vst", [2, 3])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 7, 9])
def test_no_order_stops_the_cta(vst, tiles):
    assert not stuck(None, vst, tiles)
    assert not stuck("once", vst, tiles)


@pytest.mark.parametrize("vst", [2, 3])
def test_the_barrier_of_a_stage_may_be_overtaken(vst):
    """K's tile 3 lands in stage 0 without any product of V: a V warp that has not looked
    by then waits for a phase that needs its own load."""
    assert stuck("k0", vst, 9)
    assert not stuck("k0", vst, 3)       # (three tiles never come back to a stage)
