"""How the 4-bit decode kernel cuts its work (CPU): the arithmetic of the runs, the pieces and the merge, replayed in
Python for ragged batches.  Every tile must fall into exactly one warp's run, the CTAs that the merge adds up must be
exactly those that hold tiles of the (request, head), and each of them must hold one."""
import random

import pytest

TILE, MIN_COST = 64, 4


def tiles_before(z, nt):
    return min(0 if z == 0 else max(1, z >> 1), nt)


def plan(lens, hkv, warps, sms):
    """Per CTA the warps' runs of tiles [a, b), and the CTA of every cost position."""
    nt = [-(-n // TILE) for n in lens]
    cum = [0]
    for n in nt:
        cum.append(cum[-1] + n)
    cost = (2 * cum[-1] + len(lens)) * hkv
    ctas = min(sms, max(1, cost // MIN_COST))
    each, more = divmod(cost, ctas)

    def tiles(x):
        r = max(i for i in range(len(lens)) if (2 * cum[i] + i) * hkv <= x)
        y = x - (2 * cum[r] + r) * hkv
        g = y // (2 * nt[r] + 1)
        return cum[r] * hkv + g * nt[r] + tiles_before(y - g * (2 * nt[r] + 1), nt[r])

    runs = []
    for c in range(ctas):
        n, x0 = each + (c < more), each * c + min(c, more)
        runs.append([(tiles(x0 + n * w // warps), tiles(x0 + n * (w + 1) // warps)) for w in range(warps)])
    cta_of = lambda x: x // (each + 1) if x < more * (each + 1) else more + (x - more * (each + 1)) // each
    return nt, cum, runs, cta_of


@pytest.mark.parametrize("seed", range(60))
def test_runs_cover_every_tile_once_and_the_merge_finds_its_parts(seed):
    rng = random.Random(seed)
    n, hkv, warps, sms = rng.choice([1, 1, 2, 5, 33]), rng.choice([1, 2, 3, 8]), rng.choice([8, 12]), rng.choice([4, 13, 148])
    top = rng.choice([0, 1, 64, 65, 700, 9000])
    lens = [rng.choice([0, rng.randint(0, top), top]) for _ in range(n)]
    nt, cum, runs, cta_of = plan(lens, hkv, warps, sms)
    total = cum[-1] * hkv
    if total == 0:
        return
    flat = [r for c in runs for r in c]
    assert flat[0][0] == 0 and flat[-1][1] == total
    assert all(a <= b for a, b in flat) and all(x[1] == y[0] for x, y in zip(flat, flat[1:]))
    bounds = [(c[0][0], c[-1][1]) for c in runs]
    for r in range(n):
        for g in range(hkv if nt[r] else 0):
            first = cum[r] * hkv + g * nt[r]
            stop = first + nt[r]
            holders = [c for c, (a, b) in enumerate(bounds) if a < stop and b > first]
            # the merge: from the CTA it begins in to the one in which its last tile's cost begins, all of them holders
            start = next(c for c, (a, b) in enumerate(bounds) if a <= first < b)
            last = cta_of((2 * cum[r] + r) * hkv + g * (2 * nt[r] + 1) + (0 if nt[r] == 1 else 2 * nt[r] - 1))
            assert holders == list(range(start, last + 1)), (lens, hkv, r, g)
            # a CTA continues at most one (request, head) from before and leaves at most one open
    for c, (a, b) in enumerate(bounds):
        segs = {(r, g) for r in range(n) for g in range(hkv) if nt[r] for f in [cum[r] * hkv + g * nt[r]]
                if f < b and f + nt[r] > a}
        assert sum(cum[r] * hkv + g * nt[r] < a for r, g in segs) <= 1
        assert sum(cum[r] * hkv + (g + 1) * nt[r] > b for r, g in segs) <= 1


def test_a_run_of_three_inside_a_request_has_a_tile():
    for nt in range(1, 40):
        for x in range(0, 2 * nt - 2):
            assert tiles_before(x + 3, nt) > tiles_before(x, nt)
        assert tiles_before(0, nt) == 0 and tiles_before(2 * nt + 1, nt) == nt
