"""That the sizes of test_gpu_f8_loops.py run the steady loop of every tile
kernel of the e4m3 products and, where a workgroup goes on from tile to tile,
whole tiles that another one follows."""
import numpy as np
import pytest

import test_gpu_f8_loops as loops
from test_f8_plan import KINDS, _plan

# of each tile kernel: rows of x, columns, buffers of a group of waves, groups of waves
TILES = {1: (64, 64, 4, 2), 2: (64, 128, 3, 2), 3: (128, 128, 4, 1), 4: (128, 128, 2, 1), 5: (256, 256, 2, 1)}
GOES_ON = {False: {3, 5}, True: set()}  # kernels whose workgroups take several tiles: 256 of them
CUS = 256


def _rounds(kind, k, parts):
    """Turns of the steady loop's body, for the group and part with the fewest: it runs while stages of 128 codes are left
    to load."""
    _, _, R, groups = TILES[kind]
    stages = -(-k // 128)
    fewest = None
    for part in range(parts):
        s0, s1 = stages * part // parts, stages * (part + 1) // parts
        for g in range(groups):
            mine = (s1 - s0 - g + groups - 1) // groups
            whole = (k // 128 - s0 - g + groups - 1) // groups
            turns = max(0, -(-(min(mine, whole) - (2 * R - 1)) // R))
            fewest = turns if fewest is None else min(fewest, turns)
    return fewest


def _seen(cases, swiglu, wide):
    """Of each kernel: the sets of (turns of its loop, whole K, last rows of a tile in steps of its waves), and those that
    go on with counted stores."""
    seen = {}
    for m_rows, experts, grouped, n, k, tiles, full in cases(swiglu):
        p = _plan(m_rows, experts, grouped, n, k, swiglu, wide)
        if p.kind not in TILES:
            continue
        bm, bn, _, _ = TILES[p.kind]
        cols = -(-n * (2 if swiglu else 1) // bn)
        on = p.kind in GOES_ON[wide] and tiles(bm) * cols > CUS
        seen.setdefault(p.kind, []).append((_rounds(p.kind, k, p.parts), k % 128 == 0, on, on and full(bm) and n % 8 == 0))
    return seen


def _dense(swiglu):
    for m, n, k in loops.DENSE:
        yield m, 1, False, n // 2 if swiglu else n, k, lambda bm, m=m: -(-m // bm), lambda bm, m=m: m > bm


def _grouped(swiglu):
    for tokens, top_k, E, n, k, _ in loops.GROUPED:
        flat = loops.slots_of(tokens, top_k, E).reshape(-1)
        rows = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        yield (tokens * top_k, E, True, n // 2 if swiglu else n, k, lambda bm, rows=rows: int((-(-rows // bm)).sum()),
               lambda bm, rows=rows: bool((rows >= bm).any()))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cases", [_dense, _grouped])
def test_every_steady_loop_runs(cases, wide, swiglu):
    seen = _seen(cases, swiglu, wide)
    assert set(seen) == KINDS[wide] - {0}, sorted(seen)
    for kind, runs in seen.items():
        assert max(r[0] for r in runs) > 0, (kind, runs)
        if kind in GOES_ON[wide]:
            assert any(r[3] and r[0] > 0 for r in runs), (kind, runs)  # on from a whole tile, and through the loop


def test_short_and_long_sums_on_the_way_from_tile_to_tile():
    """The counted stores with K of fewer stages than the loop needs, as many, and several rounds; K that ends inside a
    stage and at its end; without counted stores too."""
    runs = _seen(_dense, False, False)[5]
    assert {r[0] for r in runs if r[3]} >= {0, 1, 2, 3} and {r[1] for r in runs if r[3]} == {False, True}
    assert any(r[2] and not r[3] for r in runs)
    rows = {-(-(m % 256) // 64) for m, n, k in loops.DENSE if _plan(m, 1, False, n, k, False, False).kind == 5}
    assert rows == {0, 1, 2, 3, 4}, rows
