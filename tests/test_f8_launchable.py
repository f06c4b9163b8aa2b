"""A product of e4m3 codes whose fastest kernel would make more workgroups than
a launch holds runs on another kernel, where one fits (host functions alone:
nothing is enqueued)."""
import ctypes
import random

import pytest

import memory_bound_mxfp4_amd as moe
from test_f8_plan import Plan, _plan

COLUMNS = {0: 32, 1: 64, 2: 128, 3: 128, 4: 128, 5: 256}
ROWS = {0: 16, 1: 64, 2: 64, 3: 128, 4: 128, 5: 256}
MOST = 1 << 22


def _tiles(rows, experts, grouped, tile_rows):
    return rows // tile_rows + min(rows, experts + 1) if grouped else -(-rows // tile_rows)


def _launchable(plan, n, swiglu, tiles):
    moe.load()
    f = ctypes.CDLL(moe.LIB_PATH)["_ZN3moe13f8_launchableERKNS_6F8PlanEibi"]
    f.restype, f.argtypes = ctypes.c_bool, [ctypes.POINTER(Plan), ctypes.c_int, ctypes.c_bool, ctypes.c_int]
    return f(ctypes.byref(plan), n, swiglu, tiles)


def _fits(kind, rows, experts, grouped, n, swiglu):
    return -(-n * (2 if swiglu else 1) // COLUMNS[kind]) * _tiles(rows, experts, grouped, ROWS[kind]) < MOST


# slots, experts, n, k, swiglu, fp32 outputs
LARGE = [(1816, 3736, 34885, 208, True, True), (82, 389, 772384, 2288, True, False), (1270, 3217, 210551, 48, True, False),
         (1816, 3736, 34885, 208, True, False), (12025, 760, 145170, 29584, True, True)]


@pytest.mark.parametrize("rows,experts,n,k,swiglu,wide", LARGE)
def test_a_grouped_product_takes_a_kernel_that_fits(rows, experts, n, k, swiglu, wide):
    plan = _plan(rows, experts, True, n, k, swiglu, wide)
    assert _launchable(plan, n, swiglu, _tiles(rows, experts, True, plan.tile_rows)), plan.kind


def test_no_product_is_refused_that_some_kernel_takes():
    rng = random.Random(7)

    def size(low, high):
        return min(high, int(low * (high / low) ** rng.random()))

    refused = 0
    for _ in range(20000):
        grouped, swiglu, wide = rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5
        n, k = size(64, 1 << 20), 16 * size(1, 4096)
        rows, experts = (size(1, (1 << 27) - 1), size(1, 4096)) if grouped else (size(1, (1 << 24) - 1), 1)
        plan = _plan(rows, experts, grouped, n, k, swiglu, wide)
        fits = _launchable(plan, n, swiglu, _tiles(rows, experts, grouped, plan.tile_rows))
        assert plan.tile_rows == ROWS[plan.kind]
        if not fits:
            refused += 1
            few = 1 if not grouped and rows > 16 else 0  # a dense product of many rows is never a stream
            assert not any(_fits(kind, rows, experts, grouped, n, swiglu) for kind in range(few, 4 if wide else 6)), \
                (rows, experts, grouped, n, k, swiglu, wide, plan.kind)
    assert refused
