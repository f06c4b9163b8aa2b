"""Which kernel a product is given (i8_plan, a function of sizes alone): the
sizes that the GPU tests run reach every kernel there is, so that a change of
the rule's constants does not leave one untested."""
import ctypes

import memory_bound_mxfp4_amd as moe
import test_gpu_i8 as gpu

KINDS = {0, 1, 2, 3, 4, 5}  # few rows; tiles of 64 x 64, 64 x 128, 128 x 128 (one and two to a CU), 256 x 256


class Plan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("tile_rows", ctypes.c_int), ("parts", ctypes.c_int),
                ("part_bytes", ctypes.c_size_t)]


def _plan(rows, experts, grouped, n, k, swiglu):
    moe.load()
    f = ctypes.CDLL(moe.LIB_PATH)["_ZN3moe7i8_planEiibiib"]
    f.restype, f.argtypes = Plan, [ctypes.c_int, ctypes.c_int, ctypes.c_bool, ctypes.c_int, ctypes.c_int, ctypes.c_bool]
    return f(rows, experts, grouped, n, k, swiglu)


def _sizes(test, *names):
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == ",".join(names):
            return mark.args[1]
    raise AssertionError(f"{test.__name__} has no sizes {names}")


def test_every_dense_kernel_is_tested():
    seen = {}
    for m, n, k, swiglu in _sizes(gpu.test_gemm_tiles, "m", "n", "k", "swiglu"):
        p = _plan(m, 1, False, n, k, swiglu)
        seen.setdefault((p.kind, p.parts > 1), []).append(swiglu)
    assert {kind for kind, _ in seen} == KINDS
    assert set(seen[1, True]) == {False, True} and (1, False) in seen
    split = {p.parts for p in (_plan(m, 1, False, n, k, s) for m, n, k, s in _sizes(gpu.test_gemm_tiles, "m", "n", "k", "swiglu"))}
    assert len(split) > 2
    for swiglu in (False, True):
        assert {_plan(m, 1, False, n, k, swiglu).kind for m, n, k in gpu.ALL_KERNELS} == KINDS
    assert any(_plan(m, 1, False, n, k, False).parts > 1 for m, n, k in gpu.ALL_KERNELS)
    assert any(_plan(m, 1, False, n, k, True).parts > 1 for m, n, k in gpu.ALL_KERNELS)


def test_every_grouped_kernel_is_tested():
    seen = {}
    for tokens, top_k, E, n, k, swiglu in _sizes(gpu.test_experts_tiles, "tokens", "top_k", "E", "n", "k", "swiglu"):
        p = _plan(tokens * top_k, E, True, n, k, swiglu)
        assert p.parts == 1
        seen.setdefault(p.kind, []).append(swiglu)
    assert set(seen) == KINDS
