"""Which kernel a product of e4m3 codes is given (f8_plan, a function of sizes
and of the output's type): the sizes that the GPU tests run reach every kernel
there is, so that a change of the rule's constants does not leave one untested."""
import ctypes

import memory_bound_mxfp4_amd as moe
import test_gpu_f8 as gpu

# few rows; tiles of 64 x 64, 64 x 128, 128 x 128 (one and two to a CU), 256 x 256: with the products of codes (16-bit
# outputs), and with those in fp16 (fp32 outputs)
KINDS = {False: {0, 1, 2, 3, 4, 5}, True: {0, 1, 2, 3}}


class Plan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("tile_rows", ctypes.c_int), ("parts", ctypes.c_int),
                ("part_bytes", ctypes.c_size_t)]


def _plan(rows, experts, grouped, n, k, swiglu, wide):
    moe.load()
    f = ctypes.CDLL(moe.LIB_PATH)["_ZN3moe7f8_planEiibiibb"]
    i, b = ctypes.c_int, ctypes.c_bool
    f.restype, f.argtypes = Plan, [i, i, b, i, i, b, b]
    return f(rows, experts, grouped, n, k, swiglu, wide)


def _sizes(test, names):
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == names:
            return mark.args[1]
    raise AssertionError(f"{test.__name__} has no sizes {names}")


def test_every_dense_kernel_is_tested():
    outs = {o == "f32" for o in _sizes(gpu.test_gemm_exact, "out")}
    assert outs == {False, True} and set(_sizes(gpu.test_gemm_exact, "swiglu")) == {False, True}
    for wide in outs:
        for swiglu in (False, True):
            plans = [_plan(m, 1, False, n, k, swiglu, wide) for m, n, k in gpu.ALL_KERNELS]
            assert {p.kind for p in plans} == KINDS[wide], (wide, swiglu, [p.kind for p in plans])
            split = {p.parts for p in plans}
            assert 1 in split and len(split) > 1, (wide, swiglu, split)
            assert any(p.kind == 1 and p.parts == 1 for p in plans)


def test_every_grouped_kernel_is_tested():
    outs = {o == "f32" for o in _sizes(gpu.test_experts_exact, "out")}
    sizes = _sizes(gpu.test_experts_exact, "tokens,top_k,E,n,k")
    for wide in outs:
        plans = [_plan(tokens * top_k, E, True, n, k, False, wide) for tokens, top_k, E, n, k in sizes]
        assert {p.kind for p in plans} == KINDS[wide], (wide, [p.kind for p in plans])
        assert all(p.parts == 1 for p in plans)
        plans = [_plan(t * top_k, E, True, n, k, True, wide) for t, top_k, E, n, k, _ in gpu.SWIGLU_EXPERTS]
        assert {p.kind for p in plans} == KINDS[wide], (wide, [p.kind for p in plans])


def test_workspace_is_enough_for_every_output():
    """The size is asked for without the output's type; the split of K goes by it."""
    lib = moe.load()
    for m, n, k in gpu.ALL_KERNELS:
        for swiglu in (False, True):
            size = lib.gemm_f8_workspace_size(m, n, k, int(swiglu), moe.MOE_DTYPE_F8)
            assert all(size >= _plan(m, 1, False, n, k, swiglu, wide).part_bytes for wide in (False, True))
