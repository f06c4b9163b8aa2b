"""The routing and 8-bit entry points turn bad arguments down on the host,
before anything is enqueued (no GPU needed), and the binding checks what the
C interface cannot see."""
import ctypes

import pytest

import memory_bound_mxfp4_amd as moe

P = ctypes.c_void_p
BF16, F32, F16, I8 = moe.MOE_DTYPE_BF16, moe.MOE_DTYPE_F32, moe.MOE_DTYPE_F16, moe.MOE_DTYPE_I8
INVALID, UNSUPPORTED, SMALL = moe.MOE_ERR_INVALID_ARGUMENT, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE_TOO_SMALL


def _route(**over):
    a = dict(logits=P(0x1000), dtype=F32, stride=256, rows=4, bias=None, E=256, k=8, score=0, groups=8, top_groups=4,
             group_top=2, renorm=1, scale=1.0, idx=P(0x2000), gate=P(0x3000))
    a.update(over)
    p = moe.RouteParamsC(a["E"], a["k"], a["score"], a["groups"], a["top_groups"], a["group_top"], a["renorm"], a["scale"])
    return moe.load().moe_route(a["logits"], a["dtype"], a["stride"], a["rows"], a["bias"], ctypes.byref(p), a["idx"],
                                a["gate"], None)


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(idx=None), dict(gate=None), dict(dtype=I8), dict(dtype=9), dict(stride=255), dict(rows=0),
    dict(E=0), dict(k=0), dict(k=65), dict(k=129, top_groups=4), dict(score=2), dict(groups=0), dict(groups=7),
    dict(top_groups=0), dict(top_groups=9), dict(group_top=0), dict(group_top=3), dict(renorm=2),
    dict(k=33, top_groups=1), dict(logits=P(0x1002)), dict(logits=P(0x1001), dtype=F16), dict(bias=P(0x1002)),
    dict(groups=1, top_groups=2)], ids=str)
def test_route_invalid(over):
    assert _route(**over) == INVALID


def test_route_unsupported():
    assert _route(E=4104, stride=4104) == UNSUPPORTED
    assert _route(E=260, stride=260, groups=65, top_groups=65) == UNSUPPORTED
    assert _route(rows=1 << 24) == UNSUPPORTED
    assert moe.load().moe_route(P(0x1000), F32, 8, 1, None, None, P(0x2000), P(0x3000), None) == INVALID


def test_quant_refusals():
    f = moe.load().quant_rows_i8
    x, q, s = P(0x1000), P(0x2000), P(0x3000)
    for args in ((None, BF16, 64, 1, 64, q, s), (x, BF16, 64, 1, 64, None, s), (x, BF16, 64, 1, 64, q, None),
                 (x, I8, 64, 1, 64, q, s), (x, BF16, 63, 2, 64, q, s), (x, BF16, 64, 0, 64, q, s),
                 (x, BF16, 64, 1, 0, q, s), (P(0x1001), BF16, 64, 1, 64, q, s), (P(0x1002), F32, 64, 1, 64, q, s),
                 (x, BF16, 64, 1, 64, q, P(0x3002))):
        assert f(*args, None) == INVALID, args
    assert f(x, BF16, 65537, 1, 65537, q, s, None) == UNSUPPORTED
    assert f(x, BF16, 64, 1 << 24, 64, q, s, None) == UNSUPPORTED


def _gemm(**over):
    a = dict(x=P(0x1000), xd=BF16, stride=64, xs=None, m=4, k=64, w=P(0x2000), ws=P(0x3000), n=32, swiglu=0,
             y=P(0x4000), yd=BF16, work=P(0x10000), size=1 << 20)
    a.update(over)
    return moe.load().gemm_i8(a["x"], a["xd"], a["stride"], a["xs"], a["m"], a["k"], a["w"], a["ws"], a["n"], a["swiglu"],
                              a["y"], a["yd"], a["work"], a["size"], None)


BAD_PRODUCT = [
    dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(m=0), dict(n=0), dict(k=0), dict(k=8), dict(k=40),
    dict(stride=48), dict(swiglu=2), dict(xd=7), dict(yd=I8), dict(yd=5), dict(xd=I8), dict(xs=P(0x5000)),
    dict(xd=I8, xs=P(0x5000), stride=72), dict(xd=I8, xs=P(0x5000), x=P(0x1008)), dict(x=P(0x1001)),
    dict(w=P(0x2008)), dict(y=P(0x4008)), dict(ws=P(0x3002)), dict(work=None), dict(work=P(0x10010))]


@pytest.mark.parametrize("over", BAD_PRODUCT, ids=str)
def test_gemm_invalid(over):
    assert _gemm(**over) == INVALID


def test_gemm_unsupported_and_workspace():
    assert _gemm(k=65552, stride=65552) == UNSUPPORTED
    assert _gemm(n=(1 << 20) + 1) == UNSUPPORTED
    assert _gemm(m=1 << 24) == UNSUPPORTED
    need = moe.load().gemm_i8_workspace_size(4, 32, 64, 0, BF16)
    assert need > 0 and _gemm(size=need - 1) == SMALL


def test_groups_refusals():
    lib = moe.load()
    idx, buf = P(0x1000), P(0x10000)
    assert lib.moe_slot_groups_size(0, 1, 8) == 0 and lib.moe_slot_groups_size(1, 65, 8) == 0
    assert lib.moe_slot_groups_size(1, 1, 0) == 0 and lib.moe_slot_groups_size(1, 1, 4097) == 0
    assert lib.moe_slot_groups_size(1 << 23, 16, 8) == 0
    need = lib.moe_slot_groups_size(4, 2, 8)
    assert need >= 4 * 8 + 4 * 10
    assert lib.moe_group_slots(None, 4, 2, 8, buf, need, None) == INVALID
    assert lib.moe_group_slots(idx, 4, 2, 8, None, need, None) == INVALID
    assert lib.moe_group_slots(idx, 4, 2, 8, P(0x10010), need, None) == INVALID
    assert lib.moe_group_slots(P(0x1002), 4, 2, 8, buf, need, None) == INVALID
    assert lib.moe_group_slots(idx, 4, 2, 0, buf, need, None) == INVALID
    assert lib.moe_group_slots(idx, 4, 2, 8, buf, need - 1, None) == SMALL


def _experts(**over):
    a = dict(x=P(0x1000), xd=BF16, stride=64, xs=None, rows=4, k=64, g=P(0x20000), gb=1 << 20, tokens=4, top_k=2, E=8,
             w=P(0x2000), ws=P(0x3000), n=32, swiglu=0, y=P(0x4000), yd=BF16, work=P(0x10000), size=1 << 20)
    a.update(over)
    if "m" in over:
        a["rows"] = over["m"]
    return moe.load().experts_gemm_i8(a["x"], a["xd"], a["stride"], a["xs"], a["rows"], a["k"], a["g"], a["gb"],
                                      a["tokens"], a["top_k"], a["E"], a["w"], a["ws"], a["n"], a["swiglu"], a["y"],
                                      a["yd"], a["work"], a["size"], None)


@pytest.mark.parametrize("over", BAD_PRODUCT + [
    dict(g=None), dict(g=P(0x20080)), dict(rows=5), dict(rows=2), dict(tokens=0), dict(top_k=0), dict(top_k=65),
    dict(E=0), dict(E=4097)], ids=str)
def test_experts_invalid(over):
    assert _experts(**over) == INVALID


def test_experts_workspaces():
    lib = moe.load()
    assert _experts(gb=lib.moe_slot_groups_size(4, 2, 8) - 1) == SMALL
    assert _experts(size=lib.experts_gemm_i8_workspace_size(4, 2, 8, 4, 32, 64, 0, BF16) - 1) == SMALL


def test_combine_refusals():
    f = moe.load().moe_combine
    y, g, r, o = P(0x1000), P(0x2000), P(0x3000), P(0x4000)
    for args in ((None, BF16, g, 1, 2, 64, r, o), (y, BF16, None, 1, 2, 64, r, o), (y, BF16, g, 1, 2, 64, r, None),
                 (y, I8, g, 1, 2, 64, r, o), (y, BF16, g, 0, 2, 64, r, o), (y, BF16, g, 1, 0, 64, r, o),
                 (y, BF16, g, 1, 65, 64, r, o), (y, BF16, g, 1, 2, 0, r, o), (P(0x1001), BF16, g, 1, 2, 64, r, o),
                 (y, BF16, P(0x2002), 1, 2, 64, r, o), (y, BF16, g, 1, 2, 64, P(0x3002), o),
                 (y, BF16, g, 1, 2, 64, r, P(0x4002))):
        assert f(*args, None) == INVALID, args
    assert f(y, BF16, g, 1, 2, (1 << 20) + 1, r, o, None) == UNSUPPORTED
    assert f(y, BF16, g, 1 << 24, 2, 64, r, o, None) == UNSUPPORTED


def test_binding_checks():
    """What the binding sees and the C interface cannot: types, shapes, strides and devices of tensors."""
    import torch
    x, w, s = torch.zeros(4, 64), torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32)
    for call in (
            lambda: moe.gemm_i8(x, w, s),                                  # on the CPU
            lambda: moe.gemm_i8(x.double(), w, s),                         # type of x
            lambda: moe.gemm_i8(x, w.float(), s),                          # type of w
            lambda: moe.gemm_i8(x, w, s.double()),
            lambda: moe.gemm_i8(x, w[:, :48], s),                          # k of w, and not contiguous
            lambda: moe.gemm_i8(x, w, s[:31]),
            lambda: moe.gemm_i8(x, w, s, swiglu=True),                     # w needs two matrices
            lambda: moe.gemm_i8(x, w, s, x_scale=torch.zeros(4)),          # scales of rows that are no codes
            lambda: moe.gemm_i8(x.to(torch.int8), w, s),                   # codes without scales
            lambda: moe.gemm_i8(x.t(), w, s),                              # elements apart
            lambda: moe.gemm_i8(x, w, s, out=torch.zeros(4, 31)),
            lambda: moe.gemm_i8(x, w, s, out=torch.zeros(4, 32), out_dtype=torch.float16),
            lambda: moe.moe_route(x, 2, score="other"),
            lambda: moe.moe_route(x, 2, bias=torch.zeros(63)),
            lambda: moe.moe_route(x.expand(4, 64).t(), 2),
            lambda: moe.moe_route(x.to(torch.int8), 2),
            lambda: moe.moe_route(x[:1].expand(4, 64), 2),                 # rows on top of each other
            lambda: moe.quant_rows_i8(x, q=torch.zeros(4, 64)),
            lambda: moe.moe_group_slots(torch.zeros(4, 2), 8),
            lambda: moe.alloc_slot_groups(4, 2, 5000, device="cpu"),
            lambda: moe.moe_combine(torch.zeros(8, 16), torch.zeros(4, 3)),
    ):
        with pytest.raises(ValueError):
            call()
    groups = moe.alloc_slot_groups(4, 2, 8, device="cpu")
    assert groups.order.shape == (8,) and groups.offsets.shape == (10,)
    wide, scales = torch.zeros(8, 32, 64, dtype=torch.int8), torch.zeros(8, 32)
    with pytest.raises(ValueError):
        moe.experts_gemm_i8(torch.zeros(5, 64), groups, wide, scales)
    with pytest.raises(ValueError):
        moe.experts_gemm_i8(x, groups, wide[:7], scales[:7])
    with pytest.raises(ValueError):
        moe.moe_group_slots(torch.zeros(4, 2, dtype=torch.int32), 9, groups=groups)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_route_scale(scale):
    """An infinite scale would turn the gate 0 of a padded place into NaN."""
    assert _route(scale=scale) == INVALID


def test_outputs_over_inputs():
    """A product's workgroups read x while others write y; a sum's threads read y and the residual in the same way."""
    lib = moe.load()
    assert _gemm(y=P(0x1000)) == INVALID                                    # y is x
    assert _gemm(y=P(0x11F0)) == INVALID                                    # the last 16 of 512 bytes of x
    assert _gemm(x=P(0x40F0)) == INVALID                                    # x in the last 16 of 256 bytes of y
    assert _experts(y=P(0x11F0)) == INVALID
    assert _experts(x=P(0x41F0)) == INVALID                                 # 8 slots of 64 bytes
    q = lib.quant_rows_i8
    x, s = P(0x1000), P(0x9000)
    assert q(x, F32, 64, 4, 64, P(0x13FF), s, None) == INVALID              # 1024 bytes of x
    assert q(x, F32, 64, 4, 64, P(0x0F01), s, None) == INVALID
    assert q(x, F32, 64, 4, 64, P(0x8000), P(0x13FC), None) == INVALID
    c, y, g = lib.moe_combine, P(0x10000), P(0x2000)
    assert c(y, F32, g, 2, 2, 64, None, P(0x103FC), None) == INVALID        # 1024 bytes of y, 512 of out
    assert c(y, F32, g, 2, 2, 64, None, P(0x0FE04), None) == INVALID
    assert c(y, F32, g, 2, 2, 64, P(0x20000), P(0x20004), None) == INVALID  # residual, but not out itself


def test_sizes_past_32_bits():
    """Sizes whose low 32 bits would pass are turned down by the binding."""
    import torch
    big = (1 << 32) + 4
    base = torch.zeros(1, dtype=torch.bfloat16)
    rows = base.expand(big, 1)
    w, s = torch.zeros(32, 16, dtype=torch.int8), torch.zeros(32)
    for call in (
            lambda: moe.quant_rows_i8(rows),
            lambda: moe.quant_rows_i8(rows.t()),
            lambda: moe.moe_route(rows, 1),
            lambda: moe.gemm_i8(torch.zeros(4, 16), w[:1, :1].expand(big, 16), s),
            lambda: moe.moe_route(torch.zeros(4, 16), 1 << 32 | 1),
            lambda: moe.moe_route(torch.zeros(4, 16), 1, groups=(1 << 32) + 1),
            lambda: moe.alloc_slot_groups(big, 1, 8, device="cpu"),
            lambda: moe.gemm_i8_workspace_size(big, 32, 64, False, torch.bfloat16),
            lambda: moe.experts_gemm_i8_workspace_size(moe.SlotGroups(4, 2, 8, None, None, None), 4, big, 64, False,
                                                       torch.bfloat16),
            lambda: moe.moe_combine(torch.zeros(1, 1).expand(2, big), torch.zeros(1, 2)),
    ):
        with pytest.raises(ValueError):
            call()


def _routed(monkeypatch, **kw):
    """The parameters that a call of the binding hands to the C interface."""
    import torch
    seen = []

    def launch(what, device, stream, *args):
        p = args[5]._obj
        seen.append({name: getattr(p, name) for name, _ in p._fields_})

    monkeypatch.setattr(moe, "_launch", launch)
    args = dict(top_k=2)
    args.update(kw)
    moe.moe_route(torch.zeros(4, 16), **args)
    return seen[0]


def test_route_scale_is_read_in_every_call(monkeypatch):
    """A routed scaling factor held in a tensor (a module's buffer) and changed in place between two calls."""
    import torch
    scale = torch.tensor(2.5)
    assert _routed(monkeypatch, scale=scale)["scale"] == 2.5
    scale.fill_(1.0)
    assert _routed(monkeypatch, scale=scale)["scale"] == 1.0
    assert _routed(monkeypatch, scale=2)["scale"] == 2.0
    with pytest.raises((TypeError, ValueError)):
        moe.moe_route(torch.zeros(4, 16), 2, scale="2")


def test_route_sizes_are_whole_numbers(monkeypatch):
    """A float is refused whether or not the same whole number was routed with before, a number of another integer
    type is taken; a tensor's value is read in every call."""
    import numpy as np
    import torch
    assert _routed(monkeypatch, groups=4, top_groups=2)["groups"] == 4
    for over in (dict(groups=4.0, top_groups=2), dict(groups=4, top_groups=2.0), dict(groups=4, top_groups=2, group_top=1.0),
                 dict(groups=4, top_groups=2, top_k=2.0)):
        with pytest.raises(TypeError):
            _routed(monkeypatch, **over)
    got = _routed(monkeypatch, groups=np.int64(4), top_groups=np.int32(2), top_k=np.int64(3))
    assert (got["groups"], got["top_groups"], got["top_k"]) == (4, 2, 3)
    groups = torch.tensor(4)
    assert _routed(monkeypatch, groups=groups, top_groups=2)["groups"] == 4
    groups.fill_(2)
    assert _routed(monkeypatch, groups=groups, top_groups=2)["groups"] == 2


FAR = dict(x=P(0x100000), w=P(0x200000), ws=P(0x300000), y=P(0x400000), work=P(0x500000))


def test_route_outputs_over_inputs():
    """Rows are read and written by different workgroups."""
    a = dict(logits=P(0x10000), idx=P(0x20000), gate=P(0x30000), bias=P(0x40000), rows=4, stride=300)  # rows of 1024 bytes
    end = 0x10000 + 3 * 1200 + 1024
    for name in ("idx", "gate"):                                            # 4 rows of 8: 128 bytes
        for at in (0x10000, 0x10000 - 124, end - 4, 0x10000 + 1200 + 512, 0x40000, 0x40000 + 1020, 0x40000 - 124):
            assert _route(**{**a, name: P(at)}) == INVALID, (name, hex(at))
    assert _route(**{**a, "idx": P(0x30000 + 124)}) == INVALID
    assert _route(**{**a, "gate": P(0x20000)}) == INVALID


def test_product_outputs_over_inputs():
    """The output over the matrix, the scales, the workspace or the groups; the workspace over any of them."""
    need = moe.load().gemm_i8_workspace_size(4, 32, 64, 0, BF16)
    w_end, s_end = 0x200000 + 32 * 64, 0x300000 + 32 * 4
    for at in (0x200000, w_end - 16, 0x200000 - 240, 0x300000, s_end - 16, 0x500000, 0x500000 + need - 16, 0x500000 - 240):
        assert _gemm(**{**FAR, "y": P(at)}) == INVALID, hex(at)
    for at in (0x100000, 0x100200 - 256, 0x200000, w_end - 256, 0x300000, 0x400000):
        assert _gemm(**{**FAR, "work": P(at)}) == INVALID, hex(at)
    codes = {**FAR, "xd": I8, "xs": P(0x600000)}
    assert _gemm(**{**codes, "y": P(0x600000)}) == INVALID
    assert _gemm(**{**codes, "y": P(0x600000 - 240)}) == INVALID
    two = {**FAR, "swiglu": 1}
    assert _gemm(**{**two, "y": P(w_end + 32 * 64 - 16)}) == INVALID
    assert _gemm(**{**two, "y": P(s_end + 32 * 4 - 16)}) == INVALID
    # one row, which needs no workspace
    assert _gemm(**{**FAR, "m": 1, "y": P(0x200000)}) == INVALID
    assert _gemm(**{**FAR, "m": 1, "y": P(0x300000)}) == INVALID

    lib = moe.load()
    need = lib.experts_gemm_i8_workspace_size(4, 2, 8, 4, 32, 64, 0, BF16)
    groups = lib.moe_slot_groups_size(4, 2, 8)
    far = {**FAR, "g": P(0x700000), "gb": groups}
    for at in (0x200000 + 8 * 32 * 64 - 16, 0x300000 + 8 * 32 * 4 - 16, 0x500000 + need - 16, 0x700000, 0x700000 + groups - 16):
        assert _experts(**{**far, "y": P(at)}) == INVALID, hex(at)
    for at in (0x200000 + 8 * 32 * 64 - 256, 0x300000 + 8 * 32 * 4 - 256, 0x700000, 0x700000 + groups - 256):
        assert _experts(**{**far, "work": P(at)}) == INVALID, hex(at)
    one = {**far, "rows": 1, "tokens": 1}
    for at in (0x200000, 0x300000, 0x700000):
        assert _experts(**{**one, "y": P(at)}) == INVALID, hex(at)


def test_other_outputs_over_inputs():
    lib = moe.load()
    x, q, s = P(0x10000), P(0x20000), P(0x30000)
    assert lib.quant_rows_i8(x, F32, 64, 4, 64, q, P(0x20000 + 252), None) == INVALID    # 256 codes
    assert lib.quant_rows_i8(x, F32, 64, 4, 64, q, P(0x20000 - 12), None) == INVALID
    need = lib.moe_slot_groups_size(4, 2, 8)
    for at in (0x10000, 0x10000 + need - 4, 0x10000 - 28):                                # 8 slots
        assert lib.moe_group_slots(P(at), 4, 2, 8, P(0x10000), need, None) == INVALID, hex(at)
    y, g, r, o = P(0x10000), P(0x20000), P(0x30000), P(0x40000)
    for at in (0x40000, 0x40000 + 508, 0x40000 - 12):                                     # 2 tokens of 64, gates of 16 bytes
        assert lib.moe_combine(y, F32, P(at), 2, 2, 64, r, o, None) == INVALID, hex(at)
        assert lib.moe_combine(y, F32, P(at), 2, 2, 64, o, o, None) == INVALID, hex(at)
