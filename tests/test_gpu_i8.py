"""GPU parity of the 8-bit integer operators (row quantiser, product, slots by
expert, the experts' products, the gated sum) against plain 64-bit references,
and a run of them together as a layer."""
import numpy as np
import pytest

import i8_reference as ref
import memory_bound_mxfp4_amd as moe

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _x(rows, k, dtype, seed, sigma=1.0):
    """Random rows as a GPU tensor of the type, and their values in fp64."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(rows, k, generator=g) * sigma).to(ref.torch_dtype(dtype))
    return t.cuda(), t.double().numpy()


def _w(shape, seed):
    rng = np.random.default_rng(seed)
    w = np.clip(np.rint(rng.standard_normal(shape) * 40), -128, 127).astype(np.int8)
    return w, (rng.uniform(0.5, 1.5, shape[:-1]) * 1e-3).astype(np.float32)


def _close(y, want, bound, what=""):
    y = y.double().cpu().numpy()
    bad = ~(np.abs(y - want) <= bound)
    bad &= ~(np.isnan(y) & np.isnan(want))
    assert not bad.any(), (what, np.argwhere(bad)[:4], y[bad][:4], want[bad][:4])


# ---- rows to codes ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 7168), (3, 5), (7, 16), (5, 130), (2, 1000), (300, 257), (9, 2048),
                                    (4, 16384), (3, 20001), (2, 65536)])
def test_quant_rows(dtype, rows, k):
    x, v = _x(rows, k, dtype, rows * 7 + k, sigma=3.0)
    q, s = moe.quant_rows_i8(x)
    codes, scales = ref.quant(v)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales)
    assert np.array_equal(q.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quant_rows_borders(dtype):
    """Quotients on and next to the middle between two codes, rows of zeros, the smallest and largest magnitudes."""
    import torch
    k = 512
    t = torch.zeros(12, k, dtype=torch.float64)
    t[0] = torch.arange(k) / 2.0 - 127.0            # scale 1: every half
    t[0, -1] = 127.0
    t[0] = t[0].clamp(-127, 127)
    t[1] = t[0] * 0.5
    t[2] = t[0] * 3.0 / 7.0
    t[3] = 0.0
    t[4, 5] = 2.0 ** -149                           # a scale that rounds to 0
    t[5] = torch.arange(k) * 2.0 ** -149            # subnormals: codes past 127 are cut
    t[6] = (torch.arange(k) - 200) * 2.0 ** -126
    t[7] = torch.linspace(-1, 1, k) * 6e4
    t[8] = torch.linspace(-1, 1, k) * 1e38
    t[9, 0] = 3.0
    t[10] = -0.0
    t[11] = (torch.arange(k) % 255 - 127 + 0.5) * (1 + 2.0 ** -12)
    x = t.to(ref.torch_dtype(dtype))
    x = torch.where(torch.isinf(x), torch.zeros_like(x), x)
    q, s = moe.quant_rows_i8(x.cuda())
    codes, scales = ref.quant(x.double().numpy())
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales)
    assert np.array_equal(q.cpu().numpy(), codes), np.argwhere(q.cpu().numpy() != codes)[:5]


def test_quant_rows_of_nan_and_infinity():
    import torch
    x = torch.randn(5, 300)
    x[1, 299], x[2, 0], x[3, 17] = float("nan"), float("inf"), float("-inf")
    for dtype in ("bf16", "f16", "f32"):
        q, s = moe.quant_rows_i8(x.to(ref.torch_dtype(dtype)).cuda())
        assert torch.isnan(s).tolist() == [False, True, True, True, False]
        assert not q[1:4].any() and q[0].any() and q[4].any()


def test_quant_rows_strides():
    import torch
    for dtype in ("bf16", "f32"):
        wide, v = _x(6, 700, dtype, 3)
        for part, pv in ((wide[:, 1:302], v[:, 1:302]), (wide[::2, 8:520], v[::2, 8:520]), (wide[:, 3:4], v[:, 3:4])):
            q, s = moe.quant_rows_i8(part)
            codes, scales = ref.quant(pv)
            assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy().astype(np.float64), scales)
    q = torch.full((4, 64), 9, dtype=torch.int8, device="cuda")
    s = torch.full((4,), 9.0, device="cuda")
    x, v = _x(2, 64, "bf16", 1)
    moe.quant_rows_i8(x, q=q[:2], scale=s[:2])
    assert (q[2:] == 9).all() and (s[2:] == 9).all()


# ---- the dense product --------------------------------------------------------------------------------------------

SHAPES = [(1, 1, 16), (1, 16, 64), (1, 640, 7168), (2, 33, 48), (3, 17, 80), (5, 100, 1040), (16, 33, 256), (17, 100, 272),
          (31, 64, 4096), (64, 96, 528), (65, 130, 1040), (100, 515, 336), (129, 257, 528), (256, 256, 128), (300, 512, 64),
          (257, 1030, 400), (513, 770, 144), (1000, 1111, 272)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm(m, n, k, swiglu):
    kinds = ["bf16", "f16", "f32"]
    dtype, out = kinds[(m + n) % 3], kinds[(n + k // 16) % 3]
    x, v = _x(m, k, dtype, m + 3 * n + k)
    w, ws = _w((2, n, k) if swiglu else (n, k), k + n)
    y = moe.gemm_i8(x, _dev(w), _dev(ws), swiglu=swiglu, out_dtype=ref.torch_dtype(out))
    codes, scales = ref.quant(v)
    if swiglu:
        g, u = ref.product(codes, scales, w[0], ws[0]), ref.product(codes, scales, w[1], ws[1])
        _close(y, ref.silu(g) * u, ref.swiglu_bound(g, u, out))
    else:
        want = ref.product(codes, scales, w, ws)
        _close(y, want, ref.product_bound(want, out))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [1, 20, 150])
def test_gemm_types(dtype, out, m):
    n, k = 200, 320
    x, v = _x(m, k, dtype, m)
    w, ws = _w((n, k), 8)
    want = ref.product(*ref.quant(v), w, ws)
    _close(moe.gemm_i8(x, _dev(w), _dev(ws), out_dtype=ref.torch_dtype(out)), want, ref.product_bound(want, out))


@pytest.mark.parametrize("m", [1, 4, 40, 300])
def test_gemm_of_codes(m):
    """Rows that are codes already, rows apart, and the same answer as from the float rows."""
    import torch
    n, k = 150, 416
    x, v = _x(m, k, "bf16", m)
    w, ws = _w((n, k), 2)
    q, s = moe.quant_rows_i8(x)
    wide = torch.full((m, k + 48), 77, dtype=torch.int8, device="cuda")
    wide[:, :k] = q
    a = moe.gemm_i8(wide[:, :k], _dev(w), _dev(ws), x_scale=s, out_dtype=torch.float32)
    b = moe.gemm_i8(x, _dev(w), _dev(ws), out_dtype=torch.float32)
    assert torch.equal(a, b)
    want = ref.product(*ref.quant(v), w, ws)
    _close(a, want, ref.product_bound(want, "f32"))


@pytest.mark.parametrize("m", [1, 17, 200])
def test_gemm_float_rows_apart(m):
    x, v = _x(m, 300, "f32", m)
    w, ws = _w((70, 96), 4)
    want = ref.product(*ref.quant(v[:, 5:101]), w, ws)
    _close(moe.gemm_i8(x[:, 5:101], _dev(w), _dev(ws)), want, ref.product_bound(want, "bf16"))


@pytest.mark.parametrize("m", [1, 16, 130])
def test_gemm_largest_sums(m):
    """Every code at its end, K at its limit: the sums stay inside int32 and exact."""
    import torch
    n, k = 40, 65536
    q = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    q[:, ::2] = 127
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[::2] = 127
    w[3] = q[0]
    ones_m, ones_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    y = moe.gemm_i8(q, w, ones_n, x_scale=ones_m, out_dtype=torch.float32)
    want = q[:1].cpu().numpy().astype(np.float64) @ w.cpu().numpy().astype(np.float64).T
    _close(y, np.repeat(want, m, 0), np.abs(want) * 2.0 ** -24)


@pytest.mark.parametrize("m", [3, 90])
def test_gemm_bad_and_empty_rows(m):
    """A row with a NaN gives a row of NaN and no other; a row of zeros gives zeros; far gates stay finite."""
    import torch
    n, k = 64, 128
    x, _ = _x(m, k, "f32", 1)
    x[1, 5] = float("nan")
    x[2] = 0.0
    w, ws = _w((2, n, k), 2)
    y = moe.gemm_i8(x, _dev(w[0]), _dev(ws[0]), out_dtype=torch.float32)
    assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any() and (y[2] == 0).all()
    h = moe.gemm_i8(x * 3e4, _dev(w), _dev(ws), swiglu=True, out_dtype=torch.float32)
    assert torch.isnan(h[1]).all() and torch.isfinite(h[0]).all() and (h[2] == 0).all()


def test_gemm_leaves_the_rest_alone():
    import torch
    for m, n in ((1, 50), (20, 50), (70, 260), (300, 300)):
        x, _ = _x(m, 160, "bf16", m)
        w, ws = _w((n, 160), 2)
        buf = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.gemm_i8(x, _dev(w), _dev(ws), out=buf[:m * n].view(m, n))
        assert (buf[m * n:] == 7).all() and not (buf[:m * n] == 7).all()


# ---- slots by expert ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("tokens,k,E", [(1, 1, 1), (1, 16, 896), (8, 16, 128), (64, 8, 256), (3, 2, 4096), (100, 64, 1500),
                                        (1000, 6, 60), (777, 16, 896), (5000, 8, 64), (33333, 3, 1024), (40000, 8, 4096),
                                        (20000, 16, 7)])
def test_group_slots(tokens, k, E):
    rng = np.random.default_rng(tokens + E)
    idx = rng.integers(0, E, (tokens, k)).astype(np.int32)
    idx[rng.random((tokens, k)) < 0.1] = -1
    idx[rng.random((tokens, k)) < 0.02] = E
    idx[0, 0] = 2 ** 31 - 1
    order, offsets = ref.group_slots(idx, E)
    g = moe.moe_group_slots(_dev(idx), E)
    assert np.array_equal(g.offsets.cpu().numpy(), offsets)
    assert np.array_equal(g.order.cpu().numpy(), order)


@pytest.mark.parametrize("value", [-1, 0, 5])
@pytest.mark.parametrize("tokens", [1, 130, 9000])
def test_group_slots_all_alike(value, tokens):
    idx = np.full((tokens, 4), value, np.int32)
    order, offsets = ref.group_slots(idx, 6)
    g = moe.moe_group_slots(_dev(idx), 6)
    g = moe.moe_group_slots(_dev(idx), 6, groups=g)  # a buffer used again
    assert np.array_equal(g.offsets.cpu().numpy(), offsets) and np.array_equal(g.order.cpu().numpy(), order)


# ---- the experts' products ----------------------------------------------------------------------------------------


def _experts_case(tokens, top_k, E, n, k, swiglu, by_slot, dtype, out, idx=None):
    import torch
    rng = np.random.default_rng(tokens * 13 + n + k)
    if idx is None:
        idx = rng.integers(-1, E, (tokens, top_k)).astype(np.int32)
    x, v = _x(tokens * top_k if by_slot else tokens, k, dtype, tokens + k)
    w, ws = _w((E, 2, n, k) if swiglu else (E, n, k), n)
    g = moe.moe_group_slots(_dev(idx), E)
    y = torch.full((tokens * top_k + 1, n), 5.0, dtype=ref.torch_dtype(out), device="cuda")
    moe.experts_gemm_i8(x, g, _dev(w), _dev(ws), swiglu=swiglu, out=y[:-1])
    assert (y[-1] == 5).all()
    codes, scales = ref.quant(v)
    want, bound = np.zeros((tokens * top_k, n)), np.full((tokens * top_k, n), 0.0)
    flat = idx.reshape(-1)
    for s in range(tokens * top_k):
        e, r = flat[s], s if by_slot else s // top_k
        if not 0 <= e < E:
            continue
        c, sc = codes[r:r + 1], scales[r:r + 1]
        if swiglu:
            a, b = ref.product(c, sc, w[e, 0], ws[e, 0]), ref.product(c, sc, w[e, 1], ws[e, 1])
            want[s], bound[s] = (ref.silu(a) * b)[0], ref.swiglu_bound(a, b, out)[0]
        else:
            a = ref.product(c, sc, w[e], ws[e])
            want[s], bound[s] = a[0], ref.product_bound(a, out)[0]
    _close(y[:-1], want, bound)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("tokens,top_k,E,n,k", [
    (1, 1, 1, 16, 64), (1, 16, 32, 48, 272), (8, 6, 20, 33, 1040), (64, 2, 4, 130, 128), (50, 8, 3, 100, 80),
    (333, 4, 5, 64, 144), (600, 2, 2, 260, 64)])
def test_experts(tokens, top_k, E, n, k, swiglu, by_slot):
    kinds = ["bf16", "f16", "f32"]
    _experts_case(tokens, top_k, E, n, k, swiglu, by_slot, kinds[(n + E) % 3], kinds[(tokens + k // 16) % 3])


@pytest.mark.parametrize("tokens", [1, 40, 400])
@pytest.mark.parametrize("value", [-1, 2, 7])
def test_experts_all_alike(tokens, value):
    """No slot has an expert (zeros), one expert has every slot, an index that is past the last expert."""
    _experts_case(tokens, 2, 6, 96, 112, False, False, "bf16", "bf16", idx=np.full((tokens, 2), value, np.int32))


def test_experts_same_expert_twice_in_a_row():
    _experts_case(5, 3, 4, 64, 64, False, True, "f32", "f32", idx=np.array([[1, 1, 1], [3, 3, 0], [0, 0, 0], [2, 1, 2], [3, 3, 3]],
                                                                           np.int32))


def test_experts_of_codes():
    import torch
    tokens, top_k, E, n, k = 30, 4, 8, 80, 192
    idx = np.random.default_rng(0).integers(0, E, (tokens, top_k)).astype(np.int32)
    x, _ = _x(tokens, k, "bf16", 3)
    w, ws = _w((E, n, k), 1)
    q, s = moe.quant_rows_i8(x)
    g = moe.moe_group_slots(_dev(idx), E)
    a = moe.experts_gemm_i8(x, g, _dev(w), _dev(ws))
    assert torch.equal(a, moe.experts_gemm_i8(q, g, _dev(w), _dev(ws), x_scale=s))


# ---- the gated sum --------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,top_k,hidden", [(1, 1, 1), (1, 16, 7168), (3, 2, 33), (70, 8, 256), (9, 64, 100), (5, 3, 1030),
                                                 (70000, 1, 8)])
def test_combine(dtype, tokens, top_k, hidden):
    import torch
    y, v = _x(tokens * top_k, hidden, dtype, tokens)
    rng = np.random.default_rng(hidden)
    gate, res = rng.random((tokens, top_k)).astype(np.float32), rng.standard_normal((tokens, hidden)).astype(np.float32)
    terms = v.reshape(tokens, top_k, hidden) * gate[:, :, None].astype(np.float64)
    size = np.abs(terms).sum(1)
    for r in (None, res):
        want = terms.sum(1) + (0 if r is None else r)
        bound = (size + (0 if r is None else np.abs(r))) * (top_k + 1) * 2.0 ** -24
        rt = None if r is None else _dev(r)
        got = moe.moe_combine(y, _dev(gate), residual=rt)
        _close(got, want, bound)
        if rt is not None:
            moe.moe_combine(y, _dev(gate), residual=rt, out=rt)
            assert torch.equal(rt, got)


# ---- together ---------------------------------------------------------------------------------------------------------


class _Layer:
    """A mixture-of-experts block in 8 bits: routing, the experts' two products, the gated sum."""

    def __init__(self, tokens, hidden, inter, E, top_k, seed=0):
        import torch
        self.E, self.k = E, top_k
        self.w1, self.s1 = map(_dev, _w((E, 2, inter, hidden), seed))
        self.w2, self.s2 = map(_dev, _w((E, hidden, inter), seed + 1))
        self.bias = _dev((np.random.default_rng(seed).standard_normal(E) * 0.1).astype(np.float32))
        empty = lambda *s, dtype: torch.empty(s, dtype=dtype, device="cuda")
        self.idx, self.gate = empty(tokens, top_k, dtype=torch.int32), empty(tokens, top_k, dtype=torch.float32)
        self.groups = moe.alloc_slot_groups(tokens, top_k, E)
        self.h = empty(tokens * top_k, inter, dtype=torch.bfloat16)
        self.y = empty(tokens * top_k, hidden, dtype=torch.bfloat16)
        size = max(moe.experts_gemm_i8_workspace_size(self.groups, tokens, inter, hidden, True, torch.bfloat16),
                   moe.experts_gemm_i8_workspace_size(self.groups, tokens * top_k, hidden, inter, False, torch.bfloat16))
        self.ws = empty(size, dtype=torch.uint8)

    def __call__(self, logits, x, residual, out, stream=None):
        moe.moe_route(logits, self.k, bias=self.bias, score="sigmoid", groups=4, top_groups=2, group_top=2, scale=2.5,
                      idx=self.idx, gate=self.gate, stream=stream)
        moe.moe_group_slots(self.idx, self.E, groups=self.groups, stream=stream)
        moe.experts_gemm_i8(x, self.groups, self.w1, self.s1, swiglu=True, out=self.h, ws=self.ws, stream=stream)
        moe.experts_gemm_i8(self.h, self.groups, self.w2, self.s2, out=self.y, ws=self.ws, stream=stream)
        return moe.moe_combine(self.y, self.gate, residual=residual, out=out, stream=stream)

    def reference(self, logits, x, residual):
        idx, gate = ref.route(logits, self.k, bias=self.bias.cpu().numpy(), score="sigmoid", groups=4, top_groups=2,
                              group_top=2, scale=2.5)
        w1, s1, w2, s2 = (t.cpu().numpy() for t in (self.w1, self.s1, self.w2, self.s2))
        out = residual.astype(np.float64).copy()
        c, s = ref.quant(x)
        for t in range(x.shape[0]):
            for j in range(self.k):
                e = idx[t, j]
                if e < 0:
                    continue
                g, u = (ref.product(c[t:t + 1], s[t:t + 1], w1[e, p], s1[e, p]) for p in (0, 1))
                out[t] += gate[t, j] * ref.product(*ref.quant(ref.silu(g) * u), w2[e], s2[e])[0]
        return idx, out


def _layer_inputs(tokens, hidden, E, seed):
    import torch
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((tokens, E)) * 1.7).astype(np.float32)
    if tokens > 2:
        logits[tokens - 2:] = -np.inf  # padded rows
    x, v = _x(tokens, hidden, "bf16", seed)
    residual = rng.standard_normal((tokens, hidden)).astype(np.float32)
    return logits, x, v, residual


@pytest.mark.parametrize("tokens,hidden,inter", [(1, 512, 256), (7, 256, 128), (150, 256, 144)])
def test_layer(tokens, hidden, inter):
    """The operators in a row against the chain in 64 bits.  Codes of the inner rows that lie next to a border may
    fall on the other side (their bf16 rounding moves them by up to 2^-9 of a value, half a code at most): the row's
    relative error stays under 2 * 2^-9 """
    import torch
    E, k = 16, 4
    layer = _Layer(tokens, hidden, inter, E, k)
    logits, x, v, residual = _layer_inputs(tokens, hidden, E, tokens)
    out = torch.empty(tokens, hidden, device="cuda")
    layer(_dev(logits), x, _dev(residual), out)
    idx, want = layer.reference(logits, v, residual)
    assert np.array_equal(layer.idx.cpu().numpy(), idx)
    got = out.cpu().numpy().astype(np.float64)
    part = want - residual
    err = np.linalg.norm(got - want, axis=1) / np.maximum(np.linalg.norm(part, axis=1), 1e-30)
    assert (err[np.linalg.norm(part, axis=1) > 0] <= 2e-2).all(), err.max()
    empty = (idx < 0).all(1)
    assert np.array_equal(got[empty], residual[empty].astype(np.float64))


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_layer_in_a_graph_and_on_another_stream(tokens):
    """Captured once and replayed on new inputs, with the program's own eager work in between; and eagerly on a side
    stream: the same bits as an eager run."""
    import torch
    hidden, inter, E, k = 256, 128, 16, 4
    layer, check = _Layer(tokens, hidden, inter, E, k), _Layer(tokens, hidden, inter, E, k)
    ins = [_layer_inputs(tokens, hidden, E, 50 + i) for i in range(4)]
    logits, x, res, out = _dev(ins[0][0]), ins[0][1].clone(), _dev(ins[0][3]), torch.empty(tokens, hidden, device="cuda")
    want_out = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(logits, x, res, out)
    s.synchronize()
    check(logits, x, res, want_out)
    torch.cuda.synchronize()
    assert torch.equal(out, want_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer(logits, x, res, out)
    for lg, xi, _, ri in ins + ins[:2]:
        logits.copy_(_dev(lg))
        x.copy_(xi)
        res.copy_(_dev(ri))
        torch.cuda.synchronize()
        graph.replay()
        check(logits, x, res, want_out)
        torch.cuda.synchronize()
        assert torch.equal(out, want_out)


def test_two_streams_at_once():
    """Two layers with their own buffers on two streams: each has the bits of a run alone."""
    import torch
    hidden, inter, E, k, tokens = 256, 128, 16, 4, 200
    layers = [_Layer(tokens, hidden, inter, E, k, seed=i) for i in range(2)]
    ins = [_layer_inputs(tokens, hidden, E, i) for i in range(2)]
    dev = [(_dev(i[0]), i[1], _dev(i[3])) for i in ins]
    alone = [l(*d, torch.empty(tokens, hidden, device="cuda")).clone() for l, d in zip(layers, dev)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty(tokens, hidden, device="cuda") for _ in range(2)]
    for _ in range(5):
        for l, d, s, o in zip(layers, dev, streams, outs):
            l(*d, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


# ---- one float row, quantised inside the product ------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,k", [(1, 16), (40, 112), (33, 128), (100, 1040), (77, 4096), (64, 8064), (50, 16256), (50, 16272), (24, 65536)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_gemm_of_one_row(dtype, n, k, swiglu):
    """Every length of the row, past the one that a workgroup quantises too; the bits of the two calls in a row."""
    import torch
    x, v = _x(1, k, dtype, n + k, sigma=2.0)
    w, ws = _w((2, n, k) if swiglu else (n, k), k)
    y = moe.gemm_i8(x, _dev(w), _dev(ws), swiglu=swiglu, out_dtype=torch.float32)
    codes, scales = ref.quant(v)
    if swiglu:
        g, u = ref.product(codes, scales, w[0], ws[0]), ref.product(codes, scales, w[1], ws[1])
        _close(y, ref.silu(g) * u, ref.swiglu_bound(g, u, "f32"))
    else:
        want = ref.product(codes, scales, w, ws)
        _close(y, want, ref.product_bound(want, "f32"))
    q, s = moe.quant_rows_i8(x)
    assert torch.equal(y, moe.gemm_i8(q, _dev(w), _dev(ws), x_scale=s, swiglu=swiglu, out_dtype=torch.float32))


def test_gemm_of_one_row_extremes():
    import torch
    n, k = 48, 640
    w, ws = _w((n, k), 3)
    for fill in (0.0, float("nan"), float("inf"), 2.0 ** -149, 3e38):
        x = torch.zeros(1, k)
        x[0, 7] = fill
        x[0, 300] = 2.0 ** -140
        y = moe.gemm_i8(x.cuda(), _dev(w), _dev(ws), out_dtype=torch.float32)
        q, s = moe.quant_rows_i8(x.cuda())
        z = moe.gemm_i8(q, _dev(w), _dev(ws), x_scale=s, out_dtype=torch.float32)
        assert torch.equal(torch.isnan(y), torch.isnan(z)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(z))
    x = torch.randn(1, k + 3)[:, 3:].cuda()  # not 16-byte aligned
    q, s = moe.quant_rows_i8(x)
    assert torch.equal(moe.gemm_i8(x, _dev(w), _dev(ws)), moe.gemm_i8(q, _dev(w), _dev(ws), x_scale=s))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("idx", [[5], [0, 3, 5, 2], [1, -1, 1, 4], [-1, -1], [2] * 20, list(range(6)) * 8])
def test_experts_of_one_token(idx, swiglu):
    """One token: distinct experts, one that comes twice, none, more slots than a tile."""
    _experts_case(1, len(idx), 6, 50, 272, swiglu, False, "bf16", "f32", idx=np.array([idx], np.int32))


def test_memory_of_a_call_on_another_stream():
    """A call given a stream makes its outputs and workspace there: what the current stream allocates and writes while
    that stream still works never lands in them."""
    import torch
    m, n, k, top_k, E = 48, 512, 1024, 2, 4
    g = torch.Generator().manual_seed(5)
    x = torch.randn(m, k, generator=g).cuda()
    w = torch.randint(-127, 128, (E, n, k), generator=g, dtype=torch.int8).cuda()
    s = torch.rand(E, n, generator=g).cuda()
    logits = torch.randn(m, E, generator=g).cuda()

    def run(stream):
        idx, gate = moe.moe_route(logits, top_k, stream=stream)
        groups = moe.moe_group_slots(idx, E, stream=stream)
        q, qs = moe.quant_rows_i8(x, stream=stream)
        y = moe.experts_gemm_i8(x, groups, w, s, stream=stream)
        return (idx, gate, groups.order, groups.offsets, q, qs, moe.gemm_i8(x, w[0], s[0], stream=stream), y,
                moe.moe_combine(y, gate, stream=stream))

    want = [t.clone() for t in run(None)]
    need = moe.gemm_i8_workspace_size(m, n, k, False, torch.float32)
    torch.cuda.synchronize()
    for as_int in (False, True):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the calls below wait behind this
        got = run(side.cuda_stream if as_int else side)
        trash = [torch.full((size,), 0x55, dtype=torch.uint8, device="cuda")
                 for size in (need, m * k, 4 * m, 1 << 16, 1 << 12) for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        assert all(bool((t == 0x55).all()) for t in trash)


def _codes_case(rows, w_shape, k, seed):
    """Codes and scales on the GPU, and the scaled products in float64 (of whole numbers, so exact before the scales)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (rows, k), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-127, 128, w_shape + (k,), generator=g, dtype=torch.int8).cuda()
    s = (torch.rand(rows, generator=g) * 1e-3 + 1e-4).cuda()
    ws = (torch.rand(w_shape, generator=g) * 1e-3 + 1e-4).cuda()

    def product(take, w, ws):
        return (q[take].double() @ w.double().t()) * (s[take].double()[:, None] * ws.double()[None])

    return q, s, w, ws, product


@pytest.mark.parametrize("m,n,k,swiglu", [
    # few rows of a narrow matrix, and 64 x 64 tiles with K in one and in several parts
    (37, 520, 7184, False), (20, 4100, 272, False), (20, 2050, 1040, True), (70, 4100, 7184, False), (20, 4100, 7184, False),
    (20, 2050, 7184, True), (33, 3000, 7184, False), (130, 520, 7184, True), (700, 100, 7184, True), (60, 200, 16400, False),
    # 64 x 128
    (200, 4100, 80, False), (200, 4100, 272, False), (200, 4100, 7184, False), (70, 4100, 2064, True), (70, 4104, 1152, True),
    # 128 x 128, one and two to a CU
    (1000, 2050, 272, False), (1000, 2050, 7184, False), (200, 4100, 1040, True), (513, 7000, 272, False),
    (1000, 2050, 1040, True), (1000, 4100, 2064, False),
    # 256 x 256
    (1500, 7000, 80, False), (1500, 7000, 1040, False), (1500, 7000, 256, False), (700, 7000, 2064, True)])
def test_gemm_tiles(m, n, k, swiglu):
    """The sizes at which each kernel and tile is taken, with rows, columns and K that end inside one."""
    import torch
    q, s, w, ws, product = _codes_case(m, (2, n) if swiglu else (n,), k, m + n + k)
    every = slice(None)
    for out in ("f32", "bf16"):
        y = moe.gemm_i8(q, w, ws, x_scale=s, swiglu=swiglu, out_dtype=ref.torch_dtype(out))
        torch.cuda.synchronize()
        if swiglu:
            g, u = (product(every, w[i], ws[i]).cpu().numpy() for i in range(2))
            _close(y, ref.silu(g) * u, ref.swiglu_bound(g, u, out))
        else:
            want = product(every, w, ws).cpu().numpy()
            _close(y, want, ref.product_bound(want, out))


@pytest.mark.parametrize("tokens,top_k,E,n,k,swiglu", [
    (24, 2, 16, 1030, 1040, False), (20, 6, 40, 100, 7184, True), (3, 2, 2, 100, 7184, False), (60, 2, 40, 520, 1040, False),
    (160, 2, 16, 1030, 7184, False), (1400, 2, 40, 520, 272, False), (175, 2, 5, 2050, 1040, True), (60, 2, 40, 2050, 2064, False),
    (60, 2, 40, 1030, 1040, False), (800, 2, 40, 520, 7184, True), (3000, 2, 40, 1030, 272, False), (3000, 2, 40, 520, 1040, True),
    (1500, 4, 40, 1030, 2064, False)])
def test_experts_tiles(tokens, top_k, E, n, k, swiglu):
    """The same for the experts: some with many rows, some with few or none, and slots without an expert."""
    import torch
    q, s, w, ws, product = _codes_case(tokens, (E, 2, n) if swiglu else (E, n), k, tokens + n + k)
    g = torch.Generator().manual_seed(k)
    idx = (torch.rand(tokens, top_k, generator=g) ** 2 * (E + 1)).to(torch.int32) - 1
    idx[idx == E // 2] = 0
    groups = moe.moe_group_slots(idx.cuda(), E)
    for out in ("f32", "bf16"):
        y = moe.experts_gemm_i8(q, groups, w, ws, x_scale=s, swiglu=swiglu, out_dtype=ref.torch_dtype(out))
        torch.cuda.synchronize()
        flat = idx.flatten()
        assert bool((y[(flat < 0).nonzero()[:, 0].cuda()] == 0).all())
        for e in range(E):
            slots = (flat == e).nonzero()[:, 0]
            if not len(slots):
                continue
            rows = (slots // top_k).cuda()
            got = y[slots.cuda()]
            if swiglu:
                a, b = (product(rows, w[e, i], ws[e, i]).cpu().numpy() for i in range(2))
                _close(got, ref.silu(a) * b, ref.swiglu_bound(a, b, out))
            else:
                want = product(rows, w[e], ws[e]).cpu().numpy()
                _close(got, want, ref.product_bound(want, out))


def test_experts_of_one_token_with_the_widest_matrices():
    """More workgroups than the launch of a single row holds: the rows go the way of several."""
    import torch
    E, top_k, n, k = 40, 64, 1 << 20, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randint(-127, 128, (E, 2, n, k), generator=g, dtype=torch.int8, device="cuda")
    ws = torch.rand(E, 2, n, generator=g, device="cuda") * 1e-2 + 1e-3
    x, v = _x(1, k, "bf16", 3)
    idx = (torch.arange(top_k, dtype=torch.int32, device="cuda") * 7 % (E + 1) - 1)[None]
    y = moe.experts_gemm_i8(x, moe.moe_group_slots(idx, E), w, ws, swiglu=True, out_dtype=torch.float32)
    codes, scales = ref.quant(v)
    at = torch.tensor([0, 1, 15, 16, 4095, n // 2 + 3, n - 17, n - 1], device="cuda")
    for j, e in enumerate(idx[0].tolist()):
        if e < 0:
            assert bool((y[j] == 0).all())
            continue
        a, b = (ref.product(codes, scales, w[e, i, at].cpu().numpy(), ws[e, i, at].cpu().numpy()) for i in range(2))
        _close(y[j, at][None], ref.silu(a) * b, ref.swiglu_bound(a, b, "f32"))


@pytest.mark.parametrize("tokens,n,k", [(20, 1030, 1040), (800, 520, 272), (3000, 1030, 272)])
def test_experts_of_a_groups_buffer_of_any_content(tokens, n, k):
    """A buffer that was never filled: the outputs mean nothing, but no other memory is touched, and the next call
    with slots in it is right."""
    import torch
    top_k, E = 2, 40
    q, s, w, ws, product = _codes_case(tokens, (E, n), k, tokens + n)
    groups = moe.alloc_slot_groups(tokens, top_k, E)
    words = groups.buffer.view(torch.int32)
    y = torch.full((tokens * top_k + 8, n), 5.0, device="cuda")
    rng = torch.Generator(device="cuda").manual_seed(tokens)
    for fill in (-1, 0, -1331422904, 0x7FFFFFFF, None):
        if fill is None:
            words.copy_(torch.randint(-2 ** 31, 2 ** 31, words.shape, generator=rng, device="cuda").to(torch.int32))
        else:
            words.fill_(fill)
        moe.experts_gemm_i8(q, groups, w, ws, x_scale=s, out=y[4:-4])
        torch.cuda.synchronize()
        assert bool((y[:4] == 5).all()) and bool((y[-4:] == 5).all())
    idx = torch.randint(0, E, (tokens, top_k), generator=rng, dtype=torch.int32, device="cuda")
    got = moe.experts_gemm_i8(q, moe.moe_group_slots(idx, E, groups=groups), w, ws, x_scale=s, out_dtype=torch.float32)
    slots = (idx.flatten() == 3).nonzero()[:, 0]
    want = product(slots // top_k, w[3], ws[3]).cpu().numpy()
    _close(got[slots], want, ref.product_bound(want, "f32"))


# Sizes of each kernel, without and with SwiGLU: one row, few rows, 64 x 64 tiles with K in one and in parts, 64 x 128,
# 128 x 128 (one and two to a CU) and 256 x 256.
ALL_KERNELS = [(1, 520, 272), (9, 520, 272), (20, 4100, 272), (60, 200, 16400), (200, 4100, 272), (70, 4104, 1152),
               (1000, 2050, 272), (513, 7000, 272), (1500, 7000, 80)]


@pytest.mark.parametrize("size", [1e-37, 1e-36, 1e-34, 1e-20, 1e33, 1e36])
@pytest.mark.parametrize("m,n,k", ALL_KERNELS)
def test_gemm_of_small_and_large_rows(m, n, k, size):
    """Rows whose scale times a matrix scale is no normal fp32 number, or whose sums times their scale are none: the
    outputs are, and stay within the three roundings."""
    x, v = _x(m, k, "f32", m + n, sigma=size)
    w, ws = _w((n, k), k)
    at = np.unique(np.linspace(0, m - 1, 40).astype(int))
    codes, scales = ref.quant(v[at])
    want = ref.product(codes, scales, w, ws)
    y = moe.gemm_i8(x, _dev(w), _dev(ws), out_dtype=ref.torch_dtype("f32"))
    _close(y[at], want, ref.product_bound(want, "f32"))


@pytest.mark.parametrize("m,n,k", ALL_KERNELS)
def test_gemm_sum_of_zero_under_large_scales(m, n, k):
    """0 times two finite scales is 0, also where the scales' product overflows."""
    import torch
    w, _ = _w((n, k), 5)
    q = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    q[-1] = 1
    for a, b in ((8e35, 500.0), (500.0, 8e35)):
        xs, ws = torch.full((m,), a, device="cuda"), torch.full((n,), b, device="cuda")
        y = moe.gemm_i8(q, _dev(w), ws, x_scale=xs, out_dtype=torch.float32)
        assert not bool(y[:-1].any()) and not bool(y.isnan().any())
    # the same within a float row: a 1 and a -1 meet matrix rows of ones
    x = torch.zeros(m, k, device="cuda")
    x[:, 0], x[:, 1] = 1e38, -1e38
    y = moe.gemm_i8(x, torch.ones(n, k, dtype=torch.int8, device="cuda"), torch.full((n,), 1e4, device="cuda"),
                    out_dtype=torch.float32)
    assert not bool(y.any()) and not bool(y.isnan().any())


@pytest.mark.parametrize("size", [1e-36, 1e33])
@pytest.mark.parametrize("tokens,top_k,E,n,k", [(1, 4, 6, 48, 272), (20, 2, 40, 130, 1040), (3000, 2, 40, 520, 80)])
def test_experts_of_small_and_large_rows(tokens, top_k, E, n, k, size):
    x, v = _x(tokens, k, "f32", tokens, sigma=size)
    w, ws = _w((E, n, k), k)
    idx = np.random.default_rng(tokens).integers(0, E, (tokens, top_k)).astype(np.int32)
    y = moe.experts_gemm_i8(x, moe.moe_group_slots(_dev(idx), E), _dev(w), _dev(ws), out_dtype=ref.torch_dtype("f32"))
    for s in np.unique(np.linspace(0, tokens * top_k - 1, 60).astype(int)):
        codes, scales = ref.quant(v[s // top_k][None])
        e = idx.reshape(-1)[s]
        want = ref.product(codes, scales, w[e], ws[e])
        _close(y[int(s)][None], want, ref.product_bound(want, "f32"), s)


@pytest.mark.parametrize("m,n,k", ALL_KERNELS)
def test_gemm_swiglu_of_very_negative_gates(m, n, k):
    """silu(g) * u where exp(-g) overflows fp32 but silu(g), or its product with a large u, does not vanish.  The sums
    are 1 and the gates and ups the matrix scales themselves, exactly.  Below -80 the kernel takes two factors
    exp((g + 80) / 2) (2 roundings each, as any exponential), a constant and four products, so 9 roundings; above, an
    exponential, a sum, a quotient and a product, 5.  Products that end below fp32's normal numbers: half a step each."""
    import torch
    g = -np.concatenate([np.linspace(70, 104, 137), [80, 88.7, 88.75, 89, 120, 150, 174, 175, 200, 254, 300, 301, 1e4, 1e38]])
    u = np.array([1.0, -0.3, 1e-8, 1e10, -1e25, 3e38])
    g, u = (a.ravel().astype(np.float32) for a in np.meshgrid(g, u))
    at = np.resize(np.random.default_rng(1).permutation(len(g)), n)
    g, u = g[at], u[at]
    w = np.zeros((2, n, k), np.int8)
    w[0, :, 3], w[1, :, 3] = -1, 1
    q = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    q[:, 3] = 1
    y = moe.gemm_i8(q, _dev(w), _dev(np.stack([-g, u])), x_scale=torch.ones(m, device="cuda"), swiglu=True,
                    out_dtype=torch.float32)
    assert torch.equal(y, y[:1].expand(m, n))
    want = ref.silu(g.astype(np.float64)) * u.astype(np.float64)
    _close(y[:1], want[None], np.abs(want)[None] * 9 * 2.0 ** -24 * 1.001 + 4 * 2.0 ** -150)
    # one float row that the kernel quantises itself, and as one expert's row
    x = torch.zeros(1, k, device="cuda")
    x[0, 3] = 127.0
    one = moe.gemm_i8(x, _dev(w), _dev(np.stack([-g, u]) / np.float32(128)), swiglu=True, out_dtype=torch.float32)
    g, u = (127.0 * (a / np.float32(128)).astype(np.float64) for a in (g, u))
    want, turn = ref.silu(g) * u, 2 * 2.0 ** -24 * (2 + np.abs(np.minimum(-g, 400)))  # g and u with one rounding each
    _close(one, want[None], np.abs(want)[None] * (9 * 2.0 ** -24 + turn) * 1.01 + 4 * 2.0 ** -150)


@pytest.mark.parametrize("tokens,hidden,inter", [(1, 512, 256), (7, 256, 128), (150, 256, 144), (700, 256, 272)])
def test_layer_stage_by_stage(tokens, hidden, inter):
    """The operators in a row, each against its definition in 64 bits on what the one before it left: every element
    within the roundings of its own step."""
    import torch
    E, k = 16, 4
    layer = _Layer(tokens, hidden, inter, E, k)
    logits, x, v, residual = _layer_inputs(tokens, hidden, E, tokens)
    out = torch.empty(tokens, hidden, device="cuda")
    layer(_dev(logits), x, _dev(residual), out)
    idx, gate = ref.route(logits, k, bias=layer.bias.cpu().numpy(), score="sigmoid", groups=4, top_groups=2, group_top=2,
                          scale=2.5)
    assert np.array_equal(layer.idx.cpu().numpy(), idx)
    _close(layer.gate, gate, np.abs(gate) * (2.0 ** -24 + 2.0 ** -40))
    flat, codes, scales = idx.reshape(-1), *ref.quant(v)
    h, y = layer.h.double().cpu().numpy(), layer.y.double().cpu().numpy()
    hc, hs = ref.quant(h)
    w1, s1, w2, s2 = (t.cpu().numpy() for t in (layer.w1, layer.s1, layer.w2, layer.s2))
    none = flat < 0
    assert not h[none].any() and not y[none].any()
    for e in range(E):
        slots = np.flatnonzero(flat == e)
        if not len(slots):
            continue
        g, u = (ref.product(codes[slots // k], scales[slots // k], w1[e, p], s1[e, p]) for p in (0, 1))
        _close(layer.h[torch.from_numpy(slots).cuda()], ref.silu(g) * u, ref.swiglu_bound(g, u, "bf16"), ("h", e))
        want = ref.product(hc[slots], hs[slots], w2[e], s2[e])
        _close(layer.y[torch.from_numpy(slots).cuda()], want, ref.product_bound(want, "bf16"), ("y", e))
    terms = layer.gate.double().cpu().numpy()[:, :, None] * y.reshape(tokens, k, hidden)
    # k multiplications with an addition, each rounded once, and the residual's addition
    _close(out, residual + terms.sum(1), (k + 1) * 2.0 ** -24 * 1.01 * (np.abs(terms).sum(1) + np.abs(residual)))
