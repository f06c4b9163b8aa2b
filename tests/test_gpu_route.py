"""GPU parity of moe_route against the plain 64-bit reference: expert indices
exactly, gates within the roundings of their computation."""
import numpy as np
import pytest

import i8_reference as ref
import memory_bound_mxfp4_amd as moe

pytestmark = pytest.mark.gpu

# A gate is s / sum: each score one exponential (2 steps of 2^-24 and the argument's rounding, at most 0.37 of one
# weighted by its term) and, where a sum of up to 4096 terms is taken in fp32, chains of at most 16 + 10 additions;
# a quotient, a product and the final rounding: under 32 roundings in all.
GATE_REL = 32 * 2.0 ** -24


def _check(logits, dtype="f32", stride=None, idx_only=False, **kw):
    import torch
    lt = torch.from_numpy(np.ascontiguousarray(logits)).to(ref.torch_dtype(dtype)).cuda()
    seen = lt.float().cpu().numpy()
    if stride:
        wide = torch.full((lt.shape[0], stride), float("nan"), dtype=lt.dtype, device="cuda")
        wide[:, :lt.shape[1]] = lt
        lt = wide[:, :lt.shape[1]]
    bias = kw.get("bias")
    want_idx, want_gate = ref.route(seen, **kw)
    args = dict(kw)
    top_k = args.pop("top_k")
    if bias is not None:
        args["bias"] = torch.from_numpy(bias.astype(np.float32)).cuda()
    idx, gate = moe.moe_route(lt, top_k, **args)
    idx, gate = idx.cpu().numpy(), gate.cpu().numpy().astype(np.float64)
    assert np.array_equal(idx, want_idx), np.argwhere(idx != want_idx)[:5]
    bad = np.abs(gate - want_gate) > GATE_REL * np.abs(want_gate) + 2.0 ** -149
    assert not bad.any(), (np.argwhere(bad)[:5], gate[bad][:5], want_gate[bad][:5])
    return idx, gate


def _logits(rows, E, seed, sigma=1.7):
    return (np.random.default_rng(seed).standard_normal((rows, E)) * sigma).astype(np.float32)


def _bias(E, seed, sigma=0.1):
    return (np.random.default_rng(seed + 1000).standard_normal(E) * sigma).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rows,E,k,groups,top_groups,group_top", [
    (1, 1, 1, 1, 1, 1), (3, 7, 7, 1, 1, 1), (1, 896, 16, 1, 1, 1), (65, 160, 6, 8, 3, 1), (64, 256, 8, 8, 4, 2),
    (5, 63, 9, 3, 2, 2), (9, 65, 64, 1, 1, 1), (7, 320, 33, 64, 20, 2), (4, 1024, 32, 4, 1, 2), (2, 4096, 64, 1, 1, 1),
    (2, 3000, 5, 60, 7, 2), (33, 128, 1, 128 // 2, 1, 1)])
def test_route(dtype, score, biased, rows, E, k, groups, top_groups, group_top):
    seed = rows * 31 + E
    _check(_logits(rows, E, seed), dtype, top_k=k, bias=_bias(E, seed) if biased else None, score=score, groups=groups,
           top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm,scale", [(False, 1.0), (False, 16.0), (True, 2.5), (True, 0.0)])
def test_route_gates(score, renorm, scale):
    for E, biased in ((96, False), (896, True), (4096, False)):
        _check(_logits(11, E, E), top_k=12, score=score, renorm=renorm, scale=scale, bias=_bias(E, 5) if biased else None)


def test_route_row_stride():
    _check(_logits(17, 100, 3), "bf16", stride=131, top_k=4)
    _check(_logits(17, 256, 3), "f32", stride=260, top_k=4, bias=_bias(256, 3))
    _check(_logits(300, 64, 4), "f16", stride=65, top_k=3, groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("kw", [
    dict(), dict(score="sigmoid"), dict(bias=True), dict(score="sigmoid", bias=True), dict(groups=4, top_groups=2, group_top=2),
    dict(score="sigmoid", bias=True, groups=4, top_groups=3, group_top=1), dict(renorm=False)], ids=str)
def test_route_masks_and_extremes(kw):
    """Masked experts, padded rows, the lowest values, infinities and NaN: what is no candidate is never chosen."""
    E, k = 64, 6
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = _bias(E, 9)
        kw["bias"][[3, 17]] = -np.inf, np.nan
    l = _logits(16, E, 7)
    low = np.finfo(np.float32).min
    l[0] = -np.inf
    l[1] = np.nan
    l[2, :60] = -np.inf                     # four candidates for six places
    l[3, ::2] = -np.inf
    l[4, ::2] = low
    l[5] = low
    l[6, 10:50] = np.nan
    l[7, 5] = np.inf
    l[8, [5, 40]] = np.inf
    l[9, 5], l[9, 6] = np.inf, np.nan
    l[10] = 0.0
    l[11, :] = -0.0
    l[11, 3::5] = 0.0
    l[12] = np.finfo(np.float32).max
    l[13] = -1e30
    l[13, 20] = 5.0
    l[14] = np.where(np.arange(E) % 16 < 8, -np.inf, l[14])
    l[15] = np.round(l[15])                 # many ties
    _check(l, top_k=k, **kw)
    l16 = l.copy()
    l16[[4, 5, 12, 13]] = np.clip(l16[[4, 5, 12, 13]], -60000, 60000)
    _check(l16, "f16", top_k=k, **kw)
    _check(l16, "bf16", top_k=k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(score, biased):
    E = 200
    l = np.random.default_rng(3).integers(-2, 3, (40, E)).astype(np.float32)
    l[0] = 1.0
    bias = np.zeros(E, np.float32) if biased else None
    _check(l, top_k=20, score=score, bias=bias)
    _check(l, "bf16", top_k=20, score=score, bias=bias, groups=8, top_groups=3, group_top=2)
    _check(l, "bf16", top_k=20, score=score, bias=bias, groups=8, top_groups=3, group_top=1)
    _check(l[:4], top_k=64, score=score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_near_ties(score):
    """Scores that differ past the 24th bit: a comparison in fp32 would tie and take the lower index."""
    E, rows = 128, 32
    rng = np.random.default_rng(5)
    l = np.full((rows, E), -6.0, np.float32)
    bias = np.zeros(E, np.float32)
    for r in range(rows):
        at = rng.choice(E, 24, replace=False)
        base = np.float32(rng.uniform(0.5, 2.0))
        for i, e in enumerate(at):  # neighbouring fp32 logits, shuffled
            l[r, e] = base + np.float32(i) * np.spacing(base)
    _check(l, top_k=12, score=score)
    _check(l, top_k=12, score=score, bias=bias)
    _check(l, top_k=12, score=score, bias=bias, groups=16, top_groups=7, group_top=2)
    l[:, :] = rng.standard_normal((rows, 1)).astype(np.float32)  # equal logits, biases a step apart
    bias = (np.float32(0.25) + rng.permutation(E).astype(np.float32) * np.spacing(np.float32(0.25))).astype(np.float32)
    _check(l, top_k=40, score=score, bias=bias)


def test_route_bias_only_selects():
    l = _logits(6, 64, 2)
    bias = np.zeros(64, np.float32)
    bias[[60, 61]] = 1e6, -1e6
    idx, _ = _check(l, top_k=4, score="sigmoid", bias=bias)
    assert (idx[:, 0] == 60).all() and not (idx == 61).any()
    bias[60] = np.inf
    _check(l, top_k=4, score="softmax", bias=bias)


def test_route_long_prompt():
    """Every row of a long call, against its definition computed on the GPU in fp64."""
    import torch
    rows, E, k = 20011, 384, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    l = torch.randn(rows, E, generator=g, device="cuda") * 2
    b = torch.randn(E, generator=g, device="cuda") * 0.1
    idx, gate = moe.moe_route(l, k, bias=b, score="sigmoid")
    s = torch.sigmoid(l.double())
    want = torch.sort(s + b.double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx.long(), want)
    w = s.gather(1, want)
    w = w / w.sum(1, keepdim=True)
    assert ((gate.double() - w).abs() <= GATE_REL * w).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(160, 8, 3, 6), (64, 64, 5, 5), (4092, 33, 4, 16), (4096, 2, 1, 64), (96, 3, 3, 8),
                                                       (2048, 16, 2, 7)])
def test_route_groups_by_their_best(E, groups, top_groups, top_k, score, renorm):
    """Groups ranked by their best logit alone, some of them alike, some without a candidate."""
    l = _logits(40, E, E + groups)
    size = E // groups
    l[3, size:2 * size] = l[3, :size]                # two groups with the same logits
    l[4, :(groups - 1) * size] = -np.inf             # one group left
    l[5] = -np.inf                                   # none
    l[6, ::2] = np.nan
    l[7] = 1.5                                       # all alike
    _check(l, top_k=top_k, score=score, groups=groups, top_groups=top_groups, group_top=1, renorm=renorm)


def test_route_outputs_between_the_rows():
    """Outputs that lie in the gap between two rows of logits overlap neither."""
    import torch
    l = _logits(2, 64, 8)
    wide = torch.zeros(2, 100, device="cuda")
    wide[:, :64] = torch.from_numpy(l).cuda()
    idx, gate = wide[0, 64:72].view(torch.int32).view(2, 4), wide[0, 72:80].view(2, 4)
    moe.moe_route(wide[:, :64], 4, idx=idx, gate=gate)
    want_idx, want_gate = ref.route(l, top_k=4)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    assert np.allclose(gate.cpu().numpy(), want_gate, rtol=GATE_REL, atol=0)
    assert torch.equal(wide[:, :64].cpu(), torch.from_numpy(l)) and not bool(wide[1, 64:].any())
    with pytest.raises(moe.MoeError):
        moe.moe_route(wide[:, :64], 4, idx=wide[0, 60:68].view(torch.int32).view(2, 4), gate=gate)


@pytest.mark.parametrize("kw", [
    dict(), dict(scale=16.0), dict(groups=8, top_groups=3, group_top=1), dict(groups=8, top_groups=3, group_top=2),
    dict(bias=True), dict(renorm=True), dict(score="sigmoid")], ids=str)
@pytest.mark.parametrize("E,dtype", [(160, "bf16"), (896, "f32"), (2048, "f16"), (4096, "f32")])
def test_route_gates_are_rounded_once(E, dtype, kw):
    """Scores, their sum and the quotient are taken in 64 bits or close to it (a term of the sum is within 2^-29 of
    itself): a gate is half a step of fp32 off, and 2^-28 more at most."""
    import torch
    kw = dict(kw)
    kw.setdefault("renorm", False)
    l = _logits(50, E, E)
    l[1] = 0.25                             # a sum of E equal terms
    l[2, ::3] = -np.inf
    l[3, :] = np.finfo(np.float32).min if dtype == "f32" else -6e4
    l[4, :5] = 300.0, 299.5, 150.0, 80.0, 0.0
    l[5, 1:] = -90.0
    if kw.pop("bias", False):
        kw["bias"] = _bias(E, 2)
    lt = torch.from_numpy(l).to(ref.torch_dtype(dtype))
    want_idx, want = ref.route(lt.float().numpy(), top_k=8, **kw)
    args = {**kw, "bias": torch.from_numpy(kw["bias"]).cuda()} if "bias" in kw else kw
    idx, gate = moe.moe_route(lt.cuda(), 8, **args)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    off = np.abs(gate.cpu().numpy().astype(np.float64) - want)
    bound = (2.0 ** -24 + 2.0 ** -28) * np.abs(want) + 2.0 ** -150
    assert (off <= bound).all(), (off / bound).max()
