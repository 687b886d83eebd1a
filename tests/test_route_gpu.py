"""A router's choice of experts and its gradient against their definitions in 64 bits.

Ids have to be equal.  Tolerances of the computed values are derived.  expf is off by at
most 3 units in the last place, 6 * 2^-24 relative, and by the rounding of its argument,
|d| * 2^-24 for an argument of size |d|; an addition, product or quotient of float32 by
2^-24.  A weight is scale * (s / total): s and each term of the total hold one expf of a
difference of at most D (sigmoid: and a second one, at most 6 * 2^-24 of the sum it
stands in), the total adds up m terms in any order, at most m roundings.  So its relative
error is at most

    R = (2 * D + m + 32) * 2^-24 * (1 + 2^-10)

with D the largest |l - l'| that an exponent is taken of (sigmoid: the largest |l|), and
rounding to the output's type adds eps / 2 and 2^-25 at most (half of float16's smallest
subnormal); results below float32's smallest normal number may be zero (2^-126).  A
gradient is a sum of products of such weights and grad_weights: each term's relative
error is at most 2 R + (slots + 4) * 2^-24, of the magnitude that `reference_grad` adds up.
"""
from __future__ import annotations

import numpy as np
import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu

INF = float("inf")


def torch_():
    import torch
    return torch


def dtype_of(name):
    torch = torch_()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def as64(t):
    return t.detach().cpu().double().numpy()


def scores64(l, kind):
    """Scores, and the same times a number per row that keeps the largest near one."""
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        top = l.max(1, keepdims=True) if l.size else np.zeros((l.shape[0], 1))
        e = np.exp(l - np.where(top == -INF, 0, top))
        total = e.sum(1, keepdims=True)
        return e / np.where(total == 0, 1, total)


def rank_key(c, out):
    """Keys that sort descending and stably: NaN first, excluded ones (inf here) last."""
    return np.where(out, INF, np.where(np.isnan(c), -INF, np.where(c == INF, -1.7e308, -c)))


def reference_ids(l, slots, kind="softmax", bias=None, groups=1, kept=1, group_score="max"):
    t, e = l.shape
    b = np.zeros(e) if bias is None else bias
    c = scores64(l, kind) + b
    if bias is None and (kept == groups or group_score == "max"):
        c = l + 0.0  # the scores rise with the logits
    out = (l == -INF) | (b == -INF)[None]
    if kept < groups:
        size = e // groups
        cg, og = c.reshape(t, groups, size), out.reshape(t, groups, size)
        best = np.sort(np.where(og, -INF, np.where(np.isnan(cg), np.inf, cg)), 2)
        spoken = best[:, :, -1]
        if group_score == "top2" and size > 1:
            spoken = np.where(best[:, :, -2] == -INF, spoken, spoken + best[:, :, -2])
        order = np.argsort(-spoken, 1, kind="stable")
        lost = np.ones((t, groups), bool)
        np.put_along_axis(lost, order[:, :kept], False, 1)
        out = out | np.repeat(lost, size, 1)
    key = rank_key(c, out)
    ids = np.argsort(key, 1, kind="stable")[:, :slots]
    return np.where(np.take_along_axis(out, ids, 1), -1, ids)


def reference_weights(l, ids, kind, normalize, scale):
    """Weights, and their relative error R (but for the output's rounding)."""
    with np.errstate(all="ignore"):
        there = ids >= 0
        at = np.where(there, ids, 0)
        taken = np.where(there, np.take_along_axis(l, at, 1), -INF)
        if normalize:
            # proportions that no underflow reaches
            if kind == "sigmoid":
                log = np.minimum(taken, 0) - np.log1p(np.exp(-np.abs(taken)))
            else:
                log = taken
            log = np.where(there, log, -INF)
            top = np.where(there.any(1, keepdims=True), log.max(1, keepdims=True), 0)
            e = np.where(there, np.exp(log - top), 0)
            w = e / np.where(there.any(1, keepdims=True), e.sum(1, keepdims=True), 1)
            spread = taken
        else:
            w = np.where(there, np.take_along_axis(scores64(l, kind), at, 1), 0)
            spread = l
        finite = np.where(np.isfinite(spread), spread, np.nan)
        if kind == "sigmoid":
            d = np.nan_to_num(np.nanmax(np.abs(finite), 1, initial=0.0))
        else:
            d = np.nan_to_num(np.nanmax(finite, 1, initial=-1e30) - np.nanmin(finite, 1, initial=1e30)).clip(0, 120)
        d = np.minimum(d, 120)  # what is further down is zero beside the largest
        m = ids.shape[1] if normalize else l.shape[1]
        return w * scale, (2 * d + m + 32)[:, None] * 2.0**-24 * (1 + 2.0**-10)


def near(got, want, error, what=""):
    torch = torch_()
    g = as64(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    with np.errstate(all="ignore"):
        tol = error + (np.abs(want) + error) * (torch.finfo(got.dtype).eps / 2) + 2.0**-25 * (got.dtype is torch.float16) \
            + 2.0**-126
        bad = ~((np.abs(g - want) <= tol) | (np.isnan(g) & np.isnan(want)) | (g == want))
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r, expected %r" % (
        what, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), g[bad][0], want[bad][0])


def check_route(logits, slots, kind="softmax", bias=None, groups=1, kept=None, group_score="max", normalize=True,
                scale=1.0, id_type="i32", weights_dtype=None, what=""):
    torch = torch_()
    kept = groups if kept is None else kept
    ids, w = lrs.route_tokens(logits, slots, scores=kind, bias=bias, num_groups=groups, kept_groups=kept,
                              group_score=group_score, normalize=normalize, scale=scale,
                              dtype=torch.int32 if id_type == "i32" else torch.int64, weights_dtype=weights_dtype)
    l = as64(logits)
    want = reference_ids(l, slots, kind, None if bias is None else as64(bias), groups, kept, group_score)
    got = ids.cpu().numpy()
    assert got.dtype == (np.int32 if id_type == "i32" else np.int64)
    bad = got != want
    assert not bad.any(), "%s: ids of %d tokens differ, first %s: %s, expected %s" % (
        what, bad.any(1).sum(), np.argwhere(bad)[0], got[bad.any(1)][0], want[bad.any(1)][0])
    ww, r = reference_weights(l, want, kind, normalize, scale)
    near(w, ww, np.abs(ww) * r, what)
    return ids, w


def randn(shape, name, seed, scale=1.0):
    torch = torch_()
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(x).to(dtype_of(name)).cuda()


def biases(experts, seed):
    torch = torch_()
    return torch.from_numpy(np.random.default_rng(seed).integers(-100, 101, experts).astype(np.float32) * 1e-3).cuda()


EXPERTS = [1, 2, 3, 7, 8, 9, 15, 16, 60, 64, 65, 100, 127, 128, 129, 160, 250, 256, 257, 384, 512, 513, 1000, 1024, 1025,
           2047, 2048]


@pytest.mark.parametrize("experts", EXPERTS)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_route_sizes(experts, name):
    for i, (tokens, slots) in enumerate([(1, 1), (5, 2), (33, 8), (67, 13)]):
        slots = min(slots, experts)
        for kind in ("softmax", "sigmoid"):
            for bias in (None, biases(experts, i)):
                announce("route %d x %d, %d slots, %s %s bias %s" % (tokens, experts, slots, name, kind, bias is not None))
                check_route(randn((tokens, experts), name, tokens + experts), slots, kind, bias,
                            normalize=(i + (bias is None)) % 2 == 0, scale=2.5 if i % 2 else 1.0,
                            id_type="i64" if i % 2 else "i32", what="%d %d" % (tokens, slots))


@pytest.mark.parametrize("slots", [1, 16, 17, 31, 63, 64])
@pytest.mark.parametrize("experts", [64, 128, 300, 600, 2000])
def test_route_many_slots(experts, slots):
    announce("route %d of %d" % (slots, experts))
    for kind in ("softmax", "sigmoid"):
        for bias in (None, biases(experts, 1)):
            check_route(randn((40, experts), "f32", slots), slots, kind, bias, what=kind)
            check_route(randn((40, experts), "bf16", slots), slots, kind, bias, normalize=False, what=kind)


@pytest.mark.parametrize("experts,groups", [(8, 8), (64, 2), (60, 4), (160, 8), (256, 8), (256, 64), (320, 5), (512, 16),
                                            (1000, 10), (2048, 32), (66, 33), (2048, 64)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_groups(experts, groups, group_score):
    for i, kept in enumerate(sorted({1, 2, groups // 2, groups - 1, groups})):
        if kept < 1:
            continue
        slots = min(8, kept * (experts // groups))
        for kind, bias, name in (("softmax", None, "bf16"), ("sigmoid", biases(experts, 2), "f32"),
                                 ("softmax", biases(experts, 3), "f16"), ("sigmoid", None, "f32")):
            announce("groups %d of %d kept %d %s %s %s" % (groups, experts, kept, group_score, kind, name))
            check_route(randn((50, experts), name, i), slots, kind, bias, groups, kept, group_score,
                        what="%d %s" % (kept, kind))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [16, 100, 256, 512, 1024, 2048])
def test_scores_that_float32_cannot_tell_apart(kind, experts):
    """A bias that makes every sum one half to within a rounding of float32: the order is
    that of the sums in 64 bits.  And sums that are equal: the lowest id."""
    torch = torch_()
    announce("close sums %s %d" % (kind, experts))
    l = randn((1, experts), "f32", experts)
    bias = torch.from_numpy((0.5 - scores64(as64(l), kind)[0]).astype(np.float32)).cuda()
    check_route(l, min(experts, 40), kind, bias, what="close")
    check_route(l, min(experts // 4, 40), kind, bias, 4, 2, "top2", what="close groups")
    check_route(l, min(experts // 4, 40), kind, bias, 4, 1, "max", what="close groups")
    # rows of which only some are close, beside others in the same wave
    rows = torch.cat([randn((7, experts), "f32", 3), l, randn((9, experts), "f32", 4), l, l])
    check_route(rows, min(experts, 8), kind, bias, what="some close")
    # two neighbours of float32 at the border of the choice, in each order
    for up in (False, True):
        two = torch.zeros(3, experts, device="cuda") - 3
        a = np.float32(1.0)
        b = np.nextafter(a, np.float32(2.0))
        two[:, 3], two[:, 9] = (float(a), float(b)) if up else (float(b), float(a))
        ids, _ = check_route(two, 1, kind, torch.zeros(experts, device="cuda"), what="neighbours")
        assert ids.flatten().tolist() == [9 if up else 3] * 3
        check_route(two, 1, kind, None, what="neighbours")
    same = torch.full((5, experts), 0.25, device="cuda")
    for b in (None, torch.zeros(experts, device="cuda"), torch.full((experts,), -0.125, device="cuda")):
        ids, w = check_route(same, 4, kind, b, what="equal")
        assert (ids.cpu().numpy() == np.arange(4)).all() and torch.equal(w, torch.full_like(w, 0.25))
    assert (lrs.route_tokens(same, 4, kind, num_groups=4, kept_groups=2, group_score="top2")[0].cpu().numpy() ==
            np.arange(4)).all()


@pytest.mark.parametrize("experts,groups", [(16, 4), (60, 4), (160, 8), (256, 8), (512, 16), (700, 7), (2048, 32)])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_sigmoids_that_float64_holds_as_one_number(name, experts, groups):
    """Without a bias the order within the kept groups is that of the logits, whose sigmoids
    are all 1 in 64 bits from 38 on; groups of equal sums: the lowest."""
    announce("saturated sigmoids %s %d" % (name, experts))
    torch = torch_()
    rng = np.random.default_rng(experts)
    l = torch.from_numpy(40 + 20 * rng.random((9, experts))).to(dtype_of(name)).cuda()
    l[0] = torch.where(torch.arange(experts, device="cuda") % 2 == 0, 41.0, 40.0)
    l[1] = torch.arange(experts, device="cuda") * (100.0 / experts) + 40
    l[2] = l[1].flip(0)
    l[3, ::3] = -INF
    l[4, experts // 2:] = -INF
    l[5] = -l[5]  # (far apart in 64 bits; in 32 all are next to 0)
    if name == "f32":
        l[6] = -800 - l[6]
    size, x = experts // groups, as64(l)
    for kept in (2, groups - 1):
        for slots in (1, 5, 2 * size if size < 30 else 40):
            for normalize in (True, False):
                ids, w = lrs.route_tokens(l, slots, "sigmoid", num_groups=groups, kept_groups=kept, group_score="top2",
                                          normalize=normalize)
                for t in range(9):
                    best = np.sort(scores64(np.where(x[t] == -INF, 0, x[t])[None], "sigmoid")[0].reshape(groups, size) *
                                   (x[t].reshape(groups, size) != -INF), 1)[:, -2:].sum(1)
                    stay = np.argsort(-best, kind="stable")[:kept]
                    out = ~np.isin(np.arange(experts) // size, stay) | (x[t] == -INF)
                    want = np.argsort(np.where(out, INF, -x[t]), kind="stable")[:slots]
                    want = np.where(out[want], -1, want)
                    assert (ids[t].cpu().numpy() == want).all(), (t, kept, slots, ids[t].tolist(), want.tolist())
                ww, r = reference_weights(x, ids.cpu().numpy(), "sigmoid", normalize, 1.0)
                near(w, ww, np.abs(ww) * r)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [20, 128, 700])
def test_masked_experts(name, kind, experts):
    torch = torch_()
    announce("masked experts %s %s %d" % (name, kind, experts))
    lowest = torch.finfo(dtype_of(name)).min
    l = randn((12, experts), name, 5)
    l[0] = -INF                       # nothing to choose
    l[1, 3:] = -INF                   # fewer than the slots
    l[2, 1:] = lowest                 # the lowest finite value is a value
    l[3] = lowest                     # ... also where there is no other
    l[4, ::2] = -INF
    l[5, :experts // 2] = -INF        # whole groups
    l[6] = torch.where(torch.arange(experts, device="cuda") % 3 == 0, 0.0, -0.0).to(l.dtype)  # one value
    l[7] = -200.0 if kind == "sigmoid" else 30000.0  # scores below float32's smallest; large logits
    l[8, 4] = 60000.0
    l[9] = -INF
    l[9, experts - 1] = lowest
    for bias in (None, biases(experts, 4)):
        for normalize in (True, False):
            for groups, kept, how in ((1, 1, "max"), (4, 2, "max"), (4, 2, "top2"), (4, 3, "top2")):
                check_route(l, 5, kind, bias, groups, kept, how, normalize, what="%s %s %s" % (normalize, groups, how))
    ids, w = lrs.route_tokens(l, 5, kind)
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[1, 3:] == -1).all() and (w[1, 3:] == 0).all()
    assert (ids[3].cpu().numpy() == np.arange(5)).all() and (w[3] > 0).all()
    # a bias of -infinity takes an expert out of the choice, but not out of the softmax
    bias = biases(experts, 6)
    bias[::3] = -INF
    check_route(l, 5, kind, bias, normalize=False, what="bias")
    check_route(l, 5, kind, bias, 4, 2, "top2", what="bias")
    bias[:] = -INF
    ids, w = check_route(l, 5, kind, bias, what="all out")
    assert (ids == -1).all() and (w == 0).all()
    bias[:] = -1e30  # a mask by a large number: equal sums in 32 and in 64 bits
    bias[[2, 11]] = 0.0
    check_route(l[2:5], 2, kind, bias, what="large negative bias")


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_nan_and_infinity(kind):
    """NaN is the largest and shows in the weights; other tokens are not touched."""
    torch = torch_()
    announce("nan %s" % kind)
    l = randn((6, 40), "f32", 9)
    clean = l.clone()
    l[1, 7] = l[1, 30] = float("nan")
    l[2, 5] = INF
    l[3, 0] = -float("nan")
    ids, w = lrs.route_tokens(l, 3, kind)
    assert ids[1].tolist()[:2] == [7, 30] and ids[2, 0] == 5 and ids[3, 0] == 0
    assert w[1].isnan().all() and w[3].isnan().all()
    if kind == "softmax":
        assert w[2].isnan().all()
    else:
        assert torch.isfinite(w[2]).all() and w[2, 0] >= w[2, 1]
    for bias in (None, biases(40, 1)):
        for normalize in (True, False):
            got = lrs.route_tokens(l, 3, kind, bias=bias, normalize=normalize, num_groups=4, kept_groups=2,
                                   group_score="top2")
            want = lrs.route_tokens(clean, 3, kind, bias=bias, normalize=normalize, num_groups=4, kept_groups=2,
                                    group_score="top2")
            for a, b in zip(got, want):
                assert torch.equal(a[[0, 4, 5]], b[[0, 4, 5]])
            assert (got[0] >= 0).all() and (got[0] < 40).all()
            if kind == "softmax":  # the NaN is in every score of the token
                assert got[1][[1, 3]].isnan().all()
            else:
                assert got[0][1, 0] == 7 and got[1][1, 0].isnan()


def test_route_types_strides_and_shapes():
    torch = torch_()
    announce("route strides")
    for name in ("f32", "bf16", "f16"):
        for experts in (8, 60, 256):
            wide = randn((70, 2 * experts + 3), name, experts)
            for view in (wide[:, :experts], wide[:, 1:experts + 1], wide[::2, 3:experts + 3], wide[:, :experts].t().contiguous().t(),
                         wide[:1, 5:experts + 5], wide[:, 0:2 * experts:2]):
                for bias in (None, biases(experts, 1)):
                    check_route(view, 4, "sigmoid", bias, what=str(view.stride()))
            wide_bias = torch.zeros(experts, 2, device="cuda")
            wide_bias[:, 1] = biases(experts, 1)
            check_route(wide[:, :experts], 4, "sigmoid", wide_bias[:, 1], weights_dtype=torch.bfloat16)
            check_route(wide[:, :experts], 4, "softmax", weights_dtype=torch.float16, normalize=False)
            row = randn((1, experts), name, 1).expand(9, experts)  # one row for all tokens
            check_route(row, 4)
    ids, w = lrs.route_tokens(randn((0, 16), "f32", 1), 3)
    assert ids.shape == w.shape == (0, 3)
    ids, w = lrs.route_tokens(randn((5, 16), "f32", 1), 0)
    assert ids.shape == w.shape == (5, 0)
    ids, w = lrs.route_tokens(randn((5, 0), "f32", 1), 0)
    assert ids.shape == (5, 0)
    with pytest.raises(lrs.LrsError):
        lrs.route_tokens(randn((5, 2049), "f32", 1), 3)
    with pytest.raises(lrs.LrsError):
        lrs.route_tokens(randn((5, 100), "f32", 1), 65)
    # without weights, by the C call: a guard behind the ids stays as it was
    l = randn((9, 16), "f32", 2)
    ids = torch.full((9 * 2 + 4,), 77, dtype=torch.int32, device="cuda")
    lrs.lrs_route_tokens("f32", l, 16, 9, 16, 2, "softmax", None, 1, 1, "max", 1, 1.0, "i32", ids, "f32", None)
    assert torch.equal(ids[:18].view(9, 2), lrs.route_tokens(l, 2)[0]) and (ids[18:] == 77).all()


def test_route_rows_far_apart():
    """Logits beyond 2^31 elements and 2^32 bytes, and more tokens than a grid's step."""
    torch = torch_()
    announce("route far rows")
    step = (1 << 31) // 3
    buffer = torch.zeros(step * 3 + 64, device="cuda", dtype=torch.bfloat16)
    view = buffer.as_strided((4, 64), (step, 1))
    view.copy_(randn((4, 64), "bf16", 3))
    check_route(view, 4, "sigmoid", biases(64, 1))
    ids, w = lrs.route_tokens(view, 4)
    grad = torch.zeros(step * 3 + 64, device="cuda", dtype=torch.bfloat16).as_strided((4, 64), (step, 1))
    lrs.route_tokens_grad(w, view, ids, grad=grad)
    assert torch.equal(grad.contiguous(), lrs.route_tokens_grad(w, view.contiguous(), ids))
    del buffer, grad, view
    tokens = (1 << 24) + 1031  # sixteen tokens a workgroup, 2^20 of these a step
    few = randn((4099, 3), "bf16", 4)
    many = few[torch.arange(tokens, device="cuda") % 4099]
    want_ids, want_w = check_route(few, 2)
    ids, w = lrs.route_tokens(many, 2)
    at = torch.arange(tokens, device="cuda") % 4099
    assert torch.equal(ids, want_ids[at]) and torch.equal(w, want_w[at])
    assert torch.equal(lrs.route_tokens_grad(w, many, ids), lrs.route_tokens_grad(want_w, few, want_ids)[at])


# ------------------------------------------------------------------ gradient


def reference_grad(gw, l, ids, kind, normalize, scale):
    """The gradient, and the magnitudes of what each element adds up, times their
    relative error."""
    t, e = l.shape
    with np.errstate(all="ignore"):
        there = (ids >= 0) & (ids < e)
        there &= np.where(there, np.take_along_axis(l, np.where(there, ids, 0), 1), -INF) != -INF
        ids = np.where(there, ids, -1)
        w, r = reference_weights(l, ids, kind, normalize, 1.0)
        g = np.where(there, gw * scale, 0)
        taken = np.where(there, np.take_along_axis(l, np.where(there, ids, 0), 1), 0)
        dot, mag = (w * g).sum(1, keepdims=True), np.abs(w * g).sum(1, keepdims=True)
        d = w * (g - dot) if normalize else w * g
        dm = w * (np.abs(g) + mag) if normalize else np.abs(w * g)
        if kind == "sigmoid":
            less = scores64(-taken, "sigmoid")
            d, dm = d * less, dm * less
        out, total = np.zeros((t, e)), np.zeros((t, e))
        for k in range(ids.shape[1]):
            rows = np.nonzero(there[:, k])[0]
            np.add.at(out, (rows, ids[rows, k]), d[rows, k])
            np.add.at(total, (rows, ids[rows, k]), dm[rows, k])
        if kind == "softmax" and not normalize:
            s = scores64(l, "softmax")
            out -= np.where(s == 0, 0, s * dot)
            total += s * mag
    return out, total * (2 * r + (ids.shape[1] + 4) * 2.0**-24)


def check_grad(gw, logits, ids, kind, normalize, scale=1.0, what="", **kw):
    got = lrs.route_tokens_grad(gw, logits, ids, scores=kind, normalize=normalize, scale=scale, **kw)
    want, error = reference_grad(as64(gw), as64(logits), ids.cpu().numpy().astype(np.int64), kind, normalize, scale)
    assert got.dtype is logits.dtype
    near(got, want, error, what)
    return got


@pytest.mark.parametrize("experts", EXPERTS)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_route_grad(experts, name):
    torch = torch_()
    for i, (tokens, slots) in enumerate([(1, 1), (5, 2), (67, 8), (18, 40)]):
        slots = min(slots, experts)
        for kind in ("softmax", "sigmoid"):
            for normalize in (True, False):
                announce("route grad %d x %d, %d slots %s %s %s" % (tokens, experts, slots, name, kind, normalize))
                l = randn((tokens, experts), name, i)
                ids, _ = lrs.route_tokens(l, slots, kind, bias=biases(experts, i), normalize=normalize,
                                          dtype=torch.int64 if i % 2 else torch.int32)
                gw = randn((tokens, slots), ("f32", "bf16", "f16")[i % 3], 50 + i)
                check_grad(gw, l, ids, kind, normalize, 2.5 if i % 2 else 1.0, "%d %d" % (tokens, slots))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_grad_of_ids_that_take_no_part(kind, normalize):
    """Ids of no expert, masked logits, and the same expert twice."""
    torch = torch_()
    announce("grad of masked ids %s %s" % (kind, normalize))
    for experts in (10, 200, 1500):
        l = randn((9, experts), "f32", 1)
        ids = torch.from_numpy(np.random.default_rng(1).integers(0, experts, (9, 4))).cuda()
        gw = randn((9, 4), "f32", 2)
        l[0] = -INF
        ids[1] = -1
        ids[2, 1:3] = torch.tensor([experts, 2**40], device="cuda")
        l[3, ids[3, 2]] = -INF
        ids[4] = 7
        ids[5, 3] = ids[5, 0]
        l[6] = torch.finfo(torch.float32).min
        l[7, ::2] = -INF
        l[8] = -150.0
        ids[8] = torch.arange(4, device="cuda")
        out = gw.clone()
        for row, col in ((0, 0), (1, 2), (2, 1), (2, 2), (3, 2)):
            out[row, col] = float("nan")  # belongs to no part: reaches nothing
        for one in (ids, ids.clamp(-2**31, 2**31 - 1).to(torch.int32)):
            got = check_grad(gw, l, one, kind, normalize, 1.5, str(experts))
            assert torch.equal(lrs.route_tokens_grad(out, l, one, kind, normalize, 1.5), got)
        assert (got[0] == 0).all() and (got[1] == 0).all()
    none = lrs.route_tokens_grad(gw[:, :0], l, ids[:, :0], kind, normalize)
    assert none.shape == l.shape and (none == 0).all()
    assert lrs.route_tokens_grad(gw[:0], l[:0], ids[:0]).shape == (0, 1500)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_grad_against_differences(kind, normalize):
    """(f(l + h) - f(l - h)) / 2h of f = the sum of grad_weights * weights in 64 bits, the
    ids held.  Its own error: h^2 / 6 times the third derivative (at most 8 scale |g| a
    weight here) and 2^-53 |f| / h of rounding."""
    announce("grad differences %s %s" % (kind, normalize))
    l = randn((6, 12), "f32", 3)
    ids, _ = lrs.route_tokens(l, 3, kind, normalize=normalize, scale=1.5)
    gw = randn((6, 3), "f32", 4)
    got = as64(lrs.route_tokens_grad(gw, l, ids, kind, normalize, 1.5))
    l64, g64, i64 = as64(l), as64(gw), ids.cpu().numpy()
    h = 1e-4
    f = lambda x: (reference_weights(x, i64, kind, normalize, 1.5)[0] * g64).sum(1)  # noqa: E731
    bound = np.abs(g64).sum(1) * 1.5 * (8 * h * h / 6 + 2.0**-53 / h * 4 + 64 * 2.0**-24)
    for e in range(12):
        step = np.zeros(12)
        step[e] = h
        d = (f(l64 + step) - f(l64 - step)) / (2 * h)
        assert (np.abs(got[:, e] - d) <= bound).all(), (e, got[:, e], d)


def test_route_grad_strides_and_in_place():
    torch = torch_()
    announce("grad strides")
    for name in ("f32", "bf16", "f16"):
        for experts in (9, 130, 256, 600):
            for kind, normalize in (("softmax", True), ("softmax", False), ("sigmoid", True)):
                wide = randn((40, 2 * experts + 3), name, experts)
                view = wide[:, 1:experts + 1]
                ids, w = lrs.route_tokens(view, 3, kind, normalize=normalize)
                gw = randn((40, 6), "f32", 1)[:, ::2]
                want = check_grad(gw, view, ids, kind, normalize)
                before = wide.clone()
                out = lrs.route_tokens_grad(gw, view, ids, kind, normalize, grad=wide[:, experts + 2:2 * experts + 2])
                assert torch.equal(out, want)
                before[:, experts + 2:2 * experts + 2] = want
                assert torch.equal(wide, before)
                assert lrs.route_tokens_grad(gw, view, ids, kind, normalize, grad=view) is view
                before[:, 1:experts + 1] = want
                assert torch.equal(wide, before)


def test_router_block_captured_and_on_other_streams():
    """Route, group, dispatch, combine and back, as a layer runs them: eagerly against
    64 bits, captured and replayed on new inputs with eager calls between, two graphs at
    once, and on a side stream."""
    torch = torch_()
    announce("router block")

    def step(s, stream=None):
        ids, w = lrs.route_tokens(s["logits"], 4, "sigmoid", bias=s["bias"], num_groups=4, kept_groups=2,
                                  group_score="top2", scale=2.0, stream=stream)
        order, position, offsets = lrs.group_tokens(ids, 32, stream=stream)
        rows = lrs.dispatch_rows(s["x"], position, out=s["rows"], stream=stream)
        y = lrs.combine_rows(rows, position, w, stream=stream)
        grad_rows, grad_w = lrs.combine_rows_grad(s["gy"], rows, position, w, grad_rows=s["grad_rows"], stream=stream)
        grad_x = lrs.combine_rows(grad_rows, position, stream=stream)
        grad_l = lrs.route_tokens_grad(grad_w, s["logits"], ids, "sigmoid", scale=2.0, stream=stream)
        return ids, w, order, position, offsets, y, grad_w, grad_x, grad_l

    def fresh(tokens, cols, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        return {"logits": torch.randn(tokens, 32, generator=g, device="cuda"),
                "bias": torch.randint(-9, 10, (32,), generator=g, device="cuda") * 0.01,
                "x": torch.randn(tokens, cols, generator=g, device="cuda"),
                "gy": torch.randn(tokens, cols, generator=g, device="cuda"),
                "rows": torch.zeros(tokens * 4, cols, device="cuda"),
                "grad_rows": torch.zeros(tokens * 4, cols, device="cuda")}

    s = fresh(500, 72, 0)
    s["logits"][7] = -INF  # a padding token
    ids, w, _, _, _, y, grad_w, grad_x, grad_l = step(s)
    check_route(s["logits"], 4, "sigmoid", s["bias"], 4, 2, "top2", scale=2.0)
    # every expert hands its rows on unchanged: y = x * sum of weights, and what follows
    w64, x64, gy64 = as64(w), as64(s["x"]), as64(s["gy"])
    assert np.allclose(as64(y), x64 * w64.sum(1, keepdims=True), rtol=16 * 2.0**-24, atol=16 * 2.0**-24 * np.abs(x64).max() * 2)
    assert (as64(y)[7] == 0).all() and (as64(grad_l)[7] == 0).all() and (as64(grad_x)[7] == 0).all()
    dots = (x64 * gy64).sum(1, keepdims=True) * (w64 > 0)
    size = np.abs(x64 * gy64).sum(1, keepdims=True)
    assert (np.abs(as64(grad_w) - dots) <= size * 80 * 2.0**-24).all()
    check_grad(grad_w, s["logits"], ids, "sigmoid", True, 2.0)

    sizes = ((700, 264), (9000, 72))
    states, graphs, outs = [fresh(*size, 1) for size in sizes], [], []
    for s in states:
        step(s)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(s))
    for rep in range(3):
        new = [fresh(*size, 10 + rep) for size in sizes]
        for s, other, graph in zip(states, new, graphs):
            for name in s:
                s[name].copy_(other[name])
            graph.replay()
        want = [step(other) for other in new]
        torch.cuda.synchronize()
        for got, expected in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, expected)), rep
    side, big = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda")
    want = step(new[0])
    torch.cuda.synchronize()
    late = {name: torch.zeros_like(t) for name, t in new[0].items()}
    for _ in range(4):
        big @ big
    for name in late:
        late[name].copy_(new[0][name])
    got = step(late, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_route_grad_counts_as_a_write():
    torch = torch_()
    announce("versions")
    l = randn((4, 8), "f32", 1)
    ids, w = lrs.route_tokens(l, 2)
    out = torch.zeros(4, 8, device="cuda")
    y = (torch.ones(4, 8, device="cuda", requires_grad=True) * out).sum()
    lrs.route_tokens_grad(w, l, ids, grad=out)
    assert out._version == 1 and l._version == 0 and ids._version == 0 and w._version == 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("kind,biased,groups,kept", [("sigmoid", True, 8, 4), ("softmax", True, 8, 3),
                                                     ("softmax", False, 1, 1), ("sigmoid", False, 4, 2)])
def test_route_at_the_size_of_a_prompt(name, kind, biased, groups, kept):
    """Thousands of tokens, of which some have scores that only float64 tells apart; logits
    in float32 that were rounded to bfloat16 before, so that many are equal."""
    torch = torch_()
    announce("prompt %s %s %s %d" % (name, kind, biased, groups))
    for experts, tokens in ((256, 8200), (160, 4099), (512, 2051)):
        l = randn((tokens, experts), name, experts)
        bias = biases(experts, 1) if biased else None
        ids, w = check_route(l, 8, kind, bias, groups, kept, "top2", kind == "sigmoid", 2.5, "i64")
        check_grad(randn((tokens, 8), "f32", 2), l, ids, kind, kind == "sigmoid", 2.5)
        check_route(randn((tokens, experts), "bf16", 3).float(), 8, kind, bias, groups, kept, "max")


def test_nan_in_groups_of_lanes():
    """Groups that are whole vectors of neighbouring lanes: a NaN's group comes first."""
    torch = torch_()
    announce("nan in groups")
    for name in ("f32", "bf16"):
        l = randn((5, 64), name, 9)
        l[1, 37], l[3, 63] = float("nan"), INF
        for group_score in ("max", "top2"):
            for bias in (None, biases(64, 1)):
                ids, w = lrs.route_tokens(l, 4, "sigmoid", bias=bias, num_groups=4, kept_groups=1,
                                          group_score=group_score)
                assert ids[1, 0] == 37 and (ids[1] // 16 == 2).all() and w[1].isnan().all()
                assert ids[3, 0] == 63 and (ids[3] // 16 == 3).all()
                assert torch.isfinite(w[[0, 2, 3, 4]]).all()
