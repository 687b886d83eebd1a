"""The row operators against their definitions in 64 bits, on the GPU.

Tolerances are derived, not fitted.  A rounding to type T is off by at most half a
step, eps(T) / 2 relative (or half the smallest subnormal, float16's 2^-25 being the
largest of the three types).  A sum or product chain of m float32 roundings is off by
at most m * 2^-24 times the sum S of its terms' magnitudes (to first order; the
factor 1 + 2^-10 covers the rest for m <= 2^13).  So an output with the exact value
r, formed in float32 and rounded once, is within

    e + (|r| + e) * eps(T) / 2 + 2^-25,   e = m * 2^-24 * S * (1 + 2^-10).
"""
from __future__ import annotations

import numpy as np
import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu

I32MIN, I64MIN, I64MAX = -2**31, -2**63, 2**63 - 1


def torch_():
    import torch
    return torch


def dtype_of(name):
    torch = torch_()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def within(got, want, magnitude, terms, what=""):
    """got (a tensor) against want and the sum of the terms' magnitudes (float64 arrays)."""
    torch = torch_()
    g = got.detach().cpu().double().numpy()
    assert g.shape == want.shape, (g.shape, want.shape)
    e = terms * 2.0**-24 * magnitude * (1 + 2.0**-10)
    tol = e + (np.abs(want) + e) * (torch.finfo(got.dtype).eps / 2) + 2.0**-25
    off = np.abs(g - want)
    bad = ~(off <= tol)
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r, expected %r within %r" % (
        what, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), g[bad][0], want[bad][0], tol[bad][0])


def randn(shape, name, seed, scale=1.0):
    torch = torch_()
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(x).to(dtype_of(name)).cuda()


def as64(t):
    return t.detach().cpu().double().numpy()


def strided(t, layout):
    """The same matrix with its rows in a wider buffer: "pad", rows a vector apart at
    16-byte boundaries; "odd", off every 16-byte boundary, an odd stride."""
    torch = torch_()
    if layout == "packed":
        return t.contiguous()
    extra, at = (16, 0) if layout == "pad" else (5, 3)
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    if (t.shape[1] + extra) % 2 == 0 and layout == "odd":
        wide = torch.full((t.shape[0], t.shape[1] + extra + 1), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, at:at + t.shape[1]]
    view.copy_(t)
    return view


def routing(tokens, slots, experts, seed, kind="uniform", id_type="i64", first=0):
    """Distinct choices per token where a router would make them (kind: how)."""
    torch = torch_()
    rng = np.random.default_rng(seed)
    if kind == "one":  # every token chooses the same
        ids = np.full((tokens, slots), first + experts // 2)
    elif kind == "skewed":
        ids = first + (experts * rng.random((tokens, slots)) ** 4).astype(np.int64)
    elif kind == "none":
        ids = np.where(rng.random((tokens, slots)) < 0.5, first - 1, first + experts)
    elif kind == "far":  # ids far outside either way among good ones
        far = np.array([first - 1, first + experts, I32MIN, 2**31 - 1] + ([] if id_type == "i32" else [I64MIN, I64MAX]))
        ids = np.where(rng.random((tokens, slots)) < 0.4, rng.choice(far, (tokens, slots)),
                       first + rng.integers(0, max(1, experts), (tokens, slots)))
    else:
        ids = first + rng.integers(0, max(1, experts), (tokens, slots))
    return torch.from_numpy(ids.astype(np.int32 if id_type == "i32" else np.int64)).cuda()


def group_reference(ids, groups, first):
    """order, position, offsets, from python integers and a stable numpy sort."""
    flat = ids.detach().cpu().numpy().reshape(-1)
    lo = flat.astype(object) - first if flat.size < 4096 else flat.astype(np.float64) - float(first)
    inside = (lo >= 0) & (lo < groups)
    key = np.where(inside, lo, groups).astype(np.int64)
    order = np.argsort(key, kind="stable")
    position = np.empty(flat.size, dtype=np.int64)
    position[order] = np.arange(flat.size)
    position[key == groups] = -1
    counts = np.bincount(key, minlength=groups + 1)[:groups] if flat.size else np.zeros(groups, dtype=np.int64)
    return order, position.reshape(ids.shape), np.concatenate([[0], np.cumsum(counts)]), key


def check_group(ids, groups, first, got):
    order, position, offsets, _ = group_reference(ids, groups, first)
    for name, g, w in zip(("order", "position", "offsets"), got, (order, position, offsets)):
        assert g.dtype == torch_().int32 and np.array_equal(g.cpu().numpy(), w), name


# ------------------------------------------------------------------ grouping

SIZES = [0, 1, 2, 63, 64, 65, 255, 256, 1000, 1023, 1024, 1025, 2047, 4096, 4097, 8191, 8193, 16384, 16385, 40001,
         131072, 300007]


@pytest.mark.parametrize("groups,first", [(1, 0), (2, 5), (8, 0), (64, -3), (100, 1000), (255, 0), (256, 0), (257, 0),
                                          (1000, 7), (2047, 0), (2048, 0), (2049, 0), (4096, 1), (50257, 0)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "far", "one"])
def test_group_tokens(groups, first, kind):
    for i, n in enumerate(SIZES):
        id_type = "i32" if (i + groups) % 2 else "i64"
        announce("group n=%d groups=%d first=%d %s %s" % (n, groups, first, kind, id_type))
        ids = routing(n, 1, groups, n * 31 + groups, kind, id_type, first).reshape(-1)
        check_group(ids, groups, first, lrs.group_tokens(ids, groups, first_id=first))


def test_group_tokens_edges():
    torch = torch_()
    announce("group edges")
    ids = routing(37, 4, 16, 1)
    # no groups; all of no group; a window of the groups; ids at the ends of int64
    check_group(ids, 0, 0, lrs.group_tokens(ids, 0))
    check_group(routing(37, 4, 16, 1, "none"), 16, 0, lrs.group_tokens(routing(37, 4, 16, 1, "none"), 16))
    check_group(ids, 5, 3, lrs.group_tokens(ids, 5, first_id=3))
    ends = torch.tensor([I64MAX - 1, I64MIN, I64MAX - 5, 0, -1, I64MAX], device="cuda")
    check_group(ends, 5, I64MAX - 5, lrs.group_tokens(ends, 5, first_id=I64MAX - 5))
    check_group(ends, 3, I64MIN, lrs.group_tokens(ends, 3, first_id=I64MIN))
    # shapes and strides
    order, position, offsets = lrs.group_tokens(ids.t(), 16)
    assert position.shape == (4, 37)
    check_group(ids.t().contiguous(), 16, 0, (order, position, offsets))
    # a group that many slots skip: the run of equal offsets
    check_group(torch.tensor([70000, 3, 3], device="cuda"), 70001, 0, lrs.group_tokens(torch.tensor([70000, 3, 3], device="cuda"), 70001))


@pytest.mark.parametrize("groups", [5, 300, 512, 513, 2048])
def test_group_many(groups):
    """Around the sizes where blocks become larger and where the sort takes over."""
    for n in (12288, 12289, 32768, 32769, 131073, 2**20, 2**20 + 1):
        announce("group n=%d groups=%d" % (n, groups))
        for kind in ("skewed", "far"):
            ids = routing(n, 1, groups, n + groups, kind).reshape(-1)
            check_group(ids, groups, 0, lrs.group_tokens(ids, groups))


def test_first_id_beyond_int64_is_refused():
    torch = torch_()
    announce("first id beyond int64")
    ids, x = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 8, device="cuda")
    for first in (2**63, -2**63 - 1, 2**64):
        with pytest.raises(ValueError, match="int64"):
            lrs.group_tokens(ids, 4, first_id=first)
        with pytest.raises(ValueError, match="int64"):
            lrs.embedding(x, ids, first_id=first)
        with pytest.raises(ValueError, match="int64"):
            lrs.embedding_grad(x, ids, 4, first_id=first)
    for groups in (-1, 2**31):
        with pytest.raises((lrs.LrsError, RuntimeError)):
            lrs.group_tokens(ids, groups)


def test_group_outputs_are_optional_and_temp_is_reused():
    torch = torch_()
    for n, groups in ((500, 8), (30000, 100), (30000, 30000)):
        announce("group optional n=%d groups=%d" % (n, groups))
        ids = routing(n, 1, groups, 3, "far").reshape(-1)
        want = group_reference(ids, groups, 0)[:3]
        need = lrs.lrs_group_tokens(None, 0, "i64", ids, n, 0, groups, None, None, None)
        temp = torch.randint(0, 255, (need + 64,), dtype=torch.uint8, device="cuda")
        for at in (0, 1, 17):  # any alignment, whatever it held
            for which in range(8):
                outs = [torch.full((k,), -7, dtype=torch.int32, device="cuda") for k in (n, n, groups + 1)]
                given = [o if which >> i & 1 else None for i, o in enumerate(outs)]
                lrs.lrs_group_tokens(temp.data_ptr() + at, need, "i64", ids, n, 0, groups, *given)
                for i, o in enumerate(outs):
                    if which >> i & 1:
                        assert np.array_equal(o.cpu().numpy(), want[i].reshape(-1)), (at, which, i)
                    else:
                        assert bool((o == -7).all())


# ---------------------------------------------------------- sorted and back


def plan(tokens, slots, experts, seed, kind="uniform", id_type="i64", first=0):
    ids = routing(tokens, slots, experts, seed, kind, id_type, first)
    order, position, offsets = lrs.group_tokens(ids, experts, first_id=first)
    return position, position.cpu().numpy().astype(np.int64)


CASES = [  # tokens, slots, experts, kind, cols, layout
    (1, 1, 1, "uniform", 1, "packed"),
    (1, 8, 64, "uniform", 4096, "packed"),
    (3, 8, 64, "uniform", 2049, "odd"),
    (2, 1, 4, "uniform", 7, "packed"),
    (33, 2, 8, "far", 64, "packed"),
    (64, 4, 16, "skewed", 8, "packed"),
    (100, 3, 7, "uniform", 513, "odd"),
    (257, 6, 20, "far", 1000, "pad"),
    (500, 9, 32, "uniform", 136, "packed"),
    (75, 17, 40, "far", 2055, "odd"),
    (40, 2, 5, "none", 300, "packed"),
    (9, 33, 64, "uniform", 20000, "packed"),
    (2050, 2, 8, "one", 96, "pad"),
]


@pytest.mark.parametrize("row_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,slots,experts,kind,cols,layout", CASES)
def test_dispatch_rows(row_type, tokens, slots, experts, kind, cols, layout):
    torch = torch_()
    announce("dispatch %s %s" % (row_type, (tokens, slots, experts, kind, cols, layout)))
    position, pos = plan(tokens, slots, experts, 11, kind)
    x = randn((tokens, cols), row_type, 12)
    x.view(-1)[::7] = float("nan")  # copied like any value
    out = strided(torch.full((tokens * slots, cols), -3.0, dtype=x.dtype, device="cuda"), layout)
    want = out.clone()
    for t in range(tokens):
        for k in range(slots):
            if pos[t, k] >= 0:
                want[pos[t, k]] = x[t]
    word = torch.int32 if row_type == "f32" else torch.int16
    got = lrs.dispatch_rows(strided(x, layout), position, out=out)
    assert got is out and torch.equal(out.contiguous().view(word), want.contiguous().view(word))
    if layout != "packed":  # nothing beside the rows is written
        base = out._base
        assert bool(base[:, out.storage_offset() + cols:].isnan().all()) and bool(base[:, :out.storage_offset()].isnan().all())


@pytest.mark.parametrize("row_type,weight_type", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                                  ("f16", None), ("f32", None), ("f32", "f16")])
@pytest.mark.parametrize("tokens,slots,experts,kind,cols,layout", CASES)
def test_combine_rows(row_type, weight_type, tokens, slots, experts, kind, cols, layout):
    torch = torch_()
    announce("combine %s %s %s" % (row_type, weight_type, (tokens, slots, experts, kind, cols, layout)))
    position, pos = plan(tokens, slots, experts, 21, kind)
    rows = randn((tokens * slots, cols), row_type, 22)
    used = set(pos[pos >= 0].tolist())
    for r in range(rows.shape[0]):  # what no slot names is never read
        if r not in used:
            rows[r] = float("nan") if r % 2 else float("inf")
    w = None
    w64 = np.ones((tokens, slots))
    if weight_type is not None:
        w = torch.rand((tokens, slots), device="cuda").to(dtype_of(weight_type))
        w[position < 0] = float("nan")  # nor the weight of a slot without a position
        w64 = as64(w)
    r64 = as64(rows)
    want, mag = np.zeros((tokens, cols)), np.zeros((tokens, cols))
    for t in range(tokens):
        for k in range(slots):
            if pos[t, k] >= 0:
                want[t] += w64[t, k] * r64[pos[t, k]]
                mag[t] += np.abs(w64[t, k] * r64[pos[t, k]])
    out = strided(torch.full((tokens, cols), 5.0, dtype=rows.dtype, device="cuda"), layout)
    got = lrs.combine_rows(strided(rows, layout), position, w, out=out)
    assert got is out
    within(got, want, mag, slots)
    # the gradient of a dispatch is the sum without weights, in a new matrix
    if weight_type is None:
        assert torch.equal(lrs.combine_rows(rows, position), got)


@pytest.mark.parametrize("row_type,weight_type", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                                  ("f16", None)])
@pytest.mark.parametrize("tokens,slots,experts,kind,cols,layout", CASES)
def test_combine_rows_grad(row_type, weight_type, tokens, slots, experts, kind, cols, layout):
    torch = torch_()
    announce("combine grad %s %s %s" % (row_type, weight_type, (tokens, slots, experts, kind, cols, layout)))
    position, pos = plan(tokens, slots, experts, 31, kind)
    rows, gy = randn((tokens * slots, cols), row_type, 32), randn((tokens, cols), row_type, 33)
    used = set(pos[pos >= 0].tolist())
    for r in range(rows.shape[0]):
        if r not in used:
            rows[r] = float("nan")
    w = None
    w64 = np.ones((tokens, slots))
    if weight_type is not None:
        w = torch.rand((tokens, slots), device="cuda").to(dtype_of(weight_type))
        w[position < 0] = float("inf")
        w64 = as64(w)
    g64, r64 = as64(gy), as64(rows)
    want_w, mag_w = np.zeros((tokens, slots)), np.zeros((tokens, slots))
    want_r = np.full((tokens * slots, cols), 2.5)
    for t in range(tokens):
        for k in range(slots):
            if pos[t, k] >= 0:
                terms = g64[t] * r64[pos[t, k]]
                want_w[t, k], mag_w[t, k] = terms.sum(), np.abs(terms).sum()
                want_r[pos[t, k]] = w64[t, k] * g64[t]
    given = strided(torch.full((tokens * slots, cols), 2.5, dtype=rows.dtype, device="cuda"), layout)
    grad_rows, grad_w = lrs.combine_rows_grad(strided(gy, layout), strided(rows, layout), position, w, grad_rows=given)
    assert grad_rows is given
    within(grad_rows, want_r, np.abs(want_r), 1, "grad_rows")
    if w is None:
        assert grad_w is None
    else:
        assert grad_w.dtype == w.dtype
        within(grad_w, want_w, mag_w, cols, "grad_weights")
        # in place, over the rows themselves: the same answer, and what no slot names untouched
        mine = strided(rows, layout)
        before = mine.clone()
        again, again_w = lrs.combine_rows_grad(gy, mine, position, w, grad_rows=mine)
        keep = torch.tensor([r not in used for r in range(rows.shape[0])], device="cuda", dtype=torch.bool)
        assert torch.equal(again[~keep], grad_rows[~keep]) and torch.equal(again_w, grad_w)
        word = torch.int32 if row_type == "f32" else torch.int16
        assert torch.equal(again[keep].view(word), before[keep].view(word))
    # a new matrix: zeros where nothing is written
    fresh, _ = lrs.combine_rows_grad(gy, rows, position, w)
    assert torch.equal(fresh, torch.where((torch.from_numpy(want_r).cuda() == 2.5).all(1)[:, None] & ~torch.tensor(
        [r in used for r in range(rows.shape[0])], device="cuda", dtype=torch.bool)[:, None],
        torch.zeros_like(fresh), grad_rows.contiguous()))


def test_combine_grad_without_weight_gradient():
    """Through the C call: no weights' gradient wanted, the rows not even given."""
    torch = torch_()
    announce("combine grad, no weight gradient")
    position, pos = plan(50, 3, 6, 41, "far")
    gy, w = randn((50, 130), "bf16", 42), torch.rand((50, 3), device="cuda")
    out = torch.zeros(150, 130, dtype=torch.bfloat16, device="cuda")
    lrs.lrs_combine_rows_grad("bf16", gy, 130, None, 0, 150, position, "f32", w, 50, 3, 130, out, 130, None)
    want, _ = lrs.combine_rows_grad(gy, torch.zeros_like(out), position, w)
    assert torch.equal(out, want)


def test_no_slots_and_no_columns():
    torch = torch_()
    announce("no slots, no columns")
    none = torch.empty(5, 0, dtype=torch.int32, device="cuda")
    rows = torch.ones(4, 6, device="cuda")
    assert torch.equal(lrs.combine_rows(rows, none), torch.zeros(5, 6, device="cuda"))
    assert lrs.dispatch_rows(torch.ones(5, 6, device="cuda"), none).shape == (0, 6)
    position, _ = plan(5, 2, 3, 1)
    empty = torch.empty(10, 0, device="cuda")
    gr, gw = lrs.combine_rows_grad(torch.empty(5, 0, device="cuda"), empty, position, torch.ones(5, 2, device="cuda"))
    assert gr.shape == (10, 0) and torch.equal(gw, torch.zeros(5, 2, device="cuda"))
    assert lrs.combine_rows(empty, position).shape == (5, 0)
    assert lrs.embedding(empty, position).shape == (5, 2, 0)
    assert lrs.embedding_grad(torch.empty(5, 2, 0, device="cuda"), position, 7).shape == (7, 0)
    # no rows at all: every position is outside
    assert torch.equal(lrs.combine_rows(torch.empty(0, 6, device="cuda"), position), torch.zeros(5, 6, device="cuda"))


def test_positions_outside_the_rows_count_as_none():
    """Checked on the device against the number of rows: fewer rows than the plan
    names, and wild values."""
    torch = torch_()
    announce("positions outside")
    pos = torch.tensor([[0, 7], [-5, 2**31 - 1], [3, 1], [4, I32MIN], [2, 5]], dtype=torch.int32, device="cuda")
    x, rows = randn((5, 200), "f32", 51), randn((4, 200), "f32", 52)
    out = torch.full((4, 200), -1.0, device="cuda")
    lrs.dispatch_rows(x, pos, out=out)
    assert torch.equal(out, x[[0, 2, 4, 2]])
    y = lrs.combine_rows(rows, pos)
    want = torch.stack([rows[0], torch.zeros(200, device="cuda"), rows[3] + rows[1], torch.zeros(200, device="cuda"), rows[2]])
    assert torch.equal(y, want)
    w = torch.ones(5, 2, device="cuda")
    gr, gw = lrs.combine_rows_grad(x, rows, pos, w)
    assert torch.equal(gr, x[[0, 2, 4, 2]])
    assert torch.equal(gw == 0, torch.tensor([[False, True], [True, True], [False, False], [True, True], [False, True]], device="cuda"))


# ----------------------------------------------------------------- embedding

EMBED = [  # ids shape, vocab, cols, layout, kind
    ((1,), 1, 1, "packed", "uniform"),
    ((7,), 10, 3, "packed", "uniform"),
    ((2, 33), 100, 64, "pad", "far"),
    ((129,), 50, 513, "odd", "skewed"),
    ((1000,), 37, 136, "packed", "skewed"),
    ((3, 5, 41), 5000, 1000, "packed", "uniform"),
    ((2500,), 3, 200, "odd", "one"),
    ((4097,), 300, 72, "packed", "far"),
    ((64,), 70000, 24, "pad", "uniform"),
    ((300,), 40, 2100, "packed", "none"),
    ((6000,), 6000, 96, "packed", "uniform"),
    ((700,), 9, 9000, "odd", "skewed"),
]


def embed_ids(shape, vocab, kind, first, id_type):
    n = int(np.prod(shape))
    return routing(n, 1, vocab, n + vocab, kind, id_type, first).reshape(shape)


@pytest.mark.parametrize("row_type,scale,first,id_type", [("f32", 1.0, 0, "i64"), ("bf16", 1.0, 7, "i32"),
                                                          ("bf16", 22.627417, 0, "i64"), ("f16", -0.3, -4, "i64"),
                                                          ("f32", 3.3, 10**12, "i64")])
@pytest.mark.parametrize("shape,vocab,cols,layout,kind", EMBED)
def test_embedding(row_type, scale, first, id_type, shape, vocab, cols, layout, kind):
    torch = torch_()
    announce("embedding %s" % ((row_type, scale, first, id_type, shape, vocab, cols, layout, kind),))
    ids = embed_ids(shape, vocab, kind, first, id_type)
    table = randn((vocab, cols), row_type, 61)
    key = group_reference(ids, vocab, first)[3]
    t64 = np.concatenate([as64(table), np.zeros((1, cols))])
    want = (t64[key] * float(np.float32(scale))).reshape(shape + (cols,))
    out = strided(torch.full((ids.numel(), cols), 9.0, dtype=table.dtype, device="cuda"), layout)
    if len(shape) == 1:
        got = lrs.embedding(strided(table, layout), ids, scale=scale, first_id=first, out=out)
        assert got is out
    else:
        got = lrs.embedding(strided(table, layout), ids, scale=scale, first_id=first)
    within(got, want, np.abs(want), 0 if scale == 1.0 else 1)
    if scale == 1.0:
        assert np.array_equal(as64(got), want)


@pytest.mark.parametrize("row_type,grad_type,accumulate,first,id_type", [
    ("f32", "f32", False, 0, "i64"), ("bf16", "bf16", False, 7, "i32"), ("bf16", "f32", True, 0, "i64"),
    ("f16", "f16", True, -4, "i64"), ("f16", "f32", False, 0, "i32"), ("f32", "f32", True, 10**12, "i64"),
    ("bf16", "bf16", True, 3, "i32")])
@pytest.mark.parametrize("shape,vocab,cols,layout,kind", EMBED)
def test_embedding_grad(row_type, grad_type, accumulate, first, id_type, shape, vocab, cols, layout, kind):
    torch = torch_()
    announce("embedding grad %s" % ((row_type, grad_type, accumulate, first, id_type, shape, vocab, cols, layout, kind),))
    scale = 0.37
    ids = embed_ids(shape, vocab, kind, first, id_type)
    n = ids.numel()
    gy = randn((n, cols), row_type, 71)
    key = group_reference(ids, vocab, first)[3]
    gy[torch.from_numpy(key == vocab).cuda()] = float("nan")  # what belongs to no row is never read
    g64 = np.nan_to_num(as64(gy))
    total, mag = np.zeros((vocab + 1, cols)), np.zeros((vocab + 1, cols))
    np.add.at(total, key, g64)
    np.add.at(mag, key, np.abs(g64))
    s = float(np.float32(scale))
    want, mag = total[:vocab] * s, mag[:vocab] * s
    start = randn((vocab, cols), grad_type, 72)
    touched = np.bincount(key, minlength=vocab + 1)[:vocab] > 0
    untouched = torch.from_numpy(~touched).cuda()
    if accumulate:
        start[untouched] = float("nan")  # not read, not written
        old = np.nan_to_num(as64(start))
        want, mag = want + old, mag + np.abs(old)
    grad = strided(start, layout)
    most = int(np.bincount(key, minlength=vocab + 1)[:vocab].max())
    got = lrs.embedding_grad(strided(gy, layout) if len(shape) == 1 else gy.reshape(shape + (cols,)), ids, vocab,
                             scale=scale, first_id=first, dtype=dtype_of(grad_type), grad=grad, accumulate=accumulate)
    assert got is grad
    if accumulate:
        assert bool(got[untouched].isnan().all())
        got = got.clone()
        got[untouched] = 0.0
    # at most one rounding per addition, one for the scale and one for the old value
    within(got, want, mag, most + 2)
    if not accumulate:
        assert bool((got[untouched] == 0).all())
        new = lrs.embedding_grad(gy.reshape(shape + (cols,)), ids, vocab, scale=scale, first_id=first,
                                 dtype=dtype_of(grad_type))
        assert torch.equal(new, got)


def test_embedding_grad_of_no_ids():
    torch = torch_()
    announce("embedding grad of no ids")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    gy = torch.empty(0, 70, device="cuda")
    assert torch.equal(lrs.embedding_grad(gy, ids, 9), torch.zeros(9, 70, device="cuda"))
    old = randn((9, 70), "f32", 1)
    assert torch.equal(lrs.embedding_grad(gy, ids, 9, grad=old.clone(), accumulate=True), old)
    assert lrs.embedding(torch.ones(9, 70, device="cuda"), ids).shape == (0, 70)


@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_embedding_grad_of_long_runs(share):
    """Whole numbers, so that the sums are exact in any order: a share of 70,000 tokens
    is one id (a pad token), the rest spread; runs that end on and beside the
    boundaries of the pieces in which they are summed."""
    torch = torch_()
    announce("embedding grad of long runs, share %g" % share)
    n, vocab, cols = 70000, 5000, 40
    rng = np.random.default_rng(5)
    ids = rng.integers(0, vocab, n)
    ids[rng.random(n) < share] = 1234
    for at, run in ((4000, 64), (4001, 128), (4002, 32), (4003, 31), (4004, 33), (4005, 256), (4006, 1)):
        if share < 1.0:
            ids[ids == at] = 0
            ids[rng.choice(np.flatnonzero(ids < 1000), run, replace=False)] = at
    gy = rng.integers(-8, 9, (n, cols))
    want = np.zeros((vocab, cols), dtype=np.int64)
    np.add.at(want, ids, gy)
    got = lrs.embedding_grad(torch.from_numpy(gy).float().cuda(), torch.from_numpy(ids).cuda(), vocab)
    assert np.array_equal(got.cpu().numpy().astype(np.int64), want)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 31, 33, 63, 65, 127, 1023, 1024, 1025, 4096, 4097, 5000, 131072, 131073,
                               200001])
def test_embedding_grad_lengths(n):
    """Whole numbers again: both sides of every length at which the ids are ordered
    another way, ids of one to four digits, spread, in long runs, and of no row."""
    torch = torch_()
    rng = np.random.default_rng(n)
    for vocab, cols, first in ((1, 8, 0), (300, 33, -7), (3000, 64, 5), (600000, 4, 0)):
        announce("embedding grad of %d ids, vocab %d" % (n, vocab))
        for kind in ("spread", "runs", "outside"):
            ids = rng.integers(0, vocab, n)
            if kind == "runs":
                ids = ids // max(1, vocab // 5) * max(1, vocab // 5)
            if kind == "outside":
                ids = np.where(rng.random(n) < 0.9, rng.choice([-1, vocab, 2**40, -2**40], n), ids)
            gy = rng.integers(-8, 9, (n, cols))
            inside = (ids >= 0) & (ids < vocab)
            want = np.zeros((vocab, cols), dtype=np.int64)
            np.add.at(want, ids[inside], gy[inside])
            got = lrs.embedding_grad(torch.from_numpy(gy).float().cuda(), torch.from_numpy(ids + first).cuda(), vocab,
                                     first_id=first)
            assert np.array_equal(got.cpu().numpy().astype(np.int64), want), kind


@pytest.mark.parametrize("vocab", [511, 512, 1023, 1024, 2047, 2048, 2**18 - 1, 2**18, 2**20, 2**22 - 1, 2**22])
def test_embedding_grad_digits(vocab):
    """Whole numbers again: keys of every number of digits, of each width, on both
    sides of the lengths at which the digits become narrower."""
    torch = torch_()
    rng = np.random.default_rng(vocab)
    for n in (4097, 12289, 16384, 16385, 32768, 32769):
        announce("embedding grad of %d ids, vocab %d" % (n, vocab))
        for kind in ("spread", "one digit", "last"):
            ids = rng.integers(-1, vocab + 1, n)
            if kind == "one digit":
                ids = ids & ~0x3FF
            if kind == "last":
                ids = vocab - rng.integers(0, 3, n)
            gy = rng.integers(-8, 9, (n, 3))
            inside = (ids >= 0) & (ids < vocab)
            want = np.zeros((vocab, 3), dtype=np.int64)
            np.add.at(want, ids[inside], gy[inside])
            got = lrs.embedding_grad(torch.from_numpy(gy).float().cuda(), torch.from_numpy(ids).cuda(), vocab)
            assert np.array_equal(got.cpu().numpy().astype(np.int64), want), kind


# -------------------------------------------------------------------- together


@pytest.mark.parametrize("row_type", ["f32", "bf16"])
def test_mixture_of_experts_step(row_type):
    """A whole step as a training program runs it, twice over the same buffers:
    embedding, grouping, dispatch, experts (each scales its rows by its own number),
    the weighted way back; then every gradient, compared with the formula's in 64
    bits.  Values are small whole numbers and weights eighths, so that every sum is
    exact in float32 and every product exact; the only rounding is the store's."""
    torch = torch_()
    announce("mixture step %s" % row_type)
    vocab, tokens, slots, experts, cols = 97, 260, 3, 11, 88
    first, local = 2, 7  # a rank's share: the other experts' choices are dropped
    for step in range(2):
        rng = np.random.default_rng(80 + step)
        ids = rng.integers(0, vocab, tokens)
        chosen = np.stack([rng.permutation(experts)[:slots] for _ in range(tokens)])
        w64 = rng.integers(0, 9, (tokens, slots)) / 8.0
        table64 = rng.integers(-3, 4, (vocab, cols)).astype(np.float64)
        gain = rng.integers(1, 3, experts).astype(np.float64)
        gy64 = rng.integers(-2, 3, (tokens, cols)).astype(np.float64)
        dev = lambda a, t: torch.from_numpy(a).cuda().to(t)  # noqa: E731
        dt = dtype_of(row_type)
        table, gy, w = dev(table64, dt), dev(gy64, dt), dev(w64, torch.float32)
        x = lrs.embedding(table, dev(ids, torch.int64), scale=2.0)
        order, position, offsets = lrs.group_tokens(dev(chosen, torch.int64), local, first_id=first)
        rows = lrs.dispatch_rows(x, position)
        bounds = offsets.cpu().numpy()
        answers = torch.full_like(rows, float("nan"))
        for e in range(local):
            answers[bounds[e]:bounds[e + 1]] = rows[bounds[e]:bounds[e + 1]] * gain[first + e]
        y = lrs.combine_rows(answers, position, w)
        grad_answers, grad_w = lrs.combine_rows_grad(gy, answers, position, w)
        for e in range(local):
            grad_answers[bounds[e]:bounds[e + 1]] *= gain[first + e]
        grad_x = lrs.combine_rows(grad_answers, position)
        grad_table = lrs.embedding_grad(grad_x, dev(ids, torch.int64), vocab, scale=2.0, dtype=torch.float32)

        here = (chosen >= first) & (chosen < first + local)
        factor = np.where(here, w64 * gain[chosen], 0.0)  # y[t] = x[t] * sum of factors
        x64 = table64[ids] * 2.0
        half = torch.finfo(dt).eps / 2
        assert np.array_equal(as64(x), x64)
        want = x64 * factor.sum(1)[:, None]
        assert (np.abs(as64(y) - want) <= half * np.abs(want)).all()
        dots = np.where(here, (gy64[:, None, :] * x64[:, None, :]).sum(2) * gain[chosen], 0.0)
        assert np.array_equal(as64(grad_w), dots)
        want = gy64 * factor.sum(1)[:, None]
        # w * grad_y (at most 9 significant bits of 8) is exact in bfloat16 too
        assert (np.abs(as64(grad_x) - want) <= half * np.abs(want)).all()
        total = np.zeros((vocab, cols))
        np.add.at(total, ids, as64(grad_x))
        assert np.array_equal(as64(grad_table), total * 2.0)


def test_gradients_against_differences():
    """combine_rows is linear in its rows and in its weights, embedding in its table:
    a difference over a step of any length is the derivative.  The inner products are
    formed in 64 bits; each of the outputs' float32 values is off by at most
    (slots + 1) * 2^-24 of its terms' magnitudes, bounded here through the sums of
    magnitudes."""
    torch = torch_()
    announce("differences")
    tokens, slots, experts, cols = 120, 4, 9, 333
    position, pos = plan(tokens, slots, experts, 91, "far")
    rows, gy = randn((tokens * slots, cols), "f32", 92), randn((tokens, cols), "f32", 93)
    w, step_r, step_w = torch.rand((tokens, slots), device="cuda"), randn(rows.shape, "f32", 94), randn((tokens, slots), "f32", 95)
    grad_rows, grad_w = lrs.combine_rows_grad(gy, rows, position, w)

    def inner(a, b):
        return float((a.double() * b.double()).sum())

    def size(a, b):
        return float((a.double() * b.double()).abs().sum())

    # (the steps themselves are rounded: use what was added)
    up, down = rows + step_r, rows - step_r
    diff = inner(gy, lrs.combine_rows(up, position, w)) - inner(gy, lrs.combine_rows(down, position, w))
    bound = (slots + 1) * 2.0**-24 * 4 * (size(gy.abs(), lrs.combine_rows(up.abs(), position, w)) +
                                          size(gy.abs(), lrs.combine_rows(down.abs(), position, w)))
    assert abs(diff - inner(grad_rows, up.double() - down.double())) <= bound
    up, down = w + step_w, w - step_w
    diff = inner(gy, lrs.combine_rows(rows, position, up)) - inner(gy, lrs.combine_rows(rows, position, down))
    near = lrs.combine_rows(rows.abs(), position, up.abs() + down.abs())
    bound = (cols + slots + 1) * 2.0**-24 * 4 * size(gy.abs(), near)
    assert abs(diff - inner(grad_w, up.double() - down.double())) <= bound

    ids = routing(400, 1, 60, 96, "far").reshape(-1)
    table, step, gz = randn((60, cols), "f32", 97), randn((60, cols), "f32", 98), randn((400, cols), "f32", 99)
    grad = lrs.embedding_grad(gz, ids, 60, scale=1.7)
    up, down = table + step, table - step
    diff = inner(gz, lrs.embedding(up, ids, scale=1.7)) - inner(gz, lrs.embedding(down, ids, scale=1.7))
    bound = (400 + 2) * 2.0**-24 * 4 * size(gz.abs(), lrs.embedding(up.abs() + down.abs(), ids, scale=1.7))
    assert abs(diff - inner(grad, up.double() - down.double())) <= bound


def test_infinities_nan_and_subnormals():
    """What the values of real slots and rows hold reaches the results as in IEEE
    arithmetic, results below the normal range keep their bits (half the smallest
    subnormal is allowed), and a sum beyond float16 rounds to infinity."""
    torch = torch_()
    announce("special values")
    inf, nan = float("inf"), float("nan")
    for name, cols in (("f32", 5), ("bf16", 11), ("f16", 11)):
        dt = dtype_of(name)
        rows = torch.ones(4, cols, dtype=dt, device="cuda")
        rows[0, 0], rows[1, 1], rows[2, 2], rows[3, 2] = inf, nan, inf, -inf
        position = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
        y = lrs.combine_rows(rows, position)
        want = torch.full((2, cols), 2.0, dtype=dt, device="cuda")
        want[0, 0], want[0, 1], want[1, 2] = inf, nan, nan
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))
        grad = lrs.embedding_grad(rows, torch.tensor([3, 3, 1, 1], device="cuda"), 5)
        want = torch.zeros(5, cols, dtype=dt, device="cuda")
        want[3], want[1] = 2.0, 2.0
        want[3, 0], want[3, 1], want[1, 2] = inf, nan, nan
        assert torch.equal(grad.isnan(), want.isnan()) and torch.equal(grad.nan_to_num(7.0), want.nan_to_num(7.0))
    big = torch.full((2, 3), 60000.0, dtype=torch.float16, device="cuda")
    assert bool((lrs.combine_rows(big, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")) == inf).all())
    for name, scale, step in (("f32", 2.0**-140, 2.0**-149), ("bf16", 2.0**-128, 2.0**-133), ("f16", 2.0**-20, 2.0**-24)):
        table = randn((50, 40), name, 151)
        ids = torch.arange(50, device="cuda")
        want = as64(table) * scale
        assert (np.abs(as64(lrs.embedding(table, ids, scale=scale)) - want) <= step / 2).all(), name
        assert (np.abs(as64(lrs.embedding_grad(table, ids, 50, scale=scale)) - want) <= step / 2).all(), name


def test_rows_named_by_several_tokens():
    """The way back may read a row more than once, also within a token."""
    torch = torch_()
    announce("rows named twice")
    rows = randn((6, 77), "f32", 161)
    position = torch.tensor([[0, 0, 5], [5, 0, 2]], dtype=torch.int32, device="cuda")
    want = torch.stack([rows[0].double() * 2 + rows[5].double(), rows[5].double() + rows[0].double() + rows[2].double()])
    mag = torch.stack([rows[0].abs() * 2 + rows[5].abs(), rows[5].abs() + rows[0].abs() + rows[2].abs()])
    within(lrs.combine_rows(rows, position), as64(want), as64(mag), 3)


# --------------------------------------------- streams, graphs, large offsets


def whole_step(state):
    """One step through every operator, by the C calls, over the state's buffers."""
    s = state
    st = torch_().cuda.current_stream()
    lrs.lrs_group_tokens(s["temp"], s["group_need"], "i64", s["chosen"], s["chosen"].numel(), 0, 12, s["order"],
                         s["position"], s["offsets"], st)
    t, k, h = s["chosen"].shape[0], s["chosen"].shape[1], s["table"].shape[1]
    lrs.lrs_embedding("bf16", s["table"], h, s["table"].shape[0], "i64", s["ids"], t, 0, 1.5, h, s["x"], h, st)
    lrs.lrs_dispatch_rows("bf16", s["x"], h, s["position"], t, k, h, s["rows"], h, t * k, st)
    lrs.lrs_combine_rows("bf16", s["rows"], h, t * k, s["position"], "f32", s["w"], t, k, h, s["y"], h, st)
    lrs.lrs_combine_rows_grad("bf16", s["y"], h, s["rows"], h, t * k, s["position"], "f32", s["w"], t, k, h,
                              s["grad_rows"], h, s["grad_w"], st)
    lrs.lrs_combine_rows("bf16", s["grad_rows"], h, t * k, s["position"], 0, None, t, k, h, s["grad_x"], h, st)
    lrs.lrs_embedding_grad(s["temp"], s["temp"].numel(), "bf16", s["grad_x"], h, "i64", s["ids"], t, 0, 1.5, "f32",
                           s["grad"], h, s["table"].shape[0], h, 0, st)


OUTPUTS = ("order", "position", "offsets", "x", "rows", "y", "grad_rows", "grad_w", "grad_x", "grad")


def step_state(tokens, vocab, cols, seed):
    torch = torch_()
    k = 4
    s = {"chosen": routing(tokens, k, 12, seed), "ids": routing(tokens, 1, vocab, seed + 1, "skewed").reshape(-1),
         "table": randn((vocab, cols), "bf16", seed + 2), "w": torch.rand((tokens, k), device="cuda")}
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    for name, shape, dt in (("order", tokens * k, i32), ("position", (tokens, k), i32), ("offsets", 13, i32),
                            ("x", (tokens, cols), bf), ("rows", (tokens * k, cols), bf), ("y", (tokens, cols), bf),
                            ("grad_rows", (tokens * k, cols), bf), ("grad_w", (tokens, k), f32),
                            ("grad_x", (tokens, cols), bf), ("grad", (vocab, cols), f32)):
        s[name] = torch.zeros(shape, dtype=dt, device="cuda")
    s["group_need"] = lrs.lrs_group_tokens(None, 0, "i64", s["chosen"], tokens * k, 0, 12, s["order"], s["position"], s["offsets"])
    need = lrs.lrs_embedding_grad(None, 0, "bf16", s["grad_x"], cols, "i64", s["ids"], tokens, 0, 1.5, "f32", s["grad"],
                                  cols, vocab, cols, 0)
    s["temp"] = torch.empty(max(need, s["group_need"]), dtype=torch.uint8, device="cuda")
    return s


@pytest.mark.parametrize("tokens,vocab,cols", [(3, 50, 256), (700, 300, 200), (9000, 70000, 64)])
def test_captured_step_replays(tokens, vocab, cols):
    """Every operator captured into one graph and replayed on new inputs, eager work
    between the replays, each bit for bit like the eager step on those inputs."""
    torch = torch_()
    announce("captured step %s" % ((tokens, vocab, cols),))
    s = step_state(tokens, vocab, cols, 101)
    whole_step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole_step(s)
    for rep in range(4):
        other = step_state(tokens, vocab, cols, 200 + rep)
        for name in ("chosen", "ids", "table", "w"):
            s[name].copy_(other[name])
        for name in OUTPUTS + ("temp",):
            s[name].fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        (torch.arange(1 << 20, device="cuda") * 3).sum().item()
        other["temp"].fill_(rep)
        whole_step(other)
        torch.cuda.synchronize()
        for name in OUTPUTS:
            assert torch.equal(s[name], other[name]), (rep, name)


def test_two_captured_steps_share_no_state():
    """Two graphs of their own buffers, replayed on two streams at once."""
    torch = torch_()
    announce("two captured steps")
    states = [step_state(1500, 4000, 128, 300 + i) for i in range(2)]
    want = []
    for s in states:
        whole_step(s)
        torch.cuda.synchronize()
        want.append({name: s[name].clone() for name in OUTPUTS})
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            whole_step(s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in states]
    for rep in range(4):
        for s in states:
            for name in OUTPUTS:
                s[name].zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            for name in OUTPUTS:
                assert torch.equal(s[name], w[name]), (rep, name)


@pytest.mark.parametrize("as_int", [False, True])
def test_conveniences_on_a_side_stream(as_int):
    """Inputs written on the current stream just before the call, strided ones copied
    there, outputs allocated there; the result read after the side stream."""
    torch = torch_()
    announce("side stream, as int %s" % as_int)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    chosen, w = routing(3000, 2, 10, 111), torch.rand(3000, 2, device="cuda")
    ids, gy = routing(3000, 1, 500, 112).reshape(-1), randn((3000, 640), "f32", 113)
    table = randn((500, 640), "f32", 114)
    want_pos = lrs.group_tokens(chosen, 10)[1]
    x0 = lrs.embedding(table, ids)
    want_rows = lrs.dispatch_rows(x0, want_pos)
    want_y = lrs.combine_rows(want_rows, want_pos, w)
    want_gr, want_gw = lrs.combine_rows_grad(gy, want_rows, want_pos, w)
    want_g = lrs.embedding_grad(gy, ids, 500)
    for rep in range(3):
        junk = [torch.full((3000, 640), float("nan"), device="cuda") for _ in range(6)]
        torch.matmul(torch.ones(2048, 2048, device="cuda"), torch.ones(2048, 2048, device="cuda"))
        del junk  # the allocator gives this memory, still being written, to what follows
        turned = table.t().contiguous().t()  # not contiguous within a row: copied first
        _, pos, _ = lrs.group_tokens(chosen.t().contiguous().t(), 10, stream=stream)
        x = lrs.embedding(turned, ids, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        rows = lrs.dispatch_rows(x, pos, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        y = lrs.combine_rows(rows, pos, w, stream=stream)
        gr, gw = lrs.combine_rows_grad(gy.t().contiguous().t(), rows, pos, w, stream=stream)
        g = lrs.embedding_grad(gy.t().contiguous().t(), ids, 500, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        for got, want in ((pos, want_pos), (rows, want_rows), (y, want_y), (gr, want_gr), (gw, want_gw), (g, want_g)):
            assert torch.equal(got, want)


def test_calls_from_several_threads():
    """Host threads, each on a stream of its own, through the conveniences at once."""
    import threading
    torch = torch_()
    announce("several threads")
    chosen, w = [routing(1500 + 100 * i, 3, 12, 170 + i) for i in range(4)], [torch.rand(1500 + 100 * i, 3, device="cuda")
                                                                              for i in range(4)]
    x = [randn((1500 + 100 * i, 264), "bf16", 180 + i) for i in range(4)]

    def work(i):
        order, position, offsets = lrs.group_tokens(chosen[i], 12)
        rows = lrs.dispatch_rows(x[i], position)
        y = lrs.combine_rows(rows, position, w[i])
        grad_rows, grad_w = lrs.combine_rows_grad(y, rows, position, w[i])
        ids = chosen[i][:, 0].contiguous()
        return [order, position, offsets, rows, y, grad_rows, grad_w, lrs.embedding_grad(y, ids, 700 + i)]

    want = [work(i) for i in range(4)]
    torch.cuda.synchronize()
    got = [[] for _ in range(4)]

    def thread(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got[i].append(work(i))
        stream.synchronize()

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert len(got[i]) == 5
        for answers in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(answers, want[i]))


def test_tensors_of_two_devices_and_given_temp():
    torch = torch_()
    announce("two devices, given temp")
    ids, x = routing(300, 2, 9, 190), randn((300, 40), "f32", 191)
    order, position, offsets = lrs.group_tokens(ids, 9)
    rows, w = lrs.dispatch_rows(x, position), torch.rand(300, 2, device="cuda")
    flat = ids[:, 0].contiguous()
    for call in (lambda: lrs.dispatch_rows(x, position.cpu()), lambda: lrs.dispatch_rows(x.cpu(), position),
                 lambda: lrs.dispatch_rows(x, position, out=torch.zeros(600, 40)),
                 lambda: lrs.combine_rows(rows, position, w.cpu()), lambda: lrs.combine_rows(rows.cpu(), position),
                 lambda: lrs.combine_rows_grad(x.cpu(), rows, position, w), lambda: lrs.embedding(x, flat.cpu()),
                 lambda: lrs.embedding(x.cpu(), flat), lambda: lrs.embedding_grad(x, flat.cpu(), 9),
                 lambda: lrs.embedding_grad(x, flat, 9, grad=torch.zeros(9, 40)),
                 lambda: lrs.group_tokens(ids, 9, temp=torch.zeros(1 << 20)),
                 lambda: lrs.embedding_grad(x, flat, 9, temp=torch.zeros(1 << 20))):
        with pytest.raises(ValueError, match="is on|device tensors"):
            call()
    for temp in (torch.empty(1 << 22, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")):
        assert all(torch.equal(a, b) for a, b in zip(lrs.group_tokens(ids, 9, temp=temp), (order, position, offsets)))
        assert torch.equal(lrs.embedding_grad(x, flat, 9, temp=temp), lrs.embedding_grad(x, flat, 9))
    big = routing(20000, 2, 9, 192)
    temp = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(lrs.group_tokens(big, 9, temp=temp), lrs.group_tokens(big, 9)))


def test_results_are_the_same_on_every_run():
    torch = torch_()
    announce("same on every run")
    s = step_state(9000, 3000, 520, 120)
    whole_step(s)
    want = {name: s[name].clone() for name in OUTPUTS}
    for _ in range(5):
        for name in OUTPUTS + ("temp",):
            s[name].fill_(1)
        whole_step(s)
        for name in OUTPUTS:
            assert torch.equal(s[name], want[name]), name


def test_offsets_past_32_bits():
    """Tables, rows and gradients beyond 2^32 elements' bytes and 2^31 elements: rows
    at both ends of them."""
    torch = torch_()
    announce("large offsets: table and its gradient")
    cols, vocab = 32768, 70001  # 2.3e9 elements
    table = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, 65536, 65535, vocab - 1, vocab, -1], device="cuda")
    marks = randn((7, cols), "bf16", 131)
    table[ids[:4]] = marks[:4]
    y = lrs.embedding(table, ids)
    assert torch.equal(y[1:4], marks[1:4]) and torch.equal(y[0], y[4]) and torch.equal(y[0], marks[0])
    assert bool((y[5:] == 0).all())
    table.fill_(float("nan"))
    grad = lrs.embedding_grad(marks, ids, vocab, grad=table)
    assert torch.equal(grad[[0, 65536, 65535]], marks[[1, 2, 3]])
    assert torch.equal(grad[vocab - 1], (marks[0].float() + marks[4].float()).to(torch.bfloat16))
    assert int((grad != 0).any(1).sum()) == 4
    del grad, table, y
    announce("large offsets: rows by position")
    n = 70001
    rows = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[n - 1, 5], [65537, n - 2], [-1, 0]], dtype=torch.int32, device="cuda")
    x = randn((3, cols), "bf16", 132)
    lrs.dispatch_rows(x, position, out=rows)
    assert torch.equal(rows[[n - 1, 5, 65537, n - 2, 0]], x[[0, 0, 1, 1, 2]])
    w = torch.tensor([[0.5, 0.25], [1.0, 2.0], [9.0, 0.5]], device="cuda")
    y = lrs.combine_rows(rows, position, w)
    want = torch.tensor([0.75, 3.0, 0.5], device="cuda")[:, None] * x.float()
    assert bool(((y.float() - want).abs() <= want.abs() * 2.0**-8).all())
    grad_rows, _ = lrs.combine_rows_grad(x, rows, position, w, grad_rows=rows)
    assert torch.equal(grad_rows[n - 2], (2.0 * x[1].float()).to(torch.bfloat16))
    assert torch.equal(grad_rows[n - 1], (0.5 * x[0].float()).to(torch.bfloat16))


def test_many_rows_of_few_columns():
    """More row tiles than one grid dimension holds."""
    torch = torch_()
    announce("many rows")
    n = 65535 * 8 + 77
    ids = torch.arange(n, device="cuda") % 1000
    table = randn((1000, 300), "f16", 141)
    assert torch.equal(lrs.embedding(table, ids), table[ids])
    position = torch.arange(n, device="cuda", dtype=torch.int32).flip(0).reshape(n, 1)
    x = lrs.embedding(table[:, :64], ids)
    rows = lrs.dispatch_rows(x, position)
    assert torch.equal(rows, x.flip(0))
    assert torch.equal(lrs.combine_rows(rows, position), x)
