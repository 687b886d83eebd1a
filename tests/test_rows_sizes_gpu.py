"""The row operators at the sizes of prompts and training batches, where they take other
kernels than small calls do, against their definitions in 64 bits on the device.

The sizes lie on both sides of each change of path: 2,048 workgroups (a token's slots one
after another instead of at once), 32 MiB (rows past the L2s), 256 MiB of grad_y (read
past the caches), the lengths of an embedding gradient's pieces, and the rows that one
pass over a grid's limit serves.

Tolerances count roundings: an output formed in float32 by at most m roundings of terms
whose magnitudes add up to S, and rounded once to its type, is within
e + (|r| + e) * eps / 2 + 2^-25 of the exact r, e = m * 2^-24 * S * (1 + 2^-10) (half the
smallest float16 subnormal is 2^-25; the factor covers higher orders for m <= 2^13).
"""
from __future__ import annotations

import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu


def torch_():
    import torch
    return torch


def dtype_of(name):
    torch = torch_()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def within(got, want, magnitude, terms, what):
    torch = torch_()
    e = terms * 2.0**-24 * (1 + 2.0**-10) * magnitude
    tol = e + (want.abs() + e) * (torch.finfo(got.dtype).eps / 2) + 2.0**-25
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d outside, first at %s" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


def laid_out(t, layout):
    """The matrix as it is, or as columns of a wider one: "odd", off every 16-byte boundary."""
    torch = torch_()
    if layout == "packed":
        return t
    cols = t.shape[1]
    wide = torch.full((t.shape[0], cols + 6 + (cols & 1)), float("nan"), dtype=t.dtype, device="cuda")
    wide = torch.cat([wide, wide[:, :1]], 1)  # an odd stride
    view = wide[:, 3:3 + cols]
    view.copy_(t)
    return view


def routed(tokens, slots, experts, first, count, seed):
    """Positions of the slots whose expert is one of [first, first + count)."""
    torch = torch_()
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.rand(tokens, experts, generator=g, device="cuda").topk(slots, dim=1).indices
    return lrs.group_tokens(ids, count, first_id=first)[1], g


# tokens, slots, columns of 16-bit rows (half as many of float32), layout, experts, first, count
CASES = [
    (2047, 3, 2048, "packed", 8, 0, 8),    # 2,047 workgroups
    (2048, 3, 2048, "packed", 8, 0, 8),    # 2,048; 32 MiB of rows and sums, not more
    (2049, 3, 2048, "odd", 8, 0, 7),       # more than either
    (2100, 2, 1500, "odd", 7, 0, 6),       # more workgroups, the gradient's rows not past the L2s
    (300001, 1, 12, "odd", 3, 1, 2),       # the same with many rows a wave
    (2500, 8, 2056, "odd", 16, 2, 11),     # two workgroups a row, the second nearly empty
    (600, 5, 8200, "packed", 9, 0, 8),     # many columns: sums over the limit, gradients' tokens below
    (140001, 2, 24, "packed", 4, 1, 3),    # several rows a wave, the gradient just past the L2s
    (400003, 4, 22, "odd", 12, 0, 9),      # the same past the L2s
    (9000, 1, 1000, "packed", 5, 0, 4),    # one slot
]


@pytest.mark.parametrize("row_type,weight_type", [("bf16", "f32"), ("f32", "f32"), ("f16", "f16"), ("bf16", None)])
@pytest.mark.parametrize("tokens,slots,cols,layout,experts,first,count", CASES)
def test_combine_and_its_gradient(row_type, weight_type, tokens, slots, cols, layout, experts, first, count):
    torch = torch_()
    cols = cols // 2 if row_type == "f32" else cols
    announce("combine and gradient %s %s %s" % (row_type, weight_type,
                                               (tokens, slots, cols, layout, experts, first, count)))
    position, g = routed(tokens, slots, experts, first, count, tokens + cols)
    dt, n = dtype_of(row_type), tokens * slots
    rows = torch.randn(n, cols, generator=g, device="cuda").to(dt)
    grad_y = torch.randn(tokens, cols, generator=g, device="cuda").to(dt)
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    used[position[position >= 0].long()] = True
    rows[~used] = float("nan")  # what no slot names is never read
    w = None
    if weight_type is not None:
        w = torch.rand(tokens, slots, generator=g, device="cuda").to(dtype_of(weight_type))
        w[position < 0] = float("nan")
    rows = laid_out(rows, layout)
    grad_y = laid_out(grad_y, layout)

    y64 = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y64)
    grad_rows64 = torch.full((n, cols), 2.5, dtype=torch.float64, device="cuda")
    grad_w64 = torch.zeros(tokens, slots, dtype=torch.float64, device="cuda")
    grad_w_size = torch.zeros_like(grad_w64)
    for k in range(slots):
        on = (position[:, k] >= 0).nonzero()[:, 0]
        at = position[on, k].long()
        weight = w[on, k].double()[:, None] if w is not None else 1.0
        term = rows[at].double()
        gy = grad_y[on].double()
        grad_rows64[at] = weight * gy
        grad_w64[on, k] = (gy * term).sum(1)
        grad_w_size[on, k] = (gy * term).abs().sum(1)
        y64[on] += weight * term
        size[on] += (weight * term).abs()

    within(lrs.combine_rows(rows, position, w), y64, size, slots, "y")
    out = laid_out(torch.full((n, cols), 2.5, dtype=dt, device="cuda"), layout)
    grad_rows, grad_w = lrs.combine_rows_grad(grad_y, rows, position, w, grad_rows=out)
    within(grad_rows, grad_rows64, grad_rows64.abs(), 1, "grad_rows")
    assert bool((grad_rows[~used] == 2.5).all())
    if w is not None:
        within(grad_w, grad_w64, grad_w_size, cols, "grad_weights")
        assert bool((grad_w[position < 0] == 0).all())
        # over the rows themselves: the same, and what no slot names is left as it was
        again, again_w = lrs.combine_rows_grad(grad_y, rows, position, w, grad_rows=rows)
        assert torch.equal(again[used], grad_rows[used]) and torch.equal(again_w, grad_w)
        assert bool(again[~used].isnan().all())


# rows of grad_y, columns, type of grad_y, of the gradient, and what the case takes
EMBED = [
    (33100, 4096, "bf16", "f32", "pieces of 32"),
    (70001, 4096, "bf16", "bf16", "pieces of 64, past the caches"),
    (70001, 1024, "f32", "f32", "pieces of 32, past the caches"),
    (600000, 40, "f16", "f32", "pieces of 64, several in a wave, the library's sort"),
    (2200000, 64, "bf16", "bf16", "pieces of 256, several in a wave, past the caches"),
    (33100, 65536, "bf16", "f32", "pieces of 512, past the caches"),
]


@pytest.mark.parametrize("n,cols,row_type,grad_type,what", EMBED)
def test_embedding_grad_in_long_pieces(n, cols, row_type, grad_type, what):
    """Whole numbers, so that every sum is exact in float32 in any order.  Sorted, the
    ids are runs of lengths around one, two and three pieces of each length, at many
    offsets, one run of a quarter of the ids, and a tail of no row."""
    torch = torch_()
    announce("embedding grad %s" % ((n, cols, row_type, grad_type, what),))
    g = torch.Generator("cuda").manual_seed(n + cols)
    lengths = [1, 2, 3]
    for p in (16, 32, 64, 256, 512):
        lengths += [p - 1, p, p + 1, 2 * p - 1, 2 * p, 2 * p + 1, 3 * p, 3 * p + 1, 7]
    runs, total, i = [], 0, 0
    while total < n - n // 10:
        runs.append(n // 4 if len(runs) == 20 else lengths[i * 7 % len(lengths)])
        total, i = total + runs[-1], i + 1
    sorted_ids = torch.repeat_interleave(torch.arange(len(runs), device="cuda") * 2 + 1,
                                         torch.tensor(runs, device="cuda"))[:n]
    vocab = 2 * len(runs) + 3  # every other row is named by no id
    tail = torch.full((n - sorted_ids.numel(),), vocab, device="cuda")
    ids = torch.cat([sorted_ids, tail])[torch.randperm(n, generator=g, device="cuda")]
    inside = ids < vocab
    grad_y = torch.randint(-8, 9, (n, cols), generator=g, device="cuda", dtype=torch.int8).to(dtype_of(row_type))
    grad_y[~inside] = float("nan")
    dt = dtype_of(grad_type)
    start = torch.randint(-99, 100, (vocab, cols), generator=g, device="cuda", dtype=torch.int8).to(dt)
    got = lrs.embedding_grad(grad_y, ids, vocab, scale=2.0, dtype=dt)
    added = lrs.embedding_grad(grad_y, ids, vocab, scale=2.0, grad=start.clone(), accumulate=True)
    for c in range(0, cols, 4096):
        part = grad_y[:, c:c + 4096][inside].float()
        want = torch.zeros(vocab, part.shape[1], device="cuda").index_add_(0, ids[inside], part) * 2.0
        assert torch.equal(got[:, c:c + 4096], want.to(dt)), c
        assert torch.equal(added[:, c:c + 4096], (start[:, c:c + 4096].float() + want).to(dt)), c


def test_embedding_grad_of_more_rows_than_a_grid_fills():
    torch = torch_()
    announce("embedding grad of 2^24 rows and more")
    vocab = 16 * 2**20 + 77
    ids = torch.tensor([0, 2**24 + 3, vocab - 1, 2**24 + 3, vocab, 2**24 - 1], device="cuda")
    grad_y = torch.arange(24, device="cuda", dtype=torch.float32).view(6, 4)
    out = torch.full((vocab, 4), float("nan"), device="cuda")
    lrs.embedding_grad(grad_y, ids, vocab, grad=out)
    want = torch.zeros(vocab, 4, device="cuda")
    want[0], want[2**24 + 3], want[vocab - 1], want[2**24 - 1] = grad_y[0], grad_y[1] + grad_y[3], grad_y[2], grad_y[5]
    assert torch.equal(out, want)


def test_more_row_tiles_than_a_grid_holds():
    """Four rows of 300 columns a workgroup, more than 65,535 workgroups: every operator
    that steps over them, the gradient with its barriers too."""
    torch = torch_()
    tokens, slots, cols = 4 * 65535 + 77, 2, 300
    announce("more than 65,535 row tiles")
    g = torch.Generator("cuda").manual_seed(8)
    n = tokens * slots
    position = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(tokens, slots)
    position[::5, 1] = -1
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    used[position[position >= 0].long()] = True
    x = torch.randn(tokens, cols, generator=g, device="cuda", dtype=torch.float16)
    w = torch.rand(tokens, slots, generator=g, device="cuda")
    rows = torch.full((n, cols), 7.0, dtype=torch.float16, device="cuda")
    want = rows.clone()
    for k in range(slots):
        on = (position[:, k] >= 0).nonzero()[:, 0]
        want[position[on, k].long()] = x[on]
    lrs.dispatch_rows(x, position, out=rows)
    assert torch.equal(rows, want)
    rows = torch.randn(n, cols, generator=g, device="cuda", dtype=torch.float16)
    y64 = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    size, grad_w64 = torch.zeros_like(y64), torch.zeros(tokens, slots, dtype=torch.float64, device="cuda")
    grad_w_size = torch.zeros_like(grad_w64)
    grad_rows64 = torch.zeros(n, cols, dtype=torch.float64, device="cuda")
    for k in range(slots):
        on = (position[:, k] >= 0).nonzero()[:, 0]
        at = position[on, k].long()
        term, gy, weight = rows[at].double(), x[on].double(), w[on, k].double()[:, None]
        y64[on] += weight * term
        size[on] += (weight * term).abs()
        grad_rows64[at] = weight * gy
        grad_w64[on, k], grad_w_size[on, k] = (gy * term).sum(1), (gy * term).abs().sum(1)
    within(lrs.combine_rows(rows, position, w), y64, size, slots, "y")
    grad_rows, grad_w = lrs.combine_rows_grad(x, rows, position, w)
    within(grad_rows, grad_rows64, grad_rows64.abs(), 1, "grad_rows")
    within(grad_w, grad_w64, grad_w_size, cols, "grad_weights")
