"""Calls on the default stream by its handle, with another stream current."""
from __future__ import annotations

import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_default_stream_by_handle_waits_for_the_current_one():
    """Inputs written on a side stream behind long work there, the calls on handle 0:
    their results are those of the finished inputs."""
    import torch
    announce("default stream by handle")
    g = torch.Generator("cuda").manual_seed(1)
    ids = torch.randint(0, 12, (4000, 2), generator=g, device="cuda")
    x = torch.randn(4000, 520, generator=g, device="cuda")
    w = torch.rand(4000, 2, generator=g, device="cuda")
    want = lrs.group_tokens(ids, 12)
    want_rows = lrs.dispatch_rows(x, want[1])
    want_y = lrs.combine_rows(want_rows, want[1], w)
    want_grad = lrs.embedding_grad(x, ids[:, 0], 12)
    torch.cuda.synchronize()
    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    big = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for rep in range(3):
        with torch.cuda.stream(side):
            late_ids, late_x = torch.zeros_like(ids), torch.zeros_like(x)
            for _ in range(4):
                big @ big
            late_ids.copy_(ids)
            late_x.copy_(x)
            got = lrs.group_tokens(late_ids, 12, stream=0)
            side.wait_stream(default)
            rows = lrs.dispatch_rows(late_x, got[1], stream=0)
            side.wait_stream(default)
            y = lrs.combine_rows(rows, got[1], w, stream=0)
            grad = lrs.embedding_grad(late_x, late_ids[:, 0], 12, stream=0)
        default.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        assert torch.equal(rows, want_rows) and torch.equal(y, want_y) and torch.equal(grad, want_grad), rep


@pytest.mark.parametrize("as_int", [False, True])
def test_sorts_of_a_copy_made_on_the_current_stream(as_int):
    """Strided keys and values, written behind long work on the current stream and
    copied there, are sorted on a side stream."""
    import torch
    announce("sort of a copy, as int %s" % as_int)
    g = torch.Generator("cuda").manual_seed(2)
    keys = torch.randint(0, 2**31 - 1, (300001, 2), generator=g, device="cuda", dtype=torch.int32)
    values = torch.arange(600002, device="cuda", dtype=torch.int32).view(300001, 2)
    want_keys, order = torch.sort(keys[:, 1], stable=True)
    side = torch.cuda.Stream()
    big = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for rep in range(3):
        late_keys, late_values = torch.zeros_like(keys), torch.zeros_like(values)
        for _ in range(4):
            big @ big
        late_keys.copy_(keys)
        late_values.copy_(values)
        stream = side.cuda_stream if as_int else side
        alone = lrs.sort_keys(late_keys[:, 1], stream=stream)
        got_keys, got_values = lrs.sort_pairs(late_keys[:, 1], late_values.view(torch.uint32)[:, 1], stream=stream)
        side.synchronize()
        assert torch.equal(alone, want_keys) and torch.equal(got_keys, want_keys), rep
        assert torch.equal(got_values.view(torch.int32), values[:, 1][order]), rep


def test_one_row_beside_the_rows_of_its_buffer():
    """A single token's row in the columns beside those its copies go to, and the sum
    of them back to another row's."""
    import torch
    announce("one row beside others")
    wide = torch.arange(8 * 400, device="cuda", dtype=torch.float32).view(8, 400) % 97
    before = wide.clone()
    position = torch.tensor([[6, 0, 7]], dtype=torch.int32, device="cuda")
    for row in (0, 3, 7):
        wide.copy_(before)
        lrs.dispatch_rows(wide[row:row + 1, 200:], position, out=wide[:, :200])
        want = before.clone()
        want[[6, 0, 7], :200] = before[row, 200:]
        assert torch.equal(wide, want), row
        lrs.combine_rows(wide[:, :200], position, out=wide[row:row + 1, 200:])
        want[row, 200:] *= 3
        assert torch.equal(wide, want), row


def test_autograd_notices_what_the_calls_write():
    """Every tensor given to be written, here one that another gradient still needs, has
    a new version afterwards; what is only read keeps its own."""
    import torch
    announce("versions of written tensors")
    ids = torch.arange(6, device="cuda").view(3, 2) % 2
    x, w = torch.ones(3, 8, device="cuda"), torch.ones(3, 2, device="cuda")
    _, position, _ = lrs.group_tokens(ids, 2)
    rows, table = torch.ones(6, 8, device="cuda"), torch.ones(2, 8, device="cuda")
    keys, values = torch.arange(8, device="cuda", dtype=torch.int32), torch.arange(8, device="cuda").to(torch.uint32)
    read = [ids, x, w, position, rows, table, keys, values]
    versions = [t._version for t in read]
    calls = [((6, 8), lambda out: lrs.dispatch_rows(x, position, out=out)),
             ((3, 8), lambda out: lrs.combine_rows(rows, position, w, out=out)),
             ((6, 8), lambda out: lrs.combine_rows_grad(x, rows, position, w, grad_rows=out)),
             ((6, 8), lambda out: lrs.combine_rows_grad(x, out, position, w, grad_rows=out)),
             ((3, 8), lambda out: lrs.embedding(table, ids[:, 0], out=out)),
             ((3, 2, 8), lambda out: lrs.embedding(table, ids, out=out)),
             ((2, 8), lambda out: lrs.embedding_grad(x, ids[:, 0], 2, grad=out)),
             ((2, 8), lambda out: lrs.embedding_grad(x, ids[:, 0], 2, grad=out, accumulate=True)),
             ((8,), lambda out: lrs.sort_keys(torch.ones(8, device="cuda"), out=out)),
             ((8,), lambda out: lrs.sort_keys(torch.ones(8, device="cuda"), out=out, digit_bits=11)),
             ((8,), lambda out: lrs.sort_pairs(torch.ones(8, device="cuda"), values, keys_out=out))]
    for i, (shape, call) in enumerate(calls):
        leaf = torch.ones(shape, device="cuda", requires_grad=True)
        out = torch.full(shape, 2.0, device="cuda")
        y = (leaf * out).sum()
        call(out)
        assert out._version == 1, i
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    values_out = torch.empty_like(values)
    lrs.sort_pairs(keys, values, values_out=values_out)
    assert values_out._version == 1
    assert [t._version for t in read] == versions


def test_captured_conveniences_replay():
    """The conveniences captured as a program calls them, temp storage and outputs from
    the graph's own memory: replays on new inputs, with eager calls between them, give
    the eager results; two graphs of other sizes do not disturb each other."""
    import torch
    announce("captured conveniences")

    def step(s):
        order, position, offsets = lrs.group_tokens(s["ids"], 20, first_id=2)
        rows = lrs.dispatch_rows(s["x"], position, out=s["rows"])
        y = lrs.combine_rows(rows, position, s["w"])
        grad_rows, grad_w = lrs.combine_rows_grad(y, rows, position, s["w"])
        e = lrs.embedding(s["x"], s["ids"][:, 0], scale=0.5)
        grad = lrs.embedding_grad(e, s["ids"][:, 0], 24, scale=0.5, dtype=torch.float32)
        keys = lrs.sort_keys(s["ids"].view(-1))
        return order, position, offsets, rows, y, grad_rows, grad_w, e, grad, keys

    def fresh(tokens, cols, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        return {"ids": torch.randint(0, 24, (tokens, 3), generator=g, device="cuda"),
                "x": torch.randn(tokens, cols, generator=g, device="cuda", dtype=torch.bfloat16),
                "w": torch.rand(tokens, 3, generator=g, device="cuda"),
                "rows": torch.zeros(tokens * 3, cols, device="cuda", dtype=torch.bfloat16)}

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
