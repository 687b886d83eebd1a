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
