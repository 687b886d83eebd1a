"""Host-only checks of the row operators (no GPU): temp-size queries and the
refusal of bad arguments, by the C calls before any device work and by the
conveniences before they reach the library."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sorting_lsd_radix_sort_amd as lrs

# fake, well-aligned device addresses, far apart: these checks never dereference them
A, B, C, D, E, F, T = (i << 40 for i in range(1, 8))
BIG = 2**31 - 1


def group(temp=None, nbytes=0, id_type="i64", ids=A, n=1000, first=0, groups=8, order=B, position=C, offsets=D):
    return lrs.lrs_group_tokens(temp, nbytes, id_type, ids, n, first, groups, order, position, offsets, 0)


def test_group_queries_and_refusals():
    need = group()
    assert 0 < need < 2**20
    # the query depends on sizes alone
    assert group(order=None, position=None, offsets=None) == need
    assert group(id_type="i32", ids=A + 4) == need
    assert group(n=0, ids=None, order=None, position=None) > 0
    assert group(groups=0) > 0
    assert group(n=BIG, groups=131072) >= 4 * BIG
    for kw in (dict(n=-1), dict(n=2**31), dict(groups=-1), dict(groups=BIG), dict(groups=2**40), dict(id_type=2),
               dict(id_type=-1), dict(ids=None), dict(ids=A + 4), dict(ids=A + 2, id_type="i32"), dict(order=B + 1),
               dict(position=C + 2), dict(offsets=D + 3), dict(first=2**63 - 8, groups=9),
               dict(order=A), dict(position=A + 8 * 999 + 4), dict(offsets=B + 4 * 999), dict(position=B + 4)):
        with pytest.raises(lrs.LrsError) as ei:
            group(**kw)
        assert ei.value.status == lrs.LRS_ERR_INVALID_ARG, kw
    group(first=2**63 - 9, groups=8)
    group(first=-2**63, groups=8)
    need = group(n=500000)
    for temp, nbytes in ((T, need - 256), (T + 1, need - 1)):
        with pytest.raises(lrs.LrsError) as ei:
            group(temp=temp, nbytes=nbytes, n=500000)
        assert ei.value.status == lrs.LRS_ERR_TEMP_TOO_SMALL
    lib = lrs.load_library()
    assert lib.lrs_group_tokens(None, None, 0, A, 10, 0, 4, B, C, D, None) == lrs.LRS_ERR_INVALID_ARG


def dispatch(type="bf16", x=A, ld_x=64, position=C, tokens=100, slots=2, cols=64, rows=B, ld_rows=64, num_rows=200):
    lrs.lrs_dispatch_rows(type, x, ld_x, position, tokens, slots, cols, rows, ld_rows, num_rows, 0)


def combine(type="bf16", rows=A, ld_rows=64, num_rows=200, position=C, wtype="f32", weights=D, tokens=100, slots=2,
            cols=64, y=B, ld_y=64):
    lrs.lrs_combine_rows(type, rows, ld_rows, num_rows, position, wtype, weights, tokens, slots, cols, y, ld_y, 0)


def combine_grad(type="bf16", grad_y=A, ld_gy=64, rows=B, ld_rows=64, num_rows=200, position=C, wtype="f32", weights=D,
                 tokens=100, slots=2, cols=64, grad_rows=E, ld_gr=64, grad_weights=F):
    lrs.lrs_combine_rows_grad(type, grad_y, ld_gy, rows, ld_rows, num_rows, position, wtype, weights, tokens, slots,
                              cols, grad_rows, ld_gr, grad_weights, 0)


def embed(type="bf16", table=A, ld_table=64, num_ids=50, id_type="i64", ids=C, n=100, first=0, scale=1.0, cols=64, y=B,
          ld_y=64):
    lrs.lrs_embedding(type, table, ld_table, num_ids, id_type, ids, n, first, scale, cols, y, ld_y, 0)


def embed_grad(temp=None, nbytes=0, type="bf16", grad_y=A, ld_gy=64, id_type="i64", ids=C, n=100, first=0, scale=1.0,
               grad_type="bf16", grad=B, ld_grad=64, num_ids=50, cols=64, accumulate=0):
    return lrs.lrs_embedding_grad(temp, nbytes, type, grad_y, ld_gy, id_type, ids, n, first, scale, grad_type, grad,
                                  ld_grad, num_ids, cols, accumulate, 0)


COMMON = [dict(type=3), dict(type=-1), dict(cols=-1), dict(cols=2**31), dict(cols=65)]
SLOTS = [dict(tokens=-1), dict(slots=-1), dict(tokens=2**31), dict(tokens=2**16, slots=2**15), dict(position=None),
         dict(position=C + 2), dict(num_rows=-1), dict(num_rows=2**31)]


@pytest.mark.parametrize("kw", COMMON + SLOTS + [
    dict(x=None), dict(rows=None), dict(x=A + 1), dict(rows=B + 1), dict(x=A + 2, type="f32"), dict(ld_x=63),
    dict(ld_rows=63), dict(ld_rows=2**60), dict(rows=A), dict(rows=A + 2 * 64 * 99), dict(rows=A + 64),
    dict(rows=C, position=C)])
def test_dispatch_refusals(kw):
    with pytest.raises(lrs.LrsError) as ei:
        dispatch(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + SLOTS + [
    dict(rows=None), dict(y=None), dict(rows=A + 1), dict(y=B + 1), dict(ld_rows=1), dict(ld_y=63), dict(y=A),
    dict(y=D), dict(y=C), dict(wtype=3), dict(weights=D + 2), dict(weights=D + 1, wtype="f16")])
def test_combine_refusals(kw):
    with pytest.raises(lrs.LrsError) as ei:
        combine(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + SLOTS + [
    dict(grad_y=None), dict(rows=None), dict(grad_rows=None), dict(grad_y=A + 1), dict(rows=B + 1),
    dict(grad_rows=E + 1), dict(ld_gy=63), dict(ld_rows=63), dict(ld_gr=63), dict(grad_rows=A), dict(grad_rows=B + 128),
    dict(grad_rows=B, ld_gr=65), dict(grad_weights=D), dict(grad_weights=F + 2), dict(grad_weights=E),
    dict(grad_weights=B), dict(grad_weights=C), dict(wtype=-1), dict(weights=None, wtype=7), dict(weights=D + 2)])
def test_combine_grad_refusals(kw):
    with pytest.raises(lrs.LrsError) as ei:
        combine_grad(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + [
    dict(table=None), dict(y=None), dict(ids=None), dict(ids=C + 4), dict(id_type=2), dict(table=A + 1), dict(y=B + 1),
    dict(n=-1), dict(n=2**31), dict(num_ids=-1), dict(num_ids=2**31), dict(ld_table=63), dict(ld_y=63), dict(y=A),
    dict(y=A + 64), dict(y=C), dict(first=2**63 - 49)])
def test_embedding_refusals(kw):
    with pytest.raises(lrs.LrsError) as ei:
        embed(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + [
    dict(grad_y=None), dict(grad=None), dict(ids=None), dict(ids=C + 4), dict(id_type=2), dict(grad_y=A + 1),
    dict(grad=B + 1), dict(n=-1), dict(n=2**31), dict(num_ids=-1), dict(num_ids=BIG), dict(ld_gy=63), dict(ld_grad=63),
    dict(grad=A), dict(grad=C), dict(first=2**63 - 49), dict(grad_type="f16"), dict(grad_type=5),
    dict(type="f32", grad_type="bf16", grad_y=A)])
def test_embedding_grad_refusals(kw):
    with pytest.raises(lrs.LrsError) as ei:
        embed_grad(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG


def test_embedding_grad_queries():
    need = embed_grad()
    assert 0 < need < 2**24
    assert embed_grad(grad_y=A + 2, grad=B + 2) == need
    assert embed_grad(n=0, grad_y=None, ids=None) > 0
    # sorting and the sums of split runs: some words per id and a part of the rows in float32
    n, cols = 1 << 16, 4096
    assert embed_grad(n=n, num_ids=131072, cols=cols, ld_gy=cols, ld_grad=cols) < n * 64 + n * cols * 2
    with pytest.raises(lrs.LrsError) as ei:
        embed_grad(temp=T, nbytes=need - 256)
    assert ei.value.status == lrs.LRS_ERR_TEMP_TOO_SMALL
    lib = lrs.load_library()
    assert lib.lrs_embedding_grad(None, None, 1, A, 64, 1, C, 100, 0, ctypes.c_float(1), 1, B, 64, 50, 64, 0, None) == \
        lrs.LRS_ERR_INVALID_ARG


def test_empty_calls_need_no_device():
    dispatch(tokens=0, x=None, position=None)
    dispatch(slots=0, position=None)
    dispatch(cols=0, x=None, rows=None)
    dispatch(num_rows=0, rows=None)
    combine(tokens=0, position=None, weights=None, y=None)
    combine(cols=0, rows=None, y=None)
    combine_grad(tokens=0, grad_y=None, position=None, weights=None, grad_weights=None)
    combine_grad(slots=0, position=None, weights=None, grad_weights=None)
    embed(n=0, ids=None, y=None)
    embed(cols=0, table=None, y=None)
    need = embed_grad(num_ids=0, grad=None)
    assert embed_grad(temp=T, nbytes=need, num_ids=0, grad=None) == need
    need = embed_grad(cols=0, grad_y=None, ids=None, grad=None)
    assert embed_grad(temp=T, nbytes=need, cols=0, grad_y=None, ids=None, grad=None) == need
    need = embed_grad(n=0, grad_y=None, ids=None, accumulate=1)
    assert embed_grad(temp=T, nbytes=need, n=0, grad_y=None, ids=None, accumulate=1) == need


def test_interleaved_columns_are_no_overlap():
    """Two halves of one buffer's columns, row by row, share no memory, and are told
    apart from halves that meet (by the temp query, which enqueues nothing)."""
    halves = dict(grad_y=A, ld_gy=128, ld_grad=128, n=50, num_ids=50)
    assert embed_grad(grad=A + 128, **halves) > 0
    assert embed_grad(grad=A + 128 + 256 * 7, **halves) > 0
    assert embed_grad(**{**halves, "grad_y": A + 128 + 256 * 3, "grad": A}) > 0
    for grad in (A + 126, A + 130 + 256 * 7, A, A + 256):
        with pytest.raises(lrs.LrsError):
            embed_grad(grad=grad, **halves)
    with pytest.raises(lrs.LrsError):  # other strides: the halves meet somewhere
        embed_grad(grad=A + 128, **{**halves, "ld_grad": 136})


def test_conveniences_check_before_any_work():
    """With CPU tensors, so that no device is needed to reach the checks."""
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    pos, w, rows = ids.to(torch.int32), torch.zeros(4, 2), torch.zeros(8, 8)
    with pytest.raises(TypeError, match="int32 or int64"):
        lrs.group_tokens(ids.to(torch.int16), 4)
    with pytest.raises(TypeError, match="position must be int32"):
        lrs.dispatch_rows(x, ids)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        lrs.dispatch_rows(x.double(), pos)
    with pytest.raises(ValueError, match="two dimensions"):
        lrs.dispatch_rows(x[0], pos)
    with pytest.raises(ValueError, match="tokens, slots"):
        lrs.dispatch_rows(x, pos.reshape(-1))
    with pytest.raises(ValueError, match="position is for 3 tokens"):
        lrs.dispatch_rows(x, pos[:3])
    with pytest.raises(ValueError, match="out has shape"):
        lrs.dispatch_rows(x, pos, out=torch.zeros(8, 7))
    with pytest.raises(ValueError, match="out has shape"):
        lrs.dispatch_rows(x, pos, num_rows=9, out=rows)
    with pytest.raises(ValueError, match="out has dtype"):
        lrs.dispatch_rows(x, pos, out=rows.half())
    with pytest.raises(ValueError, match="contiguous"):
        lrs.dispatch_rows(x, pos, out=torch.zeros(8, 8).t())
    with pytest.raises(ValueError, match="weights have shape"):
        lrs.combine_rows(rows, pos, w[:, :1])
    with pytest.raises(TypeError, match="weights must be"):
        lrs.combine_rows(rows, pos, w.double())
    with pytest.raises(ValueError, match="out has shape"):
        lrs.combine_rows(rows, pos, w, out=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="grad_y is"):
        lrs.combine_rows_grad(torch.zeros(4, 7), rows, pos, w)
    with pytest.raises(ValueError, match="grad_y is"):
        lrs.combine_rows_grad(x.half(), rows, pos, w)
    with pytest.raises(ValueError, match="grad_rows has shape"):
        lrs.combine_rows_grad(x, rows, pos, w, grad_rows=torch.zeros(7, 8))
    with pytest.raises(ValueError, match="out has shape"):
        lrs.embedding(x, ids, out=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="contiguous"):
        lrs.embedding(x, ids, out=torch.zeros(2, 4, 8).transpose(0, 1))
    with pytest.raises(ValueError, match="grad_y has shape"):
        lrs.embedding_grad(x, ids, 4)
    with pytest.raises(TypeError, match="gradient must be"):
        lrs.embedding_grad(x.half(), ids[:, 0], 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="grad has shape"):
        lrs.embedding_grad(x, ids[:, 0], 4, grad=torch.zeros(5, 8))
    with pytest.raises(ValueError, match="accumulate needs"):
        lrs.embedding_grad(x, ids[:, 0], 4, accumulate=True)
    # well-formed CPU tensors are refused for their device, by each
    for call in (lambda: lrs.group_tokens(ids, 4), lambda: lrs.dispatch_rows(x, pos),
                 lambda: lrs.combine_rows(rows, pos, w), lambda: lrs.combine_rows_grad(x, rows, pos, w),
                 lambda: lrs.embedding(x, ids), lambda: lrs.embedding_grad(x, ids[:, 0], 4)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
