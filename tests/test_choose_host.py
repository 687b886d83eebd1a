"""Host-only checks of the operators that choose (no GPU): temp-size queries and the
refusal of bad arguments, by the C calls before any device work and by the conveniences
before they reach the library."""
from __future__ import annotations

import pytest
import torch

import sorting_lsd_radix_sort_amd as lrs

# fake, well-aligned device addresses, far apart: these checks never dereference them
A, B, C, D, E, F, G, T = (i << 44 for i in range(1, 9))


def refuses(call, **kw):
    with pytest.raises(lrs.LrsError) as ei:
        call(**kw)
    assert ei.value.status == lrs.LRS_ERR_INVALID_ARG, kw


def route(type="bf16", logits=A, ld=64, tokens=0, experts=64, slots=8, score="softmax", bias=B, groups=8, kept=4,
          group_score="max", normalize=1, scale=1.0, id_type="i32", ids=C, wtype="f32", weights=D):
    lrs.lrs_route_tokens(type, logits, ld, tokens, experts, slots, score, bias, groups, kept, group_score, normalize,
                         scale, id_type, ids, wtype, weights, 0)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(type=-1), dict(tokens=-1), dict(tokens=2**31), dict(tokens=2**28, slots=32), dict(experts=-8),
    dict(experts=2049, groups=1, kept=1, ld=2049), dict(ld=63), dict(ld=2**60), dict(slots=-1), dict(slots=65, kept=8),
    dict(slots=33), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=65), dict(groups=7), dict(kept=0),
    dict(kept=9), dict(group_score=2), dict(id_type=2), dict(wtype=3), dict(logits=None), dict(logits=A + 1),
    dict(logits=A + 2, type="f32"), dict(bias=B + 2), dict(ids=None), dict(ids=C + 2), dict(ids=C + 4, id_type="i64"),
    dict(weights=D + 2), dict(ids=A), dict(weights=A + 64 * 2 * 99), dict(ids=B), dict(weights=B + 4), dict(weights=C),
    dict(weights=C + 4 * 799)])
def test_route_refusals(kw):
    refuses(route, **{"tokens": 100, **kw})


def route_grad(type="bf16", logits=A, ld=64, tokens=100, experts=64, slots=8, score="softmax", normalize=1, scale=1.0,
               id_type="i32", ids=C, wtype="f32", gw=D, grad=E, ld_grad=64):
    lrs.lrs_route_tokens_grad(type, logits, ld, tokens, experts, slots, score, normalize, scale, id_type, ids, wtype, gw,
                              grad, ld_grad, 0)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(tokens=-1), dict(tokens=2**31), dict(experts=-1), dict(experts=2049, ld=2049, ld_grad=2049),
    dict(ld=63), dict(ld_grad=63), dict(slots=-1), dict(slots=65), dict(score=2), dict(id_type=2), dict(wtype=3),
    dict(logits=None), dict(logits=A + 1), dict(ids=None), dict(ids=C + 2), dict(gw=None), dict(gw=D + 2),
    dict(grad=None), dict(grad=E + 1), dict(grad=A + 2), dict(grad=A, ld_grad=65), dict(grad=C), dict(grad=D),
    dict(grad=A + 128)])
def test_route_grad_refusals(kw):
    refuses(route_grad, **kw)


def select(temp=None, nbytes=0, type="bf16", logits=A, ld=1000, scores=B, finished=C, end_id=2, batch=3, beams=4,
           vocab=1000, count=8, normalize=1, out_scores=D, parents=E, id_type="i32", tokens=F):
    return lrs.lrs_beam_select(temp, nbytes, type, logits, ld, scores, finished, end_id, batch, beams, vocab, count,
                               normalize, out_scores, parents, id_type, tokens, 0)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(id_type=2), dict(ld=999), dict(ld=2**60), dict(batch=-1), dict(batch=2**30), dict(beams=-1),
    dict(beams=1025), dict(vocab=0), dict(vocab=-1), dict(vocab=2**29, ld=2**29), dict(vocab=2**31, ld=2**31),
    dict(count=-1), dict(count=65), dict(end_id=-1), dict(end_id=1000), dict(logits=None), dict(logits=A + 1),
    dict(logits=A + 2, type="f32"), dict(scores=None), dict(scores=B + 2), dict(out_scores=None),
    dict(out_scores=D + 2), dict(parents=None), dict(parents=E + 1), dict(tokens=None),
    dict(tokens=F + 4, id_type="i64"), dict(out_scores=A), dict(out_scores=B + 44), dict(parents=C + 8),
    dict(tokens=A + 2000), dict(parents=D), dict(tokens=E + 92), dict(tokens=D)])
def test_beam_select_refusals(kw):
    refuses(select, **kw)


def test_beam_select_queries():
    need = select()
    assert 0 < need < 2**20
    # the query depends on sizes and types alone
    assert select(logits=A + 2, scores=B + 4, finished=None, end_id=-1, normalize=0) == need
    assert select(id_type="i64") == need
    assert select(batch=0, logits=None, scores=None, finished=None, out_scores=None, parents=None, tokens=None) >= 0
    assert select(count=0, out_scores=None, parents=None, tokens=None) > 0
    # a share of the rows' bytes
    assert select(batch=64, beams=8, vocab=131072, ld=131072, count=16) < 64 * 8 * 131072 // 8
    for temp, nbytes in ((T, need - 256), (T + 1, need - 1)):
        with pytest.raises(lrs.LrsError) as ei:
            select(temp=temp, nbytes=nbytes)
        assert ei.value.status == lrs.LRS_ERR_TEMP_TOO_SMALL
    lib = lrs.load_library()
    assert lib.lrs_beam_select(None, None, 1, A, 1000, B, None, 0, 3, 4, 1000, 8, 1, D, E, 0, F, None) == \
        lrs.LRS_ERR_INVALID_ARG
    # calls that have nothing to do need no device
    assert select(temp=T, nbytes=2**20, batch=0) == 2**20
    assert select(temp=T, nbytes=2**20, count=0) == 2**20


STEPS = (1 << 20, 1 << 16, 1 << 12, 1 << 11, 1 << 8)  # outer, batch, beam, middle, row


def reorder(src=A, src_steps=STEPS, dst=B, dst_steps=STEPS, parents=C, outer=2, batch=3, beams=4, count=4, middle=2,
            rows=5, row_bytes=256):
    lrs.lrs_beam_reorder(src, src_steps, dst, dst_steps, parents, outer, batch, beams, count, middle, rows, row_bytes, 0)


@pytest.mark.parametrize("kw", [
    dict(src=None), dict(dst=None), dict(parents=None), dict(parents=C + 2), dict(outer=-1), dict(batch=-1),
    dict(beams=-1), dict(count=-1), dict(rows=-1), dict(middle=-1), dict(row_bytes=-1), dict(outer=2**31), dict(batch=2**31),
    dict(rows=2**20, outer=2**20), dict(middle=2**29), dict(row_bytes=2**60), dict(src_steps=(-1, 1 << 16, 1 << 12, 1 << 11, 1 << 8)),
    dict(src_steps=(2**58, 1 << 16, 1 << 12, 1 << 11, 1 << 8)), dict(dst_steps=(2**58, 1 << 16, 1 << 12, 1 << 11, 1 << 8)),
    dict(dst_steps=(1 << 20, 1 << 16, 1 << 12, 1 << 11, 255)), dict(dst_steps=(1 << 20, 1 << 16, 1 << 8, 1 << 11, 1 << 8)),
    dict(dst_steps=(1 << 20, 1 << 16, 0, 1 << 11, 1 << 8)), dict(dst=A + 8), dict(dst=A, dst_steps=(1 << 21, 1 << 16, 1 << 12, 1 << 11, 1 << 8)),
    dict(dst=C), dict(parents=B + 44), dict(dst=A, count=65, beams=65, dst_steps=(1 << 30, 1 << 20, 1 << 12, 1 << 11, 1 << 8),
                                            src_steps=(1 << 30, 1 << 20, 1 << 12, 1 << 11, 1 << 8))])
def test_beam_reorder_refusals(kw):
    refuses(reorder, **kw)


@pytest.mark.parametrize("kw", [
    # a search's old beams behind the new ones are the next search's new ones
    dict(batch=4, beams=8, count=4, src_steps=(1 << 20, 4 << 12, 1 << 12, 1 << 11, 1 << 8)),
    dict(batch=4, beams=5, count=4, src_steps=(1 << 20, 4 << 12, 1 << 12, 1 << 11, 1 << 8)),
    # both steps the same
    dict(outer=1, batch=8, beams=2, count=1, middle=1, rows=1, src_steps=(0, 256, 256, 0, 0)),
    # beams that end within the next layer
    dict(outer=2, batch=1, beams=6, count=4, src_steps=(4 << 12, 0, 1 << 12, 1 << 11, 1 << 8))])
def test_beam_reorder_in_place_refuses_states_that_share_memory(kw):
    """The new states lie apart, the old ones do not: what one search writes, another would
    read.  Into other memory such states may be reordered."""
    refuses(reorder, **{"dst": A, "dst_steps": kw["src_steps"], **kw})


def test_beam_reorder_needs_layouts_and_passes_over_nothing():
    lib = lrs.load_library()
    assert lib.lrs_beam_reorder(A, None, B, None, C, 1, 1, 1, 1, 1, 1, 16, None) == lrs.LRS_ERR_INVALID_ARG
    for kw in (dict(outer=0), dict(batch=0), dict(count=0), dict(middle=0), dict(rows=0), dict(row_bytes=0)):
        reorder(src=None, dst=None, parents=None, **kw)


def test_empty_route_calls_need_no_device():
    route(tokens=0, logits=None, ids=None, weights=None, bias=None)
    route(tokens=10, slots=0, logits=None, ids=None, weights=None)
    route_grad(tokens=0, logits=None, ids=None, gw=None, grad=None)
    route_grad(experts=0, logits=None, grad=None)


def test_route_conveniences_check_before_any_work():
    """With CPU tensors, so that no device is needed to reach the checks."""
    x = torch.zeros(4, 8)
    for kw, error, match in (
            (dict(scores="tanh"), ValueError, "scores must be 'softmax' or 'sigmoid'"),
            (dict(group_score="mean"), ValueError, "group_score must be 'max' or 'top2'"),
            (dict(num_groups=3), ValueError, "do not form 3 groups"), (dict(num_groups=0), ValueError, "0 groups"),
            (dict(num_groups=2, kept_groups=3), ValueError, "of which 3"),
            (dict(num_groups=2, kept_groups=0), ValueError, "of which 0"),
            (dict(num_groups=4, kept_groups=1), ValueError, "3 slots, with 2 experts"),
            (dict(dtype=torch.int16), TypeError, "ids must be int32 or int64"),
            (dict(weights_dtype=torch.float64), TypeError, "weights must be"),
            (dict(bias=torch.zeros(8).half()), TypeError, "bias must be float32"),
            (dict(bias=torch.zeros(7)), ValueError, "bias has shape"),
            (dict(bias=torch.zeros(1, 8)), ValueError, "bias has shape"),
            (dict(), ValueError, "device tensors")):
        with pytest.raises(error, match=match):
            lrs.route_tokens(x, 3, **kw)
    with pytest.raises(ValueError, match="9 slots"):
        lrs.route_tokens(x, 9)
    with pytest.raises(ValueError, match="-1 slots"):
        lrs.route_tokens(x, -1)
    with pytest.raises(ValueError, match="two dimensions"):
        lrs.route_tokens(x[0], 2)
    with pytest.raises(TypeError, match="logits must be"):
        lrs.route_tokens(x.double(), 2)
    ids, g = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args, kw, error, match in (
            ((g, x, ids.short()), {}, TypeError, "ids must be"), ((g.double(), x, ids), {}, TypeError, "grad_weights"),
            ((g, x, ids[:3]), {}, ValueError, "ids have shape"), ((g, x, ids[0]), {}, ValueError, "ids have shape"),
            ((g[:, :1], x, ids), {}, ValueError, "grad_weights have shape"),
            ((g, x, ids), dict(scores="x"), ValueError, "scores must be"),
            ((g, x, ids), dict(grad=x.half()), ValueError, "grad has dtype"),
            ((g, x, ids), dict(grad=torch.zeros(4, 7)), ValueError, "grad has shape"),
            ((g, x, ids), dict(grad=torch.zeros(8, 4).t()), ValueError, "contiguous"),
            ((g, x, ids), {}, ValueError, "device tensors")):
        with pytest.raises(error, match=match):
            lrs.route_tokens_grad(*args, **kw)


def test_beam_conveniences_check_before_any_work():
    l, s = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    for args, kw, error, match in (
            ((l[0], s, 4), {}, ValueError, "batch, beams, vocab"), ((l.double(), s, 4), {}, TypeError, "logits must be"),
            ((l, s.half(), 4), {}, TypeError, "scores must be float32"), ((l, s[:1], 4), {}, ValueError, "scores have shape"),
            ((l, s, 4), dict(finished=s), TypeError, "finished must be"),
            ((l, s, 4), dict(finished=s[0].bool()), ValueError, "finished has shape"),
            ((l, s, 4), dict(finished=s.bool(), end_id=10), ValueError, "end_id 10"),
            ((l, s, 4), dict(finished=s.bool(), end_id=-1), ValueError, "end_id -1"),
            ((l, s, 65), {}, ValueError, "count 65"), ((l, s, -1), {}, ValueError, "count -1"),
            ((l[:, :, :0], s, 4), {}, ValueError, "vocabulary"),
            ((l, s, 4), dict(dtype=torch.uint8), TypeError, "ids must be"), ((l, s, 4), {}, ValueError, "device tensors")):
        with pytest.raises(error, match=match):
            lrs.beam_select(*args, **kw)
    st, p = torch.zeros(2, 3, 5, 7), torch.zeros(2, 4, dtype=torch.int32)
    for args, kw, error, match in (
            ((st, p.long()), {}, TypeError, "parents must be int32"), ((st, p[0]), {}, ValueError, "parents have shape"),
            ((st, p), dict(dim=1), ValueError, "parents have shape"), ((st, p), dict(dim=3), ValueError, "no batch in"),
            ((st, p), dict(dim=-5), ValueError, "no batch in"), ((st[0, 0, 0], p), {}, ValueError, "no batch in"),
            ((st, p), dict(out=st), ValueError, "out has shape"),
            ((st, p), dict(out=torch.zeros(2, 4, 5, 7).half()), ValueError, "out has dtype"),
            ((torch.zeros(2, 3, 4, 4, 4, 4)[:, :, ::2, ::2, ::2, ::2], p), {}, ValueError, "more than three dimensions"),
            ((st, p), {}, ValueError, "device tensors")):
        with pytest.raises(error, match=match):
            lrs.beam_reorder(*args, **kw)


def test_outputs_that_torch_negates_or_conjugates_when_read_are_refused():
    """What a call writes is bytes: read through such a view they would be other values."""
    def negated(*shape):
        return torch.zeros(*shape, dtype=torch.complex64).conj().imag

    x, ids, g = torch.zeros(4, 1), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1)
    assert negated(4, 1).is_neg()
    for call in (lambda: lrs.route_tokens_grad(g, x, ids, grad=negated(4, 1)),
                 lambda: lrs.dispatch_rows(x, ids, out=negated(4, 1)),
                 lambda: lrs.combine_rows(x, ids, out=negated(4, 1)),
                 lambda: lrs.combine_rows_grad(x, x, ids, None, grad_rows=negated(4, 1)),
                 lambda: lrs.embedding(x, ids[:, 0], out=negated(4, 1)),
                 lambda: lrs.embedding_grad(x, ids[:, 0], 4, grad=negated(4, 1)),
                 lambda: lrs.sort_keys(x[:1], out=negated(1)),
                 lambda: lrs.beam_reorder(torch.zeros(2, 2, 4), ids[:2], out=negated(2, 1, 4))):
        with pytest.raises(ValueError, match="view that negates"):
            call()
    z = torch.zeros(2, 2, 4, dtype=torch.complex64)
    with pytest.raises(ValueError, match="negates or conjugates"):
        lrs.beam_reorder(z, ids[:2], out=z[:, :1].conj())
    with pytest.raises(ValueError, match="negates or conjugates"):
        lrs.beam_reorder(torch.zeros(2, 2, 4), ids[:2], out=torch._neg_view(torch.zeros(2, 1, 4)))
