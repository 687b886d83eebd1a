"""The best few of a row, and what moves by the choice: a router's experts, beam search.

The ``lrs_*`` functions call the C functions of the same name
(``include/lrsort_choose.h``) with the same arguments, as the package's other
bindings do.  ``route_tokens`` and ``route_tokens_grad`` (whose ids and weights
``group_tokens`` and ``combine_rows`` take), ``beam_select`` and ``beam_reorder`` are
conveniences over them on torch tensors, in the manner of those of ``rows.py``: they
allocate outputs and temp storage, refuse tensors of the wrong shape, type or device
with ValueError or TypeError before any work, record nothing for torch's autograd but
count a tensor given as output as changed, and order a call on another stream behind
what the current one holds.
"""
from __future__ import annotations

import ctypes

from . import _as_stored, _check, _ptr, _stream, load_library
from . import rows as _r
from .rows import ID_TYPE_CODES, ROW_TYPE_CODES, _CI, _F, _I64, _SZ, _VP, _code

SCORE_CODES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE_CODES = {"max": 0, "top2": 1}


class BeamLayout(ctypes.Structure):
    """lrs_beam_layout: byte steps of a state's dimensions."""
    _fields_ = [("outer_step", _I64), ("batch_step", _I64), ("beam_step", _I64), ("middle_step", _I64),
                ("row_step", _I64)]


_PL = ctypes.POINTER(BeamLayout)
ARGTYPES = {
    "lrs_route_tokens": [_CI, _VP, _I64, _I64, _I64, _I64, _CI, _VP, _I64, _I64, _CI, _CI, _F, _CI, _VP, _CI, _VP, _VP],
    "lrs_route_tokens_grad": [_CI, _VP, _I64, _I64, _I64, _I64, _CI, _CI, _F, _CI, _VP, _CI, _VP, _VP, _I64, _VP],
    "lrs_beam_select": [_VP, _SZ, _CI, _VP, _I64, _VP, _VP, _I64, _I64, _I64, _I64, _I64, _CI, _VP, _VP, _CI, _VP, _VP],
    "lrs_beam_reorder": [_VP, _PL, _VP, _PL, _VP, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _VP],
}
CHOOSE_FUNCTIONS = tuple(ARGTYPES)


def declare(lib: ctypes.CDLL) -> None:
    """Sets the argument types of these functions on the loaded library."""
    for name, argtypes in ARGTYPES.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int


# ------------------------------------------------------------------ C calls


def lrs_route_tokens(row_type, d_logits, ld_logits, tokens, experts, slots, score, d_bias, num_groups, kept_groups,
                     group_score, normalize, scale, id_type, d_ids, weight_type, d_weights, stream=None) -> None:
    """Calls the C function of the same name.  score is an lrs_score_type code or
    "softmax" / "sigmoid", group_score an lrs_group_score code or "max" / "top2"."""
    _check(load_library().lrs_route_tokens(_code(ROW_TYPE_CODES, row_type), _ptr(d_logits), int(ld_logits), int(tokens),
                                           int(experts), int(slots), _code(SCORE_CODES, score), _ptr(d_bias),
                                           int(num_groups), int(kept_groups), _code(GROUP_SCORE_CODES, group_score),
                                           int(bool(normalize)), float(scale), _code(ID_TYPE_CODES, id_type),
                                           _ptr(d_ids), _code(ROW_TYPE_CODES, weight_type), _ptr(d_weights),
                                           _stream(stream)), "lrs_route_tokens")


def lrs_route_tokens_grad(row_type, d_logits, ld_logits, tokens, experts, slots, score, normalize, scale, id_type, d_ids,
                          weight_type, d_grad_weights, d_grad_logits, ld_grad_logits, stream=None) -> None:
    """Calls the C function of the same name."""
    _check(load_library().lrs_route_tokens_grad(_code(ROW_TYPE_CODES, row_type), _ptr(d_logits), int(ld_logits),
                                                int(tokens), int(experts), int(slots), _code(SCORE_CODES, score),
                                                int(bool(normalize)), float(scale), _code(ID_TYPE_CODES, id_type),
                                                _ptr(d_ids), _code(ROW_TYPE_CODES, weight_type), _ptr(d_grad_weights),
                                                _ptr(d_grad_logits), int(ld_grad_logits), _stream(stream)),
           "lrs_route_tokens_grad")


def lrs_beam_select(d_temp, temp_bytes, row_type, d_logits, ld_logits, d_scores, d_finished, end_id, batch, beams, vocab,
                    count, normalize, d_out_scores, d_parents, id_type, d_tokens, stream=None):
    """Calls the C function of the same name.  With d_temp None returns the temp bytes
    needed."""
    tb = ctypes.c_size_t(int(temp_bytes or 0))
    temp = _ptr(d_temp)
    st = None if temp is None else _stream(stream)
    _check(load_library().lrs_beam_select(temp, ctypes.byref(tb), _code(ROW_TYPE_CODES, row_type), _ptr(d_logits),
                                          int(ld_logits), _ptr(d_scores), _ptr(d_finished), int(end_id), int(batch),
                                          int(beams), int(vocab), int(count), int(bool(normalize)), _ptr(d_out_scores),
                                          _ptr(d_parents), _code(ID_TYPE_CODES, id_type), _ptr(d_tokens), st),
           "lrs_beam_select")
    return tb.value


def lrs_beam_reorder(d_in, in_layout, d_out, out_layout, d_parents, outer, batch, beams, count, middle, rows,
                     row_bytes, stream=None) -> None:
    """Calls the C function of the same name.  A layout is the five byte steps (outer,
    batch, beam, middle, row)."""
    _check(load_library().lrs_beam_reorder(_ptr(d_in), BeamLayout(*(int(v) for v in in_layout)), _ptr(d_out),
                                           BeamLayout(*(int(v) for v in out_layout)), _ptr(d_parents), int(outer),
                                           int(batch), int(beams), int(count), int(middle), int(rows),
                                           int(row_bytes), _stream(stream)), "lrs_beam_reorder")


# ------------------------------------------------------------- conveniences


def _name(what, codes, name) -> int:
    code = codes.get(name)
    if code is None:
        raise ValueError("%s must be %s, not %r" % (what, " or ".join(map(repr, codes)), name))
    return code


def _same_device(name, t, like):
    if t.get_device() != like.get_device():
        raise _r._elsewhere(name, t, like)


def _id_dtype(dtype):
    """(torch dtype, code) of ids to return; None is int32."""
    codes, _, int32 = _r._types or _r._type_codes()
    dtype = int32 if dtype is None else dtype
    if dtype not in codes:
        raise TypeError("ids must be int32 or int64, not %s" % dtype)
    return dtype, codes[dtype]


def route_tokens(logits, slots: int, scores: str = "softmax", bias=None, num_groups: int = 1,
                 kept_groups: int | None = None, group_score: str = "max", normalize: bool = True, scale: float = 1.0,
                 dtype=None, weights_dtype=None, stream=None):
    """The `slots` best experts of each token by its logits (tokens, experts), and their
    weights: (ids, weights), both (tokens, slots), the best first and of equal ones the
    lowest id.  scores: "softmax" over a token's experts or "sigmoid" of each.  bias
    (experts,), float32, is added to the scores for the choice only.  Of num_groups equal
    groups of consecutive experts only the kept_groups best (all by default) are chosen
    from, a group's score being that of its best expert ("max") or the sum of its two
    best ("top2").  normalize: a token's weights are divided by their sum; all are
    multiplied by `scale`.  A logit of -inf takes no part; where nothing is left to
    choose the id is -1 and the weight 0, which group_tokens passes over.  dtype of the
    ids: int32 (default) or int64; weights_dtype: float32 (default), bfloat16 or float16.
    At most 64 slots, 64 groups and 2048 experts."""
    code = _r._row_code("logits", logits.dtype)
    score, group = _name("scores", SCORE_CODES, scores), _name("group_score", GROUP_SCORE_CODES, group_score)
    tokens, experts = _r._matrix("logits", logits)
    dtype, id_code = _id_dtype(dtype)
    float32 = _r._torch.float32
    if weights_dtype is None:
        weights_dtype = float32
    weight_code = _r._row_code("weights", weights_dtype)
    slots, num_groups = int(slots), int(num_groups)
    kept_groups = num_groups if kept_groups is None else int(kept_groups)
    if num_groups < 1 or experts % num_groups or not 1 <= kept_groups <= num_groups:
        raise ValueError("%d experts do not form %d groups of which %d are kept" % (experts, num_groups, kept_groups))
    if not 0 <= slots <= kept_groups * (experts // num_groups):
        raise ValueError("%d slots, with %d experts to choose from" % (slots, kept_groups * (experts // num_groups)))
    if bias is not None:
        if bias.dtype is not float32:
            raise TypeError("bias must be float32, not %s" % bias.dtype)
        if bias.dim() != 1 or bias.shape[0] != experts:
            raise ValueError("bias has shape %s, expected (%d,)" % (tuple(bias.shape), experts))
        _same_device("bias", bias, logits)
    if not logits.is_cuda:
        raise _r._host_tensor(logits)
    logits, ld = _r._rows_in(logits, tokens, experts)
    if bias is not None:
        bias = _as_stored(bias).contiguous()
    ids = logits.new_empty(tokens, slots, dtype=dtype)
    weights = logits.new_empty(tokens, slots, dtype=weights_dtype)
    _r._run("lrs_route_tokens", stream, (logits, bias, ids, weights),
            (code, logits.data_ptr(), ld, tokens, experts, slots, score, _r._at(bias), num_groups, kept_groups, group,
             1 if normalize else 0, float(scale), id_code, ids.data_ptr(), weight_code, weights.data_ptr()))
    return ids, weights


def route_tokens_grad(grad_weights, logits, ids, scores: str = "softmax", normalize: bool = True, scale: float = 1.0,
                      grad=None, stream=None):
    """The gradient of route_tokens' weights with respect to the logits, given that of
    the weights (tokens, slots; float32, bfloat16 or float16) and the ids it returned
    (int32 or int64), with the same scores, normalize and scale.  Returns a matrix of the
    shape and type of logits, every element written: `grad` if given (which may be
    `logits` itself).  The bias and the groups have no gradient.  Ids outside the experts
    take no part."""
    code = _r._row_code("logits", logits.dtype)
    score = _name("scores", SCORE_CODES, scores)
    tokens, experts = _r._matrix("logits", logits)
    id_code, weight_code = _r._id_code(ids), _r._row_code("grad_weights", grad_weights.dtype)
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids have shape %s, expected (%d, slots)" % (tuple(ids.shape), tokens))
    if grad_weights.shape != ids.shape:
        raise ValueError("grad_weights have shape %s, ids %s" % (tuple(grad_weights.shape), tuple(ids.shape)))
    _same_device("ids", ids, logits)
    _same_device("grad_weights", grad_weights, logits)
    ld_grad = experts if grad is None else _r._rows_out("grad", grad, tokens, experts, logits)[1]
    if not logits.is_cuda:
        raise _r._host_tensor(logits)
    given = grad
    if grad is None:
        grad = logits.new_empty(tokens, experts)
    logits, ld = _r._rows_in(logits, tokens, experts)
    ids, grad_weights = ids.contiguous(), _as_stored(grad_weights).contiguous()
    _r._run("lrs_route_tokens_grad", stream, (logits, ids, grad_weights, grad),
            (code, logits.data_ptr(), ld, tokens, experts, ids.shape[1], score, 1 if normalize else 0, float(scale),
             id_code, ids.data_ptr(), weight_code, grad_weights.data_ptr(), grad.data_ptr(), ld_grad), given)
    return grad


def beam_select(logits, scores, count: int, normalize: bool = True, finished=None, end_id: int = 0, dtype=None,
                temp=None, stream=None):
    """The `count` best continuations of each search: of all totals scores[b, i] +
    log_softmax(logits[b, i])[v] (normalize False: + logits[b, i, v]) the largest, equal
    ones by the lowest i, then the largest logit, then the lowest v.  logits (batch, beams,
    vocab); scores (batch, beams), float32.  Returns (new scores, parents, tokens), each
    (batch, count): float32, the beam i as int32, the token v as `dtype` (int32 by default,
    or int64).  A beam of score -inf takes no part.  finished (batch, beams), bool or uint8:
    such a beam offers only the token end_id, at its own score.  Where nothing is left the
    score is -inf, parent and token -1.  At most 64 continuations of at most 1024 beams."""
    code = _r._row_code("logits", logits.dtype)
    if logits.dim() != 3:
        raise ValueError("logits must have the shape (batch, beams, vocab), not %s" % (tuple(logits.shape),))
    batch, beams, vocab = logits.shape
    dtype, id_code = _id_dtype(dtype)
    torch, count = _r._torch, int(count)
    if scores.dtype is not torch.float32:
        raise TypeError("scores must be float32, not %s" % scores.dtype)
    if scores.shape != (batch, beams):
        raise ValueError("scores have shape %s, expected %s" % (tuple(scores.shape), (batch, beams)))
    _same_device("scores", scores, logits)
    if finished is not None:
        if finished.dtype is not torch.bool and finished.dtype is not torch.uint8:
            raise TypeError("finished must be bool or uint8, not %s" % finished.dtype)
        if finished.shape != (batch, beams):
            raise ValueError("finished has shape %s, expected %s" % (tuple(finished.shape), (batch, beams)))
        _same_device("finished", finished, logits)
        if not 0 <= end_id < vocab:
            raise ValueError("end_id %d is no token of %d" % (end_id, vocab))
    if vocab < 1 or not 0 <= count <= 64:
        raise ValueError("count %d of a vocabulary of %d: count must be 0 to 64, the vocabulary not empty" %
                         (count, vocab))
    if not logits.is_cuda:
        raise _r._host_tensor(logits)
    logits = _as_stored(logits)
    # one row per beam, equally far apart
    to_batch, step, to_token = logits.stride()
    if beams == 1:
        step = to_batch
    rows = batch * beams
    if rows > 1 and ((batch > 1 and to_batch != beams * step) or step < vocab) or (rows and vocab > 1 and to_token != 1):
        logits, step = logits.contiguous(), vocab
    scores = _as_stored(scores).contiguous()
    if finished is not None:
        finished = finished.contiguous()
    new_scores = scores.new_empty(batch, count)
    parents = scores.new_empty(batch, count, dtype=torch.int32)
    tokens = parents.new_empty(batch, count) if id_code == 0 else scores.new_empty(batch, count, dtype=dtype)
    args = (code, logits.data_ptr(), step, scores.data_ptr(), _r._at(finished), int(end_id), batch, beams, vocab, count,
            1 if normalize else 0, new_scores.data_ptr(), parents.data_ptr(), id_code, tokens.data_ptr())
    t, size = _r._temp("lrs_beam_select", (code, batch, beams, vocab, count), args, new_scores, temp)
    _r._run("lrs_beam_select", stream, (new_scores, logits, scores, finished, t, parents, tokens),
            (t.data_ptr(), ctypes.byref(ctypes.c_size_t(size))) + args)
    return new_scores, parents, tokens


def _beam_dims(name, shape, strides, at, size):
    """Bytes of a contiguous piece of a state, and its other dimensions beside batch and
    beams, [(size, byte steps)] with the largest steps first: those that follow one another
    in all `strides` given are joined."""
    order = [d for d in range(len(shape)) if d not in (at, at + 1) and shape[d] != 1]
    order.sort(key=lambda d: strides[0][d])
    row, dims = size, []
    for d in order:
        steps = tuple(s[d] * size for s in strides)
        if not dims and all(step == row for step in steps):
            row *= shape[d]
        elif dims and all(step == dims[-1][0] * inner for step, inner in zip(steps, dims[-1][1])):
            dims[-1] = (dims[-1][0] * shape[d], dims[-1][1])
        else:
            dims.append((shape[d], steps))
    if len(dims) > 3:
        raise ValueError("%s of shape %s has more than three dimensions that neither follow one another nor are "
                         "contiguous" % (name, tuple(shape)))
    return row, dims[::-1]


_plans: dict = {}  # how states of a shape and strides are reordered, which alone decide it


def _beam_plan(shape, strides, dim, size, parents_shape, out_shape, out_strides):
    """(shape of the new states, sizes for the C call, its layouts)."""
    nd, at = len(shape), int(dim)
    at = at + nd if at < 0 else at
    if not 0 <= at < nd - 1:
        raise ValueError("states of shape %s have no batch in dimension %d with the beams behind it" %
                         (tuple(shape), dim))
    batch, beams = shape[at], shape[at + 1]
    if len(parents_shape) != 2 or parents_shape[0] != batch:
        raise ValueError("parents have shape %s, expected (%d, count)" % (tuple(parents_shape), batch))
    count = parents_shape[1]
    new_shape = (*shape[:at + 1], count, *shape[at + 2:])
    if out_shape is not None and tuple(out_shape) != new_shape:
        raise ValueError("out has shape %s, expected %s" % (tuple(out_shape), new_shape))
    if out_strides is None:
        out_strides, step = [0] * nd, 1
        for d in range(nd - 1, -1, -1):
            out_strides[d], step = step, step * max(new_shape[d], 1)
    row, dims = (0, []) if 0 in new_shape else _beam_dims("states", new_shape, (strides, out_strides), at, size)
    (outer, outer_steps), (middle, middle_steps), (n, row_steps) = [(1, (0, 0))] * (3 - len(dims)) + dims
    layouts = [BeamLayout(outer_steps[i], s[at] * size, s[at + 1] * size, middle_steps[i], row_steps[i])
               for i, s in enumerate((strides, out_strides))]
    return new_shape, (outer, batch, beams, count, middle, n, row), layouts[0], layouts[1]


def beam_reorder(states, parents, dim: int = 0, out=None, stream=None):
    """The beams' states after a step: out[..., b, j, ...] = states[..., b, parents[b, j],
    ...], zeros where a parent is outside the beams.  states: any type of 1, 2, 4, 8 or 16
    bytes, with the batch in dimension `dim` and the beams in the next; parents (batch,
    count), int32, as beam_select returns them.  Returns `out`, a tensor of that shape
    (`states` itself for the reordering in place, of at most 64 beams whose memory lies
    apart, which moves only what has another parent), or a new one.  Strides may be any
    that leave at most three dimensions beside batch, beams and a contiguous piece: the
    filled part of a cache that has room for more will do, with layers in front and heads
    before or behind the positions.  Of views that torch conjugates or negates when they
    are read the values are moved, by bytes where out is such a view too; out alone may
    not be one."""
    if parents.dtype is not (_r._types or _r._type_codes())[2]:
        raise TypeError("parents must be int32, not %s" % parents.dtype)
    key = (states.shape, states.stride(), dim, states.dtype, parents.shape,
           out is not None and (out.shape, out.stride()))
    plan = _plans.get(key)
    if plan is None:
        plan = states.is_complex(), *_beam_plan(states.shape, states.stride(), dim, states.element_size(),
                                                parents.shape,
                                                *((None, None) if out is None else (out.shape, out.stride())))
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = plan
    is_complex, shape, sizes, from_layout, to_layout = plan
    index, given = states.get_device(), out
    if parents.get_device() != index:
        raise _r._elsewhere("parents", parents, states)
    if out is not None:
        if out.dtype is not states.dtype:
            raise ValueError("out has dtype %s, expected %s" % (out.dtype, states.dtype))
        if out.get_device() != index:
            raise _r._elsewhere("out", out, states)
    if is_complex or states.is_neg() or (out is not None and out.is_neg()):
        # bytes are moved: what torch conjugates or negates when it is read has to be so on
        # both sides, or on neither
        lazy = states.is_conj(), states.is_neg()
        if lazy != ((False, False) if out is None else (out.is_conj(), out.is_neg())):
            if out is not None and (out.is_conj() or out.is_neg()):
                raise ValueError("out is a view that negates or conjugates what its memory holds")
            return beam_reorder(states.resolve_conj().resolve_neg(), parents, dim, out, stream)
    if not states.is_cuda:
        raise _r._host_tensor(states)
    if out is None:
        out = states.new_empty(shape)
    parents = parents.contiguous()
    _r._run("lrs_beam_reorder", stream, (states, out, parents),
            (states.data_ptr(), from_layout, out.data_ptr(), to_layout, parents.data_ptr(), *sizes), given)
    return out
