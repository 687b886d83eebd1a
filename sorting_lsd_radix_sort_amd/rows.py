"""Rows of a matrix moved and summed in the order of small integer keys.

The ``lrs_*`` functions call the C functions of the same name
(``include/lrsort_rows.h``) with the same arguments, as the package's other
bindings do.  ``group_tokens``, ``dispatch_rows``, ``combine_rows`` and
``combine_rows_grad`` (tokens sorted by expert and back), ``embedding`` and
``embedding_grad`` are conveniences over them on torch tensors: they allocate
outputs and temp storage, and refuse tensors of the wrong shape, type or device
with ValueError or TypeError before any work.

Matrices may have any row stride; their elements must be contiguous within a row
(inputs that are not are copied first, outputs are refused).  ``stream`` is as for
``sort_keys``: None is the current stream of the tensors' device; on any other
stream the work also waits for what the current one already holds, so that inputs
just written there can be passed.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import _check, _ptr, _stream, _temp_tensor, load_library

ID_TYPE_CODES = {"i32": 0, "i64": 1}
ROW_TYPE_CODES = {"f32": 0, "bf16": 1, "f16": 2}
_ID_SUFFIX = {"torch.int32": "i32", "torch.int64": "i64"}
_ROW_SUFFIX = {"torch.float32": "f32", "torch.bfloat16": "bf16", "torch.float16": "f16"}

_VP, _SZ, _I64, _CI, _F = (ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t), ctypes.c_int64, ctypes.c_int,
                           ctypes.c_float)
ARGTYPES = {
    "lrs_group_tokens": [_VP, _SZ, _CI, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _VP],
    "lrs_dispatch_rows": [_CI, _VP, _I64, _VP, _I64, _I64, _I64, _VP, _I64, _I64, _VP],
    "lrs_combine_rows": [_CI, _VP, _I64, _I64, _VP, _CI, _VP, _I64, _I64, _I64, _VP, _I64, _VP],
    "lrs_combine_rows_grad": [_CI, _VP, _I64, _VP, _I64, _I64, _VP, _CI, _VP, _I64, _I64, _I64, _VP, _I64, _VP, _VP],
    "lrs_embedding": [_CI, _VP, _I64, _I64, _CI, _VP, _I64, _I64, _F, _I64, _VP, _I64, _VP],
    "lrs_embedding_grad": [_VP, _SZ, _CI, _VP, _I64, _CI, _VP, _I64, _I64, _F, _CI, _VP, _I64, _I64, _I64, _CI, _VP],
}
ROW_FUNCTIONS = tuple(ARGTYPES)


def declare(lib: ctypes.CDLL) -> None:
    """Sets the argument types of the row functions on the loaded library."""
    for name, argtypes in ARGTYPES.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int


def _code(codes, t) -> int:
    return codes[t] if isinstance(t, str) else int(t)


# ------------------------------------------------------------------ C calls


def lrs_group_tokens(d_temp, temp_bytes, id_type, d_ids, n, first_id, num_groups, d_order, d_position, d_offsets,
                     stream=None):
    """Calls the C function of the same name.  id_type is an lrs_id_type code or
    "i32" / "i64".  With d_temp None returns the temp bytes needed."""
    tb = ctypes.c_size_t(int(temp_bytes or 0))
    temp = _ptr(d_temp)
    st = None if temp is None else _stream(stream)
    _check(load_library().lrs_group_tokens(temp, ctypes.byref(tb), _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n),
                                           int(first_id), int(num_groups), _ptr(d_order), _ptr(d_position),
                                           _ptr(d_offsets), st), "lrs_group_tokens")
    return tb.value


def lrs_dispatch_rows(row_type, d_x, ld_x, d_position, tokens, slots, cols, d_rows, ld_rows, num_rows,
                      stream=None) -> None:
    """Calls the C function of the same name.  row_type is an lrs_row_type code or
    "f32" / "bf16" / "f16"."""
    _check(load_library().lrs_dispatch_rows(_code(ROW_TYPE_CODES, row_type), _ptr(d_x), int(ld_x), _ptr(d_position),
                                            int(tokens), int(slots), int(cols), _ptr(d_rows), int(ld_rows),
                                            int(num_rows), _stream(stream)), "lrs_dispatch_rows")


def lrs_combine_rows(row_type, d_rows, ld_rows, num_rows, d_position, weight_type, d_weights, tokens, slots, cols, d_y,
                     ld_y, stream=None) -> None:
    """Calls the C function of the same name (d_weights None: ones)."""
    _check(load_library().lrs_combine_rows(_code(ROW_TYPE_CODES, row_type), _ptr(d_rows), int(ld_rows), int(num_rows),
                                           _ptr(d_position), _code(ROW_TYPE_CODES, weight_type), _ptr(d_weights),
                                           int(tokens), int(slots), int(cols), _ptr(d_y), int(ld_y), _stream(stream)),
           "lrs_combine_rows")


def lrs_combine_rows_grad(row_type, d_grad_y, ld_grad_y, d_rows, ld_rows, num_rows, d_position, weight_type, d_weights,
                          tokens, slots, cols, d_grad_rows, ld_grad_rows, d_grad_weights, stream=None) -> None:
    """Calls the C function of the same name."""
    _check(load_library().lrs_combine_rows_grad(_code(ROW_TYPE_CODES, row_type), _ptr(d_grad_y), int(ld_grad_y),
                                                _ptr(d_rows), int(ld_rows), int(num_rows), _ptr(d_position),
                                                _code(ROW_TYPE_CODES, weight_type), _ptr(d_weights), int(tokens),
                                                int(slots), int(cols), _ptr(d_grad_rows), int(ld_grad_rows),
                                                _ptr(d_grad_weights), _stream(stream)), "lrs_combine_rows_grad")


def lrs_embedding(row_type, d_table, ld_table, num_ids, id_type, d_ids, n, first_id, scale, cols, d_y, ld_y,
                  stream=None) -> None:
    """Calls the C function of the same name."""
    _check(load_library().lrs_embedding(_code(ROW_TYPE_CODES, row_type), _ptr(d_table), int(ld_table), int(num_ids),
                                        _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n), int(first_id), float(scale),
                                        int(cols), _ptr(d_y), int(ld_y), _stream(stream)), "lrs_embedding")


def lrs_embedding_grad(d_temp, temp_bytes, row_type, d_grad_y, ld_grad_y, id_type, d_ids, n, first_id, scale, grad_type,
                       d_grad, ld_grad, num_ids, cols, accumulate, stream=None):
    """Calls the C function of the same name.  With d_temp None returns the temp
    bytes needed."""
    tb = ctypes.c_size_t(int(temp_bytes or 0))
    temp = _ptr(d_temp)
    st = None if temp is None else _stream(stream)
    _check(load_library().lrs_embedding_grad(temp, ctypes.byref(tb), _code(ROW_TYPE_CODES, row_type), _ptr(d_grad_y),
                                             int(ld_grad_y), _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n),
                                             int(first_id), float(scale), _code(ROW_TYPE_CODES, grad_type), _ptr(d_grad),
                                             int(ld_grad), int(num_ids), int(cols), int(bool(accumulate)), st),
           "lrs_embedding_grad")
    return tb.value


# ------------------------------------------------------------- conveniences


def _id_suffix(t) -> str:
    try:
        return _ID_SUFFIX[str(t.dtype)]
    except KeyError:
        raise TypeError("ids must be int32 or int64, not %s" % t.dtype) from None


def _row_suffix(name, dtype) -> str:
    try:
        return _ROW_SUFFIX[str(dtype)]
    except KeyError:
        raise TypeError("%s must be float32, bfloat16 or float16, not %s" % (name, dtype)) from None


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _rows_in(t):
    """A matrix argument as the library reads it: elements of a row next to each
    other (a copy where they are not), any stride between rows."""
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        return t.contiguous()
    return t


def _ld(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, t.dim()))
    return t


def _out_matrix(name, t, rows, cols, dtype, device):
    """An output matrix: that shape (rows None: any number), type and device, each
    row contiguous and no two overlapping."""
    _matrix(name, t)
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape[1] != cols or (rows is not None and t.shape[0] != rows):
        raise ValueError("%s has shape %s, expected (%s, %d)" % (name, tuple(t.shape), "any" if rows is None else rows,
                                                                 cols))
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("%s must be contiguous within each row" % name)
    _same_device(device, **{name: t})
    return t


def _position(position, device):
    if str(position.dtype) != "torch.int32":
        raise TypeError("position must be int32, not %s" % position.dtype)
    if position.dim() != 2:
        raise ValueError("position must have the shape (tokens, slots), not %s" % (tuple(position.shape),))
    _same_device(device, position=position)
    return position.contiguous()


def _weights(weights, position):
    if weights is None:
        return None, 0
    if weights.shape != position.shape:
        raise ValueError("weights have shape %s, position %s" % (tuple(weights.shape), tuple(position.shape)))
    _same_device(position.device, weights=weights)
    return weights.contiguous(), ROW_TYPE_CODES[_row_suffix("weights", weights.dtype)]


class _On:
    """Where a call runs: its device made current, and the stream's handle.  On
    another stream than the current one, the work waits for what the current one
    holds (inputs copied and outputs allocated there), and `keep` records tensors
    on it, so that the caching allocator does not hand their memory on while it is
    in use there."""

    def __init__(self, device, stream):
        import torch
        if device.type != "cuda":
            raise ValueError("lrsort needs device tensors, got a tensor on %s" % device)
        self.guard = contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        current = torch.cuda.current_stream(device)
        self.side = None
        self.handle = current.cuda_stream
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            if handle != self.handle:
                self.side = torch.cuda.ExternalStream(handle, device) if isinstance(stream, int) else stream
                if self.side.device != device:
                    raise ValueError("stream is on %s, the tensors on %s" % (self.side.device, device))
                self.handle = handle
        self.current = current

    def __enter__(self):
        self.guard.__enter__()
        if self.side is not None:
            self.side.wait_stream(self.current)
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)

    def keep(self, *tensors):
        if self.side is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.side)


def group_tokens(ids, num_groups: int, first_id: int = 0, temp=None, stream=None):
    """Stable grouping of ids (int32 or int64, any shape) into groups
    first_id..first_id + num_groups - 1.  Returns (order, position, offsets), int32:
    order, the flat indices sorted by group, those of no group last; position, of
    the shape of ids, where each stands in that order, or -1; offsets
    (num_groups + 1), where each group begins and the last ends."""
    import torch
    code = ID_TYPE_CODES[_id_suffix(ids)]
    _same_device(ids.device, temp=temp)
    on = _On(ids.device, stream)
    shape = ids.shape
    ids = ids.contiguous()
    n = ids.numel()
    order = torch.empty(n, dtype=torch.int32, device=ids.device)
    position = torch.empty(shape, dtype=torch.int32, device=ids.device)
    offsets = torch.empty(max(int(num_groups), 0) + 1, dtype=torch.int32, device=ids.device)
    need = lrs_group_tokens(None, 0, code, ids, n, first_id, num_groups, order, position, offsets)
    t = _temp_tensor(need, ids.device, temp)
    with on:
        lrs_group_tokens(t, t.numel() * t.element_size(), code, ids, n, first_id, num_groups, order, position, offsets,
                         on.handle)
    on.keep(ids, t, order, position, offsets)
    return order, position, offsets


def dispatch_rows(x, position, num_rows: int | None = None, out=None, stream=None):
    """rows[position[t, k]] = x[t]: each token's row copied to its places
    (`position` from group_tokens on ids of shape (tokens, slots)).  Returns the
    rows: `out`, or a new matrix of num_rows rows (tokens * slots by default).  Rows
    that no position names are left as they were: unset in a new matrix.
    The gradient with respect to x is combine_rows(grad_rows, position)."""
    import torch
    sfx = _row_suffix("x", _matrix("x", x).dtype)
    pos = _position(position, x.device)
    if pos.shape[0] != x.shape[0]:
        raise ValueError("position is for %d tokens, x has %d" % (pos.shape[0], x.shape[0]))
    if out is not None:
        _out_matrix("out", out, num_rows, x.shape[1], x.dtype, x.device)
    on = _On(x.device, stream)
    if out is None:
        out = torch.empty(pos.numel() if num_rows is None else int(num_rows), x.shape[1], dtype=x.dtype, device=x.device)
    x = _rows_in(x)
    with on:
        lrs_dispatch_rows(ROW_TYPE_CODES[sfx], x, _ld(x), pos, x.shape[0], pos.shape[1], x.shape[1], out, _ld(out),
                          out.shape[0], on.handle)
    on.keep(x, pos, out)
    return out


def combine_rows(rows, position, weights=None, out=None, stream=None):
    """y[t] = sum over k of weights[t, k] * rows[position[t, k]] (weights None:
    ones; float32, bfloat16 or float16, of the shape of position).  Slots of
    position -1 add nothing.  Returns y, of the type of rows."""
    import torch
    sfx = _row_suffix("rows", _matrix("rows", rows).dtype)
    pos = _position(position, rows.device)
    w, wcode = _weights(weights, pos)
    if out is not None:
        _out_matrix("out", out, pos.shape[0], rows.shape[1], rows.dtype, rows.device)
    on = _On(rows.device, stream)
    if out is None:
        out = torch.empty(pos.shape[0], rows.shape[1], dtype=rows.dtype, device=rows.device)
    rows = _rows_in(rows)
    with on:
        lrs_combine_rows(ROW_TYPE_CODES[sfx], rows, _ld(rows), rows.shape[0], pos, wcode, w, pos.shape[0], pos.shape[1],
                         rows.shape[1], out, _ld(out), on.handle)
    on.keep(rows, pos, w, out)
    return out


def combine_rows_grad(grad_y, rows, position, weights, grad_rows=None, stream=None):
    """The gradient of combine_rows(rows, position, weights), given that of its
    output.  Returns (grad_rows, grad_weights): grad_rows[position[t, k]] =
    weights[t, k] * grad_y[t], in the given matrix (which may be `rows` itself: it
    is then replaced) or a new one, rows that no position names left as they were
    (zeros in a new one); grad_weights of the type of weights, zero where position
    is -1, None where weights is None."""
    import torch
    sfx = _row_suffix("rows", _matrix("rows", rows).dtype)
    pos = _position(position, rows.device)
    w, wcode = _weights(weights, pos)
    _matrix("grad_y", grad_y)
    if grad_y.dtype != rows.dtype or tuple(grad_y.shape) != (pos.shape[0], rows.shape[1]):
        raise ValueError("grad_y is %s %s, expected %s %s" % (grad_y.dtype, tuple(grad_y.shape), rows.dtype,
                                                              (pos.shape[0], rows.shape[1])))
    _same_device(rows.device, grad_y=grad_y)
    if grad_rows is not None:
        _out_matrix("grad_rows", grad_rows, rows.shape[0], rows.shape[1], rows.dtype, rows.device)
    on = _On(rows.device, stream)
    if grad_rows is None:
        grad_rows = torch.zeros(rows.shape, dtype=rows.dtype, device=rows.device)
    grad_w = None if w is None else torch.empty_like(w)
    grad_y, rows = _rows_in(grad_y), _rows_in(rows)
    with on:
        lrs_combine_rows_grad(ROW_TYPE_CODES[sfx], grad_y, _ld(grad_y), rows, _ld(rows), rows.shape[0], pos, wcode, w,
                              pos.shape[0], pos.shape[1], rows.shape[1], grad_rows, _ld(grad_rows), grad_w, on.handle)
    on.keep(grad_y, rows, pos, w, grad_rows, grad_w)
    return grad_rows, grad_w


def embedding(table, ids, scale: float = 1.0, first_id: int = 0, out=None, stream=None):
    """y[...] = scale * table[ids[...] - first_id], zeros for ids outside
    [first_id, first_id + number of rows).  ids: int32 or int64, any shape; y has
    that shape with the row length appended."""
    import torch
    sfx = _row_suffix("table", _matrix("table", table).dtype)
    code = ID_TYPE_CODES[_id_suffix(ids)]
    _same_device(table.device, ids=ids)
    n, cols, shape = ids.numel(), table.shape[1], tuple(ids.shape)
    if out is not None:
        if tuple(out.shape) != shape + (cols,):
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), shape + (cols,)))
        if out.dim() != 2 and not out.is_contiguous():
            raise ValueError("out must be contiguous")
        y = _out_matrix("out", out if out.dim() == 2 else out.view(n, cols), n, cols, table.dtype, table.device)
    on = _On(table.device, stream)
    if out is None:
        y = torch.empty(n, cols, dtype=table.dtype, device=table.device)
    table, ids = _rows_in(table), ids.contiguous()
    with on:
        lrs_embedding(ROW_TYPE_CODES[sfx], table, _ld(table), table.shape[0], code, ids, n, first_id, scale, cols, y,
                      _ld(y), on.handle)
    on.keep(table, ids, y)
    return y.view(shape + (cols,)) if out is None else out


def embedding_grad(grad_y, ids, num_ids: int, scale: float = 1.0, first_id: int = 0, dtype=None, grad=None,
                   accumulate: bool = False, temp=None, stream=None):
    """The gradient of embedding(table, ids, scale, first_id) with respect to its
    table of num_ids rows, given that of its output (of the shape of ids, the row
    length appended).  Returns a (num_ids, cols) matrix of `dtype` (grad_y's type by
    default, or float32): `grad` if given.  accumulate: the gradient is added to
    `grad`, and rows that no id names are not touched; otherwise every row is
    written."""
    import torch
    sfx = _row_suffix("grad_y", grad_y.dtype)
    code = ID_TYPE_CODES[_id_suffix(ids)]
    _same_device(grad_y.device, ids=ids, temp=temp)
    if grad_y.dim() < 1 or tuple(grad_y.shape[:-1]) != tuple(ids.shape):
        raise ValueError("grad_y has shape %s for ids of shape %s" % (tuple(grad_y.shape), tuple(ids.shape)))
    n, cols = ids.numel(), grad_y.shape[-1]
    dtype = dtype if dtype is not None else grad.dtype if grad is not None else grad_y.dtype
    if dtype not in (grad_y.dtype, torch.float32):
        raise TypeError("the gradient must be %s or float32, not %s" % (grad_y.dtype, dtype))
    if grad is not None:
        _out_matrix("grad", grad, int(num_ids), cols, dtype, grad_y.device)
    elif accumulate:
        raise ValueError("accumulate needs the gradient to add to")
    on = _On(grad_y.device, stream)
    if grad is None:
        grad = torch.empty(max(int(num_ids), 0), cols, dtype=dtype, device=grad_y.device)
    g2 = _rows_in(grad_y if grad_y.dim() == 2 else grad_y.reshape(n, cols))
    ids = ids.contiguous()
    args = (ROW_TYPE_CODES[sfx], g2, _ld(g2), code, ids, n, first_id, scale, ROW_TYPE_CODES[_row_suffix("grad", dtype)],
            grad, _ld(grad), num_ids, cols, accumulate)
    need = lrs_embedding_grad(None, 0, *args)
    t = _temp_tensor(need, grad_y.device, temp)
    with on:
        lrs_embedding_grad(t, t.numel() * t.element_size(), *args, on.handle)
    on.keep(g2, ids, t, grad)
    return grad
