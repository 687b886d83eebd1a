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

import ctypes

from . import _check, _ptr, _stream, load_library

ID_TYPE_CODES = {"i32": 0, "i64": 1}
ROW_TYPE_CODES = {"f32": 0, "bf16": 1, "f16": 2}

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
#
# A decode step's calls take a few microseconds on the GPU, so what the host does for
# each is kept short: type codes are looked up by the dtype itself, the C functions
# are called with plain addresses, and the temp bytes of a size are asked for once.

_types = None  # {torch dtype: code}: (ids, rows)
_needs: dict = {}  # temp bytes by sizes and types, which alone decide them


def _type_codes():
    global _types
    import torch
    _types = ({torch.int32: 0, torch.int64: 1}, {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}, torch.int32)
    return _types


def _id_code(t) -> int:
    code = (_types or _type_codes())[0].get(t.dtype)
    if code is None:
        raise TypeError("ids must be int32 or int64, not %s" % t.dtype)
    return code


def _row_code(name, dtype) -> int:
    code = (_types or _type_codes())[1].get(dtype)
    if code is None:
        raise TypeError("%s must be float32, bfloat16 or float16, not %s" % (name, dtype))
    return code


def _same_device(device, name, t):
    if t is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _matrix(name, t):
    """(rows, cols) of a matrix argument."""
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, t.dim()))
    return t.shape


def _row_stride(t):
    """Elements from one row to the next, or None if a row's elements are not next to
    each other or rows share memory."""
    rows, cols = t.shape
    step, one = t.stride()
    if cols > 1 and one != 1:
        return None
    if rows > 1:
        return step if step >= cols else None
    return cols


def _rows_in(t):
    """A matrix argument as the library reads it, and its row stride: a copy where a
    row's elements are not next to each other."""
    ld = _row_stride(t)
    if ld is None:
        t = t.contiguous()
        ld = t.shape[1]
    return t, ld


def _out_matrix(name, t, rows, cols, dtype, device):
    """Row stride of an output matrix, which must have that shape (rows None: any
    number), type and device."""
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    r, c = _matrix(name, t)
    if c != cols or (rows is not None and r != rows):
        raise ValueError("%s has shape %s, expected (%s, %d)" % (name, tuple(t.shape), "any" if rows is None else rows,
                                                                 cols))
    ld = _row_stride(t)
    if ld is None:
        raise ValueError("%s must be contiguous within each row" % name)
    _same_device(device, name, t)
    return ld


def _position(position, device):
    if position.dtype is not (_types or _type_codes())[2]:
        raise TypeError("position must be int32, not %s" % position.dtype)
    if position.dim() != 2:
        raise ValueError("position must have the shape (tokens, slots), not %s" % (tuple(position.shape),))
    _same_device(device, "position", position)
    return position.contiguous()


def _weights(weights, position):
    if weights is None:
        return None, 0
    if weights.shape != position.shape:
        raise ValueError("weights have shape %s, position %s" % (tuple(weights.shape), tuple(position.shape)))
    _same_device(position.device, "weights", weights)
    return weights.contiguous(), _row_code("weights", weights.dtype)


class _On:
    """Where a call runs if that is not simply the current stream of the current
    device: the tensors' device is made current, and on another stream than the
    current one the work waits for what the current one holds (inputs copied and
    outputs allocated there), and the tensors are recorded on it, so that the caching
    allocator does not hand their memory on while it is in use there."""

    def __init__(self, device, stream):
        import torch
        self.device, self.side = device, None
        self.current = torch.cuda.current_stream(device)
        self.handle = self.current.cuda_stream
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            if handle != self.handle:
                self.side = torch.cuda.ExternalStream(handle, device) if isinstance(stream, int) else stream
                if self.side.device != device:
                    raise ValueError("stream is on %s, the tensors on %s" % (self.side.device, device))
                self.handle = handle

    def call(self, fn, tensors, args) -> int:
        import torch
        if self.side is not None:
            self.side.wait_stream(self.current)
        with torch.cuda.device(self.device):
            status = fn(*args, self.handle or None)
        if self.side is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.side)
        return status


def _on(device, stream):
    """None for the current stream of the current device, else an _On."""
    import torch
    if device.type != "cuda":
        raise ValueError("lrsort needs device tensors, got a tensor on %s" % device)
    if stream is None and torch.cuda.current_device() == device.index:
        return None
    return _On(device, stream)


def _current_handle(device) -> int:
    """Handle of the device's current stream: torch's own shortcut to it where there
    is one (the Stream object that the public call builds takes 2 us)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _run(on, device, name, tensors, args) -> None:
    """Calls the C function `name` with `args` and the stream; `tensors` are in use
    until the stream has done it."""
    fn = getattr(load_library(), name)
    if on is None:
        status = fn(*args, _current_handle(device) or None)
    else:
        status = on.call(fn, tensors, args)
    if status:
        _check(status, name)


def _at(t):
    """Address of a tensor's first element (None for None and for empty tensors)."""
    return None if t is None else t.data_ptr() or None


def _temp(name, sizes, args, device, temp):
    """Temp storage for the C call `name` (args: what follows temp_bytes, without the
    stream), and its size.  `sizes`: what the size depends on."""
    import torch
    key = (name,) + sizes
    need = _needs.get(key)
    if need is None:
        tb = ctypes.c_size_t(0)
        _check(getattr(load_library(), name)(None, ctypes.byref(tb), *args, None), name)
        if len(_needs) >= 4096:
            _needs.clear()
        need = _needs[key] = tb.value
    if temp is not None:
        size = temp.numel() * temp.element_size()
        if size >= need:
            return temp, size
    return torch.empty(need, dtype=torch.uint8, device=device), need


def group_tokens(ids, num_groups: int, first_id: int = 0, temp=None, stream=None):
    """Stable grouping of ids (int32 or int64, any shape) into groups
    first_id..first_id + num_groups - 1.  Returns (order, position, offsets), int32:
    order, the flat indices sorted by group, those of no group last; position, of
    the shape of ids, where each stands in that order, or -1; offsets
    (num_groups + 1), where each group begins and the last ends."""
    import torch
    code = _id_code(ids)
    device = ids.device
    _same_device(device, "temp", temp)
    on = _on(device, stream)
    shape, n, num_groups = ids.shape, ids.numel(), int(num_groups)
    ids = ids.contiguous()
    order = torch.empty(n, dtype=torch.int32, device=device)
    position = torch.empty(shape, dtype=torch.int32, device=device)
    offsets = torch.empty(max(num_groups, 0) + 1, dtype=torch.int32, device=device)
    args = (code, _at(ids), n, int(first_id), num_groups, _at(order), _at(position), _at(offsets))
    t, size = _temp("lrs_group_tokens", (code, n, num_groups), args, device, temp)
    _run(on, device, "lrs_group_tokens", (ids, t, order, position, offsets), (_at(t), ctypes.byref(ctypes.c_size_t(size))) + args)
    return order, position, offsets


def dispatch_rows(x, position, num_rows: int | None = None, out=None, stream=None):
    """rows[position[t, k]] = x[t]: each token's row copied to its places
    (`position` from group_tokens on ids of shape (tokens, slots)).  Returns the
    rows: `out`, or a new matrix of num_rows rows (tokens * slots by default).  Rows
    that no position names are left as they were: unset in a new matrix.
    The gradient with respect to x is combine_rows(grad_rows, position)."""
    import torch
    code = _row_code("x", x.dtype)
    device = x.device
    tokens, cols = _matrix("x", x)
    pos = _position(position, device)
    if pos.shape[0] != tokens:
        raise ValueError("position is for %d tokens, x has %d" % (pos.shape[0], tokens))
    ld_out = cols if out is None else _out_matrix("out", out, num_rows, cols, x.dtype, device)
    on = _on(device, stream)
    if out is None:
        out = torch.empty(pos.numel() if num_rows is None else int(num_rows), cols, dtype=x.dtype, device=device)
    x, ld = _rows_in(x)
    _run(on, device, "lrs_dispatch_rows", (x, pos, out),
           (code, _at(x), ld, _at(pos), tokens, pos.shape[1], cols, _at(out), ld_out, out.shape[0]))
    return out


def combine_rows(rows, position, weights=None, out=None, stream=None):
    """y[t] = sum over k of weights[t, k] * rows[position[t, k]] (weights None:
    ones; float32, bfloat16 or float16, of the shape of position).  Slots of
    position -1 add nothing.  Returns y, of the type of rows."""
    import torch
    code = _row_code("rows", rows.dtype)
    device = rows.device
    num_rows, cols = _matrix("rows", rows)
    pos = _position(position, device)
    w, wcode = _weights(weights, pos)
    tokens, slots = pos.shape
    ld_out = cols if out is None else _out_matrix("out", out, tokens, cols, rows.dtype, device)
    on = _on(device, stream)
    if out is None:
        out = torch.empty(tokens, cols, dtype=rows.dtype, device=device)
    rows, ld = _rows_in(rows)
    _run(on, device, "lrs_combine_rows", (rows, pos, w, out),
           (code, _at(rows), ld, num_rows, _at(pos), wcode, _at(w), tokens, slots, cols, _at(out), ld_out))
    return out


def combine_rows_grad(grad_y, rows, position, weights, grad_rows=None, stream=None):
    """The gradient of combine_rows(rows, position, weights), given that of its
    output.  Returns (grad_rows, grad_weights): grad_rows[position[t, k]] =
    weights[t, k] * grad_y[t], in the given matrix (which may be `rows` itself: it
    is then replaced) or a new one, rows that no position names left as they were
    (zeros in a new one); grad_weights of the type of weights, zero where position
    is -1, None where weights is None."""
    import torch
    code = _row_code("rows", rows.dtype)
    device = rows.device
    num_rows, cols = _matrix("rows", rows)
    pos = _position(position, device)
    w, wcode = _weights(weights, pos)
    tokens, slots = pos.shape
    if grad_y.dtype != rows.dtype or _matrix("grad_y", grad_y) != (tokens, cols):
        raise ValueError("grad_y is %s %s, expected %s %s" % (grad_y.dtype, tuple(grad_y.shape), rows.dtype,
                                                              (tokens, cols)))
    _same_device(device, "grad_y", grad_y)
    ld_out = cols if grad_rows is None else _out_matrix("grad_rows", grad_rows, num_rows, cols, rows.dtype, device)
    on = _on(device, stream)
    if grad_rows is None:
        grad_rows = torch.zeros(num_rows, cols, dtype=rows.dtype, device=device)
    grad_w = None if w is None else torch.empty_like(w)
    grad_y, ld_y = _rows_in(grad_y)
    rows, ld = _rows_in(rows)
    _run(on, device, "lrs_combine_rows_grad", (grad_y, rows, pos, w, grad_rows, grad_w),
           (code, _at(grad_y), ld_y, _at(rows), ld, num_rows, _at(pos), wcode, _at(w), tokens, slots, cols,
            _at(grad_rows), ld_out, _at(grad_w)))
    return grad_rows, grad_w


def embedding(table, ids, scale: float = 1.0, first_id: int = 0, out=None, stream=None):
    """y[...] = scale * table[ids[...] - first_id], zeros for ids outside
    [first_id, first_id + number of rows).  ids: int32 or int64, any shape; y has
    that shape with the row length appended."""
    import torch
    code, id_code = _row_code("table", table.dtype), _id_code(ids)
    device = table.device
    num_ids, cols = _matrix("table", table)
    _same_device(device, "ids", ids)
    n, shape = ids.numel(), (*ids.shape, cols)
    y, ld_y = out, cols
    if out is not None:
        if out.shape != shape:
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), shape))
        if len(shape) != 2:
            if not out.is_contiguous():
                raise ValueError("out must be contiguous")
            y = out.view(n, cols)
        ld_y = _out_matrix("out", y, n, cols, table.dtype, device)
    on = _on(device, stream)
    if out is None:
        y = out = torch.empty(shape, dtype=table.dtype, device=device)
    table, ld = _rows_in(table)
    ids = ids.contiguous()
    _run(on, device, "lrs_embedding", (table, ids, y),
           (code, _at(table), ld, num_ids, id_code, _at(ids), n, int(first_id), float(scale), cols, _at(y), ld_y))
    return out


def embedding_grad(grad_y, ids, num_ids: int, scale: float = 1.0, first_id: int = 0, dtype=None, grad=None,
                   accumulate: bool = False, temp=None, stream=None):
    """The gradient of embedding(table, ids, scale, first_id) with respect to its
    table of num_ids rows, given that of its output (of the shape of ids, the row
    length appended).  Returns a (num_ids, cols) matrix of `dtype` (grad_y's type by
    default, or float32): `grad` if given.  accumulate: the gradient is added to
    `grad`, and rows that no id names are not touched; otherwise every row is
    written."""
    import torch
    code, id_code = _row_code("grad_y", grad_y.dtype), _id_code(ids)
    device, num_ids = grad_y.device, int(num_ids)
    _same_device(device, "ids", ids)
    _same_device(device, "temp", temp)
    if grad_y.dim() < 1 or grad_y.shape[:-1] != ids.shape:
        raise ValueError("grad_y has shape %s for ids of shape %s" % (tuple(grad_y.shape), tuple(ids.shape)))
    n, cols = ids.numel(), grad_y.shape[-1]
    if dtype is None:
        dtype = grad.dtype if grad is not None else grad_y.dtype
    if dtype not in (grad_y.dtype, torch.float32):
        raise TypeError("the gradient must be %s or float32, not %s" % (grad_y.dtype, dtype))
    if grad is not None:
        ld_grad = _out_matrix("grad", grad, num_ids, cols, dtype, device)
    elif accumulate:
        raise ValueError("accumulate needs the gradient to add to")
    on = _on(device, stream)
    if grad is None:
        grad, ld_grad = torch.empty(max(num_ids, 0), cols, dtype=dtype, device=device), cols
    g2, ld = _rows_in(grad_y if grad_y.dim() == 2 else grad_y.reshape(n, cols))
    ids = ids.contiguous()
    grad_code = _row_code("grad", dtype)
    args = (code, _at(g2), ld, id_code, _at(ids), n, int(first_id), float(scale), grad_code, _at(grad), ld_grad, num_ids,
            cols, 1 if accumulate else 0)
    t, size = _temp("lrs_embedding_grad", (code, id_code, n, grad_code, num_ids, cols), args, device, temp)
    _run(on, device, "lrs_embedding_grad", (g2, ids, t, grad), (_at(t), ctypes.byref(ctypes.c_size_t(size))) + args)
    return grad
