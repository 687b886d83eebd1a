"""Rows of a matrix moved and summed in the order of small integer keys.

The ``lrs_*`` functions call the C functions of the same name
(``include/lrsort_rows.h``) with the same arguments, as the package's other
bindings do.  ``group_tokens``, ``dispatch_rows``, ``combine_rows`` and
``combine_rows_grad`` (tokens sorted by expert and back), ``embedding`` and
``embedding_grad`` are conveniences over them on torch tensors: they allocate
outputs and temp storage, and refuse tensors of the wrong shape, type or device
with ValueError or TypeError before any work.  Gradients are calls of their own, as
in the C interface: nothing is recorded for torch's autograd, whatever the inputs
require (as under ``torch.no_grad``), but a tensor given as output counts as changed
in place, so a gradient that still needs its old values is refused by torch.

Matrices may have any row stride; their elements must be contiguous within a row
(inputs that are not are copied first, outputs are refused).  ``temp``, where a call
takes it, must be contiguous; one that is too small is not used.  ``stream`` is as for
``sort_keys``: None is the current stream of the tensors' device; on any other
stream the work also waits for what the current one already holds, so that inputs
just written there can be passed.
"""
from __future__ import annotations

import ctypes

from . import _check, _check_temp, _ptr, _stream, _stream_of, _written, load_library

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


def _int64(name, v) -> int:
    if v == 0:
        return 0
    v = int(v)
    if not -2**63 <= v < 2**63:
        raise ValueError("%s %d is no int64" % (name, v))
    return v


# ------------------------------------------------------------------ C calls


def lrs_group_tokens(d_temp, temp_bytes, id_type, d_ids, n, first_id, num_groups, d_order, d_position, d_offsets,
                     stream=None):
    """Calls the C function of the same name.  id_type is an lrs_id_type code or
    "i32" / "i64".  With d_temp None returns the temp bytes needed."""
    tb = ctypes.c_size_t(int(temp_bytes or 0))
    temp = _ptr(d_temp)
    st = None if temp is None else _stream(stream)
    _check(load_library().lrs_group_tokens(temp, ctypes.byref(tb), _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n),
                                           _int64("first_id", first_id), int(num_groups), _ptr(d_order),
                                           _ptr(d_position), _ptr(d_offsets), st), "lrs_group_tokens")
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
                                        _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n),
                                        _int64("first_id", first_id), float(scale), int(cols), _ptr(d_y), int(ld_y),
                                        _stream(stream)), "lrs_embedding")


def lrs_embedding_grad(d_temp, temp_bytes, row_type, d_grad_y, ld_grad_y, id_type, d_ids, n, first_id, scale, grad_type,
                       d_grad, ld_grad, num_ids, cols, accumulate, stream=None):
    """Calls the C function of the same name.  With d_temp None returns the temp
    bytes needed."""
    tb = ctypes.c_size_t(int(temp_bytes or 0))
    temp = _ptr(d_temp)
    st = None if temp is None else _stream(stream)
    _check(load_library().lrs_embedding_grad(temp, ctypes.byref(tb), _code(ROW_TYPE_CODES, row_type), _ptr(d_grad_y),
                                             int(ld_grad_y), _code(ID_TYPE_CODES, id_type), _ptr(d_ids), int(n),
                                             _int64("first_id", first_id), float(scale),
                                             _code(ROW_TYPE_CODES, grad_type), _ptr(d_grad), int(ld_grad), int(num_ids),
                                             int(cols), int(bool(accumulate)), st),
           "lrs_embedding_grad")
    return tb.value


# ------------------------------------------------------------- conveniences
#
# A decode step's calls take a few microseconds on the GPU, so what the host does for
# each is kept short: type codes are looked up by the dtype itself, devices compared
# by their index, the C functions called with plain addresses, and the temp bytes of
# a size asked for once.

_types = None  # ({torch dtype: code} of ids, of rows, torch.int32), once torch is there
_torch = None
_needs: dict = {}  # temp bytes by sizes and types, which alone decide them
_functions: dict = {}  # C functions of the loaded library
_current_handle = None  # device index -> handle of its current stream, once looked for


def _type_codes():
    global _types, _torch
    import torch
    _torch = torch
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


def _elsewhere(name, t, other):
    return ValueError("%s is on %s, expected %s" % (name, t.device, other.device))


def _matrix(name, t):
    """(rows, cols) of a matrix argument."""
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, t.dim()))
    return t.shape


def _row_stride(t, rows, cols):
    """Elements from one row to the next, or None if a row's elements are not next to
    each other or rows share memory."""
    if t.is_contiguous():
        return cols
    step, one = t.stride()
    if cols > 1 and one != 1:
        return None
    if rows > 1:
        return step if step >= cols else None
    return cols


def _rows_in(t, rows, cols):
    """A matrix argument as the library reads it, and its row stride: a copy where a
    row's elements are not next to each other."""
    ld = _row_stride(t, rows, cols)
    return (t, ld) if ld is not None else (t.contiguous(), cols)


def _rows_out(name, t, rows, cols, like):
    """(rows, row stride) of an output matrix, which must have that shape (rows None:
    any number) and the type and device of `like`."""
    if t.dtype is not like.dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
    r, c = _matrix(name, t)
    if c != cols or (rows is not None and r != rows):
        raise ValueError("%s has shape %s, expected (%s, %d)" % (name, tuple(t.shape), "any" if rows is None else rows,
                                                                 cols))
    ld = _row_stride(t, r, c)
    if ld is None:
        raise ValueError("%s must be contiguous within each row" % name)
    if t.get_device() != like.get_device():
        raise _elsewhere(name, t, like)
    return r, ld


def _position(position, like):
    if position.dtype is not (_types or _type_codes())[2]:
        raise TypeError("position must be int32, not %s" % position.dtype)
    if position.dim() != 2:
        raise ValueError("position must have the shape (tokens, slots), not %s" % (tuple(position.shape),))
    if position.get_device() != like.get_device():
        raise _elsewhere("position", position, like)
    return position.contiguous()


def _weights(weights, position):
    if weights is None:
        return None, 0
    if weights.shape != position.shape:
        raise ValueError("weights have shape %s, position %s" % (tuple(weights.shape), tuple(position.shape)))
    if weights.get_device() != position.get_device():
        raise _elsewhere("weights", weights, position)
    return weights.contiguous(), _row_code("weights", weights.dtype)


def _at(t):
    """Address of an optional tensor's first element."""
    return None if t is None else t.data_ptr()


def _load(name):
    fn = _functions[name] = getattr(load_library(), name)
    return fn


def _handle_lookup():
    """Finds how a device's current stream handle is had: by torch's own shortcut to it
    where there is one (the Stream object that the public call builds takes 2 us)."""
    global _current_handle
    import torch
    _current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _current_handle


def _host_tensor(t):
    return ValueError("lrsort needs device tensors, got a tensor on %s" % t.device)


def _run(name, stream, tensors, args, written=None) -> None:
    """Calls the C function `name` with `args` and the stream's handle, with the
    device of the first of `tensors` current.  None is that device's current stream.
    On another stream the work waits for what the current one holds (inputs copied
    and outputs allocated there), and the tensors are recorded on it, so that the
    caching allocator does not hand their memory on while it is in use there.
    `written`: an output that the caller gave."""
    fn = _functions.get(name) or _load(name)
    index = tensors[0].get_device()
    if stream is None and _torch.cuda.current_device() == index:
        status = fn(*args, (_current_handle or _handle_lookup())(index) or None)
        if status:
            _check(status, name)
        if written is not None:
            _written(written)
        return
    torch = _torch
    if stream is not None and not isinstance(stream, int) and stream.device.index != index:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, tensors[0].device))
    current = torch.cuda.current_stream(index)
    handle = current.cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    side = None
    if handle != current.cuda_stream:
        side = _stream_of(handle, index) if isinstance(stream, int) else stream
        side.wait_stream(current)
    with torch.cuda.device(index):
        _check(fn(*args, handle or None), name)
    if side is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(side)
    _written(written)


def _temp(name, sizes, args, like, temp):
    """Temp storage for the C call `name` (args: what follows temp_bytes, without the
    stream), and its size.  `sizes`: what the size depends on.  255 bytes are the
    alignment's alone: the call then needs no storage, and any address will do."""
    key = (name,) + sizes
    need = _needs.get(key)
    if need is None:
        tb = ctypes.c_size_t(0)
        _check((_functions.get(name) or _load(name))(None, ctypes.byref(tb), *args, None), name)
        if len(_needs) >= 4096:
            _needs.clear()
        need = _needs[key] = tb.value
    if temp is not None:
        _check_temp(temp)
        if temp.get_device() != like.get_device():
            raise _elsewhere("temp", temp, like)
        size = temp.numel() * temp.element_size()
        if size >= need:
            return temp, size
    if need <= 255:
        return like, need
    return _torch.empty(need, dtype=_torch.uint8, device=like.device), need


def group_tokens(ids, num_groups: int, first_id: int = 0, temp=None, stream=None):
    """Stable grouping of ids (int32 or int64, any shape) into groups
    first_id..first_id + num_groups - 1.  Returns (order, position, offsets), int32:
    order, the flat indices sorted by group, those of no group last; position, of
    the shape of ids, where each stands in that order, or -1; offsets
    (num_groups + 1), where each group begins and the last ends."""
    code = _id_code(ids)
    if not ids.is_cuda:
        raise _host_tensor(ids)
    ids = ids.contiguous()
    n, num_groups, int32 = ids.numel(), int(num_groups), _types[2]
    position = _torch.empty_like(ids, dtype=int32)
    order = position.new_empty(n)
    offsets = position.new_empty(num_groups + 1 if num_groups > 0 else 1)
    args = (code, ids.data_ptr(), n, _int64("first_id", first_id), num_groups, order.data_ptr(), position.data_ptr(),
            offsets.data_ptr())
    t, size = _temp("lrs_group_tokens", (code, n, num_groups), args, offsets, temp)
    _run("lrs_group_tokens", stream, (offsets, ids, t, order, position),
         (t.data_ptr(), ctypes.byref(ctypes.c_size_t(size))) + args)
    return order, position, offsets


def dispatch_rows(x, position, num_rows: int | None = None, out=None, stream=None):
    """rows[position[t, k]] = x[t]: each token's row copied to its places
    (`position` from group_tokens on ids of shape (tokens, slots)).  Returns the
    rows: `out`, or a new matrix of num_rows rows (tokens * slots by default).  Rows
    that no position names are left as they were: unset in a new matrix.
    The gradient with respect to x is combine_rows(grad_rows, position)."""
    code = _row_code("x", x.dtype)
    tokens, cols = _matrix("x", x)
    pos = _position(position, x)
    t, slots = pos.shape
    if t != tokens:
        raise ValueError("position is for %d tokens, x has %d" % (t, tokens))
    if out is not None:
        num_rows, ld_out = _rows_out("out", out, num_rows, cols, x)
    if not x.is_cuda:
        raise _host_tensor(x)
    given = out
    if out is None:
        num_rows, ld_out = t * slots if num_rows is None else int(num_rows), cols
        out = x.new_empty(num_rows, cols)
    x, ld = _rows_in(x, tokens, cols)
    _run("lrs_dispatch_rows", stream, (x, pos, out),
         (code, x.data_ptr(), ld, pos.data_ptr(), tokens, slots, cols, out.data_ptr(), ld_out, num_rows), given)
    return out


def combine_rows(rows, position, weights=None, out=None, stream=None):
    """y[t] = sum over k of weights[t, k] * rows[position[t, k]] (weights None:
    ones; float32, bfloat16 or float16, of the shape of position).  Slots of
    position -1 add nothing.  Returns y, of the type of rows."""
    code = _row_code("rows", rows.dtype)
    num_rows, cols = _matrix("rows", rows)
    pos = _position(position, rows)
    w, wcode = _weights(weights, pos)
    tokens, slots = pos.shape
    ld_out = cols if out is None else _rows_out("out", out, tokens, cols, rows)[1]
    if not rows.is_cuda:
        raise _host_tensor(rows)
    given = out
    if out is None:
        out = rows.new_empty(tokens, cols)
    rows, ld = _rows_in(rows, num_rows, cols)
    _run("lrs_combine_rows", stream, (rows, pos, w, out),
         (code, rows.data_ptr(), ld, num_rows, pos.data_ptr(), wcode, _at(w), tokens, slots, cols, out.data_ptr(),
          ld_out), given)
    return out


def combine_rows_grad(grad_y, rows, position, weights, grad_rows=None, stream=None):
    """The gradient of combine_rows(rows, position, weights), given that of its
    output.  Returns (grad_rows, grad_weights): grad_rows[position[t, k]] =
    weights[t, k] * grad_y[t], in the given matrix (which may be `rows` itself: it
    is then replaced) or a new one, rows that no position names left as they were
    (zeros in a new one); grad_weights of the type of weights, zero where position
    is -1, None where weights is None.  No two slots may have the same position
    (group_tokens gives none such)."""
    code = _row_code("rows", rows.dtype)
    num_rows, cols = _matrix("rows", rows)
    pos = _position(position, rows)
    w, wcode = _weights(weights, pos)
    tokens, slots = pos.shape
    if grad_y.dtype is not rows.dtype or _matrix("grad_y", grad_y) != (tokens, cols):
        raise ValueError("grad_y is %s %s, expected %s %s" % (grad_y.dtype, tuple(grad_y.shape), rows.dtype,
                                                              (tokens, cols)))
    if grad_y.get_device() != rows.get_device():
        raise _elsewhere("grad_y", grad_y, rows)
    ld_out = cols if grad_rows is None else _rows_out("grad_rows", grad_rows, num_rows, cols, rows)[1]
    if not rows.is_cuda:
        raise _host_tensor(rows)
    given = grad_rows
    if grad_rows is None:
        grad_rows = rows.new_zeros(num_rows, cols)
    grad_w = None if w is None else w.new_empty(tokens, slots)
    grad_y, ld_y = _rows_in(grad_y, tokens, cols)
    rows, ld = _rows_in(rows, num_rows, cols)
    _run("lrs_combine_rows_grad", stream, (rows, grad_y, pos, w, grad_rows, grad_w),
         (code, grad_y.data_ptr(), ld_y, rows.data_ptr(), ld, num_rows, pos.data_ptr(), wcode, _at(w), tokens, slots,
          cols, grad_rows.data_ptr(), ld_out, _at(grad_w)), given)
    return grad_rows, grad_w


def embedding(table, ids, scale: float = 1.0, first_id: int = 0, out=None, stream=None):
    """y[...] = scale * table[ids[...] - first_id], zeros for ids outside
    [first_id, first_id + number of rows).  ids: int32 or int64, any shape; y has
    that shape with the row length appended."""
    code, id_code = _row_code("table", table.dtype), _id_code(ids)
    num_ids, cols = _matrix("table", table)
    if ids.get_device() != table.get_device():
        raise _elsewhere("ids", ids, table)
    n, shape = ids.numel(), (*ids.shape, cols)
    given, y, ld_y = out, out, cols
    if out is not None:
        if out.shape != shape:
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), shape))
        if len(shape) != 2:
            if not out.is_contiguous():
                raise ValueError("out must be contiguous")
            y = out.view(n, cols)
        ld_y = _rows_out("out", y, n, cols, table)[1]
    if not table.is_cuda:
        raise _host_tensor(table)
    if out is None:
        y = out = table.new_empty(shape)
    table, ld = _rows_in(table, num_ids, cols)
    ids = ids.contiguous()
    _run("lrs_embedding", stream, (table, ids, y),
         (code, table.data_ptr(), ld, num_ids, id_code, ids.data_ptr(), n, _int64("first_id", first_id), float(scale),
          cols, y.data_ptr(), ld_y), given)
    return out


def embedding_grad(grad_y, ids, num_ids: int, scale: float = 1.0, first_id: int = 0, dtype=None, grad=None,
                   accumulate: bool = False, temp=None, stream=None):
    """The gradient of embedding(table, ids, scale, first_id) with respect to its
    table of num_ids rows, given that of its output (of the shape of ids, the row
    length appended).  Returns a (num_ids, cols) matrix of `dtype` (grad_y's type by
    default, or float32): `grad` if given.  accumulate: the gradient is added to
    `grad`, and rows that no id names are not touched; otherwise every row is
    written."""
    code, id_code, num_ids = _row_code("grad_y", grad_y.dtype), _id_code(ids), int(num_ids)
    if ids.get_device() != grad_y.get_device():
        raise _elsewhere("ids", ids, grad_y)
    if grad_y.dim() < 1 or grad_y.shape[:-1] != ids.shape:
        raise ValueError("grad_y has shape %s for ids of shape %s" % (tuple(grad_y.shape), tuple(ids.shape)))
    n, cols = ids.numel(), grad_y.shape[-1]
    if dtype is None:
        dtype = grad.dtype if grad is not None else grad_y.dtype
    if dtype is not grad_y.dtype and dtype is not _torch.float32:
        raise TypeError("the gradient must be %s or float32, not %s" % (grad_y.dtype, dtype))
    ld_grad = cols
    if grad is not None:
        if grad.dtype is not dtype:
            raise ValueError("grad has dtype %s, expected %s" % (grad.dtype, dtype))
        if grad.get_device() != grad_y.get_device():
            raise _elsewhere("grad", grad, grad_y)
        ld_grad = _rows_out("grad", grad, num_ids, cols, grad)[1]
    elif accumulate:
        raise ValueError("accumulate needs the gradient to add to")
    if not grad_y.is_cuda:
        raise _host_tensor(grad_y)
    given = grad
    if grad is None:
        grad = _torch.empty(num_ids if num_ids > 0 else 0, cols, dtype=dtype, device=grad_y.device)
    g2, ld = _rows_in(grad_y if grad_y.dim() == 2 else grad_y.reshape(n, cols), n, cols)
    ids = ids.contiguous()
    grad_code = _types[1][dtype]
    args = (code, g2.data_ptr(), ld, id_code, ids.data_ptr(), n, _int64("first_id", first_id), float(scale), grad_code,
            grad.data_ptr(), ld_grad, num_ids, cols, 1 if accumulate else 0)
    t, size = _temp("lrs_embedding_grad", (code, id_code, n, grad_code, num_ids, cols), args, grad, temp)
    _run("lrs_embedding_grad", stream, (g2, ids, t, grad), (t.data_ptr(), ctypes.byref(ctypes.c_size_t(size))) + args,
         given)
    return grad
