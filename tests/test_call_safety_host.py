"""What the torch conveniences refuse or arrange around a call, without a GPU: temp
storage that is not one block of memory, the stream a handle stands for, memory that
arrays share, and torch's count of writes to a tensor."""
from __future__ import annotations

import pytest
import torch

import sorting_lsd_radix_sort_amd as lrs
from sorting_lsd_radix_sort_amd import rows

# fake, well-aligned device addresses, far apart: these checks never dereference them
A, B, C, D = (i << 40 for i in range(1, 5))


# ------------------------------------------------------------------ temp storage


def scattered_temps(nbytes):
    """Tensors whose elements are as many bytes as asked for and more, but do not lie in one block."""
    return {"columns": torch.zeros(64, nbytes, dtype=torch.uint8)[:, :nbytes // 2],
            "every other": torch.zeros(4 * nbytes, dtype=torch.uint8)[::2],
            "expanded": torch.zeros(1, dtype=torch.uint8).expand(2 * nbytes),
            "turned": torch.zeros(64, nbytes, dtype=torch.uint8).t()}


@pytest.mark.parametrize("kind", ["columns", "every other", "expanded", "turned"])
def test_temp_that_is_not_one_block_is_refused(kind):
    """A call writes the bytes that follow the tensor's first element: of a column
    slice these are other columns, of an expanded element other memory."""
    need = 4096
    temp = scattered_temps(need)[kind]
    assert temp.numel() >= need and not temp.is_contiguous()
    with pytest.raises(ValueError, match="temp must be contiguous"):
        lrs._temp_tensor(need, temp.device, temp)
    like = torch.zeros(1)
    args = (1, A, 20000, 0, 8, B, C, D)
    with pytest.raises(ValueError, match="temp must be contiguous"):
        rows._temp("lrs_group_tokens", (1, 20000, 8), args, like, temp)
    # one block is taken as it is, by both
    whole = torch.zeros(1 << 20, dtype=torch.uint8)
    assert lrs._temp_tensor(need, whole.device, whole) is whole
    assert rows._temp("lrs_group_tokens", (1, 20000, 8), args, like, whole)[0] is whole


# ---------------------------------------------------------------------- streams


class FakeStream:
    def __init__(self, handle, index=0):
        self.cuda_stream = handle
        self.device = torch.device("cuda", index)
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other)


class FakeTensor:
    device = torch.device("cuda", 0)

    def __init__(self):
        self.recorded = []

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def fake_streams(monkeypatch):
    """torch's streams replaced by objects that note what is asked of them: the current
    one has the handle 5, and the default stream's handle is 0, as on a GPU.  torch's
    ExternalStream takes the handle 0 for "a new stream"."""
    import contextlib
    import types

    current, default, made = FakeStream(5), FakeStream(0), []

    def external(handle, device=None):
        made.append(FakeStream(handle if handle else 999))
        return made[-1]

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    rows._type_codes()
    monkeypatch.setattr(rows, "_current_handle", lambda index: current.cuda_stream)
    calls = []
    monkeypatch.setitem(rows._functions, "a_call", lambda *args: calls.append(args) or 0)
    return types.SimpleNamespace(current=current, default=default, made=made, calls=calls)


def test_handle_zero_is_the_default_stream(fake_streams):
    """With another stream current, work on handle 0 waits for the current stream, and
    the tensors are recorded on the default one."""
    f, t = fake_streams, FakeTensor()
    rows._run("a_call", 0, (t,), (7,))
    assert f.calls == [(7, None)]
    assert f.default.waited == [f.current] and t.recorded == [f.default] and not f.made
    assert lrs._side_stream(0) is f.default and not f.made
    # any other handle is that stream, the current one's needs nothing
    rows._run("a_call", 12, (t,), ())
    assert f.calls[-1] == (12,) and f.made[-1].cuda_stream == 12 and f.made[-1].waited == [f.current]
    assert t.recorded[-1] is f.made[-1]
    assert lrs._side_stream(12).cuda_stream == 12
    rows._run("a_call", 5, (t,), ())
    assert f.calls[-1] == (5,) and len(t.recorded) == 2
    assert lrs._side_stream(5) is None


def test_sorts_on_a_side_stream_wait_for_the_current_one(fake_streams):
    """Copies made and memory handed out on the current stream are ready there, and
    free of earlier work, only behind what it holds."""
    f, side = fake_streams, FakeStream(12)
    assert lrs._side_stream(side) is side and side.waited == [f.current]
    assert lrs._side_stream(13).waited == [f.current]
    assert lrs._side_stream(f.current) is None and not f.current.waited
    assert lrs._side_stream(None) is None


def test_default_stream_of_another_device_is_refused(fake_streams):
    """Every device's default stream has the handle 0: the device tells them apart."""
    f, t = fake_streams, FakeTensor()
    f.current.cuda_stream = 0
    rows._run("a_call", FakeStream(0, 0), (t,), ())
    assert f.calls == [(None,)]
    for other in (FakeStream(0, 1), FakeStream(12, 1)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            rows._run("a_call", other, (t,), ())
        assert not other.waited
    assert len(f.calls) == 1 and not t.recorded


# -------------------------------------------------------------- torch's bookkeeping


def test_a_written_tensor_counts_as_changed(fake_streams):
    """A tensor that a call was given to write has a new version afterwards, so that
    autograd notices if it had been saved for a gradient; also on a side stream."""
    f, t = fake_streams, FakeTensor()
    saved = torch.ones(3, requires_grad=True)
    for stream in (None, 12):
        kept = torch.full((3,), 2.0)
        y = (saved * kept).sum()
        rows._run("a_call", stream, (t,), (), kept)
        assert kept._version == 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    kept = torch.zeros(3)
    lrs._written(kept, None)
    assert kept._version == 1
    with torch.inference_mode():
        lrs._written(torch.zeros(3))  # has no version: nothing to count


# ------------------------------------------------------------------ wide numbers


@pytest.mark.parametrize("first", [2**63, -2**63 - 1, 2**64, 2**64 + 3])
def test_first_id_that_is_no_int64_is_refused_by_the_c_calls(first):
    """ctypes would keep its low 64 bits: 2**64 + 3 would be taken for 3."""
    with pytest.raises(ValueError, match="int64"):
        lrs.lrs_group_tokens(None, 0, "i64", A, 100, first, 8, B, C, D, 0)
    with pytest.raises(ValueError, match="int64"):
        lrs.lrs_embedding("bf16", A, 64, 10, "i64", B, 0, first, 1.0, 64, C, 64, 0)
    with pytest.raises(ValueError, match="int64"):
        lrs.lrs_embedding_grad(None, 0, "bf16", A, 64, "i64", B, 100, first, 1.0, "bf16", C, 64, 10, 64, 0, 0)
