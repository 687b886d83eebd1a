"""Beam search's selection and reordering against their definitions in 64 bits.

Parents and tokens have to be equal.  Scores have a derived tolerance: exp2 and its
argument are off by at most (2 |d| + 4) * 2^-24 relative for a logit d below the largest;
weighted by their shares of the sum, the |d| average to at most log(vocab) (the entropy of
the shares less the logarithm of a sum that is at least one), and up to eight of them are
added in float32, the rest in float64.  So the logarithm of the sum is off by at most
(2 log(vocab) + 12) * 2^-24, and the total, formed in float64, is rounded once.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu

INF = float("inf")


def torch_():
    import torch
    return torch


def dtype_of(name):
    torch = torch_()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def as64(t):
    return t.detach().cpu().double().numpy()


def randn(shape, name, seed, scale=2.0):
    torch = torch_()
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(x).to(dtype_of(name)).cuda()


def beam_scores(batch, beams, seed):
    torch = torch_()
    x = -np.random.default_rng(seed).random((batch, beams)).cumsum(1) * 3
    return torch.from_numpy(x.astype(np.float32)).cuda()


def reference(logits, scores, count, normalize=True, finished=None, end_id=0):
    l, s = as64(logits), as64(scores)
    b, k, v = l.shape
    with np.errstate(all="ignore"):
        total = l
        if normalize and v:
            top = l.max(2, keepdims=True)
            top = np.where(top == -INF, 0, top)
            total = l - (top + np.log(np.exp(l - top).sum(2, keepdims=True)))
        total = total + s[:, :, None]
    total[(l == -INF) | np.isnan(l)] = -INF
    total[s == -INF] = -INF
    if finished is not None:
        done = finished.cpu().numpy().astype(bool)
        total[done] = -INF
        total[done, end_id] = s[done]
    out_s, out_p, out_t = (np.full((b, count), x) for x in (-INF, -1, -1))
    for i in range(b):
        flat = total[i].reshape(-1)
        key = np.where(flat == -INF, INF, -flat)
        if flat.size > 4 * count + 1000:  # what is not among these is surely not chosen
            cut = np.partition(key, 4 * count)[4 * count]
            at = np.nonzero(key <= cut)[0]
        else:
            at = np.arange(flat.size)
        at = at[np.argsort(key[at], kind="stable")][:count]
        at = at[flat[at] != -INF]
        out_s[i, :at.size], out_p[i, :at.size], out_t[i, :at.size] = flat[at], at // v, at % v
    return out_s, out_p, out_t


def check(logits, scores, count, normalize=True, finished=None, end_id=0, id_type="i32", what=""):
    torch = torch_()
    got = lrs.beam_select(logits, scores, count, normalize=normalize, finished=finished, end_id=end_id,
                          dtype=torch.int64 if id_type == "i64" else None)
    want_s, want_p, want_t = reference(logits, scores, count, normalize, finished, end_id)
    s, p, t = (x.cpu().numpy() for x in got)
    assert p.dtype == np.int32 and t.dtype == (np.int64 if id_type == "i64" else np.int32)
    bad = (p != want_p) | (t != want_t)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError("%s: %d differ, first at %s: beam %d token %d score %r, expected %d %d %r" % (
            what, bad.sum(), i, p[tuple(i)], t[tuple(i)], s[tuple(i)], want_p[tuple(i)], want_t[tuple(i)],
            want_s[tuple(i)]))
    with np.errstate(all="ignore"):
        off = (2 * math.log(max(logits.shape[2], 1)) + 12) * 2.0**-24 if normalize else 0.0
        ok = (np.abs(s - want_s) <= off + (np.abs(want_s) + off) * 2.0**-24) | (s == want_s)
    assert ok.all(), (what, s[~ok][0], want_s[~ok][0])
    return got


VOCABS = [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 1023, 1025, 4096, 5003, 32000, 50001]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_beam_select(vocab, name):
    torch = torch_()
    for i, (batch, beams, count) in enumerate([(1, 1, 1), (1, 4, 8), (7, 5, 10), (3, 2, 64), (2, 17, 34)]):
        logits, scores = randn((batch, beams, vocab), name, vocab + i), beam_scores(batch, beams, i)
        done = torch.from_numpy(np.random.default_rng(i).random((batch, beams)) < 0.3).cuda()
        for normalize in (True, False):
            for finished in (None, done):
                announce("beam %d x %d x %d count %d %s norm %s done %s" % (batch, beams, vocab, count, name, normalize,
                                                                         finished is not None))
                check(logits, scores, count, normalize, finished, vocab // 2, "i64" if i % 2 else "i32")


@pytest.mark.parametrize("count", [1, 2, 3, 31, 32, 33, 63, 64])
def test_counts_and_parts(count):
    """Rows in one part and in many, each count."""
    for batch, beams, vocab in ((1, 1, 100003), (1, 3, 20000), (40, 8, 3001), (600, 8, 1500)):
        announce("count %d of %d x %d x %d" % (count, batch, beams, vocab))
        check(randn((batch, beams, vocab), "f32", count), beam_scores(batch, beams, count), count)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "two values", "sawtooth", "blocks"])
def test_orders_of_logits(name, kind):
    """Rows that fill the lists of the best again and again, and rows of ties."""
    torch = torch_()
    for vocab in (300, 4099, 40000):
        announce("order %s %s %d" % (kind, name, vocab))
        at = np.arange(vocab)
        x = {"rising": at * (8.0 / vocab), "falling": -at * (8.0 / vocab), "equal": at * 0.0, "two values": at % 7 == 3,
             "sawtooth": at % 97 * 0.01, "blocks": at // 64 % 5 * 1.0}[kind].astype(np.float32)
        logits = torch.from_numpy(np.tile(x, (2, 3, 1))).to(dtype_of(name)).cuda()
        scores = torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -1.5]], device="cuda")
        for count in (1, 6, 64):
            for normalize in (True, False):
                check(logits, scores, count, normalize, what="%s %d" % (kind, count))


def test_equal_rows_share_their_scores():
    """Beams of equal logits and scores, at every alignment of their rows: ties go to the
    lower beam, whatever the address its row begins at."""
    torch = torch_()
    for name in ("f32", "bf16", "f16"):
        for vocab in (129, 1001, 30007):
            announce("equal rows %s %d" % (name, vocab))
            logits = randn((1, 1, vocab), name, vocab).expand(2, 6, vocab).contiguous()
            check(logits, torch.zeros(2, 6, device="cuda"), 12, what=name)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_masked_beams_and_tokens(name):
    torch = torch_()
    announce("masked beams %s" % name)
    lowest = torch.finfo(dtype_of(name)).min
    nan = float("nan")
    for vocab in (5, 700, 6000):
        logits, scores = randn((9, 4, vocab), name, 1), beam_scores(9, 4, 1)
        scores[0, 1:] = -INF              # the first step of a search: one beam lives
        logits[0, 1:] = nan               # (and the others' logits are not read)
        scores[1] = -INF                  # none lives
        logits[2, 0] = -INF               # a beam without a token
        logits[2, 1, 1:] = -INF           # with one
        logits[3] = lowest                # nothing but the lowest finite value
        logits[4, 2] = lowest
        logits[4, 2, 3] = 1.0
        logits[5, :, ::2] = -INF
        logits[6, :, vocab // 3:] = -INF  # a vocabulary that ends early
        logits[7] = -INF
        done = torch.zeros(9, 4, dtype=torch.bool, device="cuda")
        done[8] = True
        done[7, 2] = True                 # the only continuation there is
        logits[8] = nan                   # not read
        scores[8, 3] = -INF               # finished and dead: takes no part
        for count in (1, 8, 30):
            for normalize in (True, False):
                check(logits, scores, count, normalize, done, 4, what="%d %d %s" % (vocab, count, normalize))
                check(logits, scores, count, normalize, done.to(torch.uint8) * 255, 0, what="bytes")
    s, p, t = lrs.beam_select(logits, scores, 8, finished=done, end_id=4)
    assert (p[1] == -1).all() and (t[1] == -1).all() and (s[1] == -INF).all()
    assert p[7].tolist() == [2] + [-1] * 7 and t[7, 0] == 4 and s[7, 0] == scores[7, 2]


def test_nan_and_infinity():
    torch = torch_()
    announce("beam nan")
    logits, scores = randn((6, 3, 500), "f32", 1), beam_scores(6, 3, 1)
    clean = reference(logits, scores, 6)
    logits[1, 2, 77] = float("nan")
    logits[2, 1, 5] = INF
    scores[3, 0] = float("nan")
    s, p, t = lrs.beam_select(logits, scores, 6)
    for row in (0, 4, 5):  # other searches are not touched
        assert np.array_equal(p[row].cpu(), clean[1][row]) and np.array_equal(t[row].cpu(), clean[2][row])
    for row, beam in ((1, 2), (2, 1), (3, 0)):
        assert s[row].isnan().all() and (p[row] == beam).all() and ((t[row] >= 0) & (t[row] < 500)).all()
    assert not (t[1] == 77).any()
    s, p, t = lrs.beam_select(logits, scores, 6, normalize=False)
    assert not ((t[1] == 77) & (p[1] == 2)).any() and torch.isfinite(s[1]).all()
    assert s[2, 0] == INF and t[2, 0] == 5 and p[2, 0] == 1 and torch.isfinite(s[2, 1:]).all()


def by_beam_and_logit(logits, scores, count, normalize):
    """(parents, tokens) by totals in 64 bits, equal ones by beam, then logit, then token;
    NaN totals before all others."""
    l, s = as64(logits), as64(scores)
    b, k, v = l.shape
    parents, tokens = np.full((b, count), -1), np.full((b, count), -1)
    with np.errstate(all="ignore"):
        total = l + s[:, :, None]
        if normalize:
            top = l.max(2, keepdims=True)
            total = (l - (top + np.log(np.exp(l - top).sum(2, keepdims=True)))) + s[:, :, None]
    beam, token = np.divmod(np.arange(k * v), v)
    for i in range(b):
        t, of = total[i].reshape(-1), l[i].reshape(-1)
        order = np.lexsort((token, -of, beam, np.where(np.isnan(t), 0.0, -t), ~np.isnan(t)))
        order = order[~(np.isnan(of) | (of == -INF) | (s[i][beam] == -INF))[order]][:count]
        parents[i, :order.size], tokens[i, :order.size] = beam[order], token[order]
    return parents, tokens


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normalize", [True, False])
def test_tokens_of_a_beam_go_by_their_logits(name, normalize):
    """Also where a beam's totals are one number: scores that swallow the logits, logits
    too small to change a total, NaN and infinity."""
    torch = torch_()
    lowest = torch.finfo(torch.float32).min
    for vocab in (9, 700, 33001):
        announce("swallowed logits %s %s %d" % (name, normalize, vocab))
        logits, scores = randn((8, 3, vocab), name, vocab), beam_scores(8, 3, 1)
        scores[0] = lowest
        scores[1, 1] = -1e30
        scores[2] = torch.tensor([1e30, 1e30, -INF])
        scores[3] = torch.tensor([-INF, -1e12, -INF])
        logits[4] = (randn((3, vocab), "f32", 5) * 1e-20).to(logits.dtype)  # (float16: zeros of both signs)
        scores[4] = -1.0
        scores[5, 1] = float("nan")
        scores[6] = torch.tensor([0.0, INF, -1.0])
        logits[7, 2, 4] = float("nan")
        for count in (1, 6, 64):
            got = lrs.beam_select(logits, scores, count, normalize=normalize)
            want_p, want_t = by_beam_and_logit(logits, scores, count, normalize)
            p, t = got[1].cpu().numpy(), got[2].cpu().numpy()
            for i in range(8):
                assert (p[i] == want_p[i]).all() and (t[i] == want_t[i]).all(), (vocab, count, i, p[i], t[i], want_p[i],
                                                                                 want_t[i])
            # a search gives the same alone, where its rows are cut into more parts
            for i in (0, 4, 5):
                alone = lrs.beam_select(logits[i:i + 1], scores[i:i + 1], count, normalize=normalize)
                assert all(torch.equal(a.nan_to_num(7.0), b[i:i + 1].nan_to_num(7.0)) for a, b in zip(alone, got))
    wide = randn((200, 3, 33001), name, 3)
    parked = torch.full((200, 3), lowest, device="cuda")
    got = lrs.beam_select(wide, parked, 7, normalize=normalize)
    for i in (0, 199):
        alone = lrs.beam_select(wide[i:i + 1], parked[i:i + 1], 7, normalize=normalize)
        assert all(torch.equal(a, b[i:i + 1]) for a, b in zip(alone, got))
    want_p, want_t = by_beam_and_logit(wide[:1], parked[:1], 7, normalize)
    assert (got[1][0].cpu().numpy() == want_p[0]).all() and (got[2][0].cpu().numpy() == want_t[0]).all()


def test_beam_strides_and_empty():
    torch = torch_()
    announce("beam strides")
    for name in ("f32", "bf16", "f16"):
        wide = randn((4, 6, 2050), name, 3)
        scores = beam_scores(4, 6, 3)
        for view in (wide[:, :, :2000], wide[:, :, 3:1001], wide[:, :, 1::2], wide[::2, :, :900], wide[1:2, ::3, 5:999],
                     wide[:, 2:3, :777], wide[:, :, 8:520].transpose(0, 1), wide[:1, :1, 1:], wide.permute(2, 0, 1)[:40]):
            b, k, _ = view.shape
            check(view, beam_scores(b, k, 1), 7, what=str(view.stride()))
        check(wide[0, 0, :2000].expand(3, 4, 2000), beam_scores(3, 4, 1), 9)
        strided = torch.zeros(4, 6, 2, device="cuda")
        strided[:, :, 1] = scores
        flags = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
        flags[2] = True
        check(wide, strided[:, :, 1], 5, finished=flags.t(), end_id=9)
    for shape, count in (((0, 3, 10), 4), ((3, 2, 10), 0), ((3, 0, 10), 4)):
        s, p, t = lrs.beam_select(torch.zeros(shape, device="cuda"), torch.zeros(shape[:2], device="cuda"), count)
        assert s.shape == p.shape == t.shape == (shape[0], count)
        assert (s == -INF).all() and (p == -1).all() and (t == -1).all()
    need = lrs.lrs_beam_select(None, 0, "f32", 1 << 40, 2050, 2 << 40, None, 0, 4, 6, 2050, 7, 1, 3 << 40, 4 << 40, "i32",
                               5 << 40)
    wide = randn((4, 6, 2050), "f32", 3)
    want = check(wide, scores, 7)
    for temp in (torch.empty(need + 64, dtype=torch.uint8, device="cuda")[1:], torch.empty(3, device="cuda")):
        assert all(torch.equal(a, b) for a, b in zip(lrs.beam_select(wide, scores, 7, temp=temp), want))
    # a guard behind outputs of the C call
    outs = [torch.full((4 * 7 + 5,), 9, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int64)]
    temp = torch.empty(need, dtype=torch.uint8, device="cuda")
    lrs.lrs_beam_select(temp, need, "f32", wide, 2050, scores, None, 0, 4, 6, 2050, 7, 1, outs[0], outs[1], "i64", outs[2])
    for out, w in zip(outs, want):
        assert torch.equal(out[:28].view(4, 7), w.to(out.dtype)) and (out[28:] == 9).all()


def test_many_beams_and_many_lists():
    for batch, beams, vocab, count in ((1, 1024, 700, 64), (2, 300, 5000, 64), (5, 100, 9000, 17), (2000, 1, 300, 4)):
        announce("many %d x %d x %d" % (batch, beams, vocab))
        torch = torch_()
        scores = -torch.from_numpy(np.random.default_rng(1).random((batch, beams)).astype(np.float32)).cuda()
        check(randn((batch, beams, vocab), "bf16", beams), scores, count)


def test_logits_past_32_bits():
    """Rows beyond 2^31 elements and 2^32 bytes, and a flat index close to 2^31."""
    torch = torch_()
    announce("far logits")
    step = (1 << 31) // 5
    buffer = torch.full((step * 5 + 1200,), float("nan"), device="cuda", dtype=torch.float16)
    view = buffer.as_strided((2, 3, 1200), (3 * step, step, 1))
    view.copy_(randn((2, 3, 1200), "f16", 4))
    check(view, beam_scores(2, 3, 4), 6)
    del buffer, view
    vocab = 2**31 - 1
    logits = torch.zeros(1, 1, vocab, device="cuda", dtype=torch.float16)
    best = [vocab - 1, vocab - 70, 2**30 + 5, 5]
    for i, at in enumerate(best):
        logits[0, 0, at] = 20.0 - i
    s, p, t = lrs.beam_select(logits, torch.zeros(1, 1, device="cuda"), 6)
    assert t[0].tolist() == best + [0, 1] and (p == 0).all()
    total = math.log(sum(math.exp(20.0 - i) for i in range(4)) + vocab - 4)
    want = np.array([20.0, 19.0, 18.0, 17.0, 0.0, 0.0]) - total
    off = (2 * math.log(vocab) + 12) * 2.0**-24
    assert (np.abs(as64(s)[0] - want) <= off + np.abs(want) * 2.0**-24).all()


# ----------------------------------------------------------------- reordering


def pattern(shape, dtype, seed):
    """Random bytes, so that every bit has to arrive (NaNs among them)."""
    torch = torch_()
    g = torch.Generator("cuda").manual_seed(seed)
    size = torch.empty(0, dtype=dtype).element_size()
    return torch.randint(0, 256, (*shape, size), generator=g, device="cuda", dtype=torch.uint8).view(dtype).squeeze(-1)


def bits(t):
    torch = torch_()
    t = t.contiguous()
    return t.unsqueeze(-1).view(torch.uint8)


def reordered(states, parents, dim):
    torch = torch_()
    beams = states.shape[dim + 1]
    shape = list(states.shape)
    shape[dim + 1] = parents.shape[1]
    out = bits(torch.zeros(shape, dtype=states.dtype, device="cuda"))
    old = bits(states)
    lead = (slice(None),) * dim
    for b, row in enumerate(parents.tolist()):
        for j, p in enumerate(row):
            if 0 <= p < beams:
                out[lead + (b, j)] = old[lead + (b, p)]
    return out


def parents_of(batch, beams, count, seed, wild=False):
    torch = torch_()
    rng = np.random.default_rng(seed)
    p = rng.integers(0, max(beams, 1), (batch, count))
    if wild:
        p = np.where(rng.random(p.shape) < 0.3, rng.choice([-1, beams, -2**31, 2**31 - 1], p.shape), p)
    return torch.from_numpy(p.astype(np.int32)).cuda()


SHAPES = [(1, 4, 8, 64, 16), (3, 5, 1, 129, 65), (2, 8, 3, 7, 3), (1, 1, 1, 1, 1), (4, 2, 2, 33, 31), (2, 3, 4, 1, 5)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["uint8", "int16", "bfloat16", "float32", "int64", "complex128"])
def test_beam_reorder(shape, dtype):
    torch = torch_()
    dtype = getattr(torch, dtype)
    batch, beams = shape[:2]
    for i, count in enumerate((1, beams, 2 * beams + 3)):
        for wild in (False, True):
            announce("reorder %s %s to %d wild %s" % (shape, dtype, count, wild))
            states, parents = pattern(shape, dtype, i), parents_of(batch, beams, count, i, wild)
            before = bits(states).clone()
            got = lrs.beam_reorder(states, parents)
            assert got.dtype is dtype and torch.equal(bits(got), reordered(states, parents, 0))
            assert torch.equal(bits(states), before)
            out = pattern((batch, count, *shape[2:]), dtype, 9)
            assert lrs.beam_reorder(states, parents, out=out) is out and torch.equal(bits(out), bits(got))
            if count == beams:
                assert lrs.beam_reorder(states, parents, out=states) is states
                assert torch.equal(bits(states), bits(got))


@pytest.mark.parametrize("count", [2, 4, 5, 8, 9, 16, 17, 40, 64])
def test_reorder_in_place_by_count(count):
    """Each number of beams that a lane holds: cycles, swaps, one parent for all, no
    change, no parents, and fewer beams afterwards."""
    torch = torch_()
    rng = np.random.default_rng(count)
    rows = [np.roll(np.arange(count), 1), np.roll(np.arange(count), -1), np.arange(count)[::-1], np.arange(count),
            np.zeros(count), np.full(count, count - 1), np.full(count, -1), rng.permutation(count),
            rng.integers(-1, count + 1, count)]
    parents = torch.from_numpy(np.array(rows).astype(np.int32)).cuda()
    for width in (8, 5003):
        announce("in place %d of %d" % (count, width))
        states = pattern((len(rows), count, width), torch.int16, count)
        want = reordered(states, parents, 0)
        lrs.beam_reorder(states, parents, out=states)
        assert torch.equal(bits(states), want)
        few = count // 2
        want = bits(states).clone()
        want[:, :few] = reordered(states, parents[:, :few].contiguous(), 0)
        lrs.beam_reorder(states, parents[:, :few], out=states[:, :few])
        assert torch.equal(bits(states), want)
    # more beams afterwards than before, into the memory that begins with them: a place
    # whose number is no beam is named by none
    few = max(1, count // 2)
    for width in (8, 77):
        buffer = pattern((len(rows), count, width), torch.int16, count)
        want = reordered(buffer[:, :few], parents, 0)
        lrs.beam_reorder(buffer[:, :few], parents, out=buffer)
        assert torch.equal(bits(buffer), want)
    if count == 64:
        with pytest.raises(lrs.LrsError):
            many = pattern((1, 65, 8), torch.int16, 1)
            lrs.beam_reorder(many, parents_of(1, 65, 65, 1), out=many)
        assert torch.equal(bits(lrs.beam_reorder(many, parents_of(1, 65, 130, 1))),
                           reordered(many, parents_of(1, 65, 130, 1), 0))


def test_reorder_layouts():
    """Layers first, the filled part of a cache, dimensions turned, slices of a buffer;
    what is not part of the states stays as it was."""
    torch = torch_()
    for dim, view in ((1, lambda t: t[:, :, :, :, :37]), (1, lambda t: t[..., :9]), (1, lambda t: t[1:]),
                      (2, lambda t: t.unsqueeze(0)[:, 1:, :, :, :, 3:20]), (1, lambda t: t.transpose(3, 4)),
                      (0, lambda t: t[1, :, :, 1]), (-3, lambda t: t[0, 0]), (1, lambda t: t[:, :, :, 1:2, 5:6]),
                      (1, lambda t: t[:, :, :, :1, ::2, :1]), (1, lambda t: t[:, 2:3])):
        for dtype in (torch.bfloat16, torch.float32, torch.uint8):
            buffer = pattern((3, 4, 5, 2, 50, 24), dtype, 3)
            states = view(buffer)
            at = dim % states.dim()
            batch, beams = states.shape[at:at + 2]
            parents = parents_of(batch, beams, beams, 5, True)
            announce("layout %s %s" % (tuple(states.stride()), dtype))
            want = reordered(states, parents, at)
            assert torch.equal(bits(lrs.beam_reorder(states, parents, dim=dim)), want)
            whole, expected = buffer.clone(), buffer.clone()
            view(expected).copy_(want.view(dtype).squeeze(-1))
            lrs.beam_reorder(view(whole), parents, dim=dim, out=view(whole))
            assert torch.equal(bits(whole), bits(expected))
    # beams that share their state before the step; turned states to plain ones
    shared = pattern((2, 1, 40), torch.float32, 1).expand(2, 6, 40)
    parents = parents_of(2, 6, 6, 1)
    assert torch.equal(bits(lrs.beam_reorder(shared, parents)), reordered(shared, parents, 0))
    turned = pattern((40, 6, 2), torch.float32, 1).permute(2, 1, 0)
    out = torch.zeros(2, 6, 40, device="cuda")
    lrs.beam_reorder(turned, parents, out=out)
    assert torch.equal(bits(out), reordered(turned, parents, 0))
    with pytest.raises(lrs.LrsError):  # the memory of out is shared
        lrs.beam_reorder(out.clone(), parents, out=shared)
    with pytest.raises(lrs.LrsError):  # overlapping, and not the same
        lrs.beam_reorder(out[:, 1:], parents[:, :5], out=out[:, :5])
    for shape in ((0, 3, 4), (2, 3, 0)):
        p = torch.zeros(shape[0], 5, dtype=torch.int32, device="cuda")
        assert lrs.beam_reorder(torch.zeros(shape, device="cuda"), p).shape == (shape[0], 5, shape[2])
    none = lrs.beam_reorder(torch.zeros(2, 0, 4, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda"))
    assert none.shape == (2, 5, 4) and (none == 0).all()
    assert lrs.beam_reorder(torch.zeros(2, 3, 4, device="cuda"), parents[:, :0]).shape == (2, 0, 4)


def test_reorder_of_windows():
    """States of which two searches share some: moved into other memory, refused in place."""
    torch = torch_()
    announce("windows")
    buffer = pattern((9, 40), torch.float32, 1)
    states = buffer.as_strided((8, 2, 40), (40, 40, 1))
    parents, before = parents_of(8, 2, 1, 1), bits(buffer).clone()
    with pytest.raises(lrs.LrsError):
        lrs.beam_reorder(states, parents, out=buffer[:8].unsqueeze(1))
    assert torch.equal(bits(buffer), before)
    assert torch.equal(bits(lrs.beam_reorder(states, parents)), reordered(states, parents, 0))


@pytest.mark.parametrize("beams", [3, 8, 16, 20, 40])
@pytest.mark.parametrize("width", [7, 1001])
def test_reorder_large_states(beams, width):
    """States that are read past the caches, in rows of less than a wave and more: beams
    that share a parent in one step of the kernel's and in different ones."""
    torch = torch_()
    batch, rows = 3, 176 * 2**20 // (3 * beams * width * 4) + 1
    states = pattern((batch, beams, rows, width + 1), torch.int32, beams)[..., :width]
    for count in (beams, 2 * beams + 1):
        parents = parents_of(batch, min(beams, 6), count, beams)
        parents[1, ::3], parents[2, 1] = 0, -1
        at = parents.clamp(min=0).long()
        want = torch.stack([states[b][at[b]] for b in range(batch)]) * (parents >= 0)[:, :, None, None].int()
        announce("reorder %s to %d" % (tuple(states.shape), count))
        assert torch.equal(lrs.beam_reorder(states, parents), want)
        if count == beams:
            buffer = states.clone()
            lrs.beam_reorder(buffer, parents, out=buffer)
            assert torch.equal(buffer, want)


def test_reorder_far_states_and_many_rows():
    torch = torch_()
    announce("far states")
    step = (1 << 32) // 3
    buffer = torch.zeros(4 * step + 4096, dtype=torch.uint8, device="cuda")
    states = buffer.as_strided((2, 2, 1001), (2 * step, step, 1))
    states.copy_(pattern((2, 2, 1001), torch.uint8, 3))
    parents = torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device="cuda")
    want = reordered(states, parents, 0)
    assert torch.equal(bits(lrs.beam_reorder(states, parents)), want)
    lrs.beam_reorder(states, parents, out=states)
    assert torch.equal(bits(states), want)
    del buffer, states
    many = pattern((70001, 2, 3), torch.int16, 1)  # more searches than a grid has rows
    parents = parents_of(70001, 2, 2, 1)
    want = torch.gather(many, 1, parents.long()[:, :, None].expand(-1, -1, 3))
    assert torch.equal(lrs.beam_reorder(many, parents), want)
    many = pattern((70001, 2, 600), torch.int16, 1)
    want = torch.gather(many, 1, parents.long()[:, :, None].expand(-1, -1, 600))
    lrs.beam_reorder(many, parents, out=many)
    assert torch.equal(many, want)


def test_reorder_of_as_many_rows_as_there_may_be():
    """2^31 - 1 rows of a byte: the grid that covers them is one more than an int counts."""
    torch = torch_()
    announce("2^31 - 1 rows")
    rows = 2**31 - 1
    states = torch.arange(251, device="cuda", dtype=torch.uint8).repeat(2 * rows // 251 + 1)[:2 * rows]
    states = states.view(1, 1, rows, 2)[..., 1:]
    got = lrs.beam_reorder(states, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    assert got.shape == states.shape and got.is_contiguous() and torch.equal(got, states)
    with pytest.raises(lrs.LrsError):
        lrs.beam_reorder(states.as_strided((1, 1, rows + 1, 1), (1, 1, 0, 1)),
                         torch.zeros(1, 1, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------- used together


def search_step(s, stream=None):
    """One step of a search as a program runs it: the best continuations, the sequences
    so far and the caches in their order, finished flags."""
    scores, parents, tokens = lrs.beam_select(s["logits"], s["scores"], s["count"], finished=s["done"], end_id=1,
                                              stream=stream)
    lrs.beam_reorder(s["cache"], parents, dim=1, out=s["cache"], stream=stream)
    lrs.beam_reorder(s["tokens"], parents, out=s["tokens"], stream=stream)
    done = lrs.beam_reorder(s["done"], parents, stream=stream)
    return scores, parents, tokens, done


def search_state(batch, beams, vocab, seed):
    torch = torch_()
    g = torch.Generator("cuda").manual_seed(seed)
    return {"logits": torch.randn(batch, beams, vocab, generator=g, device="cuda").bfloat16(),
            "scores": -torch.rand(batch, beams, generator=g, device="cuda"), "count": beams,
            "done": torch.rand(batch, beams, generator=g, device="cuda") < 0.2,
            "cache": torch.randn(2, batch, beams, 4, 33, 16, generator=g, device="cuda").half(),
            "tokens": torch.randint(0, vocab, (batch, beams, 19), generator=g, device="cuda")}


def test_search_against_a_plain_one():
    """Eight steps of four searches, against the same in numpy with whole sequences."""
    torch = torch_()
    announce("search")
    batch, beams, vocab, steps, end = 4, 3, 40, 8, 1
    table = randn((vocab, vocab), "f32", 1)  # the logits of a token's successors
    tokens = torch.zeros(batch, beams, steps + 1, dtype=torch.int64, device="cuda")
    tokens[:, :, 0] = torch.arange(batch, device="cuda")[:, None] + 2
    scores = torch.full((batch, beams), -INF, device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
    plain = [[(0.0, [b + 2], False)] for b in range(batch)]
    t64 = as64(table)
    logp = t64 - np.log(np.exp(t64).sum(1, keepdims=True))
    for step in range(steps):
        logits = table[tokens[:, :, step]]
        scores, parents, chosen = lrs.beam_select(logits, scores, beams, finished=done, end_id=end, dtype=torch.int64)
        lrs.beam_reorder(tokens, parents, out=tokens)
        tokens[:, :, step + 1] = chosen
        done = lrs.beam_reorder(done, parents) | (chosen == end)
        for b in range(batch):
            new = []
            for i, (s, seq, over) in enumerate(plain[b]):
                if over:
                    new.append((s, i, end, seq + [end]))
                else:
                    new += [(s + logp[seq[-1], v], i, v, seq + [v]) for v in range(vocab)]
            new.sort(key=lambda x: (-x[0], x[1], x[2]))
            plain[b] = [(s, seq, seq[-1] == end) for s, _, _, seq in new[:beams]]
            assert tokens[b, :, :step + 2].tolist() == [seq for _, seq, _ in plain[b]], (step, b)
            # each step adds one rounding of the score and one of the logarithm
            off = (step + 1) * ((2 * math.log(vocab) + 12) * 2.0**-24 + 40 * 2.0**-24)
            assert np.allclose(as64(scores)[b], [s for s, _, _ in plain[b]], rtol=0, atol=off)


def test_search_captured_and_on_other_streams():
    torch = torch_()
    announce("captured search")
    sizes = ((2, 4, 3000), (9, 8, 40000))
    states, graphs, outs = [search_state(*size, 1) for size in sizes], [], []
    names = ("logits", "scores", "done", "cache", "tokens")
    for s in states:
        search_step(s)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(search_step(s))
    for rep in range(3):
        new = [search_state(*size, 10 + rep) for size in sizes]
        for s, other, graph in zip(states, new, graphs):
            for name in names:
                s[name].copy_(other[name])
            graph.replay()
        want = [search_step(other) for other in new]
        torch.cuda.synchronize()
        for got, expected, s, other in zip(outs, want, states, new):
            assert all(torch.equal(a, b) for a, b in zip(got, expected)), rep
            assert torch.equal(s["cache"], other["cache"]) and torch.equal(s["tokens"], other["tokens"]), rep
    side, big = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda")
    for stream in (side, side.cuda_stream):
        fresh = search_state(*sizes[0], 30)
        late = {n: torch.zeros_like(fresh[n]) if n in names else fresh[n] for n in fresh}
        want_state = {n: fresh[n].clone() if n in names else fresh[n] for n in fresh}
        want = search_step(want_state)
        torch.cuda.synchronize()
        for _ in range(4):
            big @ big
        for n in names:
            late[n].copy_(fresh[n])
        got = search_step(late, stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(late["cache"], want_state["cache"]) and torch.equal(late["tokens"], want_state["tokens"])


def test_reorder_counts_as_a_write():
    torch = torch_()
    announce("reorder versions")
    states, parents = torch.zeros(2, 3, 8, device="cuda"), parents_of(2, 3, 3, 1)
    y = (torch.ones(2, 3, 8, device="cuda", requires_grad=True) * states).sum()
    lrs.beam_reorder(states, parents, out=states)
    assert states._version == 1 and parents._version == 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_served_batch_and_many_searches():
    """Rows of several parts with the largest number of vectors a lane, and more searches
    than a grid has workgroups in one step."""
    torch = torch_()
    announce("served batch")
    for name in ("bf16", "f32"):
        done = torch.from_numpy(np.random.default_rng(3).random((16, 8)) < 0.2).cuda()
        check(randn((16, 8, 128257), name, 1), beam_scores(16, 8, 1), 16, finished=done, end_id=7)
    many = (1 << 20) + 5
    announce("many searches")
    logits, scores = randn((many, 1, 5), "f32", 2), beam_scores(many, 1, 2)
    s, p, t = lrs.beam_select(logits, scores, 2)
    want = torch.topk(logits[:, 0].double(), 2, dim=1)  # (no two of these are equal)
    assert torch.equal(t.long(), want.indices) and (p == 0).all()
    total = torch.log_softmax(logits[:, 0].double(), 1).gather(1, want.indices) + scores.double()
    off = (2 * math.log(5) + 12) * 2.0**-24
    assert ((s.double() - total).abs() <= off + (total.abs() + off) * 2.0**-24).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_large_logits(name):
    """Logits whose product with log2(e) no float32 holds, beside small ones in other parts."""
    torch = torch_()
    announce("large logits %s" % name)
    logits = randn((4, 2, 20011), name, 5)
    logits[0, 0, 17000] = 3e38
    logits[1, 1, 3] = 2.9e38
    logits[1, 1, 19000] = 3e38
    logits[2] = -3e38
    logits[2, :, 40] = -2.9e38
    logits[3, 0] *= 1e37
    for normalize in (True, False):
        check(logits, beam_scores(4, 2, 1), 9, normalize)


def test_calls_at_once():
    """Calls on two streams at the same time, each with its own tensors, and temp storage
    that is not one block."""
    torch = torch_()
    announce("two streams at once")
    sizes = ((3, 4, 50001), (40, 8, 3001))
    new = [search_state(*size, 40 + i) for i, size in enumerate(sizes)]
    states = [{n: v.clone() if n != "count" else v for n, v in s.items()} for s in new]
    want = []
    for s in new:
        want.append([search_step(s) for _ in range(4)])
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(search_step(states[i]))
    torch.cuda.synchronize()
    for a, b, s, other in zip(got, want, states, new):
        assert all(torch.equal(x, y) for one, two in zip(a, b) for x, y in zip(one, two))
        assert torch.equal(s["cache"], other["cache"]) and torch.equal(s["tokens"], other["tokens"])
    with pytest.raises(ValueError, match="temp must be contiguous"):
        lrs.beam_select(states[0]["logits"], states[0]["scores"], 4,
                        temp=torch.zeros(4096, 4096, dtype=torch.uint8, device="cuda")[:, :2048])
