"""Tensors that torch conjugates or negates when they are read: calls on them give what
calls on copies of their values give."""
from __future__ import annotations

import pytest

import sorting_lsd_radix_sort_amd as lrs
from gpu_util import announce

pytestmark = pytest.mark.gpu


def torch_():
    import torch
    return torch


def negated(*shape, seed=1):
    """Imaginary parts of a conjugate: a view of the negatives."""
    torch = torch_()
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.complex64).conj().imag
    assert t.is_neg()
    return t


def same(got, want):
    torch = torch_()
    got, want = ((x,) if torch.is_tensor(x) else x for x in (got, want))
    for a, b in zip(got, want):
        assert not a.is_neg() and not a.is_conj() and torch.equal(a, b)


@pytest.mark.parametrize("cols", [1, 5])
def test_negated_values(cols):
    torch = torch_()
    announce("negated values, %d columns" % cols)
    x, w = negated(6, cols), negated(6, 1, seed=2)
    dense = torch._neg_view(torch.randn(6, cols, device="cuda"))  # (next to each other)
    ids = torch.arange(6, device="cuda", dtype=torch.int32)[:, None]
    for v in (x, dense):
        p = v.clone()
        assert not p.is_neg()
        same(lrs.sort_keys(v), lrs.sort_keys(p))
        values = torch.arange(6 * cols, device="cuda", dtype=torch.int32).view(torch.uint32).view(6, cols)
        for a, b in zip(lrs.sort_pairs(v, values), lrs.sort_pairs(p, values)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))
        same(lrs.dispatch_rows(v, ids), lrs.dispatch_rows(p, ids))
        same(lrs.combine_rows(v, ids, w), lrs.combine_rows(p, ids, w.clone()))
        same(lrs.combine_rows_grad(v, v, ids, w), lrs.combine_rows_grad(p, p, ids, w.clone()))
        same(lrs.embedding(v, ids), lrs.embedding(p, ids))
        same(lrs.embedding_grad(v, ids[:, 0], 6), lrs.embedding_grad(p, ids[:, 0], 6))
        for bias in (None, negated(cols, seed=3), torch._neg_view(torch.randn(cols, device="cuda"))):
            same(lrs.route_tokens(v, 1, "sigmoid", bias=bias, normalize=False),
                 lrs.route_tokens(p, 1, "sigmoid", bias=None if bias is None else bias.clone(), normalize=False))
        at = torch.zeros_like(ids)
        same(lrs.route_tokens_grad(w, v, at, "sigmoid", normalize=False),
             lrs.route_tokens_grad(w.clone(), p, at, "sigmoid", normalize=False))
        scores = torch._neg_view(torch.rand(3, 2, device="cuda"))
        same(lrs.beam_select(v.view(3, 2, cols), scores, 2), lrs.beam_select(p.view(3, 2, cols), scores.clone(), 2))


def test_one_negated_value():
    torch = torch_()
    announce("one negated value")
    x = negated(1)
    same(lrs.sort_keys(x), x.clone())
    l, s = negated(1, 2, 3), negated(1, 1)
    same(lrs.beam_select(l[:, :1, :1], s, 1, normalize=False), lrs.beam_select(l[:, :1, :1].clone(), s.clone(), 1,
                                                                              normalize=False))


def test_beam_reorder_of_lazy_views():
    torch = torch_()
    announce("lazy states")
    z = torch.randn(3, 4, 5, 7, device="cuda", dtype=torch.complex64)
    parents = torch.tensor([[1, 0, 3, 3], [2, 2, 2, 2], [0, 1, 2, -1]], dtype=torch.int32, device="cuda")
    at = parents.clamp(min=0).long()
    for states in (z.conj(), z.conj()[..., 1:6], z.conj().transpose(2, 3), z.imag, z.conj().imag, z.conj().real, z,
                   torch._neg_view(z.real.contiguous()), torch._neg_view(z).conj(), z.conj().unsqueeze(2)):
        plain = states.clone()
        want = torch.stack([plain[b][at[b]] for b in range(3)])
        want[2, 3] = 0
        same(lrs.beam_reorder(states, parents), want)
        out = torch.empty_like(want)
        assert lrs.beam_reorder(states, parents, out=out) is out
        same(out, want)
        # in place: the same view on both sides
        again = states.clone()
        again = torch._neg_view(again) if states.is_neg() else again
        again = again.conj() if states.is_conj() else again
        before = again.clone()
        assert lrs.beam_reorder(again, parents, out=again) is again
        want = torch.stack([before[b][at[b]] for b in range(3)])
        want[2, 3] = 0
        assert torch.equal(again, want)
    base = z.clone()
    want = torch.stack([z.conj()[b][at[b]] for b in range(3)]).resolve_conj()
    want[2, 3] = 0
    lrs.beam_reorder(base.conj(), parents, out=base)  # of one memory, read in two ways
    same(base, want)
