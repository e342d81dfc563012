"""Pins of tests/distill_ref.py: against torch's own differentiation of the loss with its clamped
rest entry, on both sides of a listed mass of 1, and against tests/student_ref.py below it."""
import pytest
import torch

import distill_ref as D
import student_ref as R


def teacher(N=6, V=40, K=7, shift=0.0, seed=1):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, dtype=torch.float64, generator=g)
    full = 3 * torch.randn(N, V, dtype=torch.float64, generator=g)
    top, index = torch.topk(full, K, dim=1)
    return z, index, top, torch.logsumexp(full / 1.7, 1) + shift


def loss_of(z, index, top, lse, tau):
    lq = torch.log_softmax(z / tau, 1)
    p = torch.exp(top / tau - lse[:, None])
    listed = torch.zeros(z.shape, dtype=torch.bool).scatter_(1, index, True)
    rest = (1 - p.sum(1)).clamp(min=0)
    qrest = torch.exp(lq).masked_fill(listed, 0.0).sum(1)
    loss = (p * (torch.log(p) - torch.gather(lq, 1, index))).sum(1)
    return loss + torch.where(rest > 0, rest * (torch.log(rest.clamp(min=1e-300)) - torch.log(qrest)),
                              torch.zeros_like(rest))


@pytest.mark.parametrize("shift", [-2.0, -0.5, 0.0, 0.5])
def test_gradient_is_that_of_the_loss(shift):
    z, index, top, lse = teacher(shift=shift)
    z.requires_grad_(True)
    up = torch.rand(6, dtype=torch.float64)
    loss = loss_of(z, index, top, lse, 1.7)
    want = torch.autograd.grad((loss * up).sum(), z)[0]
    mass = torch.exp(top / 1.7 - lse[:, None]).sum(1)
    assert shift >= 0 or bool((mass > 1).all())
    got = D.distill(z, index, top, lse, 1.7, dloss=up)
    assert torch.allclose(got["loss"][0], loss, atol=1e-12)
    assert torch.allclose(got["dlogits"][0], want, atol=1e-12)
    assert float(got["dlogits"][0].sum(1).abs().max()) < 1e-12, "adding a constant to the logits changes nothing"


@pytest.mark.parametrize("rest", [False, True])
def test_agrees_with_the_formulas_below_a_mass_of_one(rest):
    z, index, top, lse = teacher(shift=0.1)
    R.HALF_ULP[torch.float64] = R.TINY[torch.float64] = 0.0
    a, b = (f(z, index, top, lse if rest else None, 1.7) for f in (D.distill, R.distill))
    for name in a:
        assert torch.allclose(a[name][0], b[name][0], atol=1e-12), name


def test_a_list_of_everything():
    """Rounding leaves nothing for the rest entry; what the log-sum-exp says is missing is infinitely
    far from a student without a token there."""
    z, _, _, _ = teacher(V=9)
    top = torch.randn(6, 9, dtype=torch.float64)
    index = torch.arange(9).expand(6, 9)
    for shift in (-1e-7, 0.0, 1e-7):
        got = D.distill(z, index, top, torch.logsumexp(top, 1) + shift)
        p = torch.exp(top - torch.logsumexp(top, 1, keepdim=True) - shift)
        assert torch.allclose(got["loss"][0], (p * (torch.log(p) - torch.log_softmax(z, 1))).sum(1), atol=1e-12)
        assert torch.allclose(got["dlogits"][0], p.sum(1, keepdim=True) * torch.softmax(z, 1) - p, atol=1e-12)
    assert bool((D.distill(z, index, top, torch.logsumexp(top, 1) + 0.3)["loss"][0] == float("inf")).all())


def test_rows_at_one_value():
    """A constant added to a row changes nothing, also where it is the type's lowest value."""
    z, index, top, _ = teacher()
    flat = torch.zeros_like(z)
    for value in (-1e9, -1e30, -3.4028235e38, 1e30):
        a, b = D.distill(flat + value, index, top), D.distill(flat, index, top)
        assert torch.equal(a["loss"][0], b["loss"][0]) and torch.equal(a["dlogits"][0], b["dlogits"][0])
