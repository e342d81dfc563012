"""The distillation loss on the GPU where the teacher's listed mass is above 1 (its top logits
rounded to 16 bits beside the log-sum-exp of the unrounded ones)."""
import pytest
import torch

import distill_ref as D
import student_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def ops():
    from error_compensated_bit_gb300 import build, ops as mod
    build.build()
    return mod


def all_ways(ops, k):
    """The fused call, in place too, the loss alone and the autograd pair, against the formulas."""
    want = D.distill(**k)
    loss, d = ops.distill_loss_grad(**k)
    R.check(loss, want["loss"], "fused loss")
    R.check(d, want["dlogits"], "fused dlogits")
    R.check(ops.distill_loss(**k), want["loss"], "loss alone")
    z = k["logits"].detach().clone().requires_grad_(True)
    up = torch.linspace(-1.0, 2.0, z.shape[0], device="cuda")
    got = ops.distill_loss(**{**k, "logits": z})
    R.check(got, want["loss"], "loss")
    R.check(torch.autograd.grad(got, z, up)[0], D.distill(**k, dloss=up)["dlogits"], "dlogits")
    z = k["logits"].clone()
    same = ops.distill_loss_grad(**{**k, "logits": z}, out=z)
    assert torch.equal(same[0], loss) and torch.equal(z, d), "in place"
    return loss, d


def peaked(N, V, K, dtype, seed, top_dtype=BF16, tau=1.0, shift=0.0):
    """A teacher that holds nearly all of its mass in its list, and a student near it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.randn(N, V, generator=g, device="cuda")
    full[:, 5:5 + K] += 18.0 * tau + torch.randn(N, K, generator=g, device="cuda")
    top, index = torch.topk(full, K, dim=1)
    z = full + 0.1 * torch.randn(N, V, generator=g, device="cuda")
    return dict(logits=z.to(dtype), index=index, top=top.to(top_dtype), top_lse=torch.logsumexp(full / tau, 1) + shift,
                temperature=tau)


def mass_of(k):
    return torch.exp(k["top"].double() / k["temperature"] - k["top_lse"].double()[:, None]).sum(1)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("N,V,K,tau", [(12, 3001, 24, 1.0), (9, 32000, 64, 1.0), (12, 50257, 20, 2.0), (40, 1000, 200, 1.0)])
def test_rounded_teacher(ops, dtype, N, V, K, tau):
    k = peaked(N, V, K, dtype, seed=V, tau=tau)
    mass = mass_of(k)
    assert bool((mass > 1).any()) and bool((mass < 1).any())
    all_ways(ops, k)


@pytest.mark.parametrize("V,dtype", [(131072, BF16), (500009, F32)])
def test_rounded_teacher_of_long_rows(ops, V, dtype):
    """Rows over a cluster, and rows that no cluster holds."""
    all_ways(ops, peaked(4, V, 50, dtype, seed=3, top_dtype=F16, shift=-0.02))


def test_masses_far_above_one(ops):
    k = peaked(5, 700, 10, F32, seed=4, top_dtype=F32)
    k["top_lse"] -= torch.tensor([0.0, 0.3, 1.0, 3.0, 6.0], device="cuda")
    k["weight"] = torch.tensor([1.0, 0.5, 0.0, 2.0, 1e-3], device="cuda")
    k["index"][3, 4] = k["index"][3, 1]         # a token listed twice
    k["index"][4, 2] = -1
    all_ways(ops, k)


def test_gradient_sums_to_zero(ops):
    """A constant added to all logits changes no loss."""
    k = peaked(64, 2000, 30, F32, seed=5)
    assert bool((mass_of(k) > 1.001).any())
    _, d = ops.distill_loss_grad(**k)
    bound = D.distill(**k)["dlogits"][1].sum(1)
    assert bool((d.double().cpu().sum(1).abs() <= bound).all())


def test_differences(ops):
    """The gradient along a direction against central differences of the kernel's own loss."""
    k = peaked(8, 900, 12, F32, seed=6, shift=-0.1)
    assert bool((mass_of(k) > 1).all())
    step = 0.05
    _, d = ops.distill_loss_grad(**k)
    exact = D.distill(**k)
    v = torch.randn(k["logits"].shape, generator=torch.Generator().manual_seed(6)).cuda()
    hi, lo = k["logits"] + step * v, k["logits"] - step * v
    moved = (hi.double() - lo.double()).cpu()
    diff = (ops.distill_loss(**{**k, "logits": hi}).double() - ops.distill_loss(**{**k, "logits": lo}).double()).cpu()
    a, b = D.distill(**{**k, "logits": hi})["loss"], D.distill(**{**k, "logits": lo})["loss"]
    truncation = ((a[0] - b[0]) - (exact["dlogits"][0] * moved).sum(1)).abs()
    bound = truncation + a[1] + b[1] + (exact["dlogits"][1] * moved.abs()).sum(1)
    assert bool(((diff - (d.double().cpu() * moved).sum(1)).abs() <= bound).all())
