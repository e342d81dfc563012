"""The distillation loss's rest entry where nothing is left for it: lists of the whole vocabulary,
students that mask everything else; and rows without a loss whose gradient overwrites them."""
import pytest
import torch

import distill_ref as D
import student_ref as R
from test_gpu_distill_mass import all_ways, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (50, 50), (300, 300), (1000, 1024)])
def test_whole_vocabulary_listed(ops, dtype, V, K):  # noqa: F811
    N = 30
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.argsort(torch.rand(N, V, generator=g, device="cuda"), dim=1)
    top = 3 * torch.randn(N, V, generator=g, device="cuda")
    lse = torch.logsumexp(top, 1)
    if K > V:                               # tokens sent twice, with what the first entry leaves, and padding
        top[:, :10] -= 1.0
        extra = top[:, :10] + torch.log(torch.expm1(torch.ones((), device="cuda")))
        index = torch.cat([index, index[:, :10], torch.full((N, K - V - 10), -1, device="cuda")], 1)
        top = torch.cat([top, extra, torch.zeros(N, K - V - 10, device="cuda")], 1)
    z = 2 * torch.randn(N, V, generator=g, device="cuda")
    k = dict(logits=z.to(dtype), index=index, top=top, top_lse=lse)
    loss, d = all_ways(ops, k)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(d).all())
    k["top_lse"] = lse + 0.25               # mass is missing, and there is nowhere to have it
    loss, d = all_ways(ops, k)
    assert bool((loss == INF).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [400, 40000, 600000])
def test_student_masks_what_is_not_listed(ops, dtype, V):  # noqa: F811
    """Rounding is no mass; what the teacher has there in earnest makes the loss infinite."""
    N, K = 12, 40
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)])
    top = 10.0 + 3 * torch.randn(N, K, generator=g, device="cuda")
    z = torch.full((N, V), -INF, device="cuda")
    z.scatter_(1, index, top + torch.randn(N, K, generator=g, device="cuda"))
    lse = torch.logsumexp(top.double(), 1).float()
    k = dict(logits=z.to(dtype), index=index, top=top, top_lse=lse)
    loss, d = all_ways(ops, k)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(d).all())
    k["top_lse"] = lse + 0.01
    loss, d = all_ways(ops, k)
    assert bool((loss == INF).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("V", [2000, 70000])
def test_rows_without_a_loss_in_place(ops, V):  # noqa: F811
    """Rows that a long list says nothing about, or of weight 0, become zeros over their logits."""
    N, K = 700, 200
    g = torch.Generator(device="cuda").manual_seed(V)
    z = 2 * torch.randn(N, V, generator=g, device="cuda")
    index = torch.randint(0, V, (N, K), generator=g, device="cuda")
    index[::3] = V + 7                      # wholly outside the vocabulary
    top = torch.randn(N, K, generator=g, device="cuda")
    top[1::6] = -INF
    weight = torch.where(torch.rand(N, generator=g, device="cuda") < 0.2, 0.0, 1.0)
    k = dict(logits=z.to(BF16), index=index, top=top, weight=weight)
    loss, d = ops.distill_loss_grad(**k)
    few = dict(logits=k["logits"][:24], index=index[:24], top=top[:24], weight=weight[:24])
    want = D.distill(**few)
    R.check(loss[:24], want["loss"])
    R.check(d[:24], want["dlogits"])
    again = ops.distill_loss_grad(**k, out=k["logits"])
    assert torch.equal(again[0], loss) and torch.equal(again[1], d)
    dead = torch.zeros(N, dtype=torch.bool, device="cuda")
    dead[::3] = True
    dead[1::6] = True
    dead |= weight == 0
    assert not d[dead].any() and not loss[dead].any() and bool((loss[~dead] != 0).all())
