"""The distillation loss on the GPU on rows of huge or of the types' lowest values: a constant
added to a row of logits, or to a teacher's list, changes nothing."""
import pytest
import torch

import distill_ref as D
import student_ref as R
from test_gpu_distill_mass import all_ways, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


def inputs(N, V, K, dtype, rest, tau):
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)])
    top = torch.randn(N, K, generator=g, device="cuda")
    k = dict(logits=torch.zeros(N, V, dtype=dtype, device="cuda"), index=index, top=top, temperature=tau)
    if rest:
        k["top_lse"] = torch.logsumexp(top / tau, 1) + 0.3
    return k


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [9, 1000, 40001, 700001])
@pytest.mark.parametrize("rest,tau", [(False, 1.0), (True, 1.0), (True, 0.01), (False, 30.0)])
def test_rows_at_one_value(ops, dtype, V, rest, tau):  # noqa: F811
    k = inputs(7, V, 5, dtype, rest, tau)
    lowest = torch.finfo(dtype).min
    for n, value in enumerate((lowest, -lowest, 1e4, -3e4, -1e9, 1e18, -1e30)):
        k["logits"][n] = max(lowest, min(-lowest, value))
    loss, d = all_ways(ops, k)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1000, 40001, 700001])
def test_rows_mostly_at_a_mask(ops, dtype, V):  # noqa: F811
    """Masks of the lowest value beside -infinity or beside logits, whether listed or not; parts of
    a row (that different warps and blocks sum) at different huge values."""
    lowest = torch.finfo(dtype).min
    k = inputs(8, V, 5, dtype, False, 1.0)
    z, idx = k["logits"], k["index"]
    z[:] = torch.randn(z.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    z[0] = lowest
    z[0, 7] = 1.5                           # all but one token, which is listed
    idx[0] = torch.tensor([7, -1, -1, -1, -1])
    z[1] = lowest
    z[1, ::2] = -INF
    idx[1] = torch.tensor([2 * 100 + 1, 1, 3, 5, 7])
    z[2, : V // 2] = lowest                 # the masked half holds the list's tokens but one
    idx[2] = torch.tensor([V - 1, -1, -1, -1, -1])
    z[3] = -1e30
    z[3, V // 3:] = -2e30
    idx[3] = torch.arange(5)
    z[4] = lowest
    z[4, V // 2:] = lowest / 2
    idx[4] = V - 1 - torch.arange(5)
    z[5] = -INF
    z[5, 11:17] = lowest
    idx[5] = torch.arange(11, 16)
    z[6] = 1e30
    z[6, 13] = -1e30
    idx[6] = torch.arange(5)
    loss, d = all_ways(ops, k)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("V,dtype", [(500, F32), (40001, BF16)])
def test_huge_but_distinct_logits(ops, V, dtype):  # noqa: F811
    """The largest logit takes everything; the loss of the others is their distance."""
    k = inputs(6, V, 5, dtype, False, 1.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    for n, scale in enumerate((1e7, 1e9, 1e11, 1e15, 1e25, 1e35)):
        k["logits"][n] = (scale * torch.randn(V, generator=g, device="cuda")).to(dtype)
    all_ways(ops, k)


@pytest.mark.parametrize("tau", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("top_dtype", [F32, F16, BF16])
def test_teachers_at_one_value(ops, tau, top_dtype):  # noqa: F811
    """A teacher's list at any one value, its type's lowest too, is the uniform distribution."""
    k = inputs(5, 3000, 6, F32, False, tau)
    k["logits"] = torch.randn(5, 3000, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    k["top"] = torch.zeros(5, 6, dtype=top_dtype, device="cuda")
    flat = ops.distill_loss_grad(**k)
    lowest = torch.finfo(top_dtype).min
    for n, value in enumerate((lowest, -lowest, lowest / 2, 5.0, -0.1)):
        k["top"][n] = value
    loss, d = all_ways(ops, k)
    assert torch.equal(loss, flat[0]) and torch.equal(d, flat[1])
    k["top"][:, 3:] = -INF
    all_ways(ops, k)
    k["top"][:, :2] = lowest                # one entry far above the others
    k["top"][:, 2] = 0.0
    loss, _ = all_ways(ops, k)
    R.check(loss, D.distill(k["logits"], k["index"][:, 2:3], k["top"][:, 2:3], temperature=tau)["loss"])
