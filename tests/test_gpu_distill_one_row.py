"""A single row of logits, or a vocabulary of one token, with whatever strides torch gives axes of
length one."""
import pytest
import torch

import student_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def ops():
    from error_compensated_bit_gb300 import build, ops as mod
    build.build()
    return mod


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead", [(1,), (1, 1), (1, 1, 1)])
@pytest.mark.parametrize("V", [1, 333, 40001, 600001])
def test_in_place(ops, dtype, lead, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    wide = torch.randn(*lead, V + 7, generator=g, device="cuda").to(dtype)
    index = torch.randint(0, V, (*lead, 3), generator=g, device="cuda")
    top = torch.randn(*lead, 3, generator=g, device="cuda")
    z = wide[..., 3:3 + V]
    want = R.distill(z.reshape(1, V), index.view(1, 3), top.view(1, 3))
    around = torch.cat([wide[..., :3], wide[..., 3 + V:]], -1)
    loss, d = ops.distill_loss_grad(z, index, top, out=z)
    assert d is z
    R.check(loss.view(1), want["loss"], "loss")
    R.check(d.reshape(1, V), want["dlogits"], "dlogits")
    assert torch.equal(torch.cat([wide[..., :3], wide[..., 3 + V:]], -1), around)


def test_one_token(ops):
    wide = torch.randn(9, 4, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    index, top = torch.zeros(9, 1, dtype=torch.int64, device="cuda"), torch.ones(9, 1, device="cuda")
    for z in (wide[:, 1:2], wide[:, :1], wide.t()[2:3].t()):
        want = R.distill(z, index, top)
        loss, d = ops.distill_loss_grad(z, index, top, out=z)
        R.check(loss, want["loss"], "loss")
        R.check(d, want["dlogits"], "dlogits")
