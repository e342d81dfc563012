"""Decays of the scan down to float32's smallest numbers: memories without end, whose gradients by
the gate and the decay are still those of the formulas."""
import pytest
import torch

from test_gpu_scan import compare, inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 33])
def test_tiny_decays(ops, dtype, D):  # noqa: F811
    k = inputs(2, 100, D, dtype, seed=60, state=True, resets=0.02, grads=True)
    k["decay"] = torch.logspace(-44, -20, D, dtype=torch.float64).float().cuda()
    out = compare(ops, k)
    assert bool((out["dr"] != 0).any(dim=(0, 1)).all())


@pytest.mark.parametrize("D", [64, 33])
def test_huge_decays_behind_shut_gates(ops, D):  # noqa: F811
    """decay * s(r) of ordinary size from factors up to 1e28 and down to 1e-28."""
    k = inputs(2, 100, D, F32, seed=61, state=True, resets=0.02, grads=True)
    k["decay"] = torch.logspace(0, 28, D, dtype=torch.float64).float().cuda()
    k["r"] = k["r"] - torch.log(k["decay"])
    compare(ops, k)
