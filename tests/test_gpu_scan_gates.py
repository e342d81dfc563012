"""Gates of the scan far beyond where the logistic function's exponential overflows."""
import pytest
import torch

import student_ref as R
from test_gpu_scan import forward_backward, inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16

# A logistic value below float32's smallest number, 2^-149, may come out as 0: sqrt(1 - a^2) is then off by up to
# sqrt(2 * 0.9 * 2^-149) = 5e-23, with |x| < 6 and gradients below 30 less than 1e-20 in any result.
SHUT = 1e-20


def gate_values(n, dtype):
    v = torch.cat([torch.linspace(-2000.0, -60.0, n // 2), -torch.logspace(2.0, 38.5, n // 4),
                   torch.linspace(60.0, 2000.0, n // 8), torch.logspace(2.0, 38.5, n // 8)])
    return v.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max).to(dtype).cuda()


def check(got, want, name):
    R.check(got, (want[0], want[1] + SHUT), name)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("which", ["r", "i"])
def test_far_gates(ops, dtype, which):  # noqa: F811
    k = inputs(2, 128, 64, dtype, seed=40, state=True, grads=True)
    v = gate_values(128 * 64, dtype)
    k[which][0] = v.view(128, 64)
    k[which][1] = v.view(64, 128).t()
    want = R.scan(**k, backward=True)
    for name, got in forward_backward(ops, k).items():
        check(got, want[name], name)
        assert bool(torch.isfinite(got).all()), name


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D", [64, 33])
def test_far_gates_of_a_step(ops, dtype, D):  # noqa: F811
    k = inputs(64, 1, D, dtype, seed=41, state=True)
    v = gate_values(64 * 64, dtype)[:64 * D]
    k["r"][:, 0] = v.view(64, D)
    k["i"][:, 0] = v.flip(0).view(64, D)
    h = k["h0"].clone()
    want = R.scan(**k)
    y = ops.gated_scan_step(k["x"][:, 0], k["r"][:, 0], k["i"][:, 0], k["decay"], h)
    check(h, want["h"], "h")
    check(y[:, None], want["y"], "y")
