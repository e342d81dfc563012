"""What crosses a reset in the gated scan: nothing, a NaN gate included, forward and backward."""
import pytest
import torch

from test_gpu_scan import forward_backward, inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")

# one-tile items of few chains; whole chains a block (on 152 SMs); runs of tiles; single channels
SHAPES = [(2, 700, 66, F32), (3, 700, 130, BF16), (2, 700, 33, F16), (5, 300, 3200, BF16), (20, 700, 1024, BF16),
          (17, 400, 641, F16)]


def poisoned(k, row, at, channel, what="r"):
    q = dict(k)
    q[what] = k[what].clone()
    q[what][row, at, channel] = NAN
    return q


@pytest.mark.parametrize("B,T,D,dtype", SHAPES)
@pytest.mark.parametrize("begin,at,reset", [(0, 3, 40), (2, 3, 5), (0, 20, 121), (10, 100, 129), (0, 130, 255), (62, 63, 64),
                                            (0, 127, 128), (0, 5, 390), (131, 200, 250), (66, 80, 125)])
def test_a_nan_gate_stays_in_its_sequence(ops, B, T, D, dtype, begin, at, reset):  # noqa: F811
    """Everything outside the sequence, and every other channel and row, has the bits that it has
    without the NaN."""
    if reset >= T:
        pytest.skip("the row is shorter")
    k = inputs(B, T, D, dtype, seed=30, state=True, resets=0.004, grads=True)
    row, channel = B - 1, D - 2
    k["reset"][row, :] = False
    k["reset"][row, [begin, reset]] = True      # the sequence is begin .. reset - 1
    clean = forward_backward(ops, k)
    bad = forward_backward(ops, poisoned(k, row, at, channel))
    hurt = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    hurt[row, at:reset, channel] = True
    assert bool(torch.isnan(bad["y"][hurt]).all()) and torch.equal(bad["y"][~hurt], clean["y"][~hurt])
    assert torch.equal(bad["h"], clean["h"]) and torch.equal(bad["dh0"], clean["dh0"])
    hurt[row, begin:reset, channel] = True      # backward the sequence's start is reached too
    for name in ("dx", "dr", "di"):
        assert torch.equal(bad[name][~hurt], clean[name][~hurt]), name
        assert bool(torch.isnan(bad[name][row, at, channel])), name
    other = torch.arange(D, device="cuda") != channel
    assert torch.equal(bad["ddecay"][other], clean["ddecay"][other]) and bool(torch.isnan(bad["ddecay"][channel]))


@pytest.mark.parametrize("B,T,D,dtype", SHAPES)
def test_nan_gates_everywhere_but_in_one_sequence(ops, B, T, D, dtype):  # noqa: F811
    k = inputs(B, T, D, dtype, seed=31, state=True, grads=True)
    k["reset"] = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    k["reset"][:, [150, 290]] = True
    clean = forward_backward(ops, k)
    k["r"][:, :150] = NAN
    k["r"][:, 290:] = NAN
    k["h0"][:] = NAN
    bad = forward_backward(ops, k)
    for name in ("y", "dx", "dr", "di"):
        assert torch.equal(bad[name][:, 150:290], clean[name][:, 150:290]), name
    assert bool(torch.isnan(bad["y"][:, :150]).all()) and bool(torch.isnan(bad["h"]).all())
