"""What crosses a reset in the gated scan: nothing, a NaN gate included, forward and backward; and
what does not stop at one that is not there: infinities and NaN travel on however small the
decays' product becomes, the same way in every run."""
import pytest
import torch

from test_gpu_scan import forward_backward, inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")

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


@pytest.mark.parametrize("B,T,D,dtype", [(1, 4000, 66, F32), (2, 4000, 70, BF16), (1, 4000, 33, F16),
                                         (20, 900, 1024, BF16), (5, 900, 3200, BF16)])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("value", [INF, NAN])
def test_what_is_not_finite_stays(ops, B, T, D, dtype, resets, value):  # noqa: F811
    """Decays whose product over a tile is far below the smallest float32: no state is dropped by
    it, whether the row has a reset before (or after) or the batch has no flags at all."""
    k = inputs(B, T, D, dtype, seed=32, state=True, grads=True)
    k["decay"][:] = 6.0
    at, far = 300, T - 200
    if resets:
        k["reset"] = torch.zeros(B, T, dtype=torch.bool, device="cuda")
        k["reset"][:, [77, far + 100]] = True
    clean = forward_backward(ops, k)
    q = dict(k, x=k["x"].clone(), dy=k["dy"].clone())
    q["x"][:, at, ::3] = value
    q["dy"][:, far, 1::3] = value
    first = forward_backward(ops, q)
    end = far + 100 if resets else T
    hurt = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    hurt[:, at:end, ::3] = True
    assert not torch.isfinite(first["y"][hurt]).any()
    assert torch.equal(first["y"][~hurt], clean["y"][~hurt])
    back = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    back[:, 77 if resets else 0:far + 1, 1::3] = True
    assert not torch.isfinite(first["dx"][back]).any()
    if resets:
        assert torch.equal(first["dx"][~back & ~hurt], clean["dx"][~back & ~hurt]) and torch.equal(first["dh0"], clean["dh0"])
    else:
        assert not torch.isfinite(first["dh0"][:, 1::3]).any()
    for _ in range(6):
        again = forward_backward(ops, q)
        for name in first:
            a, b = first[name], again[name]
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)), name
