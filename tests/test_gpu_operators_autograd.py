"""The operators within torch: tensors that they write tell autograd so, arguments that get no
gradient are refused when they ask for one, and passes are captured in graphs."""
import pytest
import torch

from test_gpu_scan import forward_backward, inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def loss_inputs(N=6, V=500, K=5, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(N, V, generator=g, device="cuda")
    top, index = torch.topk(torch.randn(N, V, generator=g, device="cuda"), K, dim=1)
    return z, index, top


def test_a_step_raises_its_state_s_version(ops):  # noqa: F811
    k = inputs(3, 1, 40, F32, seed=50, state=True)
    args = [k[m][:, 0] for m in ("x", "r", "i")] + [k["decay"]]
    h = k["h0"].clone()
    before = h._version
    ops.gated_scan_step(*args, h)
    assert h._version > before
    w = torch.ones(3, 40, device="cuda", requires_grad=True)
    loss = (w * h).sum()                    # saves h for the gradient by w
    with torch.no_grad():
        ops.gated_scan_step(*args, h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        hi = k["h0"].clone()
        ops.gated_scan_step(*args, hi)
    assert torch.isfinite(hi).all()


def test_a_gradient_over_the_logits_raises_their_version(ops):  # noqa: F811
    z, index, top = loss_inputs()
    w = torch.randn(500, 500, device="cuda", requires_grad=True)
    capped = torch.tanh(z @ w)              # its backward pass reads its result
    _, d = ops.distill_loss_grad(capped, index, top, out=capped)
    assert d is capped
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        capped.backward(d.detach())
    logits = z @ w                          # nothing reads these again
    _, d = ops.distill_loss_grad(logits, index, top)
    want = torch.autograd.grad(logits, w, d, retain_graph=True)[0]
    _, same = ops.distill_loss_grad(logits, index, top, out=logits)
    assert torch.equal(torch.autograd.grad(logits, w, same.detach())[0], want)
    saved = (z @ w).requires_grad_(True)
    loss = ops.distill_loss(saved, index, top)
    ops.distill_loss_grad(saved, index, top, out=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    with torch.inference_mode():
        zi = z.clone()
        ops.distill_loss_grad(zi, index, top, out=zi)
    assert torch.isfinite(zi).all()


def test_a_teacher_that_asks_for_a_gradient_is_refused(ops):  # noqa: F811
    z, index, top = loss_inputs()
    z.requires_grad_(True)
    ones = torch.ones(6, device="cuda")
    for bad in (dict(top=top.clone().requires_grad_(True)), dict(top=top, weight=ones.clone().requires_grad_(True)),
                dict(top=top, top_lse=ones.clone().requires_grad_(True))):
        with pytest.raises(ValueError, match="detach"):
            ops.distill_loss(z, index, **bad)
        with torch.no_grad():
            ops.distill_loss(z, index, **bad)
        ops.distill_loss_grad(z, index, **bad)      # returns the gradient by the logits, and says so


def capture(run):
    """What run() returns eagerly, and from three replays of its graph."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        yield want, out


@pytest.mark.parametrize("T", [40, 900])
def test_training_passes_in_a_graph(ops, T):  # noqa: F811
    k = inputs(2, T, 96, BF16, seed=51, state=True, resets=0.01, grads=True)
    for want, out in capture(lambda: list(forward_backward(ops, k).values())):
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_a_step_in_a_graph(ops):  # noqa: F811
    k = inputs(5, 1, 96, BF16, seed=52, state=True)
    h = k["h0"].clone()

    def run():
        h.copy_(k["h0"])
        return [ops.gated_scan_step(k["x"][:, 0], k["r"][:, 0], k["i"][:, 0], k["decay"], h), h]

    for want, out in capture(run):
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("V", [500, 131072])
def test_losses_in_a_graph(ops, V):  # noqa: F811
    z, index, top = loss_inputs(V=V)
    z.requires_grad_(True)

    def run():
        loss = ops.distill_loss(z, index, top)
        return [loss.detach(), torch.autograd.grad(loss.sum(), z)[0], *ops.distill_loss_grad(z, index, top)]

    for want, out in capture(run):
        assert all(torch.equal(a, b) for a, b in zip(want, out))
