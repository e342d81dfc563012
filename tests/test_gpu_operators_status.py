"""Failure detection of the student-training operators, without a fault: bounded waits that run out
leave NaN and a status that Python can read, and the device stays usable."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ops():
    from error_compensated_bit_gb300 import build, ops as mod
    build.build()
    return mod


@pytest.mark.parametrize("N,V", [(1, 40000), (9, 131072), (700, 40000), (333, 70001)])
def test_a_late_block_of_a_row_is_reported(ops, N, V):
    """One block of each row's is late: the others give up, write NaN, exchange nothing more and
    stay until it is done with their memory."""
    g = torch.Generator(device="cuda").manual_seed(N)
    z = torch.randn(N, V, generator=g, device="cuda")
    top, index = torch.topk(z, 8, dim=1)
    want = ops.distill_loss_grad(z, index, top)
    assert ops.read_status() == 0 and bool(torch.isfinite(want[0]).all())
    loss, d = torch.zeros(N, device="cuda"), torch.zeros(N, V, device="cuda")
    ops._call(z.device, "ob_selftest_distill_wait", N, V, 8, z.data_ptr(), index.data_ptr(), top.data_ptr(),
              loss.data_ptr(), d.data_ptr())
    assert ops.read_status() == 1, "the waits ran out and said so"
    assert ops.read_status() == 0, "reading clears"
    assert bool(torch.isnan(loss).all()) and bool(torch.isnan(d[:, 0]).all())
    assert bool((torch.isnan(d) | (d == want[1])).all()), "what is not NaN is right"
    again = ops.distill_loss_grad(z, index, top)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert ops.read_status(z.device) == 0


def test_a_scan_s_wait_is_reported(ops):
    import ctypes
    from error_compensated_bit_gb300 import ob
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    assert ops.read_status() == 0
    ops._call(ws.device, "ob_selftest_scan_wait", ws.data_ptr(), 2_000_000)
    st = ctypes.c_uint(9)
    ops._call(ws.device, "ob_gated_scan_read_status", ws.data_ptr(), ctypes.byref(st))
    assert st.value == 1 and ops.read_status() == 1 and ops.read_status() == 0
    x = torch.ones(1, 1000, 64, device="cuda")
    y, _ = ops.gated_scan(x, x, x, torch.ones(64, device="cuda"))
    assert bool(torch.isfinite(y).all()) and ops.read_status() == 0
    assert ob.load().ob_selftest_scan_wait(ws.data_ptr(), 0, None) == ob.OB_EINVAL
    assert ob.load().ob_selftest_scan_wait(ws.data_ptr(), 3 * 10 ** 9, None) == ob.OB_EINVAL
    assert ob.load().ob_selftest_scan_wait(ws.data_ptr() + 4, 1000, None) == ob.OB_EALIGN


def test_refusals(ops):
    from error_compensated_bit_gb300 import ob
    lib, good = ob.load(), 1 << 20
    assert lib.ob_operators_read_status(None, None) == ob.OB_EINVAL
    for N, V in ((0, 40000), (4, 1000), (4, 1 << 20)):
        assert lib.ob_selftest_distill_wait(N, V, 8, good, good, good, good, good, None) == ob.OB_EINVAL
    assert lib.ob_selftest_distill_wait(4, 40000, 8, good, good, good, None, good, None) == ob.OB_EINVAL
    assert lib.ob_selftest_distill_wait(4, 40000, 8, good, good, good, good, good + 2, None) == ob.OB_EALIGN
