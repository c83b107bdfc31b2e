"""The device-side timeout paths of the gated recurrence and of the
projections, run without any fault: the test hook makes something that a
kernel waits for never happen and its waits short.  The call ends, the status
word says so, and the next call on the same workspace and GPU is right."""
import time

import pytest
import torch

import operator_refs as refs
from state_space_sequence_scan_b200 import ssd

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
TIMEOUT = 6


def runs_out(kind, ws, call):
    """The call under the fault reports the timeout, well under the 2 s of one normal wait."""
    call()
    torch.cuda.synchronize()
    assert ssd.read_device_status(ws) == 0
    ssd.set_test_fault(kind)
    try:
        t0 = time.perf_counter()
        call()
        status = ssd.read_device_status(ws)
        elapsed = time.perf_counter() - t0
    finally:
        ssd.set_test_fault(0)
    assert status == TIMEOUT and elapsed < 0.5, (status, elapsed)


# rows on 16 bytes, on pairs and on single elements; one and several groups of chunks
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("L,D", [(300, 128), (3000, 66), (1000, 65)])
def test_gated_waits_run_out(L, D, packed, dtype):
    g = torch.Generator().manual_seed(L)
    b = 2
    x, r, i, dy = (torch.randn(b, L, D, generator=g).to(dtype).cuda() for _ in range(4))
    lam, init = torch.full((D,), -4.0).cuda(), torch.randn(b, D, generator=g).cuda()
    ids = torch.cumsum(torch.rand(b, L, generator=g) < 0.01, 1).to(torch.int32).cuda() if packed else None
    wf, wb = (torch.empty(ssd.gated_scan_workspace_size(b, L, D, dtype, back), dtype=torch.uint8, device="cuda") for back in (False, True))
    states = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, seq_idx=ids)[2]

    def fwd():
        return ssd.gated_scan_fwd(x, r, i, lam, init_state=init, seq_idx=ids, workspace=wf)

    def bwd():
        return ssd.gated_scan_bwd(x, r, i, lam, states, dy, init_state=init, seq_idx=ids, workspace=wb)

    want, dwant = fwd(), bwd()
    runs_out(2, wf, fwd)
    runs_out(2, wb, bwd)
    got, dgot = fwd(), bwd()
    assert ssd.read_device_status(wf) == 0 and ssd.read_device_status(wb) == 0
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and all(torch.equal(dwant[k], dgot[k]) for k in dwant)
    h, err, _ = refs.gated(x, r, i, lam, init, ids)
    refs.check(got[0], h, err, "after the timeout")


# bf16 tiles of several widths, one and several tiles a pair and parts of k, and fp32 in parts
@pytest.mark.parametrize("M,N,K,dtype", [(300, 520, 2000, BF), (5000, 5120, 640, BF), (40, 200, 333, BF), (700, 1100, 1500, FP)])
def test_linear_waits_run_out(M, N, K, dtype):
    g = torch.Generator().manual_seed(M)
    x, w, dy = (torch.randn(*s, generator=g).to(dtype).cuda() for s in ((M, K), (N, K), (M, N)))
    wf, wb = (torch.empty(ssd.linear_workspace_size(M, N, K, dtype, back), dtype=torch.uint8, device="cuda") for back in (False, True))

    def fwd():
        return [ssd.linear_fwd(x, w, activation="silu", workspace=wf)]

    def bwd():
        d = ssd.linear_bwd(x, w, dy, workspace=wb)
        return [d["x"], d["weight"], d["bias"]]

    want, dwant = fwd(), bwd()
    runs_out(3, wf, fwd)
    runs_out(3, wb, bwd)
    got, dgot = fwd(), bwd()
    assert ssd.read_device_status(wf) == 0 and ssd.read_device_status(wb) == 0
    assert all(torch.equal(p, q) for p, q in zip(want + dwant, got + dgot))
    ref, err, _, _ = refs.linear(x, w, None, None, "silu")
    refs.check(got[0], ref, err, "after the timeout")


def test_the_hooks_leave_other_calls_alone():
    """Calls of another kind run as ever under a fault."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(300, 256, generator=g).bfloat16().cuda(), torch.randn(520, 256, generator=g).bfloat16().cuda()
    v = torch.randn(1, 700, 64, generator=g).bfloat16().cuda()
    lam = torch.full((64,), -4.0).cuda()
    y, (h, _) = ssd.linear_fwd(x, w), ssd.gated_scan_fwd(v, v, v, lam)
    try:
        for kind in (1, 2, 3):
            ssd.set_test_fault(kind)
            assert kind == 3 or torch.equal(ssd.linear_fwd(x, w), y)
            assert kind == 2 or torch.equal(ssd.gated_scan_fwd(v, v, v, lam)[0], h)
    finally:
        ssd.set_test_fault(0)
