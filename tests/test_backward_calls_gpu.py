"""The gradients as a training loop calls them: one call after another on the
same buffers."""
import pytest
import torch

import oracle
import token_dispatch_fp32_b200 as mr
from test_backward_gpu import _f32, _gate_problem, _i32
from test_rows_gpu import _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,want_dx", [(700, 1024, True), (700, 1024, False),
                                         (4000, 264, True)])
def test_gate_gradients_in_a_row_on_one_workspace(T, d, want_dx):
    """The kernels behind the logit gradients start while those are written:
    calls that take turns on one workspace read the values of their own call."""
    N_r, k = 64, 4
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=T)
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    grads = [_f32(g), _f32(-3 * g[::-1])]
    args = (_dev(x), _dev(W), _f32(L), _i32(idx))
    plan = (_i32(perm), _i32(offsets), 2.5)
    ws = torch.empty(mr.mr_router_backward_workspace_size(T, d, N_r, k), dtype=torch.uint8,
                     device="cuda")
    ref = []
    for dw in grads:
        ref.append(mr.mr_router_backward(*args, dw, *plan, want_dx=want_dx))
        torch.cuda.synchronize()
    got = [mr.mr_router_backward(*args, grads[i % 2], *plan, want_dx=want_dx, workspace=ws)
           for i in range(20)]
    torch.cuda.synchronize()
    assert mr.mr_get_error() == mr.MR_OK
    for i, (dx, dW) in enumerate(got):
        assert torch.equal(dW, ref[i % 2][1])
        assert dx is None or torch.equal(dx, ref[i % 2][0])


@pytest.mark.parametrize("d", [64, 67])
def test_an_id_named_by_four_slots_of_a_softmax_gate(d):
    """Its slots' gradients add up in slot order, in whichever lane: 2^24 + 1 -
    2^24 + 1 is 1 in fp32 (and 0, 1 or 2 in other orders).  Eight equal logits: p =
    1/8, the mean (2^24 - 2^24) / 8 + (1 + 1) / 8, the entry 2.5 / 8 * (1 - 1/4)."""
    T, N_r, k = 300, 8, 4
    idx = _i32([[t % N_r] * k for t in range(T)])
    dw = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24, 1.0], device="cuda").repeat(T, 1)
    W = torch.eye(N_r, d, device="cuda")
    dlog = torch.empty((T, N_r), device="cuda")
    dx, _ = mr.mr_router_backward(torch.zeros((T, d), device="cuda"), W,
                                  torch.zeros((T, N_r), device="cuda"), idx, dw, None, None, 2.5,
                                  flags=mr.MR_SCORE_SOFTMAX, dlogits=dlog)
    assert mr.mr_get_error() == mr.MR_OK
    assert (dlog.gather(1, idx[:, :1].long()) == 0.234375).all()
    assert torch.equal(dx[:, :N_r], dlog)


@pytest.mark.parametrize("T", [60, 900])
@pytest.mark.parametrize("place", ["first", "inside", "last"])
def test_offsets_that_overlap_or_leave_the_rows_are_flagged(T, place):
    """One row too far is enough, in a batch whose segments make one piece each
    too; the plan itself is not flagged."""
    d, N_r, k = 64, 16, 2
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=T)
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    args = (_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), _i32(perm))
    ref = mr.mr_router_backward(*args, _i32(offsets), 2.5)
    assert mr.mr_get_error() == mr.MR_OK
    bad = offsets.copy()
    if place == "first":
        bad[0] = -1
    elif place == "inside":
        bad[5] = bad[4] - 1  # the row before segment 4's is also segment 5's
    else:
        bad[N_r] += 1
    dx, _ = mr.mr_router_backward(*args, _i32(bad), 2.5)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    assert torch.equal(dx, ref[0])
