"""The gradients past 2^31 elements and on long softmax batches."""
import pytest
import torch

import gradients as gr
import token_dispatch_fp32_b200 as mr
from test_backward_gpu import _check_gate, _f32, _gate_problem, _i32
from test_rows_gpu import _dev

pytestmark = pytest.mark.gpu

T, K = 37501, 8


@pytest.fixture(scope="module", params=[7168, 7167], ids=["vectors", "elements"])
def rows(request):
    """37501 x 8 bf16 rows, more than 2^31 elements, sorted in no order."""
    d = request.param
    assert T * K * d > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(d)
    E = torch.empty((T * K, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    inv = torch.randperm(T * K, generator=gen, device="cuda").int()
    inv[:2], inv[-2:] = inv[-2:].clone(), inv[:2].clone()
    dy = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    sample = torch.cat([torch.arange(40), torch.arange(T - 40, T),
                        (inv >= T * K - 40).nonzero()[:, 0].cpu() // K]).unique().cuda()
    yield E, inv, dy, sample
    del E


def test_row_gradients_past_2_31_elements(rows):
    E, inv, dy, sample = rows
    d = E.shape[1]
    w = torch.rand((T, K), device="cuda") + 0.1
    r = inv.view(T, K)[sample].long()  # [S, K]
    dE, dw = mr.mr_combine_backward(dy, E, w, inv)
    assert mr.mr_get_error() == mr.MR_OK
    g, e, ws = dy[sample].double(), E[r].double(), w[sample].double()
    want = ws[:, :, None] * g[:, None]
    gr.check(dE[r].float().cpu().numpy(), want.cpu().numpy(),
             gr.U * want.abs().cpu().numpy(), "bf16", "dexpert")
    p = g[:, None] * e
    gr.check(dw[sample].cpu().numpy(), p.sum(2).cpu().numpy(),
             (d + 2) * gr.U * p.abs().sum(2).cpu().numpy(), "f32", "dw")
    del dE, want, p
    dx = mr.mr_gather_rows_backward(E, K, inv, add=dy)
    assert mr.mr_get_error() == mr.MR_OK
    want = e.sum(1) + g
    mag = e.abs().sum(1) + g.abs()
    gr.check(dx[sample].float().cpu().numpy(), want.cpu().numpy(),
             (K + 1) * gr.U * mag.cpu().numpy(), "bf16", "dx")


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_gate_gradient_past_2_31_elements(softmax):
    """300001 tokens of 7168 columns, all rows zero but the last 64."""
    n, d, N_r, k, m = 300001, 7168, 16, 2, 64
    assert n * d > 1 << 31
    flags = mr.MR_SCORE_SOFTMAX if softmax else 0
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    x[-m:] = torch.randn((m, d), generator=gen, device="cuda").bfloat16()
    W = torch.randn((N_r, d), generator=gen, device="cuda") / d ** 0.5
    L = torch.randn((n, N_r), generator=gen, device="cuda")
    idx = torch.rand((n, N_r), generator=gen, device="cuda").topk(k, 1).indices.int()
    g = torch.randn((n, k), generator=gen, device="cuda")
    _, offsets, perm, _ = mr.mr_dispatch(idx, N_r)
    dx, dW = mr.mr_router_backward(x, W, L, idx, g, perm, offsets, 2.5, flags=flags)
    assert mr.mr_get_error() == mr.MR_OK
    for part in (slice(0, m), slice(n - m, n)):
        dL, err = gr.dlogits(L[part].cpu().numpy(), idx[part].cpu().numpy(),
                             g[part].cpu().numpy(), 2.5, softmax)
        rx, bx, rW, bW = gr.products(dL, err, x[part].double().cpu().numpy(),
                                     W.double().cpu().numpy())
        gr.check(dx[part].float().cpu().numpy(), rx, bx, "bf16", "dx")
    gr.check(dW.cpu().numpy(), rW, bW, "f32", "dW")  # the other rows add zeros


@pytest.mark.parametrize("T,d,N_r,k,xdt", [(5000, 264, 64, 4, "bf16"), (4097, 136, 200, 8, "f32"),
                                           (6001, 67, 24, 3, "bf16")])
def test_long_softmax_batches(T, d, N_r, k, xdt):
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, xdt, "f32", 0, seed=T)
    dlog = torch.empty((T, N_r), device="cuda")
    got = mr.mr_router_backward(_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), None, None, 2.5,
                                flags=mr.MR_SCORE_SOFTMAX, dlogits=dlog)
    assert mr.mr_get_error() == mr.MR_OK
    _check_gate(x, W, L, idx, g, xdt, mr.MR_SCORE_SOFTMAX, None, (*got, dlog))
