"""The gradient formulas (tests/gradients.py) against central differences of
the oracle's forward, and the refusals of the gradients' and the 4-bit expert
layer's entry points (argument checks return before any device call)."""
import ctypes as C

import numpy as np
import pytest
import torch

import gradients as gr
import oracle
import token_dispatch_fp32_b200 as mr


def test_combine_backward_formula_is_the_oracle_combines_derivative():
    """fp32 rows: the oracle's combine is linear in E and in w, so a central
    difference is exact up to binary64 rounding of its fp32-rounded inputs."""
    rng = np.random.default_rng(0)
    T, d, k, N = 6, 5, 3, 7
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32)
    _, _, _, inv = oracle.dispatch(idx, N)
    E = rng.integers(-8, 9, (T * k, d)).astype(np.float32)
    w = (rng.integers(1, 9, (T, k)) / 8).astype(np.float32)
    dy = rng.integers(-8, 9, (T, d)).astype(np.float64)
    dE, dw, _ = gr.combine_backward(dy, E.astype(np.float64), w, inv, k)

    def loss(E, w):
        return (oracle.combine(E, w, inv, None, k)[0].astype(np.float64) * dy).sum()

    h = np.float32(0.5)
    for r, c in [(0, 0), (7, 3), (17, 4)]:
        Ep, Em = E.copy(), E.copy()
        Ep[r, c] += h
        Em[r, c] -= h
        assert (loss(Ep, w) - loss(Em, w)) == pytest.approx(dE[r, c], abs=1e-5)
    for t, j in [(0, 0), (3, 2), (5, 1)]:
        wp, wm = w.copy(), w.copy()
        wp[t, j] += h
        wm[t, j] -= h
        assert (loss(E, wp) - loss(E, wm)) == pytest.approx(dw[t, j], abs=1e-4)


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_router_backward_formula_is_the_gates_derivative(softmax):
    """Central differences of the gate's weights in binary64 with the choice
    held: error O(h^2) of the third derivative (all of order 1) plus binary64
    rounding over h."""
    rng = np.random.default_rng(1)
    T, d, N, k = 5, 12, 9, 3
    x, W = rng.standard_normal((T, d)), rng.standard_normal((N, d)) / np.sqrt(d)
    g = rng.standard_normal((T, k))
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32)

    def loss(x, W):
        L = x @ W.T
        if softmax:
            p = np.exp(L - L.max(1, keepdims=True))
            s = np.take_along_axis(p / p.sum(1, keepdims=True), idx, 1)
            w = 2.5 * s
        else:
            s = 1 / (1 + np.exp(-np.take_along_axis(L, idx, 1)))
            w = 2.5 * s / s.sum(1, keepdims=True)
        return (w * g).sum()

    dL, err = gr.dlogits(x @ W.T, idx, g, 2.5, softmax)
    dx, _, dW, _ = gr.products(dL, err, x, W)
    h = 1e-5
    for a, da in ((x, dx), (W, dW)):
        for _ in range(12):
            i = tuple(rng.integers(0, n) for n in a.shape)
            v = a[i]
            a[i] = v + h
            up = loss(x, W)
            a[i] = v - h
            down = loss(x, W)
            a[i] = v
            assert (up - down) / (2 * h) == pytest.approx(da[i], abs=1e-8)


def test_router_backward_formula_is_autograds():
    rng = np.random.default_rng(2)
    T, N, k = 20, 16, 4
    L = torch.tensor(rng.standard_normal((T, N)), requires_grad=True)
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32)
    g = rng.standard_normal((T, k))
    s = torch.sigmoid(L).gather(1, torch.from_numpy(idx).long())
    w = s / (s.sum(1, keepdim=True) + 1e-20) * 2.827
    (w * torch.from_numpy(g)).sum().backward()
    dL, _ = gr.dlogits(L.detach().numpy(), idx, g, 2.827)
    assert np.abs(dL - L.grad.numpy()).max() < 1e-14


P = C.c_void_p(64)  # never dereferenced


def test_combine_backward_refusals():
    f = mr.lib().mr_combine_backward  # dy, dtype, E, w, inv, T, d, k, dE, dw, stream
    assert f(P, 5, P, P, P, 4, 8, 2, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, -1, 8, 2, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, 4, 0, 2, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, 4, 8, 0, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, 1 << 28, 8, 8, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, 4, 8, 33, P, P, None) == mr.MR_ERR_UNSUPPORTED
    assert f(None, 1, P, P, P, 4, 8, 2, P, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, P, P, 4, 8, 2, None, None, None) == mr.MR_ERR_INVALID_ARG  # no output
    assert f(P, 1, None, P, P, 4, 8, 2, P, P, None) == mr.MR_ERR_INVALID_ARG  # dw needs the rows
    assert f(None, 1, None, None, None, 0, 8, 2, None, None, None) == mr.MR_OK


def test_gather_backward_refusals():
    f = mr.lib().mr_gather_rows_backward  # dxs, dtype, inv, add, T, d, k, dx, stream
    assert f(P, 2, P, None, 4, 8, 2, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, None, 4, -8, 2, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, None, 1 << 30, 8, 2, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, None, 4, 8, 40, P, None) == mr.MR_ERR_UNSUPPORTED
    assert f(P, 1, None, None, 4, 8, 2, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, 1, P, None, 4, 8, 2, None, None) == mr.MR_ERR_INVALID_ARG
    assert f(None, 1, None, None, 0, 8, 2, None, None) == mr.MR_OK


def _router(T=8, d=64, N=32, k=4, xdt=1, wdt=0, scale=2.5, flags=0, x=P, W=P, logits=P, idx=P,
            dw=P, perm=P, offsets=P, add=None, dlogits=P, dx=P, dW=P, ws=P, n=None):
    if n is None:
        n = mr.lib().mr_router_backward_workspace_size(T, d, N, k, flags)
    return mr.lib().mr_router_backward(x, xdt, W, wdt, logits, idx, dw, perm, offsets, T, d, N, k,
                                       scale, flags, add, dlogits, dx, dW, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1, n=0), mr.MR_ERR_INVALID_ARG),
    (dict(d=0, n=0), mr.MR_ERR_INVALID_ARG),
    (dict(xdt=3), mr.MR_ERR_INVALID_ARG),
    (dict(wdt=3), mr.MR_ERR_INVALID_ARG),
    (dict(flags=8), mr.MR_ERR_INVALID_ARG),
    (dict(scale=float("inf")), mr.MR_ERR_INVALID_ARG),
    (dict(N=513), mr.MR_ERR_UNSUPPORTED),
    (dict(k=33), mr.MR_ERR_UNSUPPORTED),
    (dict(dlogits=None, dx=None, dW=None), mr.MR_ERR_INVALID_ARG),
    (dict(logits=None), mr.MR_ERR_INVALID_ARG),
    (dict(idx=None), mr.MR_ERR_INVALID_ARG),
    (dict(dw=None), mr.MR_ERR_INVALID_ARG),
    (dict(W=None), mr.MR_ERR_INVALID_ARG),                  # dx needs W
    (dict(x=None), mr.MR_ERR_INVALID_ARG),                  # dW needs x
    (dict(perm=None), mr.MR_ERR_INVALID_ARG),               # dW of sigmoid scores needs both
    (dict(offsets=None), mr.MR_ERR_INVALID_ARG),
    (dict(ws=None), mr.MR_ERR_INVALID_ARG),
    (dict(n=16), mr.MR_ERR_INVALID_ARG),                    # workspace too small
    (dict(ws=C.c_void_p(72)), mr.MR_ERR_INVALID_ARG),       # and not aligned
    (dict(T=0, dW=None, x=None, logits=None), mr.MR_OK),
])
def test_router_backward_refusals(kw, status):
    assert _router(**kw) == status


def test_router_backward_workspace_covers_the_partial_sums():
    size = mr.lib().mr_router_backward_workspace_size
    # the slots' gradients, and one row of d per full 256 sorted rows
    assert size(1000, 64, 32, 4, 0) >= 4000 * 4 + (4000 // 256) * 64 * 4
    # softmax: the dense logit gradients
    assert size(1000, 64, 32, 4, mr.MR_SCORE_SOFTMAX) >= 4000 * 4 + 1000 * 32 * 4
    assert size(0, 64, 32, 4, 0) == 0


def test_expert_w4_refusals():
    L = mr.lib()
    size = L.mr_expert_w4_packed_bytes
    assert size(4, 64, 256, 48, 1) == 0 and size(4, 0, 256, 32, 1) == 0
    assert size(4, 64, 256, 32, 7) == 0
    n = size(4, 64, 256, 32, 1)
    assert n == 4 * 64 * 256 // 2 + 4 * 64 * 8 * 2
    # padded to 64 rows and 128 columns
    assert size(1, 1, 8, 128, 0) == 4096 + 64 * 4
    pack = L.mr_expert_pack_w4  # q, scales, sdt, N, n_out, d, group, packed, bytes, stream
    assert pack(P, P, 1, 4, 64, 256, 32, P, n - 1, None) == mr.MR_ERR_INVALID_ARG
    assert pack(P, P, 1, 4, 64, 252, 32, P, n, None) == mr.MR_ERR_UNSUPPORTED
    assert pack(P, P, 1, 4, 64, 256, 16, P, n, None) == mr.MR_ERR_UNSUPPORTED
    assert pack(P, P, 2, 4, 64, 256, 32, P, n, None) == mr.MR_ERR_INVALID_ARG
    assert pack(None, P, 1, 4, 64, 256, 32, P, n, None) == mr.MR_ERR_INVALID_ARG
    assert pack(P, P, 1, 2048, 64, 256, 32, P, 1 << 40, None) == mr.MR_ERR_UNSUPPORTED
    f = L.mr_expert_gemv_gather_w4  # x, perm, offsets, W, sdt, T, d, k, N, n_out, group, out, s
    assert f(P, P, P, P, 1, -1, 256, 2, 4, 64, 32, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, P, P, P, 1, 3, 256, 0, 4, 64, 32, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(P, P, P, P, 1, 3, 250, 2, 4, 64, 32, P, None) == mr.MR_ERR_UNSUPPORTED
    assert f(P, P, P, P, 1, 3, 256, 2, 4, 64, 33, P, None) == mr.MR_ERR_UNSUPPORTED
    assert f(P, P, None, P, 1, 3, 256, 2, 4, 64, 32, P, None) == mr.MR_ERR_INVALID_ARG
    assert f(C.c_void_p(72), P, P, P, 1, 3, 256, 2, 4, 64, 32, P, None) == mr.MR_ERR_UNSUPPORTED
    assert f(None, None, None, None, 1, 0, 256, 2, 4, 64, 32, None, None) == mr.MR_OK
