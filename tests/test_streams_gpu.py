"""Calls on a named stream: the buffers that a call allocates belong to that
stream's work."""
import numpy as np
import pytest
import torch

import oracle
import token_dispatch_fp32_b200 as mr
from test_backward_gpu import _f32, _gate_problem, _i32, _rows
from test_rows_gpu import _dev

pytestmark = pytest.mark.gpu

T, D, N_R, K, N_OUT = 700, 1024, 64, 4, 512


@pytest.fixture(scope="module")
def calls():
    """name -> call(stream=) of every step that allocates its outputs."""
    rng, x, W, L, idx, g = _gate_problem(T, D, N_R, K, "bf16", "f32", 0, seed=3)
    _, offsets, perm, inv = oracle.dispatch(idx, N_R)
    x, W, L, idx, g = _dev(x), _dev(W), _f32(L), _i32(idx), _f32(g)
    offsets, perm, inv = _i32(offsets), _i32(perm), _i32(inv)
    E = _dev(_rows(rng, (T * K, D), "bf16"))
    w = _f32(rng.uniform(0.1, 1.0, (T, K)))
    q = torch.from_numpy(rng.integers(0, 256, (N_R, N_OUT, D // 2)).astype(np.uint8)).cuda()
    sc = torch.ones((N_R, N_OUT, D // 32), dtype=torch.bfloat16, device="cuda")
    W4 = mr.mr_expert_pack_w4(q, sc, 32)
    We = _dev(_rows(rng, (N_R, N_OUT, D), "bf16"))
    x32, softmax = x.float(), mr.MR_SCORE_SOFTMAX
    return {
        "router": lambda **s: mr.mr_router_forward(x32, W, None, 1, 1, K, 2.5, mr.MR_MASK_NEG_INF,
                                                   **s),
        "dispatch": lambda **s: mr.mr_dispatch(idx, N_R, **s),
        "gather": lambda **s: mr.mr_gather_rows(x, K, perm=perm, inv_perm=inv, **s),
        "combine": lambda **s: mr.mr_combine(E, w, inv, x, **s),
        "expert": lambda **s: mr.mr_expert_gemm_gather(x, K, perm, offsets, We, **s),
        "pack_w4": lambda **s: mr.mr_expert_pack_w4(q, sc, 32, **s),
        "expert_w4": lambda **s: mr.mr_expert_gemv_gather_w4(x, K, perm, offsets, W4, N_R, N_OUT,
                                                             32, **s),
        "combine_backward": lambda **s: mr.mr_combine_backward(x, E, w, inv, **s),
        "gather_backward": lambda **s: mr.mr_gather_rows_backward(E, K, inv, **s),
        "router_backward": lambda **s: mr.mr_router_backward(x, W, L, idx, g, perm, offsets, 2.5,
                                                             **s),
        "router_backward_softmax": lambda **s: mr.mr_router_backward(
            x, W, L, idx, g, perm, offsets, 2.5, flags=softmax, **s),
    }


NAMES = ["router", "dispatch", "gather", "combine", "expert", "pack_w4", "expert_w4",
         "combine_backward", "gather_backward", "router_backward", "router_backward_softmax"]


def _tuple(r):
    return r if isinstance(r, tuple) else (r,)


def _same(got, ref):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))


def _busy():
    torch.cuda._sleep(20_000_000)  # some ten milliseconds


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_what_the_current_stream_still_writes(calls, name):
    """Buffers of the outputs' sizes, which the current stream fills late, are
    freed before the call, whose stream does not wait for that one."""
    call, s = calls[name], torch.cuda.Stream()
    ref = _tuple(call())
    torch.cuda.synchronize()
    for _ in range(2):
        junk = [torch.empty_like(o) for o in ref]
        _busy()
        for j in junk:
            j.view(torch.uint8).fill_(0xA5)
        del junk, j
        got = _tuple(call(stream=s))
        torch.cuda.synchronize()
        assert mr.mr_get_error() == mr.MR_OK
        assert _same(got, ref)
        del got


@pytest.mark.parametrize("name", NAMES)
def test_freed_outputs_do_not_reach_the_current_stream(calls, name):
    """Outputs that are dropped while the call waits to run: the current stream's
    next buffers are not written by it."""
    call, s = calls[name], torch.cuda.Stream()
    ref = _tuple(call())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        _busy()
    call(stream=s)
    junk = [torch.empty_like(o) for o in ref]
    for j in junk:
        j.view(torch.uint8).fill_(0xA5)
    torch.cuda.synchronize()
    assert all((j.view(torch.uint8) == 0xA5).all() for j in junk)
