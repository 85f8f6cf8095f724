"""The expert layer on 4-bit weights (mr_expert_gemv_gather_w4) on the GPU
against binary64 (tests/gradients.py: expert_w4).

Bound: 32 columns at a time, the kernel forms -24 sum x and adds sum (16 + u) x
to it, u the nibble: four MMA steps, each exact in its products and rounding
within 2 fp32 steps (2 * 2^-23) of its largest partial sum, which is at most
(24 + 31) sum |x|; hence 4 * 2 * 55 = 440 * 2^-23 of the scaled sum of |x|.
Groups and warps then add in fp32: at most (d / 128 + 16) * 2^-23 of the sum
of the magnitudes.  Segments of more than 32 rows: the scaled weight is exact in
two bf16 planes (fp32 scales: the fp32 product, off by 2^-24, in three), so each
of the 3 d / 16 MMA steps at most rounds within 2 fp32 steps of the sum of the
magnitudes: (3 d / 8 + 2) * 2^-23 of it.  Plus half a step of the bf16 output."""
import numpy as np
import pytest
import torch

import gradients as gr
import oracle
import token_dispatch_fp32_b200 as mr
from parity import widen
from test_backward_gpu import _f32, _i32, _ids, _rows
from test_rows_gpu import _dev, _host

pytestmark = pytest.mark.gpu


def _problem(T, k, N_r, n_out, d, group, sdt, seed, hot=0):
    rng = np.random.default_rng(seed)
    idx = _ids(rng, T, k, N_r, hot)
    _, offsets, perm, inv = oracle.dispatch(idx, N_r)
    x = _rows(rng, (T, d), "bf16")
    q = rng.integers(0, 256, (N_r, n_out, d // 2)).astype(np.uint8)
    s = _rows(rng, (N_r, n_out, -(-d // group)), sdt, 0.1)
    return x, perm, offsets, inv, q, s


def _bound(d, mag, magx):
    few = (d / 128 + 16) * mag + 440 * magx
    many = (3 * d / 8 + 2) * mag
    return np.maximum(few, many) * 2.0 ** -23


CASES = [  # T, k, N_r, n_out, d, group, scales, hot
    (1, 8, 64, 64, 7168, 32, "bf16", 0),     # one token: fewer rows than experts
    (1, 1, 1, 1, 8, 32, "bf16", 0),          # the smallest of everything
    (7, 8, 40, 96, 1024, 64, "bf16", 0),
    (16, 4, 16, 33, 520, 128, "f32", 0),     # partial group, odd n_out
    (9, 2, 8, 48, 136, 32, "f32", 0),        # one block of columns and 8 more
    (23, 3, 5, 50, 256, 64, "f32", 0),
    (64, 2, 4, 40, 384, 32, "bf16", 2),      # 64 rows on each of two experts
    (100, 1, 3, 16, 2048, 128, "bf16", 1),   # 100 rows on one
    (37, 2, 128, 31, 72, 32, "bf16", 0),
    # long segments, enough of them that the many-row kernel takes them
    (1100, 1, 1, 1000, 136, 32, "f32", 0),   # six blocks of one expert, a K tail
    (600, 4, 8, 456, 1096, 128, "bf16", 1),  # one longer than three blocks
    (193, 8, 8, 2050, 64, 64, "bf16", 0),    # two blocks each, one stage of columns
    (290, 4, 16, 1100, 200, 64, "f32", 3),   # short segments among long ones
    (500, 8, 64, 256, 512, 32, "bf16", 0),   # every segment about 60 rows
    (64, 8, 8, 2300, 72, 32, "bf16", 0),     # one block of 64 rows each
]


@pytest.mark.parametrize("T,k,N_r,n_out,d,group,sdt,hot", CASES)
def test_expert_w4(T, k, N_r, n_out, d, group, sdt, hot):
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, group, sdt, T + d, hot)
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), group)
    st = torch.bfloat16 if sdt == "bf16" else torch.float32
    out = mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(perm), _i32(offsets), W4, N_r, n_out,
                                      group, scale_dtype=st)
    assert mr.mr_get_error() == mr.MR_OK
    want, mag, magx = gr.expert_w4(widen(x), perm, offsets, q, widen(s), group, k)
    gr.check(widen(_host(out)), want, _bound(d, mag, magx), "bf16", "out")
    # rows already sorted (perm None), and a second run: bit for bit the same
    xs = _dev(np.ascontiguousarray(x[perm // k]))
    again = mr.mr_expert_gemv_gather_w4(xs, k, None, _i32(offsets), W4, N_r, n_out, group,
                                        scale_dtype=st)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_expert_w4_exact_on_integers(group):
    """Integer rows and power-of-two scales: every sum is exact in fp32, so the
    result is the exact value rounded once (to nearest even)."""
    T, k, N_r, n_out, d = 500, 2, 6, 1900, 640
    rng = np.random.default_rng(group)
    _, offsets, perm, _ = oracle.dispatch(_ids(rng, T, k, N_r, hot=1), N_r)  # 500 rows on one
    x = rng.integers(-4, 5, (T, d)).astype(np.float32)
    q = rng.integers(0, 256, (N_r, n_out, d // 2)).astype(np.uint8)
    s = (2.0 ** rng.integers(-3, 3, (N_r, n_out, d // group))).astype(np.float32)
    xb = torch.from_numpy(x).bfloat16().cuda()
    want, _, _ = gr.expert_w4(x.astype(np.float64), perm, offsets, q, s, group, k)
    for st in (torch.bfloat16, torch.float32):
        W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _f32(s).to(st), group)
        out = mr.mr_expert_gemv_gather_w4(xb, k, _i32(perm), _i32(offsets), W4, N_r, n_out, group,
                                          scale_dtype=st)
        assert torch.equal(out.cpu(), torch.from_numpy(want).float().bfloat16())


def test_expert_w4_leaves_other_rows():
    """Rows of `out` behind the last segment (assignments the dispatch dropped)
    stay as they were; the dropped rows' place in perm (-1) is not read."""
    T, k, N_r, n_out, d = 30, 2, 8, 48, 256
    x, _, _, _, q, s = _problem(T, k, N_r, n_out, d, 32, "bf16", 1)
    rng = np.random.default_rng(2)
    idx = _ids(rng, T, k, N_r)
    idx[3, 1], idx[17, 0] = N_r, -2
    _, offsets, perm, _ = mr.mr_dispatch(_i32(idx), N_r)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), 32)
    out = torch.full((T * k, n_out), 7.0, dtype=torch.bfloat16, device="cuda")
    mr.mr_expert_gemv_gather_w4(_dev(x), k, perm, offsets, W4, N_r, n_out, 32, out=out)
    assert mr.mr_get_error() == mr.MR_OK
    p, o = perm.cpu().numpy(), offsets.cpu().numpy()
    n = o[-1]
    assert n == T * k - 2
    want, mag, magx = gr.expert_w4(widen(x), p[:n], o, q, widen(s), 32, k)
    gr.check(widen(_host(out))[:n], want, _bound(d, mag, magx), "bf16", "out")
    assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("T,n_out", [(24, 32), (80, 3700)], ids=["few", "many"])
def test_expert_w4_keeps_rows_apart(T, n_out):
    """A NaN or an infinity in one token's row reaches that token's outputs
    only."""
    k, N_r, d = 4, 4, 384
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, 32, "bf16", 5)
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), 32)
    args = (k, _i32(perm), _i32(offsets), W4, N_r, n_out, 32)
    ref = mr.mr_expert_gemv_gather_w4(_dev(x), *args)
    x[5, 100], x[9, 3] = 0x7FC1, 0x7F80
    out = mr.mr_expert_gemv_gather_w4(_dev(x), *args)
    tok = torch.from_numpy(perm // k).cuda()
    hit = (tok == 5) | (tok == 9)
    assert torch.equal(out[~hit].view(torch.int16), ref[~hit].view(torch.int16))
    assert torch.isnan(out[tok == 5]).all()
    assert not torch.isfinite(out[tok == 9]).any()


@pytest.mark.parametrize("spread", [0, 12, 20, 60])
def test_expert_w4_spread_magnitudes(spread):
    """Rows whose values spread over `spread` binary orders of magnitude, rows
    of very small and very large values and a row of zeros: the bound holds,
    nothing overflows on the way."""
    T, k, N_r, n_out, d = 8, 2, 4, 64, 512
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, 32, "bf16", 6 + spread)
    rng = np.random.default_rng(spread)
    v = widen(x) * 2.0 ** rng.integers(-spread, 1, (T, d))
    v[1] *= 2.0 ** -100
    v[2] *= 2.0 ** 100
    v[3] = 0
    x = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), 32)
    out = mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(perm), _i32(offsets), W4, N_r, n_out, 32)
    want, mag, magx = gr.expert_w4(widen(x), perm, offsets, q, widen(s), 32, k)
    gr.check(widen(_host(out)), want, _bound(d, mag, magx), "bf16", "out")


@pytest.mark.parametrize("T", [5, 600], ids=["few", "many"])
@pytest.mark.parametrize("mode", ["eager", "graph"])
def test_decode_step_of_a_moe_layer(mode, T):
    """Gate, dispatch, experts on 4-bit weights, combine for a few tokens;
    against binary64 on the gate's own choice and weights."""
    d, N_r, k, n_out, group = 512, 32, 4, 512, 64
    x, _, _, _, q, s = _problem(T, k, N_r, n_out, d, group, "bf16", 9)
    rng = np.random.default_rng(3)
    Wg = _f32(rng.standard_normal((N_r, d)) / np.sqrt(d))
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), group)
    xd = _dev(x)
    ws = torch.empty(max(16, mr.mr_router_workspace_size(T, d, N_r)), dtype=torch.uint8,
                     device="cuda")

    def step():
        idx, w = mr.mr_router_forward_ex(xd, Wg, None, 4, 2, k, 2.5, mr.MR_MASK_NEG_INF,
                                         precision=mr.MR_PREC_BF16X3, workspace=ws)
        _, offsets, perm, inv = mr.mr_dispatch(idx, N_r)
        E = mr.mr_expert_gemv_gather_w4(xd, k, perm, offsets, W4, N_r, n_out, group)
        return idx, w, E, offsets, perm, inv, mr.mr_combine(E, w, inv)

    got = step()
    if mode == "graph":
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        torch.cuda.current_stream().wait_stream(st)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        got[-1].zero_()
        got[2].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert mr.mr_get_error() == mr.MR_OK
    idx, w, E, offsets, perm, inv, y = got
    want, mag, magx = gr.expert_w4(widen(x), perm.cpu().numpy(), offsets.cpu().numpy(), q, widen(s),
                             group, k)
    gr.check(widen(_host(E)), want, _bound(d, mag, magx), "bf16", "experts")
    terms = w.double()[:, :, None] * E.double()[inv.long()].reshape(T, k, -1)
    ry, mag = terms.sum(1).cpu().numpy(), terms.abs().sum(1).cpu().numpy()
    gr.check(widen(_host(y)), ry, (k + 1) * gr.U * mag, "bf16", "y")


def test_wrong_arguments_are_refused():
    q = torch.zeros((2, 16, 64), dtype=torch.uint8, device="cuda")
    s = torch.ones((2, 16, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mr.MRError):
        mr.mr_expert_pack_w4(q, s, 48)
    with pytest.raises(ValueError):
        mr.mr_expert_pack_w4(q, s, 64)  # 2 scales per row, not 4
    with pytest.raises(TypeError):
        mr.mr_expert_pack_w4(q, s.half(), 32)
    with pytest.raises(TypeError):
        mr.mr_expert_pack_w4(q.short(), s, 32)
    W4 = mr.mr_expert_pack_w4(q, s, 32)
    x = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
    perm = torch.zeros(2, dtype=torch.int32, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mr.mr_expert_gemv_gather_w4(x, 2, perm, off, W4[:-1], 2, 16, 32)
    with pytest.raises(ValueError):  # scales were packed as bf16
        mr.mr_expert_gemv_gather_w4(x, 2, perm, off, W4, 2, 16, 32, scale_dtype=torch.float32)
    with pytest.raises(TypeError):
        mr.mr_expert_gemv_gather_w4(x.float(), 2, perm, off, W4, 2, 16, 32)
    with pytest.raises(ValueError):
        mr.mr_expert_gemv_gather_w4(x, 2, perm, off[:2], W4, 2, 16, 32)
