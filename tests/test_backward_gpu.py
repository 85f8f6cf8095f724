"""Gradients of combine, gather and gate on the GPU against binary64
(tests/gradients.py), within bounds that follow from the arithmetic."""
import numpy as np
import pytest
import torch

import gradients as gr
import oracle
import token_dispatch_fp32_b200 as mr
from parity import widen
from test_rows_gpu import _dev, _host, _offset_view

pytestmark = pytest.mark.gpu


def _bits(a, dtype):
    return (a.view(np.uint32) >> 16).astype(np.uint16) if dtype == "bf16" else a


def _rows(rng, shape, dtype, scale=1.0):
    return _bits((rng.standard_normal(shape) * scale).astype(np.float32), dtype)


def _ids(rng, T, k, N_r, hot=0):
    score = rng.random((T, N_r))
    if hot:
        score[:, :hot] += 1
    return np.argsort(-score, 1)[:, :k].astype(np.int32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def _combine_problem(T, d, k, N_r, dtype, seed, hot=0):
    rng = np.random.default_rng(seed)
    idx = _ids(rng, T, k, N_r, hot)
    _, _, _, inv = oracle.dispatch(idx, N_r)
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    return rng, inv, w, _rows(rng, (T, d), dtype), _rows(rng, (T * k, d), dtype)


ROWS = [  # T, d, k, N_r, dtype
    (300, 7168, 8, 256, "bf16"),
    (257, 512, 4, 64, "f32"),
    (100, 1001, 3, 40, "bf16"),    # odd row: element path
    (50, 1000, 4, 16, "bf16"),     # 2000-byte rows: 16-byte vectors, not 32
    (51, 1004, 4, 16, "f32"),      # 4016-byte rows, the same in fp32
    (64, 37, 2, 8, "f32"),         # ragged fp32 row
    (1, 8, 1, 1, "bf16"),          # one token, one expert, one 16-byte vector
    (1, 1, 1, 3, "f32"),           # one element
    (33, 64, 9, 64, "bf16"),       # k just past one group of slots
    (65, 96, 32, 40, "f32"),       # k = 32
]


@pytest.mark.parametrize("T,d,k,N_r,dtype", ROWS)
def test_combine_backward(T, d, k, N_r, dtype):
    _, inv, w, dy, E = _combine_problem(T, d, k, N_r, dtype, seed=T + 3 * d)
    dE, dw = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(inv))
    assert mr.mr_get_error() == mr.MR_OK
    rE, rw, mag = gr.combine_backward(widen(dy), widen(E), w, inv, k)
    gr.check(widen(_host(dE)), rE, gr.U * np.abs(rE), dtype, "dexpert")
    gr.check(dw.cpu().numpy(), rw, (d + 2) * gr.U * mag, "f32", "dw")
    # one output at a time, bit for bit the same
    only, none = mr.mr_combine_backward(_dev(dy), None, _f32(w), _i32(inv), want_dw=False)
    assert none is None and torch.equal(only, dE)
    none, only = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(inv), want_dexpert=False)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("d,dtype,k", [(7168, "bf16", 8), (512, "f32", 4), (1001, "bf16", 3)])
def test_combine_backward_skips_dropped_slots(d, dtype, k):
    """A dropped slot (inv -1) writes no row and has dw 0; the expert rows no
    slot names are not read (they hold NaN), those of dexpert stay as they
    were; a token with every slot dropped has no gradient."""
    T, N_r = 300, 32
    rng, inv, w, dy, E = _combine_problem(T, d, k, N_r, dtype, seed=17)
    drop = rng.random(T * k) < 0.15
    drop[:k] = True
    lost = inv[drop]
    inv = np.where(drop, -1, inv).astype(np.int32)
    E[lost] = _bits(np.array([np.nan], np.float32), dtype)[0] if dtype == "f32" else 0x7FC1
    poison = _dev(np.full((T * k, d), 0x7FC1, np.uint16) if dtype == "bf16"
                  else np.full((T * k, d), np.nan, np.float32))
    before = _host(poison.clone())
    dE, dw = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(inv), dexpert=poison)
    rE, rw, mag = gr.combine_backward(widen(dy), widen(E), w, inv, k)
    got = _host(dE)
    kept = np.setdiff1d(np.arange(T * k), lost)
    gr.check(widen(got)[kept], rE[kept], gr.U * np.abs(rE[kept]), dtype, "dexpert")
    assert np.array_equal(got[lost].view(np.uint8), before[lost].view(np.uint8))
    gr.check(dw.cpu().numpy(), rw, (d + 2) * gr.U * mag, "f32", "dw")
    assert (dw.cpu().numpy().reshape(-1)[drop] == 0).all()


@pytest.mark.parametrize("T,d,k,N_r,dtype", ROWS)
@pytest.mark.parametrize("with_add", [True, False], ids=["add", "noadd"])
def test_gather_backward(T, d, k, N_r, dtype, with_add):
    rng = np.random.default_rng(T * 5 + d)
    _, _, _, inv = oracle.dispatch(_ids(rng, T, k, N_r), N_r)
    dxs = _rows(rng, (T * k, d), dtype)
    add = _rows(rng, (T, d), dtype) if with_add else None
    dx = mr.mr_gather_rows_backward(_dev(dxs), k, _i32(inv), None if add is None else _dev(add))
    assert mr.mr_get_error() == mr.MR_OK
    want, mag = gr.gather_backward(widen(dxs), inv, k, None if add is None else widen(add))
    gr.check(widen(_host(dx)), want, (k + 1) * gr.U * mag, dtype, "dx")
    if with_add:  # in place: add is the output
        out = _dev(add)
        mr.mr_gather_rows_backward(_dev(dxs), k, _i32(inv), add=out, dx=out)
        assert torch.equal(out, dx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gather_backward_skips_dropped_slots(dtype):
    T, d, k, N_r = 200, 512, 4, 16
    rng = np.random.default_rng(8)
    _, _, _, inv = oracle.dispatch(_ids(rng, T, k, N_r), N_r)
    dxs = _rows(rng, (T * k, d), dtype)
    drop = rng.random(T * k) < 0.2
    drop[4:8] = True  # token 1 has no slot left
    dxs[inv[drop]] = 0x7FC1 if dtype == "bf16" else np.nan  # not read
    inv = np.where(drop, -1, inv).astype(np.int32)
    dx = mr.mr_gather_rows_backward(_dev(dxs), k, _i32(inv))
    want, mag = gr.gather_backward(np.where(np.isnan(widen(dxs)), 0, widen(dxs)), inv, k)
    gr.check(widen(_host(dx)), want, (k + 1) * gr.U * mag, dtype, "dx")
    assert (widen(_host(dx))[1] == 0).all()


@pytest.mark.parametrize("d", [1, 2, 3, 509, 510, 511, 1021, 1022, 1023, 1500])
@pytest.mark.parametrize("off", [0, 1])
def test_gather_backward_of_rows_inside_words(d, off):
    """bf16 rows of any width and start, some slots dropped: what lies before
    and behind dxs and the rows of dropped slots (NaN) stay out of the sums,
    and nothing outside dx is written."""
    T, k, N_r = 90, 5, 16
    rng = np.random.default_rng(d)
    _, _, _, inv = oracle.dispatch(_ids(rng, T, k, N_r), N_r)
    dxs, add = _rows(rng, (T * k, d), "bf16"), _rows(rng, (T, d), "bf16")
    drop = rng.random(T * k) < 0.2
    drop[inv == 0] = drop[inv == T * k - 1] = False  # the first and the last row are read
    dxs[inv[drop]] = 0x7FC1
    inv = np.where(drop, -1, inv).astype(np.int32)

    def inside(a):
        buf = torch.full((a.size + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = buf[8 + off:8 + off + a.size].view(a.shape)
        view.copy_(_dev(a))
        return buf, view

    (_, src), (_, plus), (buf, out) = inside(dxs), inside(add), inside(np.zeros_like(add))
    mr.mr_gather_rows_backward(src, k, _i32(inv), add=plus, dx=out)
    assert mr.mr_get_error() == mr.MR_OK
    want, mag = gr.gather_backward(np.where(np.isnan(widen(dxs)), 0, widen(dxs)), inv, k,
                                   widen(add))
    gr.check(widen(_host(out.contiguous())), want, (k + 1) * gr.U * mag, "bf16", "dx")
    assert buf[:8 + off].isnan().all() and buf[8 + off + add.size:].isnan().all()
    mr.mr_gather_rows_backward(src, k, _i32(inv), add=plus, dx=plus)  # in place
    assert torch.equal(plus, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", [16, 4])
def test_row_gradients_on_unaligned_buffers(dtype, off):
    """Buffers 16 and 4 bytes past a 32-byte boundary: 16-byte vectors and
    elements; dexpert and dx do not depend on the path."""
    T, d, k, N_r = 77, 512, 4, 16
    rng, inv, w, dy, E = _combine_problem(T, d, k, N_r, dtype, seed=5)
    ref = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(inv))
    out = _offset_view(np.zeros_like(E), off)
    dE, dw = mr.mr_combine_backward(_offset_view(dy, off), _offset_view(E, off), _f32(w),
                                    _i32(inv), dexpert=out)
    assert torch.equal(dE, ref[0])
    _, rw, mag = gr.combine_backward(widen(dy), widen(E), w, inv, k)
    gr.check(dw.cpu().numpy(), rw, (d + 2) * gr.U * mag, "f32", "dw")
    dx = mr.mr_gather_rows_backward(_offset_view(E, off), k, _i32(inv), add=_offset_view(dy, off))
    assert torch.equal(dx, mr.mr_gather_rows_backward(_dev(E), k, _i32(inv), add=_dev(dy)))


@pytest.mark.parametrize("T,d,k,N_r,dtype", [
    (700, 2048, 6, 64, "bf16"),   # the widest rows of small CTAs, 32-byte vectors
    (700, 2064, 6, 64, "bf16"),   # one vector more
    (300, 1032, 4, 16, "f32"),    # 32-byte vectors, one more than small CTAs take
    (300, 1020, 32, 40, "f32"),   # 16-byte vectors, k = 32
    (300, 511, 5, 16, "bf16"),    # elements, small CTAs
    (300, 513, 32, 40, "bf16"),   # elements, one more
    (9000, 24, 2, 16, "bf16"),    # more tokens than CTAs at once, few vectors
])
def test_row_gradients_of_narrow_rows(T, d, k, N_r, dtype):
    test_combine_backward(T, d, k, N_r, dtype)
    test_gather_backward(T, d, k, N_r, dtype, True)


# ---- gate -----------------------------------------------------------------------------------

GATE = [  # T, d, N_r, k, x, W, hot experts
    (300, 7168, 256, 8, "bf16", "f32", 0),
    (1500, 256, 64, 2, "bf16", "f32", 2),    # segments of 1500 rows: many pieces
    (64, 512, 64, 4, "f32", "f32", 0),       # the smallest configuration
    (257, 1001, 40, 3, "bf16", "f32", 5),    # odd rows: element paths
    (61, 36, 24, 5, "f32", "bf16", 0),       # 4-column vectors only
    (130, 200, 512, 8, "bf16", "bf16", 0),   # most experts: 64-column chunks
    (75, 67, 512, 8, "f32", "f32", 40),      # the same, odd
    (200, 384, 384, 8, "bf16", "f32", 0),
    (1, 8, 1, 1, "f32", "f32", 0),           # one expert: its weight is constant
    (1, 7168, 256, 8, "bf16", "f32", 0),     # one token
    (40, 128, 48, 32, "bf16", "f32", 0),     # k = 32
    (513, 64, 16, 1, "f32", "f32", 1),       # every token on one expert
    (33, 67, 20, 3, "bf16", "bf16", 0),      # odd rows of both
    (777, 264, 21, 3, "bf16", "f32", 0),     # experts no multiple of 8, a K tail of tokens
    (1100, 520, 130, 8, "bf16", "bf16", 3),  # experts just past one tensor-core tile
]


def _gate_problem(T, d, N_r, k, xdt, wdt, hot, seed):
    rng = np.random.default_rng(seed)
    x = _rows(rng, (T, d), xdt)
    W = _rows(rng, (N_r, d), wdt, 1 / np.sqrt(d))
    L = (widen(x) @ widen(W).T).astype(np.float32)
    idx = _ids(rng, T, k, N_r, hot)
    g = rng.standard_normal((T, k)).astype(np.float32)
    return rng, x, W, L, idx, g


def _check_gate(x, W, L, idx, g, xdt, flags, add, got, scale=2.5):
    dx, dW, dlog = got
    softmax = bool(flags & mr.MR_SCORE_SOFTMAX)
    dL, err = gr.dlogits(L, idx, g, scale, softmax, 0.0 if flags & mr.MR_NORM_NO_EPS else 1e-20)
    gr.check(dlog.cpu().numpy(), dL, err, "f32", "dlogits")
    rx, bx, rW, bW = gr.products(dL, err, widen(x), widen(W), None if add is None else widen(add))
    gr.check(widen(_host(dx)), rx, bx, xdt, "dx")
    gr.check(dW.cpu().numpy(), rW, bW, "f32", "dW")


@pytest.mark.parametrize("T,d,N_r,k,xdt,wdt,hot", GATE)
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_router_backward(T, d, N_r, k, xdt, wdt, hot, softmax):
    rng, x, W, L, idx, g = _gate_problem(T, d, N_r, k, xdt, wdt, hot, seed=T + d + N_r)
    flags = mr.MR_SCORE_SOFTMAX if softmax else (mr.MR_NORM_NO_EPS if k == 3 else 0)
    add = _rows(rng, (T, d), xdt) if k % 2 == 0 else None
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    dlog = torch.empty((T, N_r), device="cuda")
    args = (_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g))
    plan = (None, None) if softmax else (_i32(perm), _i32(offsets))
    dadd = None if add is None else _dev(add)
    dx, dW = mr.mr_router_backward(*args, *plan, 2.5, flags=flags, add=dadd, dlogits=dlog)
    assert mr.mr_get_error() == mr.MR_OK
    _check_gate(x, W, L, idx, g, xdt, flags, add, (dx, dW, dlog))
    # one output at a time, and again: bit for bit the same
    ox, none = mr.mr_router_backward(*args, None, None, 2.5, flags=flags, add=dadd, want_dW=False)
    assert none is None and torch.equal(ox, dx)
    none, oW = mr.mr_router_backward(*args, *plan, 2.5, flags=flags, want_dx=False)
    assert none is None and torch.equal(oW, dW)
    if add is not None:  # in place
        mr.mr_router_backward(*args, *plan, 2.5, flags=flags, add=dadd, dx=dadd, want_dW=False)
        assert torch.equal(dadd, dx)


@pytest.mark.parametrize("T,k,hot", [(2048, 8, 0), (4096, 8, 8), (9000, 8, 9)],
                         ids=["64", "128", "256"])
def test_router_backward_piece_sizes(T, k, hot):
    """Segments in pieces of 64, 128 and 256 rows (the other cases have 32)."""
    test_router_backward(T, 2048, 24, k, "bf16", "f32", hot, False)


@pytest.mark.parametrize("d", [1, 2, 3, 1020, 1021, 1022, 1023, 2043, 2045])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("T", [1, 2, 70])
def test_gate_weight_gradient_of_rows_inside_words(T, d, off):
    """bf16 rows of any width and start: what lies before and behind x (NaN)
    and a neighbouring row's ends (infinite) stay out of a row's sums."""
    N_r, k = 6, 2
    rng, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=T + d)
    if T > 2:
        idx[:, 0], idx[:, 1] = rng.integers(0, 3, T), rng.integers(3, 5, T)  # 5: no rows
        idx[T // 2] = 0, 5  # the only row of expert 5
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    buf = torch.full((T * d + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = buf[8 + off:8 + off + T * d].view(T, d)
    view.copy_(_dev(x))
    args = (_dev(W), _f32(L), _i32(idx), _f32(g), _i32(perm), _i32(offsets), 2.5)
    dlog = torch.empty((T, N_r), device="cuda")
    _, dW = mr.mr_router_backward(view, *args, dlogits=dlog, want_dx=False)
    assert mr.mr_get_error() == mr.MR_OK
    dL, err = gr.dlogits(L, idx, g, 2.5, False, 1e-20)
    _, _, rW, bW = gr.products(dL, err, widen(x), widen(W), None)
    gr.check(dW.cpu().numpy(), rW, bW, "f32", "dW")
    if T <= 2:
        return
    t = T // 2
    view[t - 1, d - 1] = float("inf")
    view[t + 1, 0] = float("inf")
    _, dW2 = mr.mr_router_backward(view, *args, want_dx=False)
    assert torch.equal(dW2[5], dW[5])  # expert 5 has row t alone
    assert torch.equal(dW2[:, 1:d - 1], dW[:, 1:d - 1])


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_router_backward_repeated_and_bad_ids(softmax):
    """A token may name one expert in two slots (their gradients add up); a
    slot with an id out of range has none and raises the device flag; the
    dispatch drops it from the permutation."""
    T, d, N_r, k = 90, 128, 24, 4
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=3)
    idx[:, 1] = idx[:, 0]
    idx[::7, 3] = idx[::7, 0]
    idx[5, 2], idx[11, 0], idx[12] = N_r, -1, [N_r + 3, -5, 1 << 30, N_r]
    _, offsets, perm, _ = mr.mr_dispatch(_i32(idx), N_r)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    dlog = torch.empty((T, N_r), device="cuda")
    flags = mr.MR_SCORE_SOFTMAX if softmax else 0
    dx, dW = mr.mr_router_backward(_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), perm, offsets,
                                   2.5, flags=flags, dlogits=dlog)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    _check_gate(x, W, L, idx, g, "bf16", flags, None, (dx, dW, dlog))
    if not softmax:
        assert (dx[12] == 0).all()


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_router_backward_extreme_logits(softmax):
    """Logits at which sigmoid saturates either way, and softmax puts all its
    weight on one expert: no overflow, no NaN, the bound of the formula."""
    T, d, N_r, k = 32, 64, 16, 4
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "f32", "f32", 0, seed=4)
    L[0], L[1], L[2] = 60.0, -60.0, np.linspace(-80, 80, N_r)
    L[3, idx[3]] = [40.0, -40.0, 1e-30, 20.0]
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    dlog = torch.empty((T, N_r), device="cuda")
    flags = mr.MR_SCORE_SOFTMAX if softmax else 0
    got = mr.mr_router_backward(_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), _i32(perm),
                                _i32(offsets), 2.5, flags=flags, dlogits=dlog)
    _check_gate(x, W, L, idx, g, "f32", flags, None, (*got, dlog))


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_router_backward_on_unaligned_buffers(softmax, xdt):
    """x, W, add and dx 4 bytes past a 16-byte boundary: the element paths."""
    T, d, N_r, k = 150, 256, 32, 4
    rng, x, W, L, idx, g = _gate_problem(T, d, N_r, k, xdt, "f32", 0, seed=9)
    add = _rows(rng, (T, d), xdt)
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    dlog = torch.empty((T, N_r), device="cuda")
    flags = mr.MR_SCORE_SOFTMAX if softmax else 0
    out = _offset_view(np.zeros_like(x), 4)
    dx, dW = mr.mr_router_backward(_offset_view(x, 4), _offset_view(W, 4), _f32(L), _i32(idx),
                                   _f32(g), _i32(perm), _i32(offsets), 2.5, flags=flags,
                                   add=_offset_view(add, 4), dx=out,
                                   dW=_offset_view(np.zeros_like(W), 4), dlogits=dlog)
    assert mr.mr_get_error() == mr.MR_OK
    _check_gate(x, W, L, idx, g, xdt, flags, add, (dx, dW, dlog))


def test_router_backward_drops_a_bad_permutation():
    """Entries of perm out of range, and offsets that overlap, do not reach
    memory: they are flagged."""
    T, d, N_r, k = 600, 64, 16, 2
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "f32", "f32", 1, seed=2)
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    bad = perm.copy()
    bad[[0, 700]] = T * k, -7
    args = (_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g))
    mr.mr_router_backward(*args, _i32(bad), _i32(offsets), 2.5)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    over = np.where(np.arange(N_r + 1) % 2, T * k, 0)  # every second segment is everything
    mr.mr_router_backward(*args, _i32(perm), _i32(over), 2.5)
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_gradients_drop_entries_past_the_rows(dtype):
    T, d, k, N_r = 40, 64, 2, 8
    rng, inv, w, dy, E = _combine_problem(T, d, k, N_r, dtype, seed=3)
    bad = inv.copy()
    bad[7], bad[20] = T * k, 1 << 30
    ref = np.where(np.isin(np.arange(T * k), [7, 20]), -1, inv)
    got = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(bad),
                                 dexpert=_dev(np.zeros_like(E)))
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    want = mr.mr_combine_backward(_dev(dy), _dev(E), _f32(w), _i32(ref),
                                  dexpert=_dev(np.zeros_like(E)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = mr.mr_gather_rows_backward(_dev(E), k, _i32(bad))
    assert mr.mr_get_error() == mr.MR_ERR_DEVICE
    assert torch.equal(got, mr.mr_gather_rows_backward(_dev(E), k, _i32(ref)))


def test_router_backward_without_tokens():
    W = torch.randn((8, 16), device="cuda")
    e = torch.empty((0, 16), device="cuda")
    dW = torch.full((8, 16), 7.0, device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    dx, _ = mr.mr_router_backward(e, W, torch.empty((0, 8), device="cuda"), i,
                                  torch.empty((0, 2), device="cuda"), i.reshape(-1),
                                  torch.zeros(9, dtype=torch.int32, device="cuda"), 2.5, dW=dW)
    assert dx.shape == (0, 16) and (dW == 0).all()


# ---- together -------------------------------------------------------------------------------


@pytest.mark.parametrize("mode", ["eager", "graph", "streams"])
def test_training_step_of_a_moe_layer(mode):
    """Gate, dispatch, gather, experts (one linear map each, in torch), combine
    and the shared row forward; then all their gradients, against torch's
    autograd in binary64 with the choice held.  Each of the six fp32 stages is
    off by at most n u of its terms, n <= max(d, T k) = 512, so a norm-wise
    12 n u covers both directions."""
    T, d, N_r, k = 96, 512, 16, 4
    torch.manual_seed(0)
    x = torch.randn((T, d), device="cuda")
    W = torch.randn((N_r, d), device="cuda") / d ** 0.5
    A = torch.randn((N_r, d, d), device="cuda") / d ** 0.5
    shared = torch.randn((T, d), device="cuda")
    dy = torch.randn((T, d), device="cuda")
    logits = torch.empty((T, N_r), device="cuda")
    idx, w = mr.mr_router_forward_ex(x, W, None, 1, 1, k, 2.5, mr.MR_MASK_NEG_INF,
                                     precision=mr.MR_PREC_3XTF32, logits_out=logits)
    _, offsets, perm, inv = mr.mr_dispatch(idx, N_r)
    xs = mr.mr_gather_rows(x, k, perm=perm, inv_perm=inv)
    o = offsets.tolist()
    E = torch.cat([xs[o[e]:o[e + 1]] @ A[e].t() for e in range(N_r)])
    mr.mr_combine(E, w, inv, shared)
    ws = torch.empty(mr.mr_router_backward_workspace_size(T, d, N_r, k), dtype=torch.uint8,
                     device="cuda")
    dxs = torch.empty_like(xs)

    def backward():
        dE, dw = mr.mr_combine_backward(dy, E, w, inv)
        for e in range(N_r):
            if o[e] < o[e + 1]:
                torch.mm(dE[o[e]:o[e + 1]], A[e], out=dxs[o[e]:o[e + 1]])
        dx = mr.mr_gather_rows_backward(dxs, k, inv, add=dy)  # the shared expert: identity
        return (dE, dw) + mr.mr_router_backward(x, W, logits, idx, dw, perm, offsets, 2.5, add=dx,
                                                dx=dx, workspace=ws)

    if mode == "eager":
        got = backward()
    elif mode == "streams":
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = backward()
        torch.cuda.current_stream().wait_stream(s)
    else:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            backward()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = backward()
        for t in got:
            t.fill_(float("nan"))
        ws.fill_(255)
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    assert mr.mr_get_error() == mr.MR_OK

    X, Wg = x.double().requires_grad_(), W.double().requires_grad_()
    s = torch.sigmoid(X @ Wg.t()).gather(1, idx.long())
    wt = s / (s.sum(1, keepdim=True) + 1e-20) * 2.5
    wt.retain_grad()
    rows = [X[perm[o[e]:o[e + 1]].long() // k] @ A[e].double().t() for e in range(N_r)]
    Er = torch.cat(rows)
    Er.retain_grad()
    y = (wt[:, :, None] * Er[inv.long()].reshape(T, k, d)).sum(1) + X
    (y * dy.double()).sum().backward()
    for name, a, b in (("dexpert", got[0], Er.grad), ("dw", got[1], wt.grad),
                       ("dx", got[2], X.grad), ("dW", got[3], Wg.grad)):
        rel = ((a.double() - b).norm() / b.norm()).item()
        assert rel <= 12 * 512 * gr.U, (name, rel)


def test_two_gradients_at_once():
    """The same call on two streams with a workspace each, against the calls
    one after the other."""
    T, d, N_r, k = 700, 1024, 64, 4
    probs = [_gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=s) for s in (1, 2)]
    calls = []
    for _, x, W, L, idx, g in probs:
        _, offsets, perm, _ = oracle.dispatch(idx, N_r)
        calls.append((_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), _i32(perm), _i32(offsets)))
    ref = [mr.mr_router_backward(*c, 2.5) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(mr.mr_router_backward(*c, 2.5))
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        del got


@pytest.mark.parametrize("flags", [0, mr.MR_SCORE_SOFTMAX])
def test_workspace_of_a_call_on_a_named_stream(flags):
    """stream= without a workspace: the one the call allocates is not handed to
    work of the current stream while the call still waits to run."""
    T, d, N_r, k = 700, 1024, 64, 4
    _, x, W, L, idx, g = _gate_problem(T, d, N_r, k, "bf16", "f32", 0, seed=3)
    _, offsets, perm, _ = oracle.dispatch(idx, N_r)
    args = (_dev(x), _dev(W), _f32(L), _i32(idx), _f32(g), _i32(perm), _i32(offsets), 2.5, flags)
    ref = mr.mr_router_backward(*args)
    dref = mr.mr_dispatch(args[3], N_r)
    s = torch.cuda.Stream()
    size = max(mr.mr_router_backward_workspace_size(T, d, N_r, k, flags), 16)
    dsize = max(mr.mr_dispatch_workspace_size(T, k, N_r), 4)
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # some ten milliseconds
        got = mr.mr_router_backward(*args, stream=s)
        dgot = mr.mr_dispatch(args[3], N_r, stream=s)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (size, size, dsize, dsize)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        assert all(torch.equal(a, b) for a, b in zip(dgot, dref))
        del got, dgot


def test_wrong_arguments_are_refused():
    T, d, k, N_r = 4, 16, 2, 8
    dy = torch.zeros((T, d), device="cuda")
    E = torch.zeros((T * k, d), device="cuda")
    w = torch.zeros((T, k), device="cuda")
    inv = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mr.mr_combine_backward(dy, E.bfloat16(), w, inv)
    with pytest.raises(ValueError):
        mr.mr_combine_backward(dy, None, w, inv)
    with pytest.raises(ValueError):
        mr.mr_combine_backward(dy.t(), E, w, inv)
    with pytest.raises(TypeError):
        mr.mr_combine_backward(dy.half(), E.half(), w, inv)
    with pytest.raises(mr.MRError):
        mr.mr_combine_backward(dy, None, w, inv, want_dexpert=False, want_dw=False)
    with pytest.raises(ValueError):
        mr.mr_gather_rows_backward(E[:7], k, inv)
    with pytest.raises(TypeError):
        mr.mr_gather_rows_backward(E, k, inv.long())
    with pytest.raises(TypeError):
        mr.mr_gather_rows_backward(E.cpu(), k, inv)
    x, W = torch.zeros((T, d), device="cuda"), torch.zeros((N_r, d), device="cuda")
    L, idx = torch.zeros((T, N_r), device="cuda"), inv.reshape(T, k)
    off = torch.zeros(N_r + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mr.mr_router_backward(x, W, L[:, :4].contiguous(), idx, w, inv, off, 2.5)
    with pytest.raises(mr.MRError):
        mr.mr_router_backward(x, W, L, idx, w, None, None, 2.5)  # dW needs the permutation
    with pytest.raises(mr.MRError):
        mr.mr_router_backward(x, W, L, idx, w, inv, off, 2.5,
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
