"""The expert layer on 4-bit weights where segments are long or the layer is
wide: the kernel for many rows, and the choice between the two kernels."""
import numpy as np
import pytest
import torch

import gradients as gr
import token_dispatch_fp32_b200 as mr
from parity import widen
from test_backward_gpu import _i32, _rows
from test_expert_w4_gpu import _bound, _problem
from test_rows_gpu import _dev, _host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_out", [1001, 2056, 2079])
def test_columns_do_not_depend_on_the_width(n_out):
    """150 rows on each of eight experts: the last warp's lanes store only some
    columns, and every column is the one that a layer of whole warps has."""
    T, k, N_r, d, group = 200, 6, 8, 264, 32
    full = -(-n_out // 32) * 32
    x, perm, offsets, _, q, s = _problem(T, k, N_r, full, d, group, "f32", n_out)

    def layer(n):
        W4 = mr.mr_expert_pack_w4(torch.from_numpy(q[:, :n].copy()).cuda(),
                                  _dev(s[:, :n].copy()), group)
        return mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(perm), _i32(offsets), W4, N_r, n,
                                           group, scale_dtype=torch.float32)

    part, whole = layer(n_out), layer(full)
    assert torch.equal(part.view(torch.int16), whole[:, :n_out].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,k,N_r", [(16, 1, 1), (31, 1, 2), (32, 1, 1), (4, 8, 8), (33, 1, 1),
                                     (11, 3, 3)])
@pytest.mark.parametrize("n_out,d", [(32064, 72), (64064, 8)])
def test_few_rows_of_wide_layers(T, k, N_r, n_out, d):
    """Around the 32 rows from which a segment may be long, on layers of so many
    outputs (a vocabulary's) that the choice between the kernels arises."""
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, 32, "bf16", T + d)
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), 32)
    out = mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(perm), _i32(offsets), W4, N_r, n_out, 32)
    assert mr.mr_get_error() == mr.MR_OK
    want, mag, magx = gr.expert_w4(widen(x), perm, offsets, q, widen(s), 32, k)
    gr.check(widen(_host(out)), want, _bound(d, mag, magx), "bf16", "out")


def _layer(x, perm, offsets, q, s, group, k, sdt):
    N_r, n_out = q.shape[:2]
    st = torch.bfloat16 if sdt == "bf16" else torch.float32
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), group)
    return mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(perm), _i32(offsets), W4, N_r, n_out,
                                       group, scale_dtype=st)


@pytest.mark.parametrize("rows", [3, 150], ids=["few", "many"])
@pytest.mark.parametrize("group,sdt", [(32, "bf16"), (32, "f32"), (64, "f32"), (128, "bf16"),
                                       (128, "f32")])
def test_small_groups_behind_a_large_one_add_up(rows, group, sdt):
    """1 + 2^-8 from the first group, then 0.75 of fp32's step there (3 * 2^-25)
    from each of the others: exactly 1 + 2^-8 lies between two bf16 values and
    goes to the even one, 1; every addition rounded to nearest goes up, so that
    the sum ends above it and the result is 1 + 2^-7.  A sum that drops what lies
    below its last place stays where it is."""
    d, n_out, N_r = 7168, 2048, 4
    x = np.zeros((rows * N_r, d), np.float32)
    q = np.full((N_r, n_out, d // 2), 0x89, np.uint8)  # columns of weight 1 and 0
    x[:, 0], x[:, 2] = 1.0, 2.0 ** -8
    x[:, group::group] = 2.0 ** -25
    q[:, :, group // 2::group // 2] = 0x8B  # weight 3 in the first column of a group
    s = np.ones((N_r, n_out, d // group), np.float32)
    bits = lambda a: (a.view(np.uint32) >> 16).astype(np.uint16)
    offsets = np.arange(N_r + 1) * rows
    out = _layer(bits(x), np.arange(rows * N_r), offsets, q, bits(s) if sdt == "bf16" else s,
                 group, 1, sdt)
    assert mr.mr_get_error() == mr.MR_OK
    assert (out == 1 + 2.0 ** -7).all()


@pytest.mark.parametrize("T,k,N_r,n_out,d,group,sdt,hot", [
    (1100, 1, 1, 1000, 136, 32, "f32", 0),   # nine blocks of one expert, a tail of columns
    (600, 4, 8, 456, 1096, 128, "bf16", 1),  # one expert of five blocks
    (193, 8, 8, 2050, 64, 64, "bf16", 0),    # two blocks each, half a stage of columns
    (129, 8, 8, 1030, 3592, 32, "bf16", 0),  # 129 rows each, an odd number of half stages
    (64, 8, 8, 2300, 72, 32, "bf16", 0),     # one block of 64 rows each
    (33, 16, 16, 1100, 7168, 32, "bf16", 0),  # 33 rows each
    (40, 16, 16, 900, 2056, 64, "f32", 0),
    (300, 2, 6, 4100, 640, 128, "f32", 0),
])
def test_long_segments(T, k, N_r, n_out, d, group, sdt, hot):
    """Segments that all go to the many-row kernel, to its own bound: a group's
    GROUP / 16 tensor-core steps each round within 2 fp32 steps of its sum of
    magnitudes, its scaling and addition within half a step of the whole's: (GROUP
    / 8 + d / (2 GROUP) + 1) * 2^-23 of the sum of magnitudes."""
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, group, sdt, T + d, hot)
    out = _layer(x, perm, offsets, q, s, group, k, sdt)
    assert mr.mr_get_error() == mr.MR_OK
    want, mag, _ = gr.expert_w4(widen(x), perm, offsets, q, widen(s), group, k)
    assert np.diff(offsets).min() > 32
    gr.check(widen(_host(out)), want, (group / 8 + d / (2 * group) + 1) * 2.0 ** -23 * mag,
             "bf16", "out")


@pytest.mark.parametrize("T,k,N_r,n_out,d,group,sdt", [
    (1, 8, 64, 640, 7168, 32, "bf16"), (4, 8, 8, 330, 7168, 128, "f32"),
    (32, 2, 2, 96, 4104, 64, "bf16"),
])
def test_short_segments(T, k, N_r, n_out, d, group, sdt):
    """Segments of at most 32 rows, to the few-row kernel's own bound."""
    x, perm, offsets, _, q, s = _problem(T, k, N_r, n_out, d, group, sdt, T + d)
    out = _layer(x, perm, offsets, q, s, group, k, sdt)
    assert mr.mr_get_error() == mr.MR_OK
    assert np.diff(offsets).max() <= 32
    want, mag, magx = gr.expert_w4(widen(x), perm, offsets, q, widen(s), group, k)
    gr.check(widen(_host(out)), want, ((d / 128 + 16) * mag + 440 * magx) * 2.0 ** -23, "bf16",
             "out")


def test_a_thousand_long_segments():
    """34 rows on each of 1000 experts, the last 40 assignments dropped and one
    entry of perm out of range: rows behind the last segment stay, the bad entry
    is flagged and only its own row is affected."""
    N_r, n, k, n_out, d, group = 1000, 34000, 8, 96, 136, 32
    rng = np.random.default_rng(4)
    x = _rows(rng, (n // k, d), "bf16")
    q = rng.integers(0, 256, (N_r, n_out, d // 2)).astype(np.uint8)
    s = _rows(rng, (N_r, n_out, -(-d // group)), "bf16", 0.1)
    perm = rng.permutation(n).astype(np.int32)
    offsets = np.minimum(np.arange(N_r + 1) * 34, n - 40).astype(np.int32)
    W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), group)
    want, mag, _ = gr.expert_w4(widen(x), perm[:n - 40], offsets, q, widen(s), group, k)
    bound = (group / 8 + d / (2 * group) + 1) * 2.0 ** -23 * mag
    for bad in (False, True):
        p = perm.copy()
        if bad:
            p[500] = n
        out = torch.full((n, n_out), 7.0, dtype=torch.bfloat16, device="cuda")
        mr.mr_expert_gemv_gather_w4(_dev(x), k, _i32(p), _i32(offsets), W4, N_r, n_out, group,
                                    out=out)
        assert mr.mr_get_error() == (mr.MR_ERR_DEVICE if bad else mr.MR_OK)
        keep = np.arange(n - 40) != (500 if bad else -1)
        gr.check(widen(_host(out))[:n - 40][keep], want[keep], bound[keep], "bf16", "out")
        assert (out[n - 40:] == 7.0).all()


def test_two_layers_at_once():
    """Layers of long segments on two streams, each as alone."""
    probs = [_problem(600, 8, 16, 2048, 1032, 32, "bf16", seed) for seed in (1, 2)]
    calls = []
    for x, perm, offsets, _, q, s in probs:
        W4 = mr.mr_expert_pack_w4(torch.from_numpy(q).cuda(), _dev(s), 32)
        calls.append((_dev(x), 8, _i32(perm), _i32(offsets), W4, 16, 2048, 32))
    ref = [mr.mr_expert_gemv_gather_w4(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [mr.mr_expert_gemv_gather_w4(*c, stream=s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert mr.mr_get_error() == mr.MR_OK
