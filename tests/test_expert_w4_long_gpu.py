"""The expert layer on 4-bit weights where segments are long or the layer is
wide: the kernel for many rows, and the choice between the two kernels."""
import pytest
import torch

import gradients as gr
import token_dispatch_fp32_b200 as mr
from parity import widen
from test_backward_gpu import _i32
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
