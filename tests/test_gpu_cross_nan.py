"""GPU: a NaN that a query or an attended key holds is not taken for "no attended key" when the keys
of a call are split over CTAs (few queries) and the partial rows are merged: every row it enters is
NaN, with a NaN lse and NaN gradients, as in a call whose keys are not split; every other row keeps
its bits."""
import math

import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_cross import dev, rand  # noqa: F401

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def split_call(dtype, dev, D, n_kv=5000):  # noqa: F811
    """Three queries of four heads; over long keys the forward needs a workspace (its partials)."""
    op = bsa.CrossAttention(2, 3, n_kv, 4, 2, D, dtype, device=dev)
    assert op.forward_ws > 0 or n_kv < 1000
    return op, [rand(s, dtype, dev, i) for i, s in enumerate((op.q_shape, op.kv_shape, op.kv_shape, op.q_shape))]


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_kv", [300, 5000, 20000])
def test_a_nan_query(n_kv, D, dtype, dev):  # noqa: F811
    op, (q, k, v, d_o) = split_call(dtype, dev, D, n_kv)
    clean, clean_lse = op.forward(q, k, v, return_lse=True)
    q[1, 2, 3, 5] = math.nan
    o, lse = op.forward(q, k, v, return_lse=True)
    assert torch.isnan(o[1, 2, 3]).all() and torch.isnan(lse[1, 3, 2])
    keep = torch.ones(o.shape[:3], dtype=torch.bool, device=dev)
    keep[1, 2, 3] = False
    assert torch.equal(o[keep], clean[keep])
    assert torch.equal(lse[keep.transpose(1, 2)], clean_lse[keep.transpose(1, 2)])
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse)
    assert torch.isnan(dq[1, 2, 3]).all()
    assert torch.isnan(dk[1, :, 1]).all() and torch.isnan(dv[1, :, 1]).all()     # head 3 reads K/V head 1
    for t in (dq[keep], dk[0], dv[0], dk[1, :, 0], dv[1, :, 0]):
        assert torch.isfinite(t).all()


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
def test_states_that_are_all_nan(D, dtype, dev):  # noqa: F811
    op, (q, k, v, _) = split_call(dtype, dev, D)
    clean, clean_lse = op.forward(q, k, v, return_lse=True)
    k[1] = math.nan
    for length in (None, torch.tensor([5000, 4100], dtype=torch.int32, device=dev)):
        o, lse = op.forward(q, k, v, kv_len=length, return_lse=True)
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
        assert torch.equal(o[0], clean[0]) and torch.equal(lse[0], clean_lse[0])


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_lone_nan_key(where, D, dtype, dev):  # noqa: F811
    # batch element 0 attends key 10 (NaN) and key 4000, in different splits; element 1 key 10 alone
    op, (q, k, v, _) = split_call(dtype, dev, D)
    (k if where == "k" else v)[:, 10] = math.nan
    seen = torch.zeros((2, 5000), dtype=torch.bool, device=dev)
    seen[:, 10] = True
    seen[0, 4000] = True
    o, lse = op.forward(q, k, v, key_mask=seen, return_lse=True)
    assert torch.isnan(o).all()
    assert torch.isnan(lse).all() if where == "k" else torch.isfinite(lse).all()
    # hidden, it leaves no trace: element 1 then attends nothing
    seen[:, 10] = False
    o, lse = op.forward(q, k, v, key_mask=seen, return_lse=True)
    # P = 1, so O = V: exactly in bf16; in fp32 V's low part (below 2^-10 of it) is cut to 11 bits
    want = v[0, 4000].repeat_interleave(2, dim=0).expand(3, -1, -1)
    assert ((o[0] - want).abs() <= (2.0 ** -20 if dtype == torch.float32 else 0.0) * want.abs()).all()
    assert not o[1].any() and bool((lse[1] == -math.inf).all())


@DTYPES
def test_a_nan_value_of_no_weight(dtype, dev):  # noqa: F811
    # key 10 holds NaN in V; its probability is far below the smallest number, and 0 NaN is NaN
    op, (q, k, v, _) = split_call(dtype, dev, 64)
    q[:] = 1.0
    k[:] = 0.0
    k[:, 10] = -64.0            # logit -64 * 64 / 8 = -512
    k[:, 4000] = 64.0
    v[:, 10] = math.nan
    seen = torch.zeros((2, 5000), dtype=torch.bool, device=dev)
    seen[:, 10] = seen[:, 4000] = True
    assert torch.isnan(op.forward(q, k, v, key_mask=seen)).all()
