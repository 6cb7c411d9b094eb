"""GPU: gradients where a key mask leaves few of many keys and the attended keys are not gathered
(fewer than 2048 query rows to a K/V head).  One attended key has probability 1 whatever its logit,
so that its dQ and dK are exactly zero, however many keys the mask hides."""
import math

import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_cross import check, dev, oracle, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q,n_kv,H,hkv", [(200, 300, 2, 2), (1, 129, 4, 1), (2, 5000, 4, 2), (700, 1111, 2, 1)])
def test_one_attended_key_among_many(n_q, n_kv, H, hkv, D, dtype, dev):  # noqa: F811
    B = 4
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
    q, d_o = rand((B, n_q, H, D), dtype, dev, 1, 3.0), rand((B, n_q, H, D), dtype, dev, 4)
    k, v = rand((B, n_kv, hkv, D), dtype, dev, 2), rand((B, n_kv, hkv, D), dtype, dev, 3)
    # one key in the first tile, one in the last, one of two left by the length, and two
    mask = torch.zeros((B, n_kv), dtype=torch.bool, device=dev)
    mask[0, 7] = mask[1, n_kv - 1] = mask[2, 3] = mask[2, n_kv - 2] = mask[3, 0] = mask[3, n_kv - 1] = True
    m = {"key_mask": mask, "kv_len": torch.tensor([n_kv, n_kv, n_kv - 2, n_kv], dtype=torch.int32, device=dev)}
    o, lse = op.forward(q, k, v, return_lse=True, **m)
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse, **m)
    op.check_status()
    ref = oracle(q, k, v, d_o, **m)
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, t, ref[name])
    assert not dq[:3].any() and not dk[:3].any()
    assert dq[3].any() and dk[3].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_replayed_graph_counts_the_keys_anew(dtype, dev):  # noqa: F811
    B, n_q, n_kv, H, D = 2, 130, 4500, 1, 64
    op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, device=dev)
    x = [rand(s, dtype, dev, i) for i, s in enumerate((op.q_shape, op.kv_shape, op.kv_shape, op.q_shape))]
    mask = torch.ones((B, n_kv), dtype=torch.bool, device=dev)
    o, lse = op.forward(*x[:3], key_mask=mask, return_lse=True)
    op.backward(x[3], *x[:3], o, lse, key_mask=mask)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = op.forward(*x[:3], key_mask=mask, return_lse=True)
        dq, dk, dv = op.backward(x[3], *x[:3], o, lse, key_mask=mask)
    for keys in ([4499], [0, 4499], [17], []):
        mask.zero_()
        mask[1, keys] = True
        mask[0, 5:400] = True
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle(*x, key_mask=mask)
        for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            check(name, t, ref[name])
        assert bool(dq[1].any()) == bool(dk[1].any()) == (len(keys) > 1) and dq[0].any()


@pytest.mark.parametrize("n_kv", [1, 40, 300])
def test_a_single_key_that_is_nan_shows(n_kv, dev):  # noqa: F811
    # bf16 (fp32 asks for finite values at attended keys)
    op = bsa.CrossAttention(1, 200, n_kv, 1, 1, 64, torch.bfloat16, device=dev)
    q, k, v, d_o = (rand(s, torch.bfloat16, dev, i)
                    for i, s in enumerate((op.q_shape, op.kv_shape, op.kv_shape, op.q_shape)))
    at = n_kv // 2
    k[0, at] = math.nan
    mask = torch.zeros((1, n_kv), dtype=torch.bool, device=dev)
    mask[0, at] = True
    o, lse = op.forward(q, k, v, key_mask=mask, return_lse=True)
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse, key_mask=mask)
    for t in (o, lse, dq, dk[0, at], dv[0, at]):
        assert torch.isnan(t).all()
    rest = torch.arange(n_kv, device=dev) != at
    assert not dk[0, rest].any() and not dv[0, rest].any()
