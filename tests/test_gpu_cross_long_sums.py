"""GPU: long sums of terms of one sign, whose roundings must not all go one way.

The tensor core rounds each addition toward zero, so a sum that it carries over n products loses about
n 2^-25 of itself; added up tile by tile in fp32 (to nearest) the errors cancel like a random walk.
Bound for fp32, relative in norm: the products lose up to 1.75 2^-20 (both low parts of a product are
cut) of a term, twice (in the logit, times its size of at most 1, and in the product that is summed),
the exponential, lse and scale 2^-20, a tile's own additions 4 2^-23, the random walk of 4096 tiles
64 2^-24: together below 1e-5.  A sum carried over 32 768 rows would be off by 1e-4.
For bf16: half a step of the output (2^-8) and as much again for P.
"""
import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_cross import dev  # noqa: F401

pytestmark = pytest.mark.gpu

ALLOWED = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -7}


def draw(shape, dtype, dev, seed, scale=1.0, positive=False):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
    return (x.abs_() if positive else x).mul_(scale).to(dtype)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype,n_q,heads", [(torch.float32, 32768, 37), (torch.bfloat16, 131072, 37)],
                         ids=["f32", "bf16"])
def test_gradients_over_many_rows(dtype, n_q, heads, dev):  # noqa: F811
    # 37 heads of 512 keys: as many CTAs as the GPU takes at a time, so that rows are not split
    n_kv, D = 512, 64
    op = bsa.CrossAttention(1, n_q, n_kv, heads, heads, D, dtype, device=dev)
    q, k = draw(op.q_shape, dtype, dev, 1, 0.25), draw(op.kv_shape, dtype, dev, 2, 0.25)
    v, d_o = draw(op.kv_shape, dtype, dev, 3), draw(op.q_shape, dtype, dev, 4, 1.0, True)
    q += 0.25                           # with dO of one sign dS has a part of one sign for each key: dK is a long sum too
    o, lse = op.forward(q, k, v, return_lse=True)
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse)
    op.check_status()
    for h in (0, heads - 1):
        Q, K, V, G = (t[0, :, h].double() for t in (q, k, v, d_o))
        P = torch.softmax(Q @ K.T * D ** -0.5, dim=-1)
        assert off(dv[0, :, h], P.T @ G) <= ALLOWED[dtype]
        dS = G @ V.T
        dS = P.mul_(dS - (P * dS).sum(-1, keepdim=True)) * D ** -0.5
        assert off(dk[0, :, h], dS.T @ Q) <= ALLOWED[dtype]
        assert off(dq[0, :, h], dS @ K) <= ALLOWED[dtype]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_forward_and_dq_over_many_keys(dtype, dev):  # noqa: F811
    # 111 heads of 256 query rows fill the GPU three times over: keys are not split
    n_q, n_kv, heads, D = 256, 32768, 111, 64
    op = bsa.CrossAttention(1, n_q, n_kv, heads, heads, D, dtype, device=dev)
    q, k = draw(op.q_shape, dtype, dev, 1, 0.25), draw(op.kv_shape, dtype, dev, 2, 0.25)
    v, d_o = draw(op.kv_shape, dtype, dev, 3, 1.0, True), draw(op.q_shape, dtype, dev, 4)
    o, lse = op.forward(q, k, v, return_lse=True)
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse)
    op.check_status()
    for h in (0, heads - 1):
        Q, K, V, G = (t[0, :, h].double() for t in (q, k, v, d_o))
        S = Q @ K.T * D ** -0.5
        P = torch.softmax(S, dim=-1)
        assert off(o[0, :, h], P @ V) <= ALLOWED[dtype]
        assert off(lse[0, h], torch.logsumexp(S, dim=-1)) <= 2.0 ** -20
        assert off(dv[0, :, h], P.T @ G) <= ALLOWED[dtype]
