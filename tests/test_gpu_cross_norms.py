"""Cross attention's outputs and gradients against the formula in 64 bits, in norm: per batch element,
head and tile of 128 tokens (of Q for o and dq, of K and V for dk and dv), so that a row, a split or a
tile that is lost shows, and so does an error of a per cent that has the same sign everywhere.  (Bounds
per element have to allow for every rounding at its worst at once.)

A rounding to bf16 is off by at most h = 2^-8 of the value, h / sqrt(3) in the root mean square, and
independent roundings add in their squares.  Such are, with bf16:
  P as an operand          error of O: sqrt(sum P^2 V^2), of dV: sqrt(sum P^2 dO^2)      (times h / sqrt(3))
  dS as an operand         error of dQ: scale sqrt(sum dS^2 K^2), of dK alike
  O, read for delta with more than 128 keys (its own P and its rounding):
      r = sqrt(sum P^2 dP^2 + sum dO^2 O^2) of a row; error of dQ: scale r |sum P K|, of dK: scale sqrt(sum P^2 r^2 Q^2)
  every output             its size
Twice their root of the sum of squares, in norm over a tile, covers a single rounding at its worst (sqrt(3)
of its root mean square) and any number of them together; 1e-4 beside it the sums in fp32.
fp32: 1e-5 of the norm of the result and of the root of the sum of the squares that make it up: a
product of three tf32 ones is within 1.75 2^-20 of its size, twice in a row (P or dS, then the sum),
and a logit of up to 16 brings 16 times its relative error of 2^-22 (random, over D products) into P.
"""
import math

import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_cross import SHAPES, masks, rand

TILE = 128
STEP = 2.0 ** -8 / math.sqrt(3.0)


def tiles_norm(x):
    """x [B, n, heads, D] -> the norm of each (batch element, tile of tokens, head)."""
    n = x.shape[1]
    x = torch.nn.functional.pad(x.double(), (0, 0, 0, 0, 0, -n % TILE))
    return x.unflatten(1, (-1, TILE)).square().sum((2, 4)).sqrt()


def formula(q, k, v, d_o, kv_len=None, key_mask=None):
    """{name: (value, size, noise)} in 64 bits: size is the root of the sum of the squares of the
    terms, noise that of the roundings to bf16 over STEP."""
    n_q, H, D = q.shape[1:]
    n_kv, G = k.shape[1], H // k.shape[2]
    scale = D ** -0.5
    seen = torch.ones((q.shape[0], n_kv), dtype=torch.bool, device=q.device)
    if kv_len is not None:
        seen &= torch.arange(n_kv, device=q.device)[None] < kv_len[:, None]
    if key_mask is not None:
        seen &= key_mask.bool()
    h = lambda x: x.double().transpose(1, 2)                       # noqa: E731
    back = lambda x: x.transpose(1, 2)                             # noqa: E731
    share = lambda x: x.unflatten(1, (H // G, G)).sum(2)           # noqa: E731
    sq, T = torch.square, lambda x: x.transpose(2, 3)              # noqa: E731
    Q, K, V, dO = h(q), h(k).repeat_interleave(G, 1), h(v).repeat_interleave(G, 1), h(d_o)
    S = (Q @ T(K) * scale).masked_fill(~seen[:, None, None, :], -math.inf)
    P = torch.softmax(S, dim=-1).nan_to_num(0.0)                   # a row without keys: zeros
    O, dP = P @ V, dO @ T(V)
    delta = (P * dP).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    r2 = (sq(P) * sq(dP)).sum(-1, keepdim=True) + (sq(dO) * sq(O)).sum(-1, keepdim=True)
    if n_kv <= TILE:                                               # delta from P and dP in fp32
        r2 = torch.zeros_like(r2)
    mag2 = sq(P) * (sq(dP) + sq(delta) + sq(dO) @ T(sq(V)))
    dQ, dK, dV = scale * dS @ K, share(scale * T(dS) @ Q), share(T(P) @ dO)
    o2, dv2 = sq(P) @ sq(V), share(T(sq(P)) @ sq(dO))
    out = {"o": (O, o2, o2 + sq(O)),
           "dq": (dQ, scale ** 2 * mag2 @ sq(K), scale ** 2 * (sq(dS) @ sq(K) + r2 * sq(P @ K)) + sq(dQ)),
           "dk": (dK, share(scale ** 2 * T(mag2) @ sq(Q)),
                  share(scale ** 2 * T(sq(dS) + sq(P) * r2) @ sq(Q)) + sq(dK)),
           "dv": (dV, dv2, dv2 + sq(dV))}
    return {n: (back(x), back(y.sqrt()), back(z.sqrt())) for n, (x, y, z) in out.items()}


def too_far(got, x, m):
    """{name: worst norm of the difference over what is allowed} of the outputs `got` ({name: tensor})
    for the inputs x = (q, k, v, d_o) and masks m."""
    want = formula(*x, **m)
    worst = {}
    for name, t in got.items():
        value, size, noise = want[name]
        allowed = tiles_norm(value) + tiles_norm(size)
        allowed = 1e-4 * allowed + 2 * STEP * tiles_norm(noise) if x[0].dtype == torch.bfloat16 else 1e-5 * allowed
        d = tiles_norm(t.double() - value)
        if not bool(torch.isfinite(d).all()):
            worst[name] = math.inf
        else:                                                      # where nothing is allowed, nothing may differ
            worst[name] = float(torch.where(d == 0, 0.0, d / allowed).max())
    return worst


IDS = ["x".join(map(str, s)) for s in SHAPES]


def inputs(shape, dtype, dev):
    B, n_q, n_kv, H, hkv, D, kind = shape
    x = [rand(s, dtype, dev, 20 + i, 2.0 if i == 1 else 1.0)
         for i, s in ((1, (B, n_q, H, D)), (2, (B, n_kv, hkv, D)), (3, (B, n_kv, hkv, D)), (4, (B, n_q, H, D)))]
    return x, masks(kind, B, n_kv, dev)


# few keys; shared heads; many query rows; rows that share heads; few queries
MISTAKES = [(1, 700, 5, 12, 12, 128, "none"), (4, 33, 40, 32, 1, 64, "length"), (2, 513, 226, 4, 4, 128, "length"),
            (1, 512, 700, 8, 2, 128, "holes"), (2, 3, 900, 8, 2, 64, "length")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", MISTAKES, ids=["x".join(map(str, s)) for s in MISTAKES])
def test_the_bound_sees_mistakes(shape, dtype):
    """On the CPU: the rounded results of the formula pass; with a mistake of 1.5% they do not."""
    (q, k, v, d_o), m = inputs(shape, dtype, "cpu")
    good = {n: x.to(dtype) for n, (x, _, _) in formula(q, k, v, d_o, **m).items()}
    assert max(too_far(good, (q, k, v, d_o), m).values()) <= 1.0
    for name in good:                                              # 1.5% too large everywhere
        bad = {name: (good[name].double() * 1.015).to(dtype)}
        assert too_far(bad, (q, k, v, d_o), m)[name] > 1.0, name
    less = d_o.clone()                                             # the last query row leaves dK and dV
    less[:, -1] = 0.0
    bad = formula(q, k, v, less, **m)
    for name in ("dk", "dv"):
        assert too_far({name: bad[name][0].to(dtype)}, (q, k, v, d_o), m)[name] > 1.0, name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_gradients_in_norm(shape, dtype):
    dev = torch.device("cuda", 0)
    B, n_q, n_kv, H, hkv, D, _ = shape
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
    (q, k, v, d_o), m = inputs(shape, dtype, dev)
    o, lse = op.forward(q, k, v, return_lse=True, **m)
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse, **m)
    op.check_status()
    worst = too_far({"o": o, "dq": dq, "dk": dk, "dv": dv}, (q, k, v, d_o), m)
    assert max(worst.values()) <= 1.0, worst
