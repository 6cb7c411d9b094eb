"""GPU: cross attention (CrossAttention.forward, .backward) against the formula in 64 bits.

Tolerances.  u is half a step of the tensors' type relative to the value (bf16 2^-8, fp32 2^-24);
for bf16 the probabilities P and their gradients dS are rounded to bf16 as operands of the matrix
products, for fp32 they are not (up = u or 0).  e bounds the relative error of a probability: a logit
is a sum of D products (each rounded at most twice, 2^-23 relative) and is scaled and shifted by the
maximum or the lse (a few roundings of numbers below |s| + |lse|), the exponential is within 2^-21.
Every other fp32 sum of n terms is within n 2^-24 of the sum of their magnitudes.
  O    off by  A (up + 2 e + n 2^-23),             A = P |V|;  then u |O|
  dV   off by  sum P |dO| (up + e + n 2^-23),      then u |dV|
  dS   off by  P t + |dS| (up + e),                t = errors of dP and of D = rowsum(dO O), where O
       comes rounded from the forward: 2^-23 D (|dO| |V|) + |dO| err(O) + D 2^-23 |dO| |O|
  dQ   off by  scale (errors of dS) |K| + n 2^-23 scale |dS| |K|, then u |dQ|;  dK alike.
For fp32 a product is three tf32 products, within 2^-20 of its size: for a logit that is inside
the D 2^-23 above (D >= 64), for the other products inside e >= 2^-20.
"""
import math
import random

import pytest
import torch

import block_sparse_attention_permute_b200 as bsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bsa.load()
    return torch.device("cuda", 0)


def rand(shape, dtype, dev, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)


def oracle(q, k, v, d_o=None, kv_len=None, key_mask=None, scale=None):
    """{name: (value, allowed error)} in 64 bits, from the definition."""
    B, n_q, H, D = q.shape
    n_kv, G = k.shape[1], H // k.shape[2]
    dt = q.dtype
    u = torch.finfo(dt).eps / 2
    up = u if dt == torch.bfloat16 else 0.0
    scale = D ** -0.5 if scale is None else scale
    dev = q.device
    seen = torch.ones((B, n_kv), dtype=torch.bool, device=dev)
    if kv_len is not None:
        seen &= torch.arange(n_kv, device=dev)[None] < kv_len[:, None]
    if key_mask is not None:
        seen &= key_mask.bool()
    h = lambda x: x.double().transpose(1, 2)                       # noqa: E731  [B, heads, n, D]
    wide = lambda x: h(x).repeat_interleave(G, dim=1)              # noqa: E731
    Q, K, V = h(q), wide(k), wide(v)
    hide = ~seen[:, None, :, None]
    K, V = K.masked_fill(hide, 0.0), V.masked_fill(hide, 0.0)
    S = (Q @ K.transpose(2, 3) * scale).masked_fill(~seen[:, None, None, :], -math.inf)
    lse = torch.logsumexp(S, dim=-1)
    some = lse > -math.inf
    P = torch.where(some[..., None], torch.exp(S - torch.where(some, lse, 0.0)[..., None]), 0.0)
    mag = Q.abs() @ K.abs().transpose(2, 3) * scale
    top = torch.where(seen[:, None, None, :], mag, 0.0).amax(dim=-1, keepdim=True)
    e = (D + 8) * 2.0 ** -23 * (top + torch.where(some, lse.abs(), 0.0)[..., None]) + 2.0 ** -20
    f = n_kv * 2.0 ** -23
    O, A = P @ V, P @ V.abs()
    eO = A * (up + 2 * e + f)
    eO = eO + u * (O.abs() + eO)
    back = lambda x: x.transpose(1, 2)                             # noqa: E731
    out = {"o": (back(O), back(eO)),
           "lse": (lse, e[..., 0] + f + 2.0 ** -22 * torch.where(some, lse.abs(), 0.0))}
    if d_o is None:
        return out
    dO = h(d_o)
    n = n_q * G * 2.0 ** -23
    dP = dO @ V.transpose(2, 3)
    delta = (dO * O).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    t = D * 2.0 ** -23 * (dO.abs() @ V.abs().transpose(2, 3)) + (dO.abs() * eO).sum(-1, keepdim=True) \
        + D * 2.0 ** -23 * (dO.abs() * O.abs()).sum(-1, keepdim=True)
    edS = P * t * (1 + e) + dS.abs() * (up + e) + P * t * up
    share = lambda x: x.unflatten(1, (H // G, G)).sum(2)           # noqa: E731
    for name, val, err in (
            ("dq", scale * dS @ K, scale * (edS @ K.abs() + f * (dS.abs() + edS) @ K.abs())),
            ("dk", share(scale * dS.transpose(2, 3) @ Q),
             share(scale * (edS.transpose(2, 3) @ Q.abs() + n * (dS.abs() + edS).transpose(2, 3) @ Q.abs()))),
            ("dv", share(P.transpose(2, 3) @ dO),
             share((P * (up + e + n) * (1 + e)).transpose(2, 3) @ dO.abs()))):
        out[name] = (back(val), back(err + u * (val.abs() + err)))
    return out


def check(name, got, want):
    val, tol = want
    got = got.double()
    assert got.shape == val.shape
    inf = torch.isinf(val)
    assert torch.equal(got[inf], val[inf]), name
    # 2^-130: results below the smallest normal number
    bad = ~((got - val)[~inf].abs() <= tol[~inf] + 2.0 ** -130)
    assert not bad.any(), (name, int(bad.sum()), float((got - val)[~inf].abs().max()),
                           float(((got - val)[~inf].abs() / (tol[~inf] + 1e-30)).max()))


def masks(kind, B, n_kv, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return {}
    if kind == "length":
        n = torch.randint(0, n_kv + 1, (B,), generator=g, dtype=torch.int32)
        n[-1] = n_kv if B > 1 else max(1, n_kv - 1)
        return {"kv_len": n.to(dev)}
    m = torch.rand((B, n_kv), generator=g) < 0.6
    if kind == "empty":                     # no key at all in the first batch element
        m[0] = False
    if kind == "one":
        m[:] = False
        m[:, n_kv // 2] = True
    out = {"key_mask": m.to(dev)}
    if kind == "both":
        out["kv_len"] = torch.full((B,), max(0, n_kv - 3), dtype=torch.int32, device=dev)
    return out


# B, n_q, n_kv, heads, heads_kv, head_dim, mask
SHAPES = [
    (1, 1, 1, 1, 1, 64, "none"),
    (2, 1, 129, 4, 1, 128, "length"),
    (1, 2, 63, 3, 3, 64, "holes"),
    (2, 63, 64, 2, 2, 128, "none"),
    (1, 64, 65, 6, 2, 64, "length"),
    (3, 65, 77, 5, 1, 128, "holes"),
    (1, 127, 128, 2, 1, 64, "both"),
    (2, 128, 127, 2, 2, 128, "empty"),
    (1, 129, 257, 3, 1, 128, "holes"),
    (2, 200, 300, 8, 2, 64, "one"),
    (1, 255, 256, 1, 1, 128, "none"),
    (1, 257, 511, 2, 2, 64, "length"),
    (2, 513, 226, 4, 4, 128, "length"),
    (1, 700, 5, 12, 12, 128, "none"),
    (1, 1300, 1, 2, 2, 64, "none"),
    (1, 3, 2000, 40, 8, 128, "length"),
    (2, 1, 5001, 6, 2, 64, "holes"),
    (1, 17, 9000, 1, 1, 128, "both"),
    (4, 33, 40, 256, 1, 64, "length"),
    (1, 1, 300, 127, 1, 64, "holes"),
    (2, 2, 150, 96, 1, 128, "length"),
    (3, 1, 1, 2, 1, 128, "none"),
    (1, 3000, 129, 1, 1, 64, "empty"),
    (2, 2100, 300, 2, 2, 128, "holes"),
    (2, 1050, 513, 4, 2, 64, "both"),
    (2, 2048, 1500, 1, 1, 128, "empty"),
    (2, 2048, 200, 3, 3, 64, "one"),
    (1, 512, 2300, 8, 2, 128, "holes"),
]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_gradients(shape, dtype, dev):
    B, n_q, n_kv, H, hkv, D, kind = shape
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
    q = rand((B, n_q, H, D), dtype, dev, 1, 2.0)
    k, v = rand((B, n_kv, hkv, D), dtype, dev, 2), rand((B, n_kv, hkv, D), dtype, dev, 3)
    d_o = rand((B, n_q, H, D), dtype, dev, 4)
    m = masks(kind, B, n_kv, dev)
    o, lse = op.forward(q, k, v, return_lse=True, **m)
    op.check_status()
    ref = oracle(q, k, v, d_o, **m)
    check("o", o, ref["o"])
    check("lse", lse, ref["lse"])
    assert torch.equal(op.forward(q, k, v, **m), o)
    g = op.backward(d_o, q, k, v, o, lse, **m)
    op.check_status()
    for name, x in zip(("dq", "dk", "dv"), g):
        check(name, x, ref[name])
    for x, y in zip(g, op.backward(d_o, q, k, v, o, lse, **m)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n_q", [1, 150, 1100])
def test_masked_keys_may_hold_anything(n_q, dtype, dev):
    B, n_kv, H, hkv, D = 2, 200, 4, 2, 64
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
    q, d_o = rand((B, n_q, H, D), dtype, dev, 1), rand((B, n_q, H, D), dtype, dev, 4)
    k, v = rand((B, n_kv, hkv, D), dtype, dev, 2), rand((B, n_kv, hkv, D), dtype, dev, 3)
    for kind in ("length", "holes"):
        m = masks(kind, B, n_kv, dev, 5)
        hide = torch.arange(n_kv, device=dev)[None] >= m["kv_len"][:, None] if kind == "length" else ~m["key_mask"]
        o, lse = op.forward(q, k, v, return_lse=True, **m)
        g = op.backward(d_o, q, k, v, o, lse, **m)
        for junk in (math.nan, math.inf, torch.finfo(dtype).min):
            k2, v2 = k.clone(), v.clone()
            k2[hide], v2[hide] = junk, junk
            o2, lse2 = op.forward(q, k2, v2, return_lse=True, **m)
            assert torch.equal(o2, o) and torch.equal(lse2, lse), (kind, junk)
            for x, y in zip(g, op.backward(d_o, q, k2, v2, o, lse, **m)):
                assert torch.equal(x, y), (kind, junk)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_views_of_fused_projections(dtype, dev):
    B, n_q, n_kv, H, D = 2, 140, 90, 3, 128
    op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, device=dev)
    kv = rand((B, n_kv, 2, H, D), dtype, dev, 1)
    k, v = kv[:, :, 0], kv[:, :, 1]
    q = rand((B, H, n_q, D), dtype, dev, 2).transpose(1, 2)        # heads before tokens
    one = rand((1, n_q, H, D), dtype, dev, 3).expand(B, -1, -1, -1)  # the same gradient for all
    o, lse = op.forward(q, k, v, return_lse=True)
    want = op.forward(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(o, want)
    # into a strided buffer, whose other elements stay
    buf = torch.full((B, n_q, 2, H, D), 7.0, dtype=dtype, device=dev)
    op.forward(q, k, v, out=buf[:, :, 1])
    assert torch.equal(buf[:, :, 1], o) and bool((buf[:, :, 0] == 7.0).all())
    g = op.backward(one, q, k, v, o, lse)
    g2 = op.backward(one.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), o, lse)
    dkv = torch.empty_like(kv)
    dq = torch.empty((B, H, n_q, D), dtype=dtype, device=dev).transpose(1, 2)
    op.backward(one, q, k, v, o, lse, out=(dq, dkv[:, :, 0], dkv[:, :, 1]))
    for x, y, z in zip(g, g2, (dq, dkv[:, :, 0], dkv[:, :, 1])):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_shared_states_of_a_broadcast_batch(dev):
    # the same encoder states for every batch element, without a copy
    B, n_q, n_kv, H, D = 3, 70, 130, 2, 128
    for dtype in (torch.float32, torch.bfloat16):
        op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, device=dev)
        q, d_o = rand((B, n_q, H, D), dtype, dev, 1), rand((B, n_q, H, D), dtype, dev, 2)
        k, v = (rand((1, n_kv, H, D), dtype, dev, s).expand(B, -1, -1, -1) for s in (3, 4))
        o, lse = op.forward(q, k, v, return_lse=True)
        assert torch.equal(o, op.forward(q, k.contiguous(), v.contiguous()))
        ref = oracle(q, k, v, d_o)
        for name, x in zip(("dq", "dk", "dv"), op.backward(d_o, q, k, v, o, lse)):
            check(name, x, ref[name])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "length", "one", "few queries", "many queries"])
def test_one_key_has_no_gradient_of_its_logit(kind, dtype, dev):
    # softmax over one key is 1 whatever its logit: O = V, dQ = dK = 0 exactly
    # (few queries: the keys are split over CTAs; many: the attended keys are gathered)
    B, H, D = 2, 2, 64
    n_q, n_kv = {"few queries": (2, 5000), "many queries": (2100, 300), "none": (130, 1)}.get(kind, (130, 40))
    op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, device=dev)
    q, d_o = rand((B, n_q, H, D), dtype, dev, 1, 3.0), rand((B, n_q, H, D), dtype, dev, 4)
    k, v = rand((B, n_kv, H, D), dtype, dev, 2), rand((B, n_kv, H, D), dtype, dev, 3)
    m = {"kv_len": torch.ones(B, dtype=torch.int32, device=dev)} if kind in ("length", "few queries") else \
        masks("one", B, n_kv, dev) if kind in ("one", "many queries") else {}
    o, lse = op.forward(q, k, v, return_lse=True, **m)
    ref = oracle(q, k, v, d_o, **m)
    check("o", o, ref["o"])
    dq, dk, dv = op.backward(d_o, q, k, v, o, lse, **m)
    assert not dq.any() and not dk.any()
    check("dv", dv, ref["dv"])


@pytest.mark.parametrize("scale", [0.02, 1.5])
def test_scale_and_peaked_rows(scale, dev):
    B, n_q, n_kv, H, D = 1, 100, 150, 2, 64
    for dtype in (torch.float32, torch.bfloat16):
        op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, scale=scale, device=dev)
        q, d_o = rand((B, n_q, H, D), dtype, dev, 1, 3.0), rand((B, n_q, H, D), dtype, dev, 2)
        k, v = rand((B, n_kv, H, D), dtype, dev, 3), rand((B, n_kv, H, D), dtype, dev, 4)
        o, lse = op.forward(q, k, v, return_lse=True)
        ref = oracle(q, k, v, d_o, scale=scale)
        check("o", o, ref["o"])
        check("lse", lse, ref["lse"])
        for name, x in zip(("dq", "dk", "dv"), op.backward(d_o, q, k, v, o, lse)):
            check(name, x, ref[name])


def test_gradient_against_differences(dev):
    # f(x) = <O(x), w>; the central difference with step h is off by h^2 / 6 of the third derivative,
    # which for logits below 1 in size and unit-size v, w is below 10 per direction of unit length;
    # h = 2^-5 gives 2^-10 10 / 6 < 0.0017.  fp32 sums: f is a sum of N = 2560 products of fp32
    # outputs within 2^-20 of values of size 1, its difference over 2 h adds 2^-20 N / 2^-4 < 0.04,
    # with random signs far less; the gradient itself is within 2^-18 of |g|.
    B, n_q, n_kv, H, hkv, D = 1, 5, 9, 8, 4, 64
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, torch.float32, device=dev)
    x = [rand((B, n_q, H, D), torch.float32, dev, 1, 0.3), rand((B, n_kv, hkv, D), torch.float32, dev, 2, 0.3),
         rand((B, n_kv, hkv, D), torch.float32, dev, 3)]
    w = rand((B, n_q, H, D), torch.float32, dev, 4)
    o, lse = op.forward(*x, return_lse=True)
    g = op.backward(w, *x, o, lse)
    h = 2.0 ** -5
    for i in range(3):
        d = rand(x[i].shape, torch.float32, dev, 10 + i)
        d /= d.norm()
        f = []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * h * d
            f.append(float((op.forward(*y).double() * w.double()).sum()))
        slope = (f[0] - f[1]) / (2 * h)
        assert abs(slope - float((g[i].double() * d.double()).sum())) <= 0.0417, i


def test_captured_in_a_graph(dev):
    B, n_q, n_kv, H, hkv, D = 2, 150, 200, 4, 2, 128
    for dtype in (torch.float32, torch.bfloat16):
        op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
        q, d_o = rand((B, n_q, H, D), dtype, dev, 1), rand((B, n_q, H, D), dtype, dev, 4)
        k, v = rand((B, n_kv, hkv, D), dtype, dev, 2), rand((B, n_kv, hkv, D), dtype, dev, 3)
        n = torch.tensor([200, 17], dtype=torch.int32, device=dev)
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            o, lse = op.forward(q, k, v, kv_len=n, return_lse=True)
            op.backward(d_o, q, k, v, o, lse, kv_len=n)
        torch.cuda.current_stream(dev).wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = op.forward(q, k, v, kv_len=n, return_lse=True)
            g = op.backward(d_o, q, k, v, o, lse, kv_len=n)
        q.copy_(rand(q.shape, dtype, dev, 8))
        n.copy_(torch.tensor([0, 150]))
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = op.forward(q, k, v, kv_len=n, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for x, y in zip(g, op.backward(d_o, q, k, v, o2, lse2, kv_len=n)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gathered_keys_in_a_graph_with_another_mask(dtype, dev):
    B, n_q, n_kv, H, D = 2, 2050, 260, 1, 64
    op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, dtype, device=dev)
    x = [rand(s, dtype, dev, i) for i, s in enumerate((op.q_shape, op.kv_shape, op.kv_shape, op.q_shape))]
    m = masks("holes", B, n_kv, dev)
    o, lse = op.forward(*x[:3], return_lse=True, **m)
    op.backward(x[3], *x[:3], o, lse, **m)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = op.forward(*x[:3], return_lse=True, **m)
        g = op.backward(x[3], *x[:3], o, lse, **m)
    for key_mask in (masks("holes", B, n_kv, dev, 9)["key_mask"], masks("empty", B, n_kv, dev, 3)["key_mask"],
                     torch.ones((B, n_kv), dtype=torch.bool, device=dev)):
        m["key_mask"].copy_(key_mask)
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle(*x, **m)
        for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *g)):
            check(name, t, ref[name])


def test_nan_in_an_attended_key_shows(dev):
    for dtype in (torch.float32, torch.bfloat16):
        op = bsa.CrossAttention(1, 140, 200, 1, 1, 64, dtype, device=dev)
        q, k, v = (rand(s, dtype, dev, i) for i, s in enumerate((op.q_shape, op.kv_shape, op.kv_shape)))
        k[0, 150, 0, 3] = math.nan
        assert torch.isnan(op.forward(q, k, v)).all()


def test_offsets_past_32_bits(dev):
    # K and V of 2.5e9 elements, one query token: the last keys count as much as the first
    n_kv, H, D = 600_000, 32, 128
    op = bsa.CrossAttention(1, 1, n_kv, H, H, D, torch.bfloat16, device=dev)
    kv = [torch.empty((1, n_kv, H, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    g = torch.Generator(device=dev).manual_seed(1)
    for t in kv:
        for i in range(0, n_kv, 50_000):
            t[:, i:i + 50_000].copy_(torch.randn((1, 50_000, H, D), generator=g, device=dev))
    q = rand((1, 1, H, D), torch.bfloat16, dev, 2, 3.0)
    o, lse = op.forward(q, *kv, return_lse=True)
    op.check_status()
    for h in (0, 17, 31):
        ref = oracle(q[:, :, h:h + 1], kv[0][:, :, h:h + 1], kv[1][:, :, h:h + 1])
        check("o", o[:, :, h:h + 1], ref["o"])
        check("lse", lse[:, h:h + 1], ref["lse"])


def test_lengths_out_of_range_are_clamped_and_reported(dev):
    op = bsa.CrossAttention(2, 4, 10, 1, 1, 64, torch.bfloat16, device=dev)
    q, k, v = (rand((2, n, 1, 64), torch.bfloat16, dev, s) for s, n in ((1, 4), (2, 10), (3, 10)))
    o = op.forward(q, k, v, kv_len=torch.tensor([11, -1], dtype=torch.int32, device=dev))
    with pytest.raises(bsa.BsaError, match="kv_len") as err:
        op.check_status()
    assert err.value.status == 6
    assert torch.equal(o, op.forward(q, k, v, kv_len=torch.tensor([10, 0], dtype=torch.int32, device=dev)))
    op.check_status()


def test_writes_only_its_buffers(dev):
    for dtype in (torch.float32, torch.bfloat16):
        for shape in ((1, 130, 70, 2, 1, 64), (2, 1, 900, 4, 2, 128), (1, 2050, 140, 1, 1, 64)):
            B, n_q, n_kv, H, hkv, D = shape
            op = bsa.CrossAttention(*shape, dtype, device=dev)
            q, d_o = rand((B, n_q, H, D), dtype, dev, 1), rand((B, n_q, H, D), dtype, dev, 4)
            k, v = rand((B, n_kv, hkv, D), dtype, dev, 2), rand((B, n_kv, hkv, D), dtype, dev, 3)

            def guarded(shape, dt):
                n = math.prod(shape) * torch.empty((), dtype=dt).element_size()
                raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=dev)
                return raw, raw[4096:4096 + n].view(dt).view(shape)

            bufs = [guarded(s, dtype) for s in (q.shape, q.shape, k.shape, v.shape)]
            ws = [guarded((max(n, 256),), torch.uint8) for n in (op.forward_ws, op.backward_ws)]
            m = masks("holes", B, n_kv, dev)
            _, lse = op.forward(q, k, v, out=bufs[0][1], return_lse=True, workspace=ws[0][1], **m)
            op.backward(d_o, q, k, v, bufs[0][1], lse, out=tuple(b[1] for b in bufs[1:]), workspace=ws[1][1], **m)
            op.check_status()
            for raw, body in bufs + ws:
                n = body.numel() * body.element_size()
                assert bool((raw[:4096] == 0xA5).all()) and bool((raw[4096 + n:] == 0xA5).all())
            o, lse = op.forward(q, k, v, return_lse=True, **m)
            for x, y in zip((o, *op.backward(d_o, q, k, v, o, lse, **m)), (b[1] for b in bufs)):
                assert torch.equal(x, y)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes_views_and_masks(seed, dev):
    rng = random.Random(seed)
    dtype, D = rng.choice((torch.float32, torch.bfloat16)), rng.choice((64, 128))
    B, hkv, G = rng.randint(1, 3), rng.choice((1, 2, 3)), rng.choice((1, 1, 2, 3, 5, 8))
    n_q = rng.choice((1, 2, 7, 31, 128, 129, 260, 511))
    n_kv = rng.choice((1, 2, 31, 64, 127, 128, 129, 383, 384, 385, 1500))
    H = hkv * G

    def view(n, heads, s, scale=1.0):
        kind = rng.randint(0, 3)
        x = rand((B, n, heads, D), dtype, dev, 100 * seed + s, scale)
        if kind == 1:        # heads before tokens
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if kind == 2:        # every other head of a wider tensor, more tokens behind
            wide = rand((B, n + 3, heads * 2, D), dtype, dev, 7)
            wide[:, :n, ::2] = x
            return wide[:, :n, ::2]
        if kind == 3:        # the same for the whole batch
            return x[:1].expand(B, -1, -1, -1)
        return x

    q, k, v, d_o = view(n_q, H, 1, 2.0), view(n_kv, hkv, 2), view(n_kv, hkv, 3), view(n_q, H, 4)
    m = masks(rng.choice(("none", "length", "holes", "both", "empty")), B, n_kv, dev, seed)
    op = bsa.CrossAttention(B, n_q, n_kv, H, hkv, D, dtype, device=dev)
    ref = oracle(q, k, v, d_o, **m)
    o, lse = op.forward(q, k, v, return_lse=True, **m)
    check("o", o, ref["o"])
    check("lse", lse, ref["lse"])
    for name, x in zip(("dq", "dk", "dv"), op.backward(d_o, q, k, v, o, lse, **m)):
        check(name, x, ref[name])
    op.check_status()


def test_two_objects_on_two_streams(dev):
    # calls that overlap on the GPU, each with its own workspace
    shapes = ((2, 300, 500, 4, 2, 128), (1, 1, 20000, 8, 2, 64))
    for dtype in (torch.float32, torch.bfloat16):
        streams = [torch.cuda.Stream(dev) for _ in shapes]
        work = []
        for i, s in enumerate(shapes):
            B, n_q, n_kv, H, hkv, D = s
            op = bsa.CrossAttention(*s, dtype, device=dev)
            x = [rand(t, dtype, dev, 10 * i + j) for j, t in enumerate((op.q_shape, op.kv_shape, op.kv_shape, op.q_shape))]
            o, lse = op.forward(*x[:3], return_lse=True)
            work.append((op, x, o, lse, op.backward(x[3], *x[:3], o, lse)))
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(3):
            for i, st in enumerate(streams):
                op, x, _, _, _ = work[i]
                with torch.cuda.stream(st):
                    o, lse = op.forward(*x[:3], return_lse=True)
                    got[i].append((o, lse, *op.backward(x[3], *x[:3], o, lse)))
        torch.cuda.synchronize()
        for i in range(2):
            for run in got[i]:
                for a, b in zip(run, (work[i][2], work[i][3], *work[i][4])):
                    assert torch.equal(a, b)


def test_a_wait_that_runs_out_is_reported(dev):
    # the first CTA leaves out its n-th K/V copy: the waits end at their limit, the call with a
    # status, and the object works again afterwards
    B, n_q, n_kv, H, D = 1, 300, 700, 2, 64
    op = bsa.CrossAttention(B, n_q, n_kv, H, H, D, torch.bfloat16, device=dev)
    q, d_o = rand((B, n_q, H, D), torch.bfloat16, dev, 1), rand((B, n_q, H, D), torch.bfloat16, dev, 4)
    k, v = rand((B, n_kv, H, D), torch.bfloat16, dev, 2), rand((B, n_kv, H, D), torch.bfloat16, dev, 3)
    length = torch.full((B,), n_kv - 1, dtype=torch.int32, device=dev)
    o, lse = op.forward(q, k, v, kv_len=length, return_lse=True)
    g = op.backward(d_o, q, k, v, o, lse, kv_len=length)
    op.check_status()
    for n in (1, 2):
        op.set_watchdog(20_000_000, n)
        for call in (lambda: op.forward(q, k, v, kv_len=length),
                     lambda: op.backward(d_o, q, k, v, o, lse, kv_len=length)):
            call()
            with pytest.raises(bsa.BsaError, match="wait") as err:
                op.check_status()
            assert err.value.status == 4
    op.set_watchdog()
    assert torch.equal(op.forward(q, k, v, kv_len=length), o)
    for x, y in zip(g, op.backward(d_o, q, k, v, o, lse, kv_len=length)):
        assert torch.equal(x, y)
    op.check_status()


def test_refusals(dev):
    op = bsa.CrossAttention(1, 4, 3000, 2, 1, 64, torch.bfloat16, device=dev)
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device=dev)
    k = torch.zeros((1, 3000, 1, 64), dtype=torch.bfloat16, device=dev)
    for bad in ((q.float(), k, k), (q, k[:, :9], k), (q, k, k.cpu()), (k, k, k)):
        with pytest.raises(bsa.BsaError):
            op.forward(*bad)
    with pytest.raises(bsa.BsaError, match="kv_len"):
        op.forward(q, k, k, kv_len=torch.zeros(1, dtype=torch.int64, device=dev))
    with pytest.raises(bsa.BsaError, match="key_mask"):
        op.forward(q, k, k, key_mask=torch.ones((1, 2999), dtype=torch.bool, device=dev))
    with pytest.raises(bsa.BsaError, match="overlap"):
        op.forward(q, k, k, out=q[:, :1].expand(-1, 4, -1, -1))
    o, lse = op.forward(q, k, k, return_lse=True)
    with pytest.raises(bsa.BsaError, match="lse"):
        op.backward(q, q, k, k, o, lse[:, :1])
    with pytest.raises(bsa.BsaError, match="same memory"):
        op.backward(q, q, k, k, o, lse, out=(torch.empty_like(q), k, k))
    with pytest.raises(bsa.BsaError) as err:
        op.backward(q, q, k, k, o, lse, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert err.value.status == 5
    if op.forward_ws:
        with pytest.raises(bsa.BsaError) as err:
            op.forward(q, k, k, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
        assert err.value.status == 5
    for bad in ((q[:, :1].expand(-1, 4, -1, -1), k, k), (q, k[:, :1].expand(-1, 3000, -1, -1), k),
                (q[:, :, :1].expand(-1, -1, 2, -1), k, k)):
        with pytest.raises(bsa.BsaError, match="repeats") as err:
            op.forward(*bad)
        assert err.value.status == 2
    with pytest.raises(bsa.BsaError, match="scale"):
        bsa.CrossAttention(1, 4, 4, 2, 1, 64, scale=0.0)
    torch.cuda.synchronize()


def test_refuses_workspace_and_status_elsewhere(dev):
    """Working memory and a status word that no kernel could write."""
    op = bsa.CrossAttention(1, 4, 3000, 2, 1, 64, torch.bfloat16, device=dev)
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device=dev)
    k = torch.zeros((1, 3000, 1, 64), dtype=torch.bfloat16, device=dev)
    room = max(op.forward_ws, op.backward_ws, 256)
    o, lse = op.forward(q, k, k, return_lse=True)
    for bad in (torch.empty(room, dtype=torch.uint8), torch.empty(2 * room, dtype=torch.uint8, device=dev)[::2], room):
        with pytest.raises(bsa.BsaError, match="workspace must be"):
            op.forward(q, k, k, workspace=bad)
        with pytest.raises(bsa.BsaError, match="workspace must be"):
            op.backward(q, q, k, k, o, lse, workspace=bad)
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device=dev),
                torch.zeros(0, dtype=torch.int32, device=dev)):
        with pytest.raises(bsa.BsaError, match="dev_status must be"):
            op.forward(q, k, k, dev_status=bad)
        with pytest.raises(bsa.BsaError, match="dev_status must be"):
            op.backward(q, q, k, k, o, lse, dev_status=bad)
    torch.cuda.synchronize()


def test_refuses_outputs_over_inputs(dev):
    """Tiles of an output are written while others of the inputs are still to be read."""
    op = bsa.CrossAttention(1, 300, 300, 2, 2, 64, torch.bfloat16, device=dev)
    q, k, v, do = (torch.zeros((1, 300, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(4))
    for out in (q, k, v):
        with pytest.raises(bsa.BsaError, match="memory of an input"):
            op.forward(q, k, v, out=out)
    o, lse = op.forward(q, k, v, return_lse=True)
    new = [torch.empty_like(q) for _ in range(3)]
    for at in range(3):
        for t in (q, k, v, o, do):
            with pytest.raises(bsa.BsaError, match="memory of an input"):
                op.backward(do, q, k, v, o, lse, out=tuple(t if i == at else x for i, x in enumerate(new)))
    torch.cuda.synchronize()


def test_rotary_self_attention_cross_attention_together(dev):
    """One block's attention path: rotate Q and K of a fused projection, block-sparse self-attention
    over the rotated tensors, cross attention of its output over text states, and the gradients back
    to the unrotated Q of the cross attention's queries."""
    grid, heads, D, n_kv = (4, 16, 32), 3, 128, 77
    plan = bsa.Plan(1, *grid, 1, 8, 16, heads, D, 0, torch.bfloat16, dev)
    n = plan.info.n_tot
    rope = plan.rope((44, 42, 42))
    qkv = rand((1, n, 3, heads, D), torch.bfloat16, dev, 1)
    q, k = rope.apply(qkv[:, :, 0], qkv[:, :, 1])
    v = qkv[:, :, 2].contiguous()
    x = plan.forward(q, k, v, bsa.TOPK, 1.0)                        # density 1: dense attention
    plan.check_status()
    s = (q.double().transpose(1, 2) @ k.double().transpose(1, 2).transpose(2, 3)) * D ** -0.5
    dense = (torch.softmax(s, -1) @ v.double().transpose(1, 2)).transpose(1, 2)
    assert float((x.double() - dense).abs().max()) <= 2e-2         # the forward's documented tolerance
    cross = plan.cross(n_kv)
    tk, tv = rand((1, n_kv, heads, D), torch.bfloat16, dev, 2), rand((1, n_kv, heads, D), torch.bfloat16, dev, 3)
    length = torch.tensor([50], dtype=torch.int32, device=dev)
    o, lse = cross.forward(x, tk, tv, kv_len=length, return_lse=True)
    d_o = rand(o.shape, torch.bfloat16, dev, 4)
    ref = oracle(x, tk, tv, d_o, kv_len=length)
    check("o", o, ref["o"])
    dx, dk, dv = cross.backward(d_o, x, tk, tv, o, lse, kv_len=length)
    for name, t in (("dq", dx), ("dk", dk), ("dv", dv)):
        check(name, t, ref[name])
    back = rope.backward(dx)
    assert torch.allclose(rope.apply(back).float(), dx.float(), atol=2.0 ** -6, rtol=2.0 ** -6)
    cross.check_status()
