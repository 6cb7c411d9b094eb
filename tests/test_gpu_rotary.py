"""GPU: rotary positions (Plan.rope, Rope.apply, Rope.backward) against the formula in 64 bits.

Tolerance of one output: the angle is reduced in double and rounded once to fp32 as a turn in
[-1/2, 1/2] (off by at most 2^-26 turns, 2 pi 2^-26 < 2^-23 radians), sincospif is within 1 ulp
(2^-23), mscale and the two products and their sum round four times more (2^-24 each, relative to
|a| + |b|): together below 2^-20 mscale (|a| + |b|), plus half a step of the output's type.
"""
import itertools
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_permute_b200 as bsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bsa.load()
    return torch.device("cuda", 0)


def frequencies(dims, theta, scaling, factor, orig_len, beta=(32.0, 1.0)):
    f, axis = [], []
    for x, d in enumerate(dims):
        for i in range(d // 2):
            th = theta * factor ** (d / (d - 2)) if scaling == "ntk" and d > 2 else theta
            w = th ** (-2 * i / d)
            if scaling == "linear":
                w /= factor
            if scaling == "yarn":
                g = min(1.0, max(0.0, (orig_len * w / math.tau - beta[1]) / (beta[0] - beta[1])))
                w = (1 - g) * w / factor + g * w
            f.append(w)
            axis.append(x)
    return np.array(f), np.array(axis)


def oracle(x, grid, dims, layout, origin=None, theta=10000.0, scaling="none", factor=1.0, orig_len=0.0,
           mscale=1.0, backward=False):
    """The rotation in 64 bits and, per output, mscale (|a| + |b|) (0 where passed through)."""
    T, H, W = grid
    x = x.double().cpu().numpy()
    out, mag = x.copy(), np.zeros_like(x)
    f, axis = frequencies(dims, theta, scaling, factor, orig_len)
    P = len(f)
    ea = np.arange(P) * 2 if layout == "interleaved" else np.arange(P)
    eb = ea + 1 if layout == "interleaved" else ea + P
    for b in range(x.shape[0]):
        t, y, xx = np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij")
        pos = np.stack([t.ravel().astype(np.float64) + (0 if origin is None else int(origin[b])),
                        y.ravel(), xx.ravel()])
        w = pos[axis].T * f                                        # [n_video, P]
        c, s = np.cos(w)[:, None], np.sin(w)[:, None] * (-1 if backward else 1)
        nv = T * H * W
        u, v = x[b, :nv][..., ea], x[b, :nv][..., eb]
        o = out[b, :nv]
        o[..., ea], o[..., eb] = mscale * (u * c - v * s), mscale * (u * s + v * c)
        m = mag[b, :nv]
        m[..., ea] = m[..., eb] = mscale * (np.abs(u) + np.abs(v))
    return torch.from_numpy(out), torch.from_numpy(mag)


def check(got, ref, mag, dtype):
    got = got.double().cpu()
    step = torch.finfo(dtype).eps / 2
    tol = 2.0 ** -20 * mag + step * (ref.abs() + 2.0 ** -20 * mag)
    tol[mag == 0] = 0                                              # passed through: the same bits
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


def rand(shape, dtype, dev, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(dev)


# grid, text tokens, heads, heads_k, head_dim, dims
SHAPES = [
    ((1, 1, 1), 0, 1, 1, 64, (64, 0, 0)),
    ((1, 1, 1), 3, 8, 2, 128, (128, 0, 0)),
    ((3, 5, 7), 0, 3, 3, 128, (44, 42, 42)),
    ((2, 9, 11), 5, 2, 1, 128, (16, 56, 56)),
    ((4, 8, 8), 0, 2, 2, 64, (16, 24, 24)),
    ((5, 1, 3), 1, 4, 4, 128, (32, 32, 32)),
    ((1, 6, 2), 2, 5, 5, 64, (0, 2, 0)),
    ((2, 3, 4), 0, 1, 1, 128, (2, 0, 60)),
    ((130, 1, 1), 0, 7, 7, 64, (36, 0, 0)),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_rotation_and_its_transpose(k, layout, dtype, dev):
    grid, text, heads, hk, D, dims = SHAPES[k]
    B = 2
    plan = bsa.Plan(B, *grid, 1, 1, 1, heads, D, text, dtype, dev)
    rope = plan.rope(dims, layout=layout, heads_k=hk)
    N = grid[0] * grid[1] * grid[2] + text
    q, kk = rand((B, N, heads, D), dtype, dev, k), rand((B, N, hk, D), dtype, dev, 100 + k)
    for f, backward in ((rope.apply, False), (rope.backward, True)):
        qo, ko = f(q, kk)
        check(qo, *oracle(q, grid, dims, layout, backward=backward), dtype)
        check(ko, *oracle(kk, grid, dims, layout, backward=backward), dtype)
        # alone, in place, and into views of one buffer
        assert torch.equal(f(q), qo)
        q2, k2 = q.clone(), kk.clone()
        assert f(q2, k2, out=(q2, k2))[0] is q2
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
@pytest.mark.parametrize("dims", [(44, 42, 42), (2, 6, 96)])
def test_scaled_frequencies(scaling, dims, dev):
    grid = (40, 2, 3)
    plan = bsa.Plan(1, *grid, 4, 4, 8, 2, 128, 0, torch.float32, dev)
    rope = plan.rope(dims, theta=500.0, scaling=scaling, factor=4.0, orig_len=21, mscale=1.25)
    q = rand((1, 240, 2, 128), torch.float32, dev, 3)
    more = dict(theta=500.0, scaling=scaling, factor=4.0, orig_len=21, mscale=1.25)
    check(rope.apply(q), *oracle(q, grid, dims, "interleaved", **more), torch.float32)
    check(rope.backward(q), *oracle(q, grid, dims, "interleaved", backward=True, **more), torch.float32)


def test_far_origins_of_each_batch_element(dev):
    # f / (2 pi) and the turn round to 2^-53 of up to 2^22 turns, the oracle's angle to 2^-53 of
    # up to 1.7e7 radians: below 2^-28 radians, inside the tolerance's 2^-20
    plan = bsa.Plan(3, 3, 1, 1, 1, 1, 1, 2, 128, 0, torch.float32, dev)
    rope = plan.rope((128, 0, 0), theta=10000.0, layout="half")
    origin = torch.tensor([0, 999_983, 16_777_217], device=dev)
    q = rand((3, 3, 2, 128), torch.float32, dev, 5)
    ref, mag = oracle(q, (3, 1, 1), (128, 0, 0), "half", origin=origin)
    check(rope.apply(q, t_origin=origin), ref, mag, torch.float32)


def test_strided_views_of_a_fused_projection(dev):
    grid, B, heads, D = (3, 4, 5), 2, 3, 128
    plan = bsa.Plan(B, *grid, 1, 4, 4, heads, D, 7, torch.bfloat16, dev)
    for layout, dims in itertools.product(("interleaved", "half"), ((44, 42, 42), (32, 32, 32))):
        rope = plan.rope(dims, layout=layout)
        qkv = rand((B, 67, 3, heads, D), torch.bfloat16, dev, 9)
        q, k = qkv[:, :, 0], qkv[:, :, 1]
        qo, ko = rope.apply(q, k)
        assert qo.is_contiguous()
        check(qo, *oracle(q, grid, dims, layout), torch.bfloat16)
        check(ko, *oracle(k, grid, dims, layout), torch.bfloat16)
        # heads before tokens, and in place inside the projection: V stays as it was
        v = qkv[:, :, 2].clone()
        qh = q.transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(rope.apply(qh), qo)
        rope.apply(q, k, out=(q, k))
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, :, 2], v)


def test_infinities_and_nans_stay_in_their_pair(dev):
    # elements past R and text tokens are copied as bits, whatever their neighbours hold
    plan = bsa.Plan(1, 1, 2, 2, 1, 1, 1, 1, 64, 1, torch.float32, dev)
    for layout in ("interleaved", "half"):
        rope = plan.rope((2, 4, 4), layout=layout)
        q = rand((1, 5, 1, 64), torch.float32, dev, 4)
        q[0, 1, 0, 10:] = math.inf
        q[0, 4] = math.nan
        o = rope.apply(q)
        assert torch.equal(o[0, :4, 0, 10:], q[0, :4, 0, 10:])
        assert torch.isfinite(o[0, :4, 0, :10]).all() and torch.isnan(o[0, 4]).all()


def test_transpose_is_the_adjoint(dev):
    # <R x, y> = <x, R^T y>: both sums have n terms, each product off by at most 2^-19 relative
    plan = bsa.Plan(1, 5, 3, 4, 1, 1, 1, 3, 64, 2, torch.float32, dev)
    rope = plan.rope((24, 20, 10), layout="half", scaling="linear", factor=2.0, mscale=1.5)
    x, y = (rand((1, 62, 3, 64), torch.float32, dev, s) for s in (1, 2))
    a = (rope.apply(x).double() * y.double())
    b = (x.double() * rope.backward(y).double())
    assert abs(float(a.sum() - b.sum())) <= 2.0 ** -19 * 1.5 * 2 * float(x.double().norm() * y.double().norm())


def test_captured_in_a_graph_reads_new_inputs(dev):
    plan = bsa.Plan(2, 2, 3, 4, 1, 1, 1, 4, 64, 0, torch.bfloat16, dev)
    rope = plan.rope((16, 24, 24))
    q, k = (rand((2, 24, 4, 64), torch.bfloat16, dev, s) for s in (1, 2))
    origin = torch.zeros(2, dtype=torch.int64, device=dev)
    out = torch.empty_like(q), torch.empty_like(k)
    rope.apply(q, k, t_origin=origin, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(q, k, t_origin=origin, out=out)
    q.copy_(rand(q.shape, q.dtype, dev, 7))
    origin.copy_(torch.tensor([5, 70000]))
    g.replay()
    torch.cuda.synchronize()
    got = out[0].clone(), out[1].clone()
    want = rope.apply(q, k, t_origin=origin)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits(dev):
    # 500 000 tokens of 40 heads of 128: the last token turns like one of a small grid at its place
    grid, heads, D = (100, 50, 100), 40, 128
    plan = bsa.Plan(1, *grid, 4, 4, 8, heads, D, 0, torch.bfloat16, dev)
    rope = plan.rope((44, 42, 42))
    q = torch.empty((1, 500_000, heads, D), dtype=torch.bfloat16, device=dev)
    q[0, :499_000].fill_(1.0)
    q[0, 499_000:].copy_(rand((1000, heads, D), torch.bfloat16, dev, 3))
    tail = q[:, -100:].clone()
    rope.apply(q, out=q)
    small = bsa.Plan(1, 1, 50, 100, 4, 4, 8, heads, D, 0, torch.bfloat16, dev)
    x = torch.zeros((1, 5000, heads, D), dtype=torch.bfloat16, device=dev)
    x[:, -100:] = tail
    want = small.rope((44, 42, 42)).apply(x, t_origin=torch.tensor([99], device=dev))
    assert torch.equal(q[:, -100:], want[:, -100:])
    del q


def test_refusals(dev):
    plan = bsa.Plan(1, 2, 2, 2, 1, 1, 1, 2, 64, 0, torch.bfloat16, dev)
    rope = plan.rope((16, 24, 24))
    q = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16, device=dev)
    for bad in (q.float(), q[:, :7], q.cpu(), q.transpose(2, 3)):
        with pytest.raises(bsa.BsaError):
            rope.apply(bad)
    buf = torch.zeros((1, 8, 2, 65), dtype=torch.bfloat16, device=dev)
    with pytest.raises(bsa.BsaError, match="16 bytes"):
        rope.apply(buf[..., :64])
    with pytest.raises(bsa.BsaError, match="aligned"):
        rope.apply(torch.zeros(8 * 128 + 1, dtype=torch.bfloat16, device=dev)[1:].view(1, 8, 2, 64))
    with pytest.raises(bsa.BsaError, match="overlap"):
        rope.apply(q, out=q[:, :1].expand(-1, 8, -1, -1))
    with pytest.raises(bsa.BsaError, match="other strides"):
        big = torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16, device=dev)
        rope.apply(big[:, :, :2], out=big.flatten()[: 8 * 128].view(1, 8, 2, 64))
    with pytest.raises(bsa.BsaError, match="t_origin"):
        rope.apply(q, t_origin=torch.zeros(2, dtype=torch.int64, device=dev))
    # an input may repeat its values
    one = rand((1, 1, 2, 64), torch.bfloat16, dev, 1).expand(-1, 8, -1, -1)
    assert torch.equal(rope.apply(one), rope.apply(one.contiguous()))


@pytest.mark.parametrize("kw", [dict(dims=(16, 24, 26)), dict(dims=(0, 0, 0)), dict(dims=(15, 24, 24)),
                                dict(theta=1.0), dict(scaling="linear", factor=0.5), dict(mscale=0.0),
                                dict(scaling="yarn", factor=2.0), dict(layout="other"), dict(heads_k=300),
                                dict(scaling="yarn", orig_len=5, beta_fast=1.0)])
def test_bad_configurations_are_refused(kw, dev):
    plan = bsa.Plan(1, 2, 2, 2, 1, 1, 1, 2, 64, 0, torch.bfloat16, dev)
    kw.setdefault("dims", (16, 24, 24))
    with pytest.raises(bsa.BsaError):
        plan.rope(**kw)
