"""GPU: rotary positions at the far end of their range, |t_origin + t| up to 2^30.

The angle is a turn pos f / (2 pi): f, 2 pi, their quotient and the product are within 2^-53 of
themselves each, so that 2^30 radians are off by at most 2^30 4 2^-53 = 2^-21; the rest is at most 2^-21
of |a| + |b| (turn to fp32, sincospif, mscale, two products and a sum): together 2^-20.  The oracle works
in 64-bit mantissas (x87): its angle is off by 2^-34.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_rotary import dev, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_positions_up_to_the_end_of_the_range(layout, dev):  # noqa: F811
    assert np.finfo(np.longdouble).nmant >= 63
    B, T, D = 4, 3, 128
    plan = bsa.Plan(B, T, 1, 1, 1, 1, 1, 2, D, 0, torch.float32, dev)
    rope = plan.rope((D, 0, 0), theta=10000.0, layout=layout)
    origin = torch.tensor([2 ** 30 - T, 2 ** 29 + 12345, 1 - 2 ** 30, 0], device=dev)
    q = rand((B, T, 2, D), torch.float32, dev, 6)
    got = rope.apply(q, t_origin=origin).double().cpu().numpy()
    x = q.double().cpu().numpy()
    f = np.power(np.longdouble(10000.0), -np.arange(0, D, 2).astype(np.longdouble) / D)
    ea = np.arange(D // 2) * 2 if layout == "interleaved" else np.arange(D // 2)
    eb = ea + 1 if layout == "interleaved" else ea + D // 2
    for b in range(B):
        for t in range(T):
            w = np.longdouble(int(origin[b]) + t) * f
            c, s = np.cos(w).astype(np.float64), np.sin(w).astype(np.float64)
            u, v = x[b, t][:, ea], x[b, t][:, eb]
            tol = (np.abs(u) + np.abs(v)) * 2.0 ** -20
            assert (np.abs(got[b, t][:, ea] - (u * c - v * s)) <= tol).all()
            assert (np.abs(got[b, t][:, eb] - (u * s + v * c)) <= tol).all()
