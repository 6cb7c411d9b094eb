"""GPU: rotary outputs that lie over the other tensor's input are refused (the kernel would write Q
before it has read K); rotations in place, also of one tensor's two parts, are not."""
import pytest
import torch

import block_sparse_attention_permute_b200 as bsa
from test_gpu_rotary import dev, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_refuses_an_output_over_the_other_input(layout, dev):  # noqa: F811
    plan = bsa.Plan(1, 2, 3, 4, 1, 1, 1, 2, 64, 0, torch.bfloat16, dev)
    rope = plan.rope((16, 24, 24), layout=layout)
    q, k = (rand((1, 24, 2, 64), torch.bfloat16, dev, s) for s in (1, 2))
    was = q.clone(), k.clone()
    new = torch.empty_like(q)
    for f in (rope.apply, rope.backward):
        for out in ((k, q), (k, new), (new, q)):
            with pytest.raises(bsa.BsaError, match="memory of") as err:
                f(q, k, out=out)
            assert err.value.status == 1
        with pytest.raises(bsa.BsaError, match="memory of"):       # one tensor as both, Q in place
            f(q, q, out=(q, new))
    torch.cuda.synchronize()
    assert torch.equal(q, was[0]) and torch.equal(k, was[1])
    want = rope.apply(q, k)
    qkv = torch.stack((q, k), dim=2)
    rope.apply(qkv[:, :, 0], qkv[:, :, 1], out=(qkv[:, :, 0], qkv[:, :, 1]))
    assert torch.equal(qkv[:, :, 0], want[0]) and torch.equal(qkv[:, :, 1], want[1])
    both = rope.apply(q, q)
    assert torch.equal(both[0], want[0]) and torch.equal(both[1], want[0])
