"""GPU: the binding refuses lengths, masks and origins that are no tensors with its own error."""
import pytest
import torch

import block_sparse_attention_permute_b200 as bsa

pytestmark = pytest.mark.gpu


def test_lengths_masks_and_origins_have_to_be_tensors():
    dev = torch.device("cuda", 0)
    op = bsa.CrossAttention(2, 4, 9, 2, 2, 64, device=dev)
    q, k = (torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in (op.q_shape, op.kv_shape))
    o, lse = op.forward(q, k, k, return_lse=True)
    for kw in ({"kv_len": [9, 9]}, {"kv_len": 9}, {"key_mask": [[True] * 9] * 2}):
        name = next(iter(kw))
        with pytest.raises(bsa.BsaError, match=name):
            op.forward(q, k, k, **kw)
        with pytest.raises(bsa.BsaError, match=name):
            op.backward(q, q, k, k, o, lse, **kw)
    plan = bsa.Plan(2, 1, 2, 2, 1, 1, 1, 2, 64, 0, torch.bfloat16, dev)
    rope = plan.rope((16, 24, 24))
    for origin in ([1, 2], 3):
        with pytest.raises(bsa.BsaError, match="t_origin"):
            rope.apply(q, t_origin=origin)
    torch.cuda.synchronize()
