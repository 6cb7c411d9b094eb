"""GPU: cross attention's C entry points refuse addresses that a kernel could not read or write as
numbers (host checks: nothing is launched)."""
import ctypes

import pytest
import torch

import block_sparse_attention_permute_b200 as bsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["kv_len", "lse", "dev_status"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_misaligned_addresses_are_refused(name, dtype):
    dev = torch.device("cuda", 0)
    L = bsa.load()
    op = bsa.CrossAttention(1, 4, 9, 2, 2, 64, dtype, device=dev)
    q, o, dq, d_o = (torch.zeros(op.q_shape, dtype=dtype, device=dev) for _ in range(4))
    k, v, dk, dv = (torch.zeros(op.kv_shape, dtype=dtype, device=dev) for _ in range(4))
    keep, at = bsa._views(q, k, v, o, d_o, dq, dk, dv)
    room = torch.zeros(1024, dtype=torch.uint8, device=dev)
    ws = torch.empty(max(op.forward_ws, op.backward_ws, 256), dtype=torch.uint8, device=dev)
    good = {"kv_len": torch.full((1,), 9, dtype=torch.int32, device=dev),
            "lse": torch.zeros(op.lse_shape, device=dev), "dev_status": torch.zeros(1, dtype=torch.int32, device=dev)}
    for off in (1, 2, 3):
        a = {n: ctypes.c_void_p(t.data_ptr()) for n, t in good.items()}
        a[name] = ctypes.c_void_p(room.data_ptr() + off)
        rc = L.bsa_cross_attention(op._h, *at[:3], a["kv_len"], None, at[3], a["lse"], ws.data_ptr(), ws.numel(),
                                   a["dev_status"], None)
        assert rc == 1 and f"{name} must be 4-byte aligned" in L.bsa_last_error_string().decode()
        rc = L.bsa_cross_attention_backward(op._h, *at[:3], a["kv_len"], None, at[3], a["lse"], *at[4:], ws.data_ptr(),
                                            ws.numel(), a["dev_status"], None)
        assert rc == 1 and f"{name} must be 4-byte aligned" in L.bsa_last_error_string().decode()
    torch.cuda.synchronize()
    assert not room.any()
