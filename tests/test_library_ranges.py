"""Host-side tests (no GPU needed): numbers that the kernels would hold in fp32 as 0 or infinity are
refused.  A scale that became 0 would make a masked logit -inf * 0 = NaN, one that became infinite
every logit."""
import ctypes

import pytest

import block_sparse_attention_permute_b200 as bsa
from block_sparse_attention_permute_b200 import build as bsa_build


@pytest.fixture(scope="module")
def lib():
    bsa_build.build()
    return bsa.load()


@pytest.mark.parametrize("scale", [1e-300, 1e-46, 1e-39, 2.4e38, 1e39, 1e300])
@pytest.mark.parametrize("dtype", [0, 1])
def test_cross_scale_outside_fp32(lib, scale, dtype):
    h = ctypes.c_void_p()
    assert lib.bsa_cross_create(ctypes.byref(h), 1, 4, 4, 2, 2, 64, dtype, scale) == 1
    assert "scale" in lib.bsa_last_error_string().decode()
    assert not h.value


@pytest.mark.parametrize("scale", [0.0, 1.2e-38, 1e-6, 2.0, 1e30])
def test_cross_scale_inside_fp32(lib, scale):
    h = ctypes.c_void_p()
    st = lib.bsa_cross_create(ctypes.byref(h), 1, 4, 4, 2, 2, 64, 1, scale)
    assert st in (0, 3), lib.bsa_last_error_string().decode()      # 3: no device here
    if st == 0:
        lib.bsa_cross_destroy(h)


@pytest.mark.parametrize("mscale", [1e-300, 1e-46, 1e-39, 1e39, 1e300])
def test_rope_mscale_outside_fp32(lib, mscale):
    h = ctypes.c_void_p()
    cfg = bsa.RopeConfig()
    cfg.dim[:] = (4, 0, 0)
    cfg.theta = 100.0
    cfg.mscale = mscale
    assert lib.bsa_rope_create(ctypes.byref(h), None, ctypes.byref(cfg)) == 1
    assert "mscale" in lib.bsa_last_error_string().decode()
    cfg.mscale = 1.0                                               # then the plan is what is missing
    assert lib.bsa_rope_create(ctypes.byref(h), None, ctypes.byref(cfg)) == 1
    assert "plan" in lib.bsa_last_error_string().decode()
