"""Addresses that the operators around the layer cannot use are refused on the host (CPU only: refused before the context
is used, so a block of zeros stands in for it and made-up addresses for the tensors)."""
import ctypes
import os
import shutil

import pytest

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from varlen_grouped_gemm_gb300 import build
    build.build()
    import varlen_grouped_gemm_gb300 as vgg
    return vgg.lib()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_norm_rstd_is_a_float_address(L, off):
    fake = ctypes.cast(ctypes.create_string_buffer(4096), ctypes.c_void_p)
    status = L.moe_add_rmsnorm(fake, A, 64, A, 64, 0, A, 0, 4, 64, 1e-6, A, 64, A, 64, A + off, 0, None, None, None)
    assert status == 1
