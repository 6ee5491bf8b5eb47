"""Row statistics at an address that is not their type's: the C ABI refuses them
before anything is launched (the scalar unit would read the word below)."""
import ctypes

import pytest

import stable_variance_amd as sv

INVALID = 1
P = ctypes.c_void_p(0x10000)  # never dereferenced: the calls fail on the host


@pytest.fixture(scope="module")
def L():
    return sv.capi()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_root_mean_square_norm(L, off):
    odd = ctypes.c_void_p(0x20000 + off)
    for n, dtype in ((8, 0), (4096, 1), (40000, 2)):
        for call, name in (
                (lambda r: L.sv_rms_norm(P, n, None, n, dtype, dtype, 4, n, None, dtype, 1e-6, P, n, None, n, r, None),
                 b"sv_rms_norm:"),
                (lambda r: L.sv_rms_norm_fp8(P, n, None, n, dtype, dtype, 4, n, None, dtype, 1e-6, 3, 128, P, n, P, None,
                                             n, r, None), b"sv_rms_norm_fp8:"),
                (lambda r: L.sv_rms_norm_backward(P, n, P, n, None, n, dtype, dtype, 4, n, None, dtype, r, P, n, None, n,
                                                  P, P, 1 << 30, None), b"sv_rms_norm_backward:")):
            assert call(odd) == INVALID
            assert L.sv_last_error_message() == name + b" rstd is not aligned to its type"
    # without rows nothing is read or written
    assert L.sv_rms_norm(P, 8, None, 8, 0, 0, 0, 8, None, 0, 1e-6, P, 8, None, 8, odd, None) == 0


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", ["mean", "rstd"])
def test_layer_norm(L, off, name):
    odd = ctypes.c_void_p(0x20000 + off)
    stats = (odd, P) if name == "mean" else (P, odd)
    for n, dtype in ((8, 0), (4096, 1), (40000, 2)):
        assert L.sv_layer_norm(P, dtype, 4, n, n, None, None, dtype, 1e-5, P, n, *stats, None) == INVALID
        assert L.sv_last_error_message() == f"sv_layer_norm: {name} is not aligned to its type".encode()
        assert L.sv_layer_norm_backward(P, n, P, n, dtype, 4, n, None, dtype, *stats, P, n, P, P, P, 1 << 30, None) == INVALID
        assert L.sv_last_error_message() == f"sv_layer_norm_backward: {name} is not aligned to its type".encode()
