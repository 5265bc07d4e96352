"""Scales whose products pass fp32's range are refused before any launch: scores or results would be infinite times
zero (no GPU)."""
import ctypes

import pytest

from paged_kv_decode_21_gb300 import build as pkd_build

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced on the failing paths
F = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    pkd_build.build()
    from paged_kv_decode_21_gb300 import ops
    return ops.lib()


@pytest.mark.parametrize("scale,ks,vs,want", [
    (0.1, 1e37, 1.0, 2), (-0.1, 3e38, 1.0, 2), (0.1, 1.0, 2e36, 2), (1e38, 10.0, 1.0, 2), (-1e38, 1.0, 1.0, 2),
    (1e35, 1.0, 1.0, 0), (0.1, 1e36, 1e36, 0), (0.1, 1e-45, 1e-45, 0), (0.0, 1e36, 1.0, 0)])
def test_decode(L, scale, ks, vs, want):
    # with no sequences there is nothing to launch: what is not refused returns PKD_OK
    assert L.paged_decode_attention_int4(*[FAKE] * 6, 0, 1, 8, 2, 128, 16, 64, 64, 1000, F(scale), F(ks), F(vs), 0, FAKE,
                                         1 << 30, None, None) == want


@pytest.mark.parametrize("kind,scale,ks,want", [
    (0, 3e38, 1.0, 2), (0, 1e38, 1.0, 0), (1, 1e20, 1e19, 2), (1, -1e20, 1e18, 0), (2, 1e36, 1.0, 2), (2, 1e35, 1.0, 0),
    (2, 0.1, 1e37, 2), (2, 0.1, 1e36, 0), (0, 1e-38, 1e-38, 0)])
def test_weights(L, kind, scale, ks, want):
    assert L.paged_kv_attention_weights(*[FAKE] * 6, 0, 1, 8, 2, 128, 16, 64, 64, 1000, F(scale), F(ks), F(1.0), kind, FAKE,
                                        1 << 30, None, None) == want
