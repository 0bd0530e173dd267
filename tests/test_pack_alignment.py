"""Scales that are not aligned to their own type are refused before the repack kernels would load them (fake pointers
that are never followed)."""
import ctypes

import pytest

hq = pytest.importorskip("quantized_gemm_dequant_gb300")

CODES, SCALES, ZEROS, GLOBAL, PACKED = (0x10000 * i for i in range(1, 6))


@pytest.mark.parametrize("wfmt,size", [("e4m3_block", 4), ("uint4_zp", 2), ("int4_sym", 2), ("int8_sym", 2), ("e4m3", 2),
                                       ("uint2_zp", 2), ("uint1_zp", 2), ("uint3_zp", 2)])
def test_scales(wfmt, size):
    f = hq.make_format(wfmt, 256, 256)
    for off in range(1, size):
        s = SCALES + off
        assert hq._lib.hq_pack_weights(ctypes.byref(f), CODES, s, ZEROS, None, PACKED, None) == hq.HQ_ERR_ALIGNMENT
        assert hq._lib.hq_unpack_weights(ctypes.byref(f), PACKED, CODES, s, ZEROS, None, None) == hq.HQ_ERR_ALIGNMENT


def test_global_scale():
    f = hq.make_format("nvfp4", 256, 256)
    for off in (1, 2, 3):
        g = GLOBAL + off
        assert hq._lib.hq_pack_weights(ctypes.byref(f), CODES, SCALES, None, g, PACKED, None) == hq.HQ_ERR_ALIGNMENT
        assert hq._lib.hq_unpack_weights(ctypes.byref(f), PACKED, CODES, SCALES, None, g, None) == hq.HQ_ERR_ALIGNMENT
