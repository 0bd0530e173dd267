"""Every finite eps that is not negative is taken by the norm, and nothing else (no rows: nothing reaches a device)."""
import ctypes

import pytest

hq = pytest.importorskip("quantized_gemm_dequant_gb300")

LARGEST = 3.4028234663852886e38  # fp32's


def _norm(eps):
    n = hq.Norm(act_type=hq.HQ_A_BF16, eps=eps, T=0, K=256, x_stride=256)
    return hq._lib.hq_add_rms_norm(ctypes.byref(n), None)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-6, 1.0, 3.4e38, 3.402e38, LARGEST])
def test_taken(eps):
    assert _norm(eps) == hq.HQ_OK


@pytest.mark.parametrize("eps", [-1e-45, -1.0, float("inf"), float("-inf"), float("nan")])
def test_refused(eps):
    assert _norm(eps) == hq.HQ_ERR_INVALID_ARG
