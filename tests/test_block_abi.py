"""Refusals of the operators with block scales, before anything touches a device (fake pointers are never followed)."""
import ctypes

import pytest
import torch

hq = pytest.importorskip("quantized_gemm_dequant_gb300")

X, R, W, RO, D, S = (0x10000 * i for i in range(1, 7))


def _norm(**kw):
    a = dict(act_type=hq.HQ_A_E4M3_BLOCK, eps=1e-6, T=4, K=256, x=X, x_stride=256, residual=R, residual_stride=256,
             weight=W, residual_out=RO, residual_out_stride=256, out_data=D, out_scale=S)
    a.update(kw)
    n = hq.Norm(**a)
    return hq._lib.hq_add_rms_norm(ctypes.byref(n), None)


@pytest.mark.parametrize("status,changed", [
    ("UNSUPPORTED", dict(act_type=hq.HQ_A_NVFP4)), ("UNSUPPORTED", dict(act_type=0)),
    ("INVALID_ARG", dict(T=-1)), ("INVALID_ARG", dict(K=0)), ("INVALID_ARG", dict(eps=-1.0)),
    ("INVALID_ARG", dict(eps=float("nan"))), ("INVALID_ARG", dict(eps=float("inf"))), ("ALIGNMENT", dict(K=200)),
    ("ALIGNMENT", dict(act_type=hq.HQ_A_E4M3_TOKEN, K=24)), ("ALIGNMENT", dict(act_type=hq.HQ_A_BF16, K=12)),
    ("UNSUPPORTED", dict(K=32768 + 128, x_stride=1 << 16, residual_stride=1 << 16, residual_out_stride=1 << 16)),
    ("INVALID_ARG", dict(residual=None)), ("INVALID_ARG", dict(residual_out=None)),
    ("INVALID_ARG", dict(x_stride=248)), ("INVALID_ARG", dict(residual_stride=128)),
    ("INVALID_ARG", dict(residual_out_stride=0)), ("ALIGNMENT", dict(x_stride=260)),
    ("INVALID_ARG", dict(x=None)), ("INVALID_ARG", dict(weight=None)), ("INVALID_ARG", dict(out_data=None)),
    ("INVALID_ARG", dict(out_scale=None)), ("ALIGNMENT", dict(x=X + 2)), ("ALIGNMENT", dict(residual=R + 8)),
    ("ALIGNMENT", dict(weight=W + 4)), ("ALIGNMENT", dict(residual_out=RO + 8)), ("ALIGNMENT", dict(out_data=D + 1)),
    ("ALIGNMENT", dict(out_scale=S + 4)), ("OK", dict(T=0, x=None, out_data=None))])
def test_norm(status, changed):
    assert _norm(**changed) == getattr(hq, "HQ_" + ("OK" if status == "OK" else "ERR_" + status))


def test_norm_no_struct():
    assert hq._lib.hq_add_rms_norm(None, None) == hq.HQ_ERR_INVALID_ARG


def test_swiglu_quantize():
    f = hq._lib.hq_swiglu_quantize
    B, T = hq.HQ_A_E4M3_BLOCK, hq.HQ_A_E4M3_TOKEN
    assert f(hq.HQ_A_BF16, X, 4, 256, D, S, None) == hq.HQ_ERR_UNSUPPORTED
    assert f(B, X, -1, 256, D, S, None) == hq.HQ_ERR_INVALID_ARG
    assert f(B, X, 4, 0, D, S, None) == hq.HQ_ERR_INVALID_ARG
    assert f(B, X, 4, 192, D, S, None) == hq.HQ_ERR_ALIGNMENT
    assert f(T, X, 4, 200, D, S, None) == hq.HQ_ERR_ALIGNMENT
    assert f(T, X, 4, 32768 + 16, D, S, None) == hq.HQ_ERR_UNSUPPORTED
    for bad in ((None, D, S), (X, None, S), (X, D, None)):
        assert f(T, bad[0], 4, 256, bad[1], bad[2], None) == hq.HQ_ERR_INVALID_ARG
    for bad in ((X + 8, D, S), (X, D + 8, S), (X, D, S + 4)):
        assert f(B, bad[0], 4, 256, bad[1], bad[2], None) == hq.HQ_ERR_ALIGNMENT
    assert f(B, None, 0, 256, None, None, None) == hq.HQ_OK


def test_quantize_act_block():
    f = hq._lib.hq_quantize_act
    B = hq.HQ_A_E4M3_BLOCK
    assert f(B, X, 4, 192, None, D, S, None, None, 0, None) == hq.HQ_ERR_ALIGNMENT
    assert f(B, X + 8, 4, 256, None, D, S, None, None, 0, None) == hq.HQ_ERR_ALIGNMENT
    assert f(B, X, 4, 256, None, D, None, None, None, 0, None) == hq.HQ_ERR_INVALID_ARG
    assert f(B, None, 0, 256, None, None, None, None, None, 0, None) == hq.HQ_OK
    assert hq.quantize_act_workspace_bytes("e4m3_block", 8192, 7168) == 0


def test_format():
    f = hq.make_format("e4m3_block", 300, 256)
    # 3 tiles x 2 blocks of 16 KB, then 6 scales in a 256-byte unit
    assert hq.packed_bytes(f) == 3 * 2 * 16384 + 256
    for bad in (dict(num_experts=2), dict(act_type=hq.HQ_A_BF16), dict(scale_type=hq.HQ_S_BF16), dict(group_size=64),
                dict(has_zero=1), dict(has_global_scale=1)):
        g = hq.make_format("e4m3_block", 300, 256, **({} if "num_experts" in bad else bad))
        if "num_experts" in bad:
            g.num_experts = 2
        assert hq.packed_bytes(g) == 0, bad
    assert hq.packed_bytes(hq.make_format("e4m3_block", 300, 200)) == 0
    # E4M3 weights for bf16 activations are what they were
    assert hq.packed_bytes(hq.make_format("e4m3", 300, 256)) == 3 * 2 * (16384 + 256)
    assert hq.workspace_bytes(f, 100) > 0 and hq.workspace_bytes(f, 100, topk=2) == 0
    assert hq.kernels_per_call(f, 100) == 1 and hq.kernels_per_call(f, 100, moe=True) == 0
    with pytest.raises(hq.HQError):
        hq.launch_plan(f, 100, moe=True)


def test_gemm():
    f = hq.make_format("e4m3_block", 256, 256)
    ok = dict(data=X, scale=S, c=D, ws=R, bytes=1 << 20, M=4)

    def call(**kw):
        v = {**ok, **kw}
        A = hq.Act(v["data"], v["scale"], None)
        return hq._lib.hq_gemm(ctypes.byref(f), ctypes.byref(A), W, None, v["c"], v["M"], 256, 256, v["ws"], v["bytes"],
                               None)

    assert call(scale=None) == hq.HQ_ERR_INVALID_ARG
    assert call(data=None) == hq.HQ_ERR_INVALID_ARG
    assert call(M=-1) == hq.HQ_ERR_INVALID_ARG
    assert call(scale=S + 4) == hq.HQ_ERR_ALIGNMENT
    assert call(c=D + 2) == hq.HQ_ERR_ALIGNMENT
    assert call(M=0) == hq.HQ_OK
    A = hq.Act(X, S, None)
    for fn in (hq._lib.hq_moe_gemm, hq._lib.hq_moe_gemm_combine):
        assert fn(ctypes.byref(f), ctypes.byref(A), W, R, None, 4, 1, D, RO, 1 << 20, None) == hq.HQ_ERR_UNSUPPORTED


def _raises(fn, *words):
    with pytest.raises(hq.HQArgError) as e:
        fn()
    for w in words:
        assert w in str(e.value), str(e.value)


def test_binding():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    x, w = bf(4, 256), bf(256)
    n = hq.add_rms_norm
    _raises(lambda: n("nvfp4", x, w), "afmt")
    _raises(lambda: n("e4m3_block", x[0], w), "2-D")
    _raises(lambda: n("e4m3_block", x, None), "weight")
    _raises(lambda: n("e4m3_block", x.float(), w), "x", "dtype")
    _raises(lambda: n("e4m3_block", x, w[:200]), "weight", "bytes")
    _raises(lambda: n("e4m3_block", x, w, residual=bf(4, 128)), "residual")
    _raises(lambda: n("e4m3_block", x, w, residual=bf(3, 256)), "rows")
    _raises(lambda: n("e4m3_block", x, w, residual_out=x), "residual_out")
    _raises(lambda: n("e4m3_block", x, w, residual=x, residual_out=bf(5, 256)), "rows")
    _raises(lambda: n("e4m3_block", bf(256, 4).t(), w), "contiguous")
    _raises(lambda: n("e4m3_block", bf(4, 1).expand(4, 256), w), "contiguous")
    _raises(lambda: n("e4m3_block", x[:1].expand(4, 256), w), "overlap")
    _raises(lambda: n("e4m3_block", x, w, out={"data": bf(4, 256)}), "out")
    _raises(lambda: n("e4m3_block", x, w, out={"data": bf(4, 256), "scale": torch.zeros(4, 2)}), "out['data']", "dtype")
    u8 = torch.zeros(4, 256, dtype=torch.uint8)
    _raises(lambda: n("e4m3_block", x, w, out={"data": u8, "scale": torch.zeros(4)}), "out['scale']", "bytes")
    _raises(lambda: n("e4m3_block", x, w), "device memory")
    s = hq.swiglu_quantize
    _raises(lambda: s("bf16", x), "afmt")
    _raises(lambda: s("e4m3_tok", bf(4, 255)), "2-D")
    _raises(lambda: s("e4m3_tok", x.half()), "dtype")
    _raises(lambda: s("e4m3_tok", x, out={"data": u8[:1], "scale": torch.zeros(4)}), "out['data']", "bytes")
    _raises(lambda: s("e4m3_tok", x), "device memory")
    f = hq.make_format("e4m3_block", 300, 256)
    codes = torch.zeros(300, 256, dtype=torch.uint8)
    _raises(lambda: hq.pack_weights(f, codes, torch.zeros(2, 2)), "scales", "bytes")
    _raises(lambda: hq.pack_weights(f, codes, torch.zeros(3, 2, dtype=torch.bfloat16)), "scales", "dtype")
    _raises(lambda: hq.pack_weights(f, codes[:, :255], torch.zeros(3, 2)), "codes", "contiguous")
    packed = torch.zeros(hq.packed_bytes(f), dtype=torch.uint8)
    act = {"data": torch.zeros(4, 256, dtype=torch.uint8), "scale": torch.zeros(4, 2)}
    _raises(lambda: hq.gemm(f, {**act, "scale": torch.zeros(4)}, packed, 4), "act['scale']", "bytes")
    _raises(lambda: hq.gemm(f, {**act, "scale": torch.zeros(4, 2, dtype=torch.float64)}, packed, 4), "act['scale']", "dtype")
    _raises(lambda: hq.gemm(f, act, packed, 4), "device memory")
