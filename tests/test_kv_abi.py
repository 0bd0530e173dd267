"""Host checks of the paged key-value cache's entry points (no GPU: nothing is launched on these paths)."""
import ctypes

import pytest
import torch


def _hq():
    import quantized_gemm_dequant_gb300 as hq
    return hq


def _fmt(hq, **over):
    f = dict(kind=hq.HQ_KV_E4M3, page_size=16, num_heads=2, head_dim=128, num_pages=8, **{})
    f.update(over)
    return hq.KVFormat(**f)


def test_formats_are_checked():
    hq = _hq()
    L = hq._lib
    size = lambda **k: L.hq_kv_workspace_bytes(ctypes.byref(_fmt(hq, **k)), 0, 0)  # noqa: E731
    assert size() >= 4
    for over in (dict(kind=0), dict(kind=4), dict(head_dim=96), dict(head_dim=0), dict(page_size=0), dict(page_size=24),
                 dict(page_size=2048), dict(num_heads=0), dict(num_heads=2000), dict(num_pages=0),
                 dict(num_pages=1 << 31), dict(num_pages=1 << 27, num_heads=16)):
        assert size(**over) == 0, over
    f = ctypes.byref(_fmt(hq))
    assert L.hq_kv_workspace_bytes(f, -1, 8) == 0 and L.hq_kv_workspace_bytes(f, 4, 3) == 0
    assert L.hq_kv_workspace_bytes(f, 64, 8) >= L.hq_kv_workspace_bytes(f, 0, 0)
    assert L.hq_kv_workspace_bytes(None, 0, 0) == 0


def test_attention_arguments_are_checked():
    hq = _hq()
    L, f = hq._lib, _fmt(hq)
    c = hq.KVPools(0x10000, 0x20000, 0x30000, 0x40000, None, None)
    ok = dict(q=0x50000, page_table=0x60000, table_stride=4, lens=0x70000, B=0, window=0, num_q_heads=8, scale=1.0,
              softcap=0.0, out=0x80000, lse=None)

    def call(fmt=ctypes.byref(f), cache=ctypes.byref(c), ws=0x90000, n=1 << 40, **k):
        return L.hq_paged_attention(fmt, cache, ctypes.byref(hq.KVAttention(**{**ok, **k})), ws, n, None)
    assert ctypes.sizeof(hq.KVAttention) == hq._KV_ATTENTION.size and ctypes.sizeof(hq.KVRows) == hq._KV_ROWS.size
    assert call() == hq.HQ_OK  # no sequences
    assert L.hq_paged_attention(ctypes.byref(f), ctypes.byref(c), None, 0x90000, 1 << 40, None) == hq.HQ_ERR_INVALID_ARG
    bad = ctypes.byref(hq.KVPools(0x10008, 0x20000, 0x30000, 0x40000, None, None))
    none = ctypes.byref(hq.KVPools(0x10000, 0x20000, None, 0x40000, None, None))
    for over, code in ((dict(fmt=None), hq.HQ_ERR_INVALID_ARG), (dict(num_q_heads=7), hq.HQ_ERR_INVALID_ARG),
                       (dict(B=-1), hq.HQ_ERR_INVALID_ARG), (dict(window=-1), hq.HQ_ERR_INVALID_ARG),
                       (dict(scale=float("nan")), hq.HQ_ERR_INVALID_ARG), (dict(softcap=-1.0), hq.HQ_ERR_INVALID_ARG),
                       (dict(B=2, cache=None), hq.HQ_ERR_INVALID_ARG), (dict(B=2, cache=none), hq.HQ_ERR_INVALID_ARG),
                       (dict(B=2, cache=bad), hq.HQ_ERR_ALIGNMENT), (dict(B=2, q=None), hq.HQ_ERR_INVALID_ARG),
                       (dict(B=2, page_table=None), hq.HQ_ERR_INVALID_ARG), (dict(B=2, q=0x50002), hq.HQ_ERR_ALIGNMENT),
                       (dict(B=2, ws=None), hq.HQ_ERR_WORKSPACE), (dict(B=2, n=8), hq.HQ_ERR_WORKSPACE),
                       (dict(B=1 << 29), hq.HQ_ERR_INVALID_ARG)):
        assert call(**over) == code, over


def test_write_arguments_are_checked():
    hq = _hq()
    L, f = hq._lib, _fmt(hq)
    c = ctypes.byref(hq.KVPools(0x10000, 0x20000, 0x30000, 0x40000, None, None))
    ok = dict(qkv=0x50000, row_stride=12 * 128, T=0, num_q_heads=8, rotary_dim=64, interleaved=0, eps=1e-6, q_norm=None,
              k_norm=None, cos_sin=0x60000, num_positions=4, positions=0x70000, slots=0x80000, q_out=0x90000)
    call = lambda ws=0xA0000, n=1 << 20, **k: L.hq_kv_write(  # noqa: E731
        ctypes.byref(f), c, ctypes.byref(hq.KVRows(*{**ok, **k}.values())), ws, n, None)
    assert call() == hq.HQ_OK  # no rows
    for over, code in ((dict(T=-1), hq.HQ_ERR_INVALID_ARG), (dict(num_q_heads=3), hq.HQ_ERR_INVALID_ARG),
                       (dict(rotary_dim=144), hq.HQ_ERR_INVALID_ARG), (dict(rotary_dim=8), hq.HQ_ERR_ALIGNMENT),
                       (dict(row_stride=128), hq.HQ_ERR_INVALID_ARG), (dict(row_stride=12 * 128 + 4), hq.HQ_ERR_ALIGNMENT),
                       (dict(interleaved=2), hq.HQ_ERR_INVALID_ARG), (dict(eps=float("inf")), hq.HQ_ERR_INVALID_ARG),
                       (dict(T=1, slots=None), hq.HQ_ERR_INVALID_ARG), (dict(T=1, positions=None), hq.HQ_ERR_INVALID_ARG),
                       (dict(T=1, num_positions=0), hq.HQ_ERR_INVALID_ARG), (dict(T=1, qkv=0x50008), hq.HQ_ERR_ALIGNMENT),
                       (dict(T=1, ws=None), hq.HQ_ERR_WORKSPACE)):
        assert call(**over) == code, over


def test_read_arguments_are_checked():
    hq = _hq()
    L, f = hq._lib, _fmt(hq)
    c = ctypes.byref(hq.KVPools(0x10000, 0x20000, 0x30000, 0x40000, None, None))
    ok = dict(page_table=0x50000, table_stride=4, starts=0x60000, first=None, B=2, total=0, k_out=0x70000, v_out=0x80000)
    call = lambda ws=0x90000, n=1 << 20, **k: L.hq_kv_read(  # noqa: E731
        ctypes.byref(f), c, ctypes.byref(hq.KVRead(**{**ok, **k})), ws, n, None)
    assert ctypes.sizeof(hq.KVRead) == hq._KV_READ.size
    assert call() == hq.HQ_OK and call(B=0, total=5) == hq.HQ_OK
    assert L.hq_kv_read(ctypes.byref(f), c, None, 0x90000, 1 << 20, None) == hq.HQ_ERR_INVALID_ARG
    for over, code in ((dict(B=-1), hq.HQ_ERR_INVALID_ARG), (dict(total=-1), hq.HQ_ERR_INVALID_ARG),
                       (dict(total=3, starts=None), hq.HQ_ERR_INVALID_ARG), (dict(total=3, k_out=None), hq.HQ_ERR_INVALID_ARG),
                       (dict(total=3, v_out=0x80008), hq.HQ_ERR_ALIGNMENT), (dict(total=3, ws=None), hq.HQ_ERR_WORKSPACE)):
        assert call(**over) == code, over


def test_cache_handles_are_checked():
    """Shapes, types and the pools a format needs; host tensors are refused after them."""
    hq = _hq()
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    k8, s8 = z(2, 3, 16, 64), z(2, 3, 16, dt=torch.float32)
    for bad in (dict(kind="int8", k=k8, v=k8), dict(kind="e4m3", k=k8[0], v=k8), dict(kind="e4m3", k=k8, v=k8),
                dict(kind="e4m3", k=k8, v=k8[:1], k_scale=s8, v_scale=s8),
                dict(kind="e4m3", k=k8, v=k8, k_scale=s8, v_scale=s8[:1]),
                dict(kind="e4m3", k=k8.float(), v=k8, k_scale=s8, v_scale=s8),
                dict(kind="bf16", k=k8.bfloat16(), v=k8.bfloat16(), k_scale=s8, v_scale=s8),
                dict(kind="nvfp4", k=k8, v=k8, k_scale=z(2, 3, 16, 8), v_scale=z(2, 3, 16, 8)),
                dict(kind="e4m3", k=k8, v=k8, k_scale=s8, v_scale=s8)):  # the last is right, but on the host
        with pytest.raises(hq.HQArgError):
            hq.KVCache(**bad)
    with pytest.raises(hq.HQArgError):
        hq.make_kv_cache("nvfp4", 2, 16, 2, 64, device="cpu")
    with pytest.raises(hq.HQArgError):
        hq.paged_attention(None, None, None, None)
