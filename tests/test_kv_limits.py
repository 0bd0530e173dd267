"""Limits of the paged key-value cache's entry points that the host sees (no GPU: nothing is launched on these paths)."""
import ctypes

import pytest


@pytest.mark.parametrize("kind,dim,extra", [("BF16", 64, 20), ("BF16", 256, 5), ("E4M3", 64, 18), ("E4M3", 128, 19),
                                            ("NVFP4", 64, 21), ("NVFP4", 128, 10)])
@pytest.mark.parametrize("heads,q_heads,tiles", [(1, 1, 1), (1, 8, 1), (2, 4, 2), (4, 68, 8)])
def test_a_batch_past_the_count_of_work_is_refused(kind, dim, extra, heads, q_heads, tiles):
    """Each (sequence, head, 16 query heads) is `extra` units and one at least for its tokens; they are counted in 31
    bits.  One sequence fewer than too many has a workspace, and passes on to the checks that follow."""
    import quantized_gemm_dequant_gb300 as hq
    f = ctypes.byref(hq.KVFormat(getattr(hq, "HQ_KV_" + kind), 16, heads, dim, 8))
    most = (2 ** 31 - 1) // (extra + 1) // tiles
    rows = 2 ** 30 // q_heads  # the other limit, of batch * query heads
    c = ctypes.byref(hq.KVPools(0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000))

    def call(batch):
        x = hq.KVAttention(q=0x70000, page_table=0x80000, table_stride=4, lens=0x90000, B=batch, window=0,
                           num_q_heads=q_heads, scale=1.0, softcap=0.0, out=0xA0000, lse=None)
        return hq._lib.hq_paged_attention(f, c, ctypes.byref(x), None, 0, None)
    if most < rows:
        assert hq._lib.hq_kv_workspace_bytes(f, most, q_heads) > 0 and call(most) == hq.HQ_ERR_WORKSPACE
        assert hq._lib.hq_kv_workspace_bytes(f, most + 1, q_heads) == 0
        assert call(most + 1) == hq.HQ_ERR_INVALID_ARG
    else:
        assert hq._lib.hq_kv_workspace_bytes(f, rows, q_heads) > 0 and call(rows) == hq.HQ_ERR_WORKSPACE


@pytest.mark.parametrize("name,layout", [("KVRows", "_KV_ROWS"), ("KVRead", "_KV_READ"), ("KVAttention", "_KV_ATTENTION")])
def test_packed_arguments_are_the_structures(name, layout):
    """What a call packs is, byte for byte, the structure with the same fields."""
    import quantized_gemm_dequant_gb300 as hq
    s, layout = getattr(hq, name), getattr(hq, layout)
    values = [0.5 + i if t is ctypes.c_float else 1000 + i for i, (_, t) in enumerate(s._fields_)]
    assert layout.size == ctypes.sizeof(s) and layout.pack(*values) == bytes(s(*values))
