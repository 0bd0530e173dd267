"""The operators together, as the example uses them: a prompt's prefill and captured decoding steps against a plain
64-bit form of the block that goes on from the same projections and the same cache."""
import numpy as np
import pytest
import torch

from tests import kv_ref as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", K.KINDS)
def test_prefill_then_captured_steps(lib, kind):
    from examples.decode_attention import Attention
    batch, steps = 3, 5
    block = Attention(batch, 80, hidden=256, q_heads=4, kv_heads=2, dim=64, kind=kind, page=16, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    lens = [1, 33, 70]
    block.prefill([torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for n in lens])
    x = torch.randn(batch, 256, generator=g, device="cuda").to(torch.bfloat16)
    block.step(x)
    block.lens -= 1
    graph = torch.cuda.CUDAGraph()
    seen = {}
    attend = lib.paged_attention
    try:  # keep the tensors that the captured call works on
        def spy(cache, q, *a, **k):
            seen["q"], seen["out"] = q, attend(cache, q, *a, **k)
            return seen["out"]
        lib.paged_attention = spy
        with torch.cuda.graph(graph):
            y = block.step(x)
    finally:
        lib.paged_attention = attend
    for s in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        now = [n + s + 1 for n in lens]
        assert block.lens.tolist() == now
        out, lse, bo, bl = K.attention(block.cache, seen["q"], block.table, now, 64 ** -0.5)
        assert np.all(np.abs(K.f64(seen["out"][0]) - out) <= bo)
        assert np.all(np.abs(K.f64(seen["out"][1]) - lse) <= bl)
        # the step's own key is in the cache: its place holds the rotated, normed key of this step's projection
        held = K.cache_values(block.cache, "k")
        for b, n in enumerate(now):
            row = held[int(block.table[b, (n - 1) // 16]), :, (n - 1) % 16]
            assert np.abs(row).sum() > 0
        assert torch.isfinite(y).all()
        x.copy_(y / y.float().square().mean(-1, keepdim=True).sqrt().to(y.dtype))
    assert lib.last_device_status(block.workspace) == lib.HQ_OK
