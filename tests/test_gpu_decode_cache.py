"""What the example's captured decoding steps leave in the cache, against the 64-bit norm and rotation of the steps' own
projections, at the sequences' own positions."""
import pytest
import torch

from tests import kv_ref as K
from tests.test_gpu_kv_cache import _check_held, _magnitude

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", K.KINDS)
def test_captured_steps_append_the_projections_rows(lib, kind):
    from examples.decode_attention import Attention
    batch, q_heads, heads, D = 3, 4, 2, 64
    block = Attention(batch, 80, hidden=256, q_heads=q_heads, kv_heads=heads, dim=D, kind=kind, page=16, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    lens = [1, 33, 70]
    block.prefill([torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for n in lens])
    x = torch.randn(batch, 256, generator=g, device="cuda").to(torch.bfloat16)
    block.step(x)
    block.lens -= 1
    graph, seen, write = torch.cuda.CUDAGraph(), {}, lib.kv_write

    def spy(cache, qkv, *a, **k):  # keep the projection that the captured call works on
        seen["qkv"] = qkv
        return write(cache, qkv, *a, **k)
    try:
        lib.kv_write = spy
        with torch.cuda.graph(graph):
            block.step(x)
    finally:
        lib.kv_write = write
    table = block.table.cpu()
    for s in range(4):
        graph.replay()
        torch.cuda.synchronize()
        at = torch.tensor([n + s for n in lens])
        slots = table.gather(1, (at // 16)[:, None])[:, 0].long() * 16 + at % 16
        h = seen["qkv"].cpu().view(batch, q_heads + 2 * heads, D)
        k, v, w, cs = h[:, q_heads:q_heads + heads], h[:, q_heads + heads:], block.k_norm.cpu(), block.cos_sin.cpu()
        _check_held(block.cache, "k", slots, K.norm_rotate(k, w, 1e-6, cs, at, False), _magnitude(k, w, 1e-6, D, False))
        _check_held(block.cache, "v", slots, K.f64(v), abs(K.f64(v)))
        x.copy_(torch.randn(batch, 256, generator=g, device="cuda"))
