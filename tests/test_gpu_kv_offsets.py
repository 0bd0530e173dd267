"""Writing and reading the paged cache at offsets past 2^32: pools, strided rows and outputs."""
import pytest
import torch

from tests import kv_ref as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", K.KINDS)
def test_pools_past_32_bits(lib, kind):
    """Pools of over 2^32 bytes, the tokens' pages at their end: codes, scales and rows read back are bit for bit those
    of a small cache, and the page before the tokens' is as it was."""
    T, Hq, heads, D, page, used = 150, 8, 8, 128, 64, 4
    row = {"bf16": 256, "e4m3": 128, "nvfp4": 64}[kind]
    pages = (1 << 32) // (row * heads * page) + 40
    base = pages - used
    small = lib.make_kv_cache(kind, used, page, heads, D, k_amax=30.0, v_amax=30.0)
    big = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        t = getattr(small, n)
        if t is not None:
            big[n] = torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
            big[n][base - 1:] = 0
    c = lib.KVCache(kind, **big, k_global=small.k_global, v_global=small.v_global)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, (Hq + 2 * heads) * D, generator=g).to(torch.bfloat16).cuda()
    slots = torch.randperm(used * page, generator=g)[:T].cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    a = lib.kv_write(small, x, slots, Hq, q_norm=w, k_norm=w)
    b = lib.kv_write(c, x, slots + base * page, Hq, q_norm=w, k_norm=w)
    table, n = torch.arange(used, dtype=torch.int32, device="cuda")[None], used * page
    starts = torch.tensor([0, n], device="cuda")
    ra, rb = lib.kv_read(small, table, starts, n), lib.kv_read(c, table + base, starts, n)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(i, j) for i, j in zip(ra, rb))
    for name, t in big.items():
        assert torch.equal(t[base:], getattr(small, name)) and not t[base - 1].any()


def test_rows_past_32_bits(lib):
    """Rows 2^30 elements apart, so that the last begins at 2^32."""
    T, Hq, H, D = 5, 4, 2, 64
    row = (Hq + 2 * H) * D
    wide = torch.empty(((T - 1) << 30) + row, dtype=torch.bfloat16, device="cuda").as_strided((T, row), (1 << 30, 1))
    x = torch.randn(T, row, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    wide.copy_(x)
    a, b = (lib.make_kv_cache("e4m3", 1, 16, H, D) for _ in range(2))
    slots = torch.arange(T).cuda()
    qa, qb = lib.kv_write(a, x, slots, Hq), lib.kv_write(b, wide, slots, Hq)
    torch.cuda.synchronize()
    assert torch.equal(qa, qb)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name))


def test_outputs_past_32_bits(lib):
    """Rows read to 2^32 elements from the outputs' start, and the row before them is as it was."""
    heads, D, page, n = 8, 128, 64, 100
    c = lib.make_kv_cache("e4m3", 2, page, heads, D)
    K.fill(c, 3)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    want = lib.kv_read(c, table, torch.tensor([0, n], device="cuda"), n)
    first = (1 << 32) // (heads * D)
    out = tuple(torch.empty((first + n, heads, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in out:
        t[first - 1] = 7.0
    lib.kv_read(c, table, torch.tensor([first, first + n], device="cuda"), first + n, out=out)
    torch.cuda.synchronize()
    for t, w in zip(out, want):
        assert torch.equal(t[first:], w) and bool((t[first - 1] == 7.0).all())
