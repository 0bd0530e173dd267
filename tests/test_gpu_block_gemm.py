"""The product of e4m3 activations and weights with fp32 scales per block of 128, against a plain 64-bit form."""
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu


def _call(lib, ops, M, N, K, **kw):
    a, sa, w, sw, b = ops
    fmt = lib.make_format("e4m3_block", N, K)
    return lib.gemm(fmt, {"data": a, "scale": sa}, lib.pack_weights(fmt, w, sw), M, bias=b, **kw)


def _check(lib, M, N, K, bias=False, seed=0):
    ops = B.operands(seed, M, N, K, bias)
    got = _call(lib, ops, M, N, K)
    want, size = B.product(*ops)
    B.check_product(got, want, size, K // 128, ops[4])


# one token; the edges of every token tile; more than one tile of tokens
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1030])
def test_rows(lib, M):
    _check(lib, M, 384, 512, seed=M)


# one output feature, odd ones, a last tile with one row, several tiles
@pytest.mark.parametrize("N", [1, 3, 7, 127, 128, 129, 130, 255, 257, 1001, 2048])
@pytest.mark.parametrize("M", [1, 40, 200, 700])
def test_features(lib, M, N):
    _check(lib, M, N, 256, bias=True, seed=N)


# one K block, odd numbers of them, more than a ring, more than a chunk of scales
@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152, 2176, 7168, 16384])
@pytest.mark.parametrize("M", [1, 20, 96, 300])
def test_depths(lib, M, K):
    _check(lib, M, 256, K, seed=K)


# enough tiles that a CTA (pair) takes several, or that clusters of every size are chosen
@pytest.mark.parametrize("M,N,K", [(5, 14336, 1024), (64, 4096, 7168), (100, 16500, 512), (900, 9000, 384),
                                   (2500, 4100, 640), (4096, 2048, 1024)])
def test_large(lib, M, N, K):
    _check(lib, M, N, K, bias=True)


# every kernel and every way of splitting a tile, at sizes that the planner would give to another
@pytest.mark.parametrize("choice", ["kernel=0,bt=128", "kernel=0,bt=256", "kernel=1,bt=16", "kernel=1,bt=32,sk=1",
                                    "kernel=1,bt=64,sk=8", "kernel=1,bt=128,sk=4", "kernel=1,bt=16,sk=2"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (3, 130, 1024), (129, 257, 1152), (257, 1001, 1280), (1030, 700, 2048)])
def test_choices(lib, monkeypatch, choice, M, N, K):
    monkeypatch.setenv("HQ_TUNE", choice)
    _check(lib, M, N, K, bias=True, seed=N)


def test_pack_is_inverted(lib):
    for N, K in ((1, 128), (130, 256), (384, 1152)):
        _, _, w, sw, _ = B.operands(3, 1, N, K)
        fmt = lib.make_format("e4m3_block", N, K)
        w2, s2 = torch.zeros_like(w), torch.zeros_like(sw)
        lib.unpack_weights(fmt, lib.pack_weights(fmt, w, sw), w2, s2)
        assert torch.equal(w, w2) and torch.equal(sw, s2)
    odd = torch.zeros(w.numel() + 1, dtype=torch.uint8, device="cuda")[1:]  # codes that are not 16-byte aligned
    odd.copy_(w.flatten())
    assert torch.equal(lib.pack_weights(fmt, w, sw), lib.pack_weights(fmt, odd.view(N, K), sw))
    odd.zero_()
    lib.unpack_weights(fmt, lib.pack_weights(fmt, w, sw), odd.view(N, K), s2)
    assert torch.equal(w.flatten(), odd)


def test_block_sums_are_exact_integers(lib):
    """Small integer codes and scales of one: every sum fits fp32, so the product is the integers' own, rounded once."""
    g = torch.Generator().manual_seed(0)
    for M, N, K in ((9, 200, 1024), (130, 130, 512), (400, 300, 2048)):
        a, w = (torch.randint(-8, 9, s, generator=g).float() for s in ((M, K), (N, K)))
        ops = [t.to(torch.float8_e4m3fn).view(torch.uint8).cuda() for t in (a, w)]
        one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
        got = _call(lib, (ops[0], one(M, K // 128), ops[1], one(-(-N // 128), K // 128), None), M, N, K)
        assert torch.equal(got.cpu(), (a.double() @ w.double().T).to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("M", [3, 100, 300])
def test_scales_far_apart(lib, M):
    """Scales of zero, tiny and huge ones in one row: blocks keep to themselves."""
    N, K = 260, 1024
    a, sa, w, sw, _ = B.operands(5, M, N, K)
    sa[:, 1] = 0
    sa[:, 2] *= 1e-30
    sa[:, 3] *= 1e18
    sa[M // 2, 3] = 0
    sw[:, 5] *= 1e15
    want, size = B.product(a, sa, w, sw)
    B.check_product(_call(lib, (a, sa, w, sw, None), M, N, K), want, size, K // 128)


@pytest.mark.parametrize("M", [3, 100, 300])
def test_nan_and_infinity_stay_in_their_row_and_column(lib, M):
    N, K = 200, 512
    a, sa, w, sw, _ = B.operands(6, M, N, K)
    a[1, 200] = 0x7F        # a NaN code
    w[150, 300] = 0xFF
    sa[2, 1] = float("inf")
    got = _call(lib, (a, sa, w, sw, None), M, N, K).float()
    ok = torch.ones(M, N, dtype=torch.bool, device="cuda")
    ok[1] = ok[2] = False
    ok[:, 150] = False
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, 150]).all() and not torch.isfinite(got[2]).any()
    clean = _call(lib, (a.clone().index_fill_(0, torch.tensor([1], device="cuda"), 0), sa.clone().clamp(max=1e30),
                        w.clone().index_fill_(0, torch.tensor([150], device="cuda"), 0), sw, None), M, N, K).float()
    assert torch.equal(got[ok], clean[ok])


def test_runs_agree_and_rows_do_not_depend_on_the_batch_they_are_in(lib):
    """Sums are taken in a fixed order: two runs give the same bits."""
    for M, N, K in ((1, 4096, 7168), (64, 1024, 4096), (700, 1000, 1024)):
        ops = B.operands(7, M, N, K)
        assert torch.equal(_call(lib, ops, M, N, K), _call(lib, ops, M, N, K))


def test_zero_rows_and_reused_workspace(lib):
    N, K = 256, 384
    a, sa, w, sw, _ = B.operands(8, 90, N, K)
    fmt = lib.make_format("e4m3_block", N, K)
    packed, ws = lib.pack_weights(fmt, w, sw), lib.make_workspace(fmt, 90)
    out = torch.full((90, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.gemm(fmt, {"data": a, "scale": sa}, packed, 0, out=out, workspace=ws)
    assert bool((out == 7).all())
    for M in (1, 50, 90, 17):  # rows past M are left as they were
        out.fill_(7)
        lib.gemm(fmt, {"data": a, "scale": sa}, packed, M, out=out, workspace=ws)
        want, size = B.product(a[:M], sa[:M], w, sw)
        B.check_product(out[:M], want, size, K // 128)
        assert bool((out[M:] == 7).all())
    assert lib.last_device_status(ws) == lib.HQ_OK


def test_streams_graphs_and_static_scratch(lib):
    """Two streams at once with a workspace each, a captured call replayed on new data, and the fixed scratch."""
    M, N, K = 48, 1024, 2048
    a, sa, w, sw, b = B.operands(9, M, N, K, bias=True)
    fmt = lib.make_format("e4m3_block", N, K)
    packed = lib.pack_weights(fmt, w, sw)
    act = {"data": a, "scale": sa}
    want = lib.gemm(fmt, act, packed, M, bias=b)
    assert torch.equal(want, lib.gemm_static_scratch(fmt, act, packed, M, bias=b))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [lib.make_workspace(fmt, M) for _ in streams]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(want) for _ in range(8)] for _ in streams]
    for i in range(8):
        for s, ws, o in zip(streams, spaces, outs):
            lib.gemm(fmt, act, packed, M, bias=b, out=o[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for os in outs for o in os)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        lib.gemm(fmt, act, packed, M, bias=b, out=out, workspace=spaces[0])
    a2, sa2, *_ = B.operands(10, M, N, K)
    a.copy_(a2)
    sa.copy_(sa2)
    graph.replay()
    ref, size = B.product(a2, sa2, w, sw, b)
    B.check_product(out, ref, size, K // 128, b)


def test_no_moe_form(lib):
    fmt = lib.make_format("e4m3_block", 256, 256)
    a, sa, w, sw, _ = B.operands(0, 4, 256, 256)
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.HQError) as e:
        lib.moe_gemm(fmt, {"data": a, "scale": sa}, lib.pack_weights(fmt, w, sw), ids, workspace=ws)
    assert e.value.code == lib.HQ_ERR_UNSUPPORTED
    assert torch.isfinite(lib.gemm(fmt, {"data": a, "scale": sa}, lib.pack_weights(fmt, w, sw), 4).float()).all()
