"""RMS norm with the residual's addition, SwiGLU and plain rows, each with an 8-bit output, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu

FORMATS = {"bf16": 8, "e4m3_tok": 16, "e4m3_block": 128}


def _rows(seed, T, K, scale=1.0):
    """bf16 rows on the CPU with strong channels; a row of zeros and one of a single value where there are enough."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(0.7 * torch.randn(K, generator=g)) * scale
    if T > 3:
        x[1] = 0
        x[2] = 0
        x[2, K // 3] = -37.0
    return x.to(torch.bfloat16)


def _weight(seed, K):
    return (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def _check_norm(afmt, act, x, r, w, eps, res=None):
    total = B.f64(x) + (B.f64(r) if r is not None else 0.0)
    want = B.norm(total, B.f64(w)[None], eps)
    if afmt == "bf16":
        B.check_bf16(act["data"], want)
    else:
        B.check_act(act, want, afmt == "e4m3_block")
    if r is not None:
        B.check_bf16(res, total)


# widths: one chunk, odd numbers of chunks, the edges of every thread layout; rows: one, odd ones, many
@pytest.mark.parametrize("afmt,K", [(f, K) for f in FORMATS for K in (8, 16, 48, 128, 1000, 1024, 1040, 2048, 4096, 4112,
                                                                      7168, 8192, 8200, 16384, 16640, 20000, 32768)
                                    if K % FORMATS[f] == 0])
@pytest.mark.parametrize("T", [1, 5, 333])
@pytest.mark.parametrize("add", [True, False])
def test_norm(lib, afmt, K, T, add):
    x, w = _rows(K + T, T, K, 0.5), _weight(K, K)
    r = _rows(K - T, T, K, 3.0) if add else None
    act, res = lib.add_rms_norm(afmt, x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), eps=1e-6)
    assert (res is None) == (r is None)
    _check_norm(afmt, act, x, r, w, 1e-6, res)


# enough rows for warps to take rows of their own, and for several turns of every CTA
@pytest.mark.parametrize("afmt,T,K", [("bf16", 2048, 64), ("e4m3_tok", 9001, 256), ("e4m3_block", 5000, 128),
                                      ("e4m3_block", 4099, 1024), ("bf16", 3001, 1000), ("e4m3_tok", 6000, 4096),
                                      ("e4m3_block", 6000, 2048)])
def test_norm_many_rows(lib, afmt, T, K):
    x, w, r = _rows(1, T, K, 0.5), _weight(2, K), _rows(3, T, K, 2.0)
    act, res = lib.add_rms_norm(afmt, x.cuda(), w.cuda(), residual=r.cuda())
    _check_norm(afmt, act, x, r, w, 1e-6, res)


@pytest.mark.parametrize("afmt", FORMATS)
def test_norm_strided_rows_and_in_place(lib, afmt):
    """Rows of wider tensors on every side, the residual updated in place, or over x; what lies between stays."""
    T, K = 37, 1280
    x, w, r = _rows(4, T, K, 0.5), _weight(5, K), _rows(6, T, K)
    wide = [torch.full((T, 2 * K + 8 * i), 5.0, dtype=torch.bfloat16, device="cuda") for i in range(3)]
    vx, vr, vo = (t[:, 8 * (i + 1):8 * (i + 1) + K] for i, t in enumerate(wide))
    vx.copy_(x)
    vr.copy_(r)
    act, res = lib.add_rms_norm(afmt, vx, w.cuda(), residual=vr, residual_out=vo)
    _check_norm(afmt, act, x, r, w, 1e-6, res)
    assert res.data_ptr() == vo.data_ptr() and torch.equal(vx.cpu(), x) and torch.equal(vr.cpu(), r)
    for i, t in enumerate(wide):
        assert bool((t[:, :8 * (i + 1)] == 5).all()) and bool((t[:, 8 * (i + 1) + K:] == 5).all())
    want, _ = lib.add_rms_norm(afmt, vx, w.cuda(), residual=vr)
    for over in ("residual", "x"):
        cx, cr = x.cuda(), r.cuda()
        act2, res2 = lib.add_rms_norm(afmt, cx, w.cuda(), residual=cr, residual_out=cr if over == "residual" else cx)
        assert all(torch.equal(want[k], act2[k]) for k in want) and torch.equal(res2, res)
        assert torch.equal((cx if over == "residual" else cr).cpu(), x if over == "residual" else r)


@pytest.mark.parametrize("afmt", FORMATS)
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e19, 1e30, 1e38])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_at_the_ends_of_the_range(lib, afmt, size, eps):
    """Squares that leave fp32's range, with and without an eps that covers them."""
    T, K = 6, 2048
    g = torch.Generator().manual_seed(11)
    x = (size * (0.2 + torch.rand(T, K, generator=g)) * torch.sign(torch.randn(T, K, generator=g))).to(torch.bfloat16)
    x[0] *= 2.0 ** -4
    x[1, 3:] = 0
    w = _weight(12, K)
    act, _ = lib.add_rms_norm(afmt, x.cuda(), w.cuda(), eps=eps)
    want = B.norm(B.f64(x), B.f64(w)[None], eps)
    if afmt == "bf16":
        B.check_bf16(act["data"], want, tiny=2.0 ** -132)
    else:
        B.check_act(act, want, afmt == "e4m3_block")


def test_norm_mean_and_eps_that_overflow_together(lib):
    """Squares whose sum still fits fp32, and an eps with which their mean does not."""
    x = torch.tensor([[6e18, -6e18] * 4, [1e18] * 8]).to(torch.bfloat16)
    w = _weight(1, 8)
    act, _ = lib.add_rms_norm("bf16", x.cuda(), w.cuda(), eps=3.2e38)
    B.check_bf16(act["data"], B.norm(B.f64(x), B.f64(w)[None], float(np.float32(3.2e38))))


@pytest.mark.parametrize("afmt", ["e4m3_tok", "e4m3_block"])
def test_not_numbers_make_their_scale_not_a_number(lib, afmt):
    T, K = 5, 512
    x = _rows(13, T, K)
    x[0, 200] = float("nan")
    x[3, 300] = float("inf")
    act, _ = lib.add_rms_norm(afmt, x.cuda(), _weight(1, K).cuda())
    v = B.decode(act["data"]) * np.repeat(B.f64(act["scale"]).reshape(T, -1), 128 if afmt == "e4m3_block" else K, axis=1)
    assert np.isnan(v[0]).all() and np.isnan(v[3, 300]) and np.isfinite(v[[2, 4]]).all()
    q = lib.swiglu_quantize(afmt, x.cuda())
    v = B.decode(q["data"]) * np.repeat(B.f64(q["scale"]).reshape(T, -1), 128 if afmt == "e4m3_block" else K // 2, axis=1)
    assert np.isnan(v[0, 200]) and np.isfinite(v[[2, 4]]).all() and not np.isfinite(v[3, 44])


@pytest.mark.parametrize("afmt,I", [(f, I) for f in ("e4m3_tok", "e4m3_block") for I in
                                    (16, 128, 768, 1024, 1040, 4096, 7168, 14336, 16400, 32768) if I % FORMATS[f] == 0])
@pytest.mark.parametrize("R", [1, 3, 300])
def test_swiglu(lib, afmt, I, R):
    x = _rows(I + R, R, 2 * I)
    B.check_act(lib.swiglu_quantize(afmt, x.cuda()), B.swiglu(B.f64(x)), afmt == "e4m3_block")


@pytest.mark.parametrize("afmt,R,I", [("e4m3_tok", 5001, 768), ("e4m3_tok", 3000, 2064), ("e4m3_block", 4097, 640)])
def test_swiglu_many_rows(lib, afmt, R, I):
    x = _rows(1, R, 2 * I)
    B.check_act(lib.swiglu_quantize(afmt, x.cuda()), B.swiglu(B.f64(x)), afmt == "e4m3_block")


@pytest.mark.parametrize("afmt", ["e4m3_tok", "e4m3_block"])
def test_swiglu_every_gate(lib, afmt):
    """Every finite bf16 gate in [-86, 3e38], one to a row of its own scale, so that no other value hides its error."""
    g = torch.arange(1 << 16).to(torch.int32).to(torch.int16).view(torch.bfloat16).float()
    g = g[torch.isfinite(g) & (g >= -86) & ((g.abs() > 2.0 ** -100) | (g == 0))].to(torch.bfloat16)
    x = torch.zeros(len(g), 256, dtype=torch.bfloat16)
    x[:, 7] = g
    x[:, 135] = 0.75
    B.check_act(lib.swiglu_quantize(afmt, x.cuda()), B.swiglu(B.f64(x)), afmt == "e4m3_block")
    low = torch.tensor([-87.0, -89.0, -1e4, -3e38, float("-inf"), float("inf")], dtype=torch.bfloat16)
    x = torch.zeros(len(low), 256, dtype=torch.bfloat16)
    x[:, 7] = low
    x[:, 135] = 1
    q = lib.swiglu_quantize(afmt, x.cuda())
    s = B.f64(q["scale"]).flatten()
    assert np.all(s[:4] <= 1e-35) and np.isnan(s[4]) and np.isinf(s[5])


@pytest.mark.parametrize("M,K", [(1, 128), (3, 384), (130, 2048), (17, 7168), (3000, 640)])
def test_quantize_act_block(lib, M, K):
    """The codes and scales are hq_quantize_act's own of every 128 elements taken as a row."""
    x = _rows(M, M, K).cuda()
    got, rows = lib.quantize_act("e4m3_block", x), lib.quantize_act("e4m3_tok", x.view(-1, 128))
    assert got["scale"].shape == (M, K // 128)
    assert torch.equal(got["data"].view(-1, 128), rows["data"]) and torch.equal(got["scale"].flatten(), rows["scale"])
    B.check_act(got, B.f64(x), True, rows_of_zeros=(1,) if M > 3 else ())


def test_outputs_given_and_rows_of_none(lib):
    T, K = 9, 256
    x, w = _rows(1, T, 2 * K).cuda(), _weight(2, K).cuda()
    for afmt in ("e4m3_tok", "e4m3_block"):
        want = lib.swiglu_quantize(afmt, x)
        out = {k: torch.full((t.numel() + 64,), 9, dtype=t.dtype, device="cuda") for k, t in want.items()}
        assert lib.swiglu_quantize(afmt, x, out=out) is out
        for k, t in want.items():  # what lies behind the rows is left as it was
            assert torch.equal(out[k][:t.numel()], t.flatten()) and bool((out[k][t.numel():] == 9).all())
        none = lib.swiglu_quantize(afmt, x[:0])
        assert none["data"].shape == (0, K)
        act, res = lib.add_rms_norm(afmt, x[:0, :K], w, residual=x[:0, K:])
        assert act["data"].shape == (0, K) and res.shape == (0, K)
    assert lib.quantize_act("e4m3_block", x[:0])["data"].shape == (0, 2 * K)


def test_streams_and_graphs(lib):
    """Calls on another stream than the current one, and captured ones replayed on new rows."""
    T, K = 70, 1024
    x, w, r = _rows(1, T, K).cuda(), _weight(2, K).cuda(), _rows(3, T, K).cuda()
    want, res = lib.add_rms_norm("e4m3_block", x, w, residual=r)
    sw = lib.swiglu_quantize("e4m3_tok", x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, res2 = lib.add_rms_norm("e4m3_block", x, w, residual=r, stream=side)
    sw2 = lib.swiglu_quantize("e4m3_tok", x, stream=side)
    side.synchronize()
    assert torch.equal(res, res2) and all(torch.equal(want[k], got[k]) and torch.equal(sw[k], sw2[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, res2 = lib.add_rms_norm("e4m3_block", x, w, residual=r)
        sw2 = lib.swiglu_quantize("e4m3_tok", x)
    x.copy_(_rows(7, T, K))
    graph.replay()
    want, res = lib.add_rms_norm("e4m3_block", x, w, residual=r)
    sw = lib.swiglu_quantize("e4m3_tok", x)
    assert torch.equal(res, res2) and all(torch.equal(want[k], got[k]) and torch.equal(sw[k], sw2[k]) for k in want)
