"""The row operators at the ends of what their arguments may be, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu

FORMATS = {"bf16": 8, "e4m3_tok": 16, "e4m3_block": 128}


# a warp a row, a CTA a row with one, two and four chunks a thread, and rows past the registers' prefetch
@pytest.mark.parametrize("T,K", [(2100, 256), (5, 256), (400, 1024), (400, 4096), (3, 32768)])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1e-38, 1.2e-38, 1e-30])
@pytest.mark.parametrize("afmt", FORMATS)
@pytest.mark.parametrize("add", [True, False])
def test_norm_rows_of_zeros_with_a_tiny_eps(lib, afmt, eps, T, K, add):
    """0 / sqrt(0 + eps) is 0 for every eps above 0, fp32's subnormals among them; other rows keep to the formula."""
    eps = float(np.float32(eps))
    g = torch.Generator().manual_seed(K)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16)
    zeros = list(range(0, T, 3))
    x[zeros] = 0
    x[1] *= 1e-22  # squares of eps's own size
    r = torch.zeros(T, K, dtype=torch.bfloat16)
    if add:  # sums that cancel are zeros as well
        r[zeros] = torch.randn(len(zeros), K, generator=g).to(torch.bfloat16)
        x[zeros] = -r[zeros]
    w = (1 + 0.3 * torch.randn(K, generator=g)).to(torch.bfloat16)
    act, res = lib.add_rms_norm(afmt, x.cuda(), w.cuda(), residual=r.cuda() if add else None, eps=eps)
    total = B.f64(x) + B.f64(r)
    want = B.norm(total, B.f64(w)[None], eps)
    if afmt == "bf16":
        B.check_bf16(act["data"], want)
        assert not act["data"][zeros].any()
    else:
        B.check_act(act, want, afmt == "e4m3_block", rows_of_zeros=zeros)
    if add:
        B.check_bf16(res, total)


@pytest.mark.parametrize("afmt", FORMATS)
def test_norm_rows_of_zeros_without_eps(lib, afmt):
    """0 / sqrt(0) is no number."""
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    x[1] = 3
    act, _ = lib.add_rms_norm(afmt, x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), eps=0.0)
    y = act["data" if afmt == "bf16" else "scale"].float()
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()


# every layout of the rows: a warp a row, a CTA a row, and the kernel with a scale per 128
@pytest.mark.parametrize("afmt,copies,I", [("e4m3_tok", 1, 128), ("e4m3_tok", 16, 128), ("e4m3_tok", 1, 4096),
                                           ("e4m3_tok", 0, 4096), ("e4m3_tok", 1, 16400), ("e4m3_block", 0, 128),
                                           ("e4m3_block", 1, 128), ("e4m3_block", 16, 256)])
def test_swiglu_gates_far_below_zero(lib, afmt, copies, I):
    """silu(g) for gates whose sigmoid leaves fp32's normal range is still a number that `up` can make large: every bf16
    gate in [-210, -86] with ups up to bf16's largest, alone in its row or block and beside an ordinary value."""
    g = torch.arange(1 << 16).to(torch.int32).to(torch.int16).view(torch.bfloat16).float()
    g = g[(g >= -210) & (g <= -86)]
    up = torch.tensor([1.0, -1e10, 1e30, 1e38, -3.3e38])
    pairs = torch.cartesian_prod(g, up).repeat(max(copies, 1), 1).to(torch.bfloat16)
    if copies == 0:
        pairs = pairs[::7]
    x = torch.zeros(len(pairs), 2 * I, dtype=torch.bfloat16)
    x[:, 7], x[:, I + 7] = pairs[:, 0], pairs[:, 1]
    x[::2, 9], x[::2, I + 9] = 4, 3
    x[3::5, 7] = 1.5  # rows without such a gate between the others
    B.check_act(lib.swiglu_quantize(afmt, x.cuda()), B.swiglu(B.f64(x)), afmt == "e4m3_block")


@pytest.mark.parametrize("afmt", FORMATS)
def test_norm_with_the_largest_eps(lib, afmt):
    """fp32's largest eps, with means that change the sum, that take it past fp32, that do not count, and of zero."""
    eps = float(np.finfo(np.float32).max)
    x = torch.tensor([[1e19], [6e18], [1e12], [1.0], [0.0]]) * torch.tensor([1.0, -2.0] * 64)
    x, w = x.to(torch.bfloat16), torch.linspace(0.5, 1.5, 128).to(torch.bfloat16)
    act, _ = lib.add_rms_norm(afmt, x.cuda(), w.cuda(), eps=eps)
    want = B.norm(B.f64(x), B.f64(w)[None], eps)
    if afmt == "bf16":
        B.check_bf16(act["data"], want)
    else:
        B.check_act(act, want, afmt == "e4m3_block", rows_of_zeros=(4,))


@pytest.mark.parametrize("T,K", [(3, 4096), (500, 1024), (3000, 512), (700, 7168), (3, 32768)])
def test_two_calls_give_the_same_bits(lib, T, K):
    g = torch.Generator().manual_seed(T)
    x, r = (torch.randn(T, K, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.randn(K, generator=g).to(torch.bfloat16).cuda()
    for afmt in FORMATS:
        a, b = (lib.add_rms_norm(afmt, x, w, residual=r) for _ in range(2))
        assert torch.equal(a[1], b[1]) and all(torch.equal(a[0][k], b[0][k]) for k in a[0])
    for afmt in ("e4m3_tok", "e4m3_block"):
        a, b = (lib.swiglu_quantize(afmt, x) for _ in range(2))
        assert all(torch.equal(a[k], b[k]) for k in a)
