"""The paged cache's operators at the ends of their ranges, against plain 64-bit forms: huge finite inputs, caps far above
the scores, value scales and weights far apart.  The bounds are derived beside each test."""
import numpy as np
import pytest
import torch

from tests import kv_ref as K

pytestmark = pytest.mark.gpu


def _e4m3_codes(x):
    """fp32 numpy -> e4m3 bytes, nearest even, saturating."""
    return torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _e2m1_codes(x):
    """numpy -> e2m1 codes: ties to the even code, saturating, no negative zero."""
    a = np.abs(x)
    m = sum((a > t).astype(np.uint8) if i % 2 == 0 else (a >= t).astype(np.uint8)
            for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    return np.where((x < 0) & (m > 0), m + 8, m).astype(np.uint8)


def _nvfp4(x, g):
    """fp32 numpy [..., dims] -> (codes [..., dims], scale bytes [..., dims / 16]) by IEEE fp32 steps."""
    b, g = x.reshape(*x.shape[:-1], -1, 16), np.float32(g)
    with np.errstate(over="ignore", under="ignore", divide="ignore", invalid="ignore"):
        sb = _e4m3_codes(np.abs(b).max(-1) / (np.float32(6.0) * g))
        d = (K._e4m3(sb).astype(np.float32) * g)[..., None]
        codes = _e2m1_codes(np.where(d > 0, b / d, np.float32(0.0)))
    return codes.reshape(x.shape), sb


def _held_nvfp4(c, side, T):
    """(codes [T, heads, dims], scale bytes) of slots 0 .. T - 1 of a cache with one page."""
    z = getattr(c, side)[0, :, :T].cpu().numpy().transpose(1, 0, 2)
    codes = np.empty((*z.shape[:-1], c.head_dim), np.uint8)
    codes[..., 0::2], codes[..., 1::2] = z & 15, z >> 4
    return codes, getattr(c, side + "_scale")[0, :, :T].cpu().numpy().transpose(1, 0, 2)


@pytest.mark.parametrize("big", [2.0, 5e36, 1.9e37, 3e37, 1e38, 3.3e38, float("inf")])
@pytest.mark.parametrize("k_amax,v_amax", [(24.0, 8.0), (0.01, 2688.0)])
def test_huge_nvfp4_values_saturate(lib, big, k_amax, v_amax):
    """Values far above the calibrated ones, up to infinity, saturate: the largest block scale, the largest codes with
    their signs; whatever their size, codes and scales are those of IEEE divisions, bit for bit."""
    T, H, D = 6, 2, 64
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, 3 * H, D, generator=g)
    x[0, H:, 5], x[1, H:, 20], x[2, H:, 0], x[2, H:, 1] = big, -big, -big, big
    x[3, H:, 48:] *= big if np.isfinite(big) else 1.0
    x = x.clamp(-3.38e38, 3.38e38) if np.isfinite(big) else x
    x = x.to(torch.bfloat16)
    c = lib.make_kv_cache("nvfp4", 1, 16, H, D, k_amax=k_amax, v_amax=v_amax)
    lib.kv_write(c, x.reshape(T, -1).cuda(), torch.arange(T).cuda(), H)
    torch.cuda.synchronize()
    rows = x.float().numpy()
    for side, at in (("k", H), ("v", 2 * H)):
        want, sb = _nvfp4(rows[:, at:at + H], getattr(c, side + "_global").cpu().numpy()[0])
        got, got_sb = _held_nvfp4(c, side, T)
        assert np.array_equal(got_sb, sb), side
        assert np.array_equal(got, want), side
        if big > 1e6:
            assert (got_sb[0, :, 0] == 0x7E).all() and (got[0, :, 5] == 7).all() and (got[1, :, 20] == 15).all()
            assert (got[2, :, 0] == 15).all() and (got[2, :, 1] == 7).all()


@pytest.mark.parametrize("power", [-110, -98, -92, 100, 119, 122, 124])
def test_nvfp4_globals_at_the_ends(lib, power):
    """Global scales and values at the ends of fp32's range: codes and scales are those of IEEE divisions, bit for bit."""
    T, H, D = 16, 2, 128
    x = torch.randn(T, 3 * H, D, generator=torch.Generator().manual_seed(12)).clamp(-3.9, 3.9)
    x = (x.double() * 2.0 ** (power + 2)).to(torch.bfloat16)
    c = lib.make_kv_cache("nvfp4", 1, 16, H, D, k_amax=1.0, v_amax=1.0)
    c.k_global.fill_(2.0 ** power)
    c.v_global.fill_(1.7 * 2.0 ** power)
    lib.kv_write(c, x.reshape(T, -1).cuda(), torch.arange(T).cuda(), H)
    torch.cuda.synchronize()
    rows = x.float().numpy()
    for side, at in (("k", H), ("v", 2 * H)):
        want, sb = _nvfp4(rows[:, at:at + H], getattr(c, side + "_global").cpu().numpy()[0])
        got, got_sb = _held_nvfp4(c, side, T)
        assert np.array_equal(got_sb, sb) and np.array_equal(got, want), side
