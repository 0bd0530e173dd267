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


def _exact_cache(lib, kind, n, D, seed):
    """One sequence of n tokens whose values (0, +-.5, .. +-2) every format holds exactly, and queries in eighths: with
    64 dims all products and their sums are whole multiples of 1/16 below 2^11, exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    page = 16
    pages = -(-n // page)
    c = lib.make_kv_cache(kind, pages, page, 1, D, k_amax=2688.0, v_amax=2688.0)
    for side in ("k", "v"):
        code = torch.randint(0, 5, (pages, 1, page, D), generator=g)
        x = code * 0.5 * (1 - 2 * torch.randint(0, 2, code.shape, generator=g))
        if kind == "bf16":
            getattr(c, side).copy_(x)
        elif kind == "e4m3":
            getattr(c, side).copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
            getattr(c, side + "_scale").fill_(1.0)
        else:
            e = (code + 8 * (x < 0)).to(torch.uint8)
            getattr(c, side).copy_(e[..., 0::2] | (e[..., 1::2] << 4))
            getattr(c, side + "_scale").fill_(0x38)
    q = (torch.randint(-32, 33, (1, 2, D), generator=g) / 8).to(torch.bfloat16)
    return c, q, torch.randperm(pages, generator=g).to(torch.int32)[None]


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("softcap", [1e-39, 1e-3, 0.7, 30.0, 1e3, 1e5, 1e7, 1e30, 3.4e38])
def test_caps_of_any_size(lib, kind, softcap):
    """softcap * tanh(s / softcap) to a relative error: a cap far above the scores is no cap.

    The dot products are exact here, so a score's error is that of the cap's evaluation, relative to the score.  Below
    a quarter of the cap: a series whose remainder is under 2^-26, and at most eight roundings of 2^-24.  Above:
    1 - 2 / (1 + e^2t) with exp2 within 2^-22 and its argument's rounding, |2t log2 e| 2^-24, times the derivative, the
    approximate division within 2 ulp: under 2^-21 in all, of tanh t >= 0.2449.  So 2^-18 of the score is ample."""
    n, D, scale = 300, 64, 0.125
    c, q, table = _exact_cache(lib, kind, n, D, 21)
    out, lse = lib.paged_attention(c, q.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), scale=scale,
                                   softcap=softcap)
    torch.cuda.synchronize()
    k, v = (K.rows_of(K.cache_values(c, side), table[0].numpy(), c.page_size, 0, n)[:, 0] for side in ("k", "v"))
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    cap = float(np.float32(softcap))
    for h in range(2):
        s = cap * np.tanh((k @ K.f64(q)[0, h] * scale) / cap)
        ds = np.abs(s).max() * (2.0 ** -18 + 2.0 ** -21)
        e = np.exp(s - s.max())
        want, wl = e @ v / e.sum(), s.max() + np.log(e.sum())
        bound = 2.0 ** -8 * np.abs(want) + (u + 2 * ds + 2.0 ** -18) * (e @ np.abs(v)) / e.sum()
        assert abs(float(lse[0, h]) - wl) <= ds + 2.0 ** -18 + abs(wl) * 2.0 ** -22
        assert np.all(np.abs(K.f64(out)[0, h] - want) <= bound)


@pytest.mark.parametrize("n,heads,group,D", [(33, 1, 1, 64), (70, 2, 4, 128), (5000, 1, 8, 256), (5000, 1, 16, 256),
                                             (60001, 1, 4, 128)])
@pytest.mark.parametrize("low,high", [(None, 50), (None, 100), (-60, 70), (-120, 100), (100, -120), (-100, -100)])
def test_value_scales_rise_and_fall(lib, n, heads, group, D, low, high):
    """e4m3: all of the first half's values have a scale of 2^low (None: 0, rows of zeros), the second half's 2^high,
    or half of either where the other would be out of reach.  The scores are ordinary, so every token's weight counts
    in the sum of weights whatever its values' scale is."""
    table, pages = K.tables([n], 16, spare=0)
    c = lib.make_kv_cache("e4m3", pages, 16, heads, D)
    K.fill(c, 31)
    half = n // 2 // 16
    for j in range(table.shape[1]):
        p = int(table[0, j])
        if (low if j < half else high) is None:
            c.v[p], c.v_scale[p] = 0, 0.0
        else:
            c.v_scale[p] = 2.0 ** (low if j < half else high)
    q = torch.randn(1, heads * group, D, generator=torch.Generator().manual_seed(32)).to(torch.bfloat16)
    out, lse = lib.paged_attention(c, q.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    want, wl, bo, bl = K.attention(c, q, table, [n], D ** -0.5)
    assert np.all(np.abs(K.f64(lse) - wl) <= bl)
    assert np.all(np.abs(K.f64(out) - want) <= bo)


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("above", [12.0, 16.0, 17.0, 18.0, 19.0])
@pytest.mark.parametrize("at", [0, 500])
def test_a_sink_without_values(lib, kind, above, at):
    """One token holds nearly all of the weight, `above` nats over the others, and has values of zero: the output is
    what the others bring.  Their weights are rounded to the 16-bit type: bf16 (in two parts) to 2^-15 of each; f16 to
    2^-11 of each, or, scaled so that the largest is 2^7 at least, to 2^-32 of the largest where that is more."""
    n, D, page = 512, 64, 16
    c = lib.make_kv_cache(kind, n // page, page, 1, D, k_amax=2688.0, v_amax=2688.0)
    x = torch.zeros(n, 3, D)
    x[at, 1] = 6.0  # (the formats hold these exactly, e4m3 to its scale's rounding)
    x[:, 2] = 6.0
    x[at, 2] = 0.0
    if kind == "e4m3":
        x[at, 2, 1] = 6.0  # the row's scale is as the others': its zeros are codes
    lib.kv_write(c, x.to(torch.bfloat16).reshape(n, -1).cuda(), torch.arange(n).cuda(), 1)
    q = torch.full((1, 1, D), 1.0, dtype=torch.bfloat16)
    out, lse = lib.paged_attention(c, q.cuda(), torch.arange(n // page, dtype=torch.int32)[None].cuda(),
                                   torch.tensor([n], dtype=torch.int32).cuda(), scale=above / (6 * D))
    torch.cuda.synchronize()
    w = np.exp(-float(np.float32(above / (6 * D))) * 6 * D)
    z = 1.0 + (n - 1) * w
    want = np.full(D, 6 * (n - 1) * w / z)
    if kind == "e4m3":
        want[1] = 6.0
    u, sub = (2.0 ** -15, 0.0) if kind == "bf16" else (2.0 ** -11, 2.0 ** -32)
    # the scores' error: above 2^-21 from the product with log2 e and exp2's argument; exp2 and sums 2^-18
    bound = 2.0 ** -8 * want + (u + 2 * above * 2.0 ** -21 + 2.0 ** -18) * want + sub * 6 * (n - 1) / z
    assert np.all(np.abs(K.f64(out)[0, 0] - want) <= bound)
    assert abs(float(lse[0, 0]) - (above + np.log(z))) <= above * 2.0 ** -21 + 2.0 ** -18


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("power", [10, 18, 24, 28])
def test_queries_with_one_huge_element(lib, kind, power):
    """One dim of the queries is 2^power, the keys hold zeros there: the scores come from the other dims, in full.  The
    others are multiples of 2^-8, so that none needs more than f16's bits at the row's scale; the matrix unit aligns a step's products to the largest exponent, where
    a zero key may count as f16's smallest normal: 2^-23 of that for each of the dims."""
    lens, D = [300, 33], 64
    table, pages = K.tables(lens, 16)
    c = lib.make_kv_cache(kind, pages, 16, 2, D, k_amax=168.0, v_amax=168.0)
    K.fill(c, 41)
    if kind == "nvfp4":
        c.k[..., 8] &= 0xF0  # dim 16
    else:
        c.k[..., 16] = 0
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(42)).mul(256).round().div(256).to(torch.bfloat16)
    q[..., 16] = 2.0 ** power
    out, lse = lib.paged_attention(c, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    want, wl, bo, bl = K.attention(c, q, table, lens, D ** -0.5)
    ds = 0.0
    if kind != "bf16":
        top = c.k_scale.max().item() if kind == "e4m3" else float(c.k_global)
        ds = D * 2.0 ** -23 * 2.0 ** (power - 14) * top * D ** -0.5
    v = np.abs(K.cache_values(c, "v")).max()
    assert np.all(np.abs(K.f64(lse) - wl) <= bl + ds)
    assert np.all(np.abs(K.f64(out) - want) <= bo + 2 * ds * v)


@pytest.mark.parametrize("D,heads,group", [(64, 2, 4), (128, 1, 16), (128, 2, 3), (256, 1, 8), (256, 1, 12)])
def test_bf16_weights_keep_15_bits(lib, D, heads, group):
    """The weights enter a bf16 cache's products as two bf16 numbers, within 2^-15 of themselves (the second is 2^-7 of a
    weight at most): where values cancel in the output, nothing else is left to err than the scores, exp2 and the sums."""
    lens, page = [64, 300, 2000], 16
    table, pages = K.tables(lens, page)
    c = lib.make_kv_cache("bf16", pages, page, heads, D)
    K.fill(c, 51)
    q = torch.randn(len(lens), heads * group, D, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16)
    out, _ = lib.paged_attention(c, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    keys, values = K.cache_values(c, "k"), K.cache_values(c, "v")
    for b, n in enumerate(lens):
        k, v = (K.rows_of(x, table[b].clamp(min=0).numpy(), page, 0, n) for x in (keys, values))
        for h in range(heads * group):
            kk, vv, qq = k[:, h // group], v[:, h // group], K.f64(q)[b, h]
            s = kk @ qq * D ** -0.5
            # sums of D products in fp32, the matrix unit's truncated ones twice that; log2 e and exp2's argument
            ds = 2 * D * 2.0 ** -24 * np.max(np.abs(kk) @ np.abs(qq)) * D ** -0.5 + np.abs(s).max() * 2.0 ** -21
            e = np.exp(s - s.max())
            want = e @ vv / e.sum()
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2 * ds + 2.0 ** -18) * (e @ np.abs(vv)) / e.sum()
            assert np.all(np.abs(K.f64(out)[b, h] - want) <= bound)


@pytest.mark.parametrize("D,group,n", [(64, 4, 40), (128, 16, 300), (256, 8, 20000)])
def test_infinite_bf16_values_stay_infinite(lib, D, group, n):
    """An infinite value in a seen place makes its dim of its heads' outputs infinite with its sign; opposite ones in one
    dim make it NaN.  The other dims and the other head are as without them."""
    heads, page = 2, 16
    table, pages = K.tables([n], page)
    c = lib.make_kv_cache("bf16", pages, page, heads, D)
    K.fill(c, 61)
    q = (0.1 * torch.randn(1, heads * group, D, generator=torch.Generator().manual_seed(62))).to(torch.bfloat16)
    at = lambda j: (int(table[0, j // page]), 0, j % page)  # noqa: E731
    args = (q.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    was, _ = lib.paged_attention(c, *args)
    inf = float("inf")
    for j, dim, x in ((3, 5, inf), (n - 1, 6, -inf), (n // 2, 7, inf), (n // 2 + 1, 7, inf), (1, 9, inf), (n - 2, 9, -inf)):
        c.v[(*at(j), dim)] = x
    out, lse = lib.paged_attention(c, *args)
    torch.cuda.synchronize()
    got, want = out.cpu()[0], was.cpu()[0].clone()
    want[:group, 5] = want[:group, 7] = inf
    want[:group, 6] = -inf
    want[:group, 9] = float("nan")
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)) and torch.equal(got.isnan(), want.isnan())
    assert torch.isfinite(lse).all()
