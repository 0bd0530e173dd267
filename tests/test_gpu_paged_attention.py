"""Attention of one new token over the paged cache against a plain 64-bit form, within bounds derived in kv_ref."""
import numpy as np
import pytest
import torch

from tests import kv_ref as K

pytestmark = pytest.mark.gpu

# lengths around the 16-token block, the page and the work split; zero and one among them
LENS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 300]


def _cache(lib, kind, pages, page, heads, dim, seed, poison=()):
    c = lib.make_kv_cache(kind, pages, page, heads, dim, k_amax=168.0, v_amax=168.0)
    K.fill(c, seed, poison)
    return c


def _q(seed, B, Hq, D, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (gain * torch.randn(B, Hq, D, generator=g)).to(torch.bfloat16).cuda()


def _check(got, want, what=""):
    out, lse = K.f64(got[0]), K.f64(got[1])
    ro, rl, bo, bl = want
    assert out.shape == ro.shape and lse.shape == rl.shape
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty), what
    assert not out[empty].any(), what
    r = np.abs(out - ro) / np.where(bo > 0, bo, 1.0)
    assert np.all(np.abs(out - ro) <= bo), f"{what}: output error {np.max(r):.3f} of the bound"
    with np.errstate(invalid="ignore"):
        d = np.where(empty, 0.0, np.abs(lse - rl))
    assert np.all(d <= bl), f"{what}: lse error {np.max(d / np.where(bl > 0, bl, 1)):.3f} of the bound"


def _case(lib, kind, D, heads, group, page, lens, seed=0, window=0, softcap=0.0, scale=None, gain=1.0):
    table, pages = K.tables(lens, page, seed)
    c = _cache(lib, kind, pages, page, heads, D, seed, poison=(0,))
    K.poison_tail(c, table, lens)
    q = _q(seed + 1, len(lens), heads * group, D, gain)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = lib.make_kv_workspace(c, len(lens), heads * group)
    got = lib.paged_attention(c, q, table.cuda(), n, scale=scale, window=window, softcap=softcap, workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_OK
    want = K.attention(c, q, table, lens, D ** -0.5 if scale is None else scale, window, softcap)
    return got, want


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group,page", [(2, 4, 16), (1, 1, 48), (3, 8, 32)])
def test_against_plain_form(lib, kind, D, heads, group, page):
    """Unowned pages and the places past each length hold NaN: masked places must not reach a result."""
    _check(*_case(lib, kind, D, heads, group, page, LENS))


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("group", [2, 3, 5, 7, 9, 16, 17, 40])
def test_group_sizes(lib, kind, group):
    _check(*_case(lib, kind, 128, 2, group, 64, [33, 257, 5]))


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("window", [1, 15, 16, 100, 299, 300, 5000])
def test_window(lib, kind, window):
    _check(*_case(lib, kind, 64, 2, 4, 16, LENS, window=window), f"window {window}")


def test_pages_before_the_window_may_be_gone(lib):
    """A server frees a page once the window has left it: its table entry is not read."""
    lens, page, window = [300, 100, 17], 16, 40
    table, pages = K.tables(lens, page)
    c = _cache(lib, "e4m3", pages, page, 2, 64, 3)
    gone = table.clone()
    for b, n in enumerate(lens):
        gone[b, :max(0, n - window) // page] = -1
    q, ws = _q(1, 3, 8, 64), lib.make_kv_workspace(c, 3, 8)
    got = lib.paged_attention(c, q, gone.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), window=window, workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_OK
    _check(got, K.attention(c, q, table, lens, 64 ** -0.5, window))


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("softcap", [0.5, 30.0])
def test_softcap(lib, kind, softcap):
    _check(*_case(lib, kind, 128, 2, 8, 32, LENS, softcap=softcap, gain=3.0), f"cap {softcap}")


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (-0.1, 1.0), (1.0, 4.0), (2.0 ** -40, 2.0 ** 38), (2.0 ** 30, 2.0 ** -32)])
def test_scales(lib, kind, scale, gain):
    """Flat, reversed and peaked scores, and queries whose magnitudes leave the f16 range."""
    _check(*_case(lib, kind, 128, 1, 4, 16, [1, 40, 200], scale=scale, gain=gain), f"scale {scale} gain {gain}")


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("lens,heads,group", [([20011], 1, 8), ([9000, 1, 0, 4097, 2], 2, 3),
                                              ([700] * 40, 4, 2), (list(range(200)), 1, 4),
                                              ([30000, 1, 25003], 1, 2), ([60001], 1, 9), ([3, 9000, 12000, 8000], 1, 1)])
def test_long_and_many(lib, kind, lens, heads, group):
    """Lengths split over many CTAs (a few parts, and so many that they are joined in groups first), and many sequences
    in one CTA's share."""
    _check(*_case(lib, kind, 128, heads, group, 16, lens))


def test_value_scales_far_apart(lib):
    """e4m3 values whose scales span 2^60, tokens with a zero scale among them: a token's weight and its value scale
    are both in the weighted sum, and neither may push the other out of a 16-bit type's range."""
    lens = [200, 33]
    table, pages = K.tables(lens, 16)
    c = _cache(lib, "e4m3", pages, 16, 2, 64, 3)
    g = torch.Generator().manual_seed(5)
    c.v_scale.copy_(torch.exp2(torch.randint(-30, 31, c.v_scale.shape, generator=g).float()))
    zero = torch.rand(c.v_scale.shape, generator=g) < 0.2
    c.v_scale[zero.cuda()] = 0.0
    c.v[zero.cuda()] = 0
    q = _q(1, 2, 8, 64)
    got = lib.paged_attention(c, q, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    _check(got, K.attention(c, q, table, lens, 64 ** -0.5))


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("power", [-126, -110, 110, 126])
def test_queries_of_any_magnitude(lib, kind, power):
    """Queries at the ends of bf16's range: with scores below 2^-90 the weights are equal; with scores far apart (keys
    +-1 in one dim, or its block) the larger one's value is the result."""
    D, n = 64, 20
    c = lib.make_kv_cache(kind, 2, 16, 1, D, k_amax=1.0, v_amax=4.0)
    x = torch.zeros(n, 3, D)
    x[:, 1, 3] = -1.0
    x[7, 1, 3] = 1.0
    x[:, 2] = torch.randn(n, D, generator=torch.Generator().manual_seed(1)).clamp(-4, 4)
    lib.kv_write(c, x.to(torch.bfloat16).reshape(n, -1).cuda(), torch.arange(n).cuda(), 1)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16)
    q[0, 0, 3] = 2.0 ** power
    out, lse = lib.paged_attention(c, q.cuda(), torch.tensor([[0, 1]], dtype=torch.int32).cuda(),
                                   torch.tensor([n], dtype=torch.int32).cuda(), scale=0.25)
    torch.cuda.synchronize()
    v = K.cache_values(c, "v").transpose(0, 2, 1, 3).reshape(32, D)[:n]
    want = v[7] if power > 0 else v.mean(0)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11  # the weights' roundings, then the output's
    assert np.all(np.abs(K.f64(out)[0, 0] - want) <= 2.0 ** -8 * np.abs(want) + (u + 2.0 ** -18) * np.abs(v).max())
    want = 2.0 ** (power - 2) * K.cache_values(c, "k")[0, 0, 7, 3] if power > 0 else np.log(n)
    assert abs(float(lse) - want) <= 2.0 ** -18 * want


def test_zero_values_of_the_longest_sequences(lib):
    """e4m3, one page named over and over: 2^29 tokens of equal scores and values with a zero scale."""
    page, n = 1024, 2 ** 29
    c = lib.make_kv_cache("e4m3", 1, page, 1, 64)
    table = torch.zeros(1, n // page, dtype=torch.int32).cuda()
    out, lse = lib.paged_attention(c, _q(1, 1, 2, 64), table, torch.tensor([n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert not out.any() and torch.all((lse.cpu() - 29 * np.log(2.0)).abs() <= 2.0 ** -18 + 29 * 2.0 ** -22)


@pytest.mark.parametrize("kind", K.KINDS)
def test_all_value_scales_zero(lib, kind):
    lens = [50]
    table, pages = K.tables(lens, 16)
    c = _cache(lib, kind, pages, 16, 1, 128, 3)
    c.v.zero_()
    if c.v_scale is not None:
        c.v_scale.zero_()
    q = _q(1, 1, 4, 128)
    got = lib.paged_attention(c, q, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    _check(got, K.attention(c, q, table, lens, 128 ** -0.5))


@pytest.mark.parametrize("kind", K.KINDS)
def test_bad_indices_are_left_out_and_reported(lib, kind):
    """A page id outside the pools leaves its tokens out; a length past the table or below zero is clamped."""
    lens, page = [100, 64, 64, 5], 16
    table, pages = K.tables(lens, page)
    c = _cache(lib, kind, pages, page, 2, 64, 7)
    bad = table.clone()
    bad[0, 2], bad[0, 5], bad[1, :4] = -5, pages, 2 ** 31 - 1
    q = _q(2, 4, 8, 64)
    ws = lib.make_kv_workspace(c, 4, 8)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got = lib.paged_attention(c, q, bad.cuda(), n, workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_ERR_INVALID_ARG
    t = bad.numpy()
    drop = lambda b, j: (t[b, j // page] < 0) | (t[b, j // page] >= pages)  # noqa: E731
    ok = torch.where((bad >= 0) & (bad < pages), bad, 0)
    _check(got, K.attention(c, q, ok, lens, 64 ** -0.5, drop=drop))
    # the status is cleared, and lengths outside the table are taken as its ends
    cols = table.shape[1] * page
    tab = table.clone()
    tab[tab < 0] = 0
    got = lib.paged_attention(c, q, tab.cuda(), torch.tensor([cols + 1, -3, 2 ** 31 - 1, 5], dtype=torch.int32).cuda(),
                              workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_ERR_INVALID_ARG
    _check(got, K.attention(c, q, tab, [cols, 0, cols, 5], 64 ** -0.5))
    got = lib.paged_attention(c, q, table.cuda(), n, workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_OK
    _check(got, K.attention(c, q, table, lens, 64 ** -0.5))


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_nan_in_a_seen_place_is_not_hidden(lib, kind, softcap):
    """A NaN key makes its heads' rows NaN, a NaN value its dims', in that sequence and key-value head alone."""
    lens, page, D = [300, 300, 40], 16, 64
    table, pages = K.tables(lens, page)
    c = _cache(lib, kind, pages, page, 2, D, 7)
    for b, side, j in ((0, "k", 290), (1, "v", 5)):  # (sequence 0, head 0, key 290), (sequence 1, head 1, value 5)
        p, o = int(table[b, j // page]), j % page
        if kind == "bf16":
            getattr(c, side)[p, b, o, 3] = float("nan")
        elif kind == "e4m3":
            getattr(c, side)[p, b, o, 3] = 0x7F
        else:  # e2m1 has no NaN: the block's scale
            getattr(c, side + "_scale")[p, b, o, 0] = 0x7F
            getattr(c, side)[p, b, o, :8] = 0x11  # codes that are not zero
    q = _q(2, 3, 8, D)
    out, lse = lib.paged_attention(c, q, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), softcap=softcap)
    torch.cuda.synchronize()
    want, wl, bo, bl = K.attention(c, q, table, lens, D ** -0.5, softcap=softcap)
    got = K.f64(out)
    nan = np.zeros_like(got, bool)
    nan[0, :4] = True
    nan[1, 4:, 3 if kind != "nvfp4" else slice(0, 16)] = True
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(np.isnan(K.f64(lse)), nan.all(-1))
    assert np.all(np.abs(got - want)[~nan] <= bo[~nan])


def test_nan_value_scale_is_not_hidden(lib):
    lens = [20, 20]
    table, pages = K.tables(lens, 16)
    c = _cache(lib, "e4m3", pages, 16, 1, 64, 7)
    c.v_scale[int(table[0, 1]), 0, 2] = float("nan")
    out, _ = lib.paged_attention(c, _q(2, 2, 2, 64), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert out[0].isnan().all() and not out[1].isnan().any()


def test_empty_batch_and_empty_table(lib):
    c = _cache(lib, "bf16", 2, 16, 2, 64, 0)
    out, lse = lib.paged_attention(c, _q(0, 0, 4, 64), torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                                   torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = lib.paged_attention(c, _q(0, 3, 4, 64), torch.empty((3, 0), dtype=torch.int32, device="cuda"),
                                   torch.zeros(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", K.KINDS)
def test_same_bits_every_time(lib, kind):
    """The split and the order of joining do not depend on timing, on the workspace's history or on the stream."""
    lens = [5000, 3, 1200, 0, 40000]
    table, pages = K.tables(lens, 32)
    c = _cache(lib, kind, pages, 32, 4, 128, 1)
    q, n, t = _q(1, 5, 16, 128), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    ws = lib.make_kv_workspace(c, 64, 64)
    first = lib.paged_attention(c, q, t, n, workspace=ws)
    lib.paged_attention(c, q[:2].contiguous(), t[:2].contiguous(), n[:2].contiguous(), window=77, workspace=ws)
    for _ in range(5):
        again = lib.paged_attention(c, q, t, n, workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = lib.paged_attention(c, q, t, n, stream=s)
    s.synchronize()
    for got in (again, other):
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_graph_replay_follows_the_lengths(lib):
    """A captured call reads lengths and tables at replay: one graph serves a growing context."""
    page, cols = 16, 20
    table, pages = K.tables([cols * page] * 3, page)
    c = _cache(lib, "e4m3", pages, page, 2, 128, 2)
    q, t, n = _q(4, 3, 8, 128), table.cuda(), torch.tensor([7, 0, 100], dtype=torch.int32).cuda()
    ws = lib.make_kv_workspace(c, 3, 8)
    out, lse = lib.paged_attention(c, q, t, n, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.paged_attention(c, q, t, n, out=out, lse=lse, workspace=ws)
    for lens in ([1, 0, 320], [64, 63, 65], [0, 0, 0]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _check((out, lse), K.attention(c, q, table, lens, 128 ** -0.5), f"lengths {lens}")


@pytest.mark.parametrize("kind", K.KINDS)
def test_offsets_past_32_bits(lib, kind):
    """Pools of over 2^32 bytes, the sequence's pages at their end."""
    D, heads, page = 128, 8, 64
    row = {"bf16": 256, "e4m3": 128, "nvfp4": 64}[kind]
    pages = (1 << 32) // (row * heads * page) + 40
    small = _cache(lib, kind, 12, page, heads, D, 9)
    big = {}
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(small, name)
        if t is not None:
            big[name] = torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
            big[name][pages - 12:] = t
    c = lib.KVCache(kind, **big, k_global=small.k_global, v_global=small.v_global)
    lens = [500, 190]
    table, n = K.tables(lens, page, spare=0)
    assert n <= 12
    q, lt = _q(3, 2, 16, D), torch.tensor(lens, dtype=torch.int32).cuda()
    a = lib.paged_attention(small, q, table.cuda(), lt)
    b = lib.paged_attention(c, q, torch.where(table >= 0, table + pages - 12, table).cuda(), lt)
    torch.cuda.synchronize()
    _check(a, K.attention(small, q, table, lens, D ** -0.5))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refuses(lib):
    c = _cache(lib, "e4m3", 3, 16, 2, 64, 0)
    q, t, n = _q(0, 2, 8, 64), torch.zeros((2, 2), dtype=torch.int32, device="cuda"), \
        torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[:, :, :32].contiguous()), dict(page_table=t.long()), dict(page_table=t[:1]),
           dict(lens=n.long()), dict(lens=n[:1]), dict(lens=n.cpu()), dict(q=q.transpose(0, 1)),
           dict(out=torch.empty(2, 8, 32, dtype=torch.bfloat16, device="cuda"))]
    for over in bad:
        with pytest.raises(lib.HQArgError):
            lib.paged_attention(c, **{**dict(q=q, page_table=t, lens=n), **over})
    for over, code in ((dict(q=_q(0, 2, 3, 64)), lib.HQ_ERR_INVALID_ARG), (dict(window=-1), lib.HQ_ERR_INVALID_ARG),
                       (dict(softcap=float("nan")), lib.HQ_ERR_INVALID_ARG),
                       (dict(scale=float("inf")), lib.HQ_ERR_INVALID_ARG),
                       (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), lib.HQ_ERR_WORKSPACE)):
        with pytest.raises(lib.HQError) as e:
            lib.paged_attention(c, **{**dict(q=q, page_table=t, lens=n), **over})
        assert e.value.code == code
