"""Writing the paged cache (norm, rotation, quantisation) and reading it back, against plain 64-bit forms.

Values without a norm or rotation are quantised from bf16 inputs by single IEEE fp32 steps, so their codes are compared
bit for bit with the oracle's activation quantisers.  After a norm and a rotation the fp32 value itself is off by a few
2^-24, and what is held is compared with the 64-bit value: within half a step of the format plus that.
"""
import numpy as np
import pytest
import torch

import oracle
from tests import kv_ref as K
from tests import ref_helpers as R

pytestmark = pytest.mark.gpu

# relative error of the fp32 norm and rotation: mean of D squares (each add within 2^-24; trees of depth <= 12), rsqrtf
# within 2 ulp, products and the rotation's two products and sum; relative to |a| + |b| of the rotated pair
F32 = 32 * 2.0 ** -24


def _rows(seed, T, Hq, H, D, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * H, D, generator=g) * torch.exp(torch.randn(T, Hq + 2 * H, 1, generator=g))
    x[:, :, D // 3] *= 8.0
    if T > 2:
        x[1, Hq:] = 0.0  # rows of zeros: scale 0, zero codes
    return (gain * x).to(torch.bfloat16).reshape(T, -1)


def _angles(P, R, seed=0):
    a = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def _weight(seed, D):
    return (1 + 0.4 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def _slots(T, pages, page, seed):
    s = torch.randperm(pages * page, generator=torch.Generator().manual_seed(seed))[:T].to(torch.int64)
    if T > 4:
        s[T // 2] = -1
    return s


def _call(lib, c, x, slots, Hq, **k):
    ws = lib.make_kv_workspace(c)
    k = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in k.items()}
    q = lib.kv_write(c, x, slots.cuda(), Hq, workspace=ws, **k)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_OK
    return q


def _magnitude(x, w, eps, R, interleaved):
    """|a| + |b| of each dim's rotated pair after the norm (|x| where it is not rotated)."""
    y = np.abs(K.norm_rotate(x, w, eps, None, None, False))
    z = y.copy()
    if R:
        i = np.arange(R // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        z[..., ia] = z[..., ib] = y[..., ia] + y[..., ib]
    return z


def _check_held(c, side, slots, want, mag):
    """Rows `want` (float64 [T, H, D]) against what the pool holds in their slots; mag: magnitudes of fp32 errors."""
    keep = slots.numpy() >= 0
    p, o = slots.numpy()[keep] // c.page_size, slots.numpy()[keep] % c.page_size
    got, want, slack = K.cache_values(c, side)[p, :, o], want[keep], F32 * mag[keep] + 1e-37
    if c.kind == "bf16":
        step = 2.0 ** -8 * np.abs(want)
    elif c.kind == "e4m3":
        s = K.f64(getattr(c, side + "_scale"))[p, :, o]
        top = np.abs(want).max(-1)
        assert np.all(np.abs(s - top / 448) <= (F32 * mag[keep].max(-1) + 2.0 ** -23 * top) / 448 + 1e-37)
        step = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s[..., None]) * (1 + 2.0 ** -20)
    else:
        g = float(getattr(c, side + "_global").cpu()[0])
        sb = K._e4m3(getattr(c, side + "_scale").cpu().numpy()[p, :, o])
        top = np.abs(want).reshape(*want.shape[:-1], -1, 16).max(-1)
        ideal = np.minimum(top / (6 * g), 448.0)
        loose = (F32 * mag[keep].reshape(*want.shape[:-1], -1, 16).max(-1) + 2.0 ** -22 * top) / (6 * g)
        assert np.all(np.abs(sb - ideal) <= np.maximum(2.0 ** -4 * ideal, 2.0 ** -10) + loose)
        d = np.repeat(sb * g, 16, axis=-1)
        # half the gap between neighbours of |y / d|, or what lies past the largest code
        step = np.maximum(np.maximum(0.25 * d, 0.25 * np.abs(want)), np.abs(want) - 6 * d) * (1 + 2.0 ** -20)
    err = np.abs(got - want)
    assert np.all(err <= step + slack), f"{side}: {np.max(err / (step + slack)):.3f} of the bound"


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("D,R,interleaved,norm", [(64, 64, False, True), (128, 128, False, True), (256, 256, False, True),
                                                  (128, 64, True, True), (64, 32, False, False), (256, 0, False, True),
                                                  (128, 16, True, False), (64, 48, False, True), (128, 0, False, False)])
@pytest.mark.parametrize("T,heads,group", [(1, 1, 1), (7, 2, 3), (130, 3, 2)])
def test_write(lib, kind, D, R, interleaved, norm, T, heads, group):
    Hq, page, pages = heads * group, 16, 12
    c = lib.make_kv_cache(kind, pages, page, heads, D, k_amax=30.0, v_amax=60.0)
    x, slots = _rows(1, T, Hq, heads, D), _slots(T, pages, page, 2)
    pos = torch.randint(0, 500, (T,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    cs = _angles(500, R) if R else None
    wq, wk = (_weight(4, D), _weight(5, D)) if norm else (None, None)
    more = dict(positions=pos, cos_sin=cs) if R else {}
    q = _call(lib, c, x.cuda(), slots, Hq, q_norm=wq, k_norm=wk, eps=1e-5, interleaved=interleaved, **more)
    h = x.view(T, -1, D)
    want = K.norm_rotate(h[:, :Hq], wq, 1e-5, cs, pos, interleaved)
    slack = F32 * _magnitude(h[:, :Hq], wq, 1e-5, R, interleaved)
    err = np.abs(K.f64(q) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + slack + 1e-37)
    k = h[:, Hq:Hq + heads]
    _check_held(c, "k", slots, K.norm_rotate(k, wk, 1e-5, cs, pos, interleaved),
                _magnitude(k, wk, 1e-5, R, interleaved))
    v = h[:, Hq + heads:]
    _check_held(c, "v", slots, K.f64(v), np.abs(K.f64(v)))
    # places that no token was written to are as they were
    used = np.zeros(pages * page, bool)
    used[slots.numpy()[slots.numpy() >= 0]] = True
    for side in ("k", "v"):
        rest = K.cache_values(c, side).transpose(0, 2, 1, 3).reshape(pages * page, heads, D)[~used]
        assert not rest.any()


@pytest.mark.parametrize("D,heads,group", [(256, 2, 9), (256, 5, 8), (128, 4, 10), (64, 16, 9)])
def test_write_many_heads(lib, D, heads, group):
    """More query heads than a CTA keeps in registers (one step over, and many), more key heads than one step."""
    T, Hq, page, pages = 5, heads * group, 16, 2
    c = lib.make_kv_cache("e4m3", pages, page, heads, D)
    x, slots, pos = _rows(1, T, Hq, heads, D), torch.arange(T), torch.arange(T, dtype=torch.int32) * 7
    w, cs = _weight(4, D), _angles(50, D)
    q = _call(lib, c, x.cuda(), slots, Hq, q_norm=w, k_norm=w, positions=pos, cos_sin=cs)
    h = x.view(T, -1, D)
    for got, part in ((K.f64(q), h[:, :Hq]), (None, h[:, Hq:Hq + heads])):
        want = K.norm_rotate(part, w, 1e-6, cs, pos, False)
        mag = _magnitude(part, w, 1e-6, D, False)
        if got is not None:
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + F32 * mag + 1e-37)
        else:
            _check_held(c, "k", slots, want, mag)
    v = K.f64(h[:, Hq + heads:])
    _check_held(c, "v", slots, v, np.abs(v))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_are_the_oracles(lib, D):
    """No norm, no rotation: codes and scales bit for bit those of the oracle's quantisers, keys and values alike."""
    T, heads, page, pages = 40, 3, 16, 4
    x = _rows(7, T, heads, heads, D, gain=0.3)
    x[5] = x[5] * 1e-30
    slots = _slots(T, pages, page, 1)
    keep = slots.numpy() >= 0
    p, o = slots.numpy()[keep] // page, slots.numpy()[keep] % page
    rows = x.view(T, 3 * heads, D)
    for kind in ("e4m3", "nvfp4"):
        c = lib.make_kv_cache(kind, pages, page, heads, D, k_amax=2.75, v_amax=11.0)
        _call(lib, c, x.cuda(), slots, heads)
        for side, at, amax in (("k", heads, 2.75), ("v", 2 * heads, 11.0)):
            bits = R.np_bits(rows[:, at:at + heads].reshape(T * heads, D).contiguous())
            if kind == "e4m3":
                codes, s = oracle.quantize_act_e4m3_per_token(bits)
                want_s = s.reshape(T, heads)[keep].view(np.uint32)
                got_s = getattr(c, side + "_scale").cpu().numpy()[p, :, o].view(np.uint32)
            else:
                g32 = getattr(c, side + "_global").cpu().numpy()[0]
                codes, sb, g = oracle.quantize_act_nvfp4(bits, global_amax=np.float32(amax))
                if np.float32(g).view(np.uint32) != g32.view(np.uint32):
                    pytest.fail("the oracle's global scale is another one")
                want_s, got_s = sb.reshape(T, heads, -1)[keep], getattr(c, side + "_scale").cpu().numpy()[p, :, o]
            assert np.array_equal(got_s, want_s), (kind, side)
            got = getattr(c, side).cpu().numpy()[p, :, o]
            assert np.array_equal(got, codes.reshape(T, heads, -1)[keep]), (kind, side)


def test_infinities_and_nan_in_a_row(lib):
    """An infinite value makes its e4m3 row's scale infinite and itself NaN, the others' codes zero, as x / s does; a NaN
    is itself alone.  Other rows are as without it."""
    T, H, D = 4, 1, 64
    x = _rows(3, T, H, H, D)
    x = torch.where(x == 0, torch.ones_like(x), x)
    clean = lib.make_kv_cache("e4m3", 1, 16, H, D)
    _call(lib, clean, x.cuda(), torch.arange(T), H)
    x.view(T, 3, D)[1, 1:, 5] = float("inf")
    x.view(T, 3, D)[2, 1:, 7] = float("nan")
    c = lib.make_kv_cache("e4m3", 1, 16, H, D)
    _call(lib, c, x.cuda(), torch.arange(T), H)
    for side in ("k", "v"):
        codes, s, was = getattr(c, side)[0, 0].cpu(), getattr(c, side + "_scale")[0, 0].cpu(), getattr(clean, side)[0, 0].cpu()
        assert torch.isinf(s[1]) and (codes[1, 5] & 0x7F) == 0x7F
        rest = torch.arange(D) != 5
        assert not (codes[1][rest] & 0x7F).any()
        assert torch.isfinite(s[2]) and (codes[2, 7] & 0x7F) == 0x7F and ((codes[2][torch.arange(D) != 7] & 0x7F) != 0x7F).all()
        assert torch.equal(codes[[0, 3]], was[[0, 3]])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kind", K.KINDS)
def test_nan_is_kept(lib, kind, norm):
    """A NaN is read back as one: alone (of NVFP4 with its block of 16 dims), among zeros, in a row of nothing else; a
    norm makes the key's whole row NaN.  Other heads and rows are as without it."""
    T, Hq, H, D = 4, 2, 2, 64
    x = _rows(3, T, Hq, H, D)
    w = _weight(4, D) if norm else None
    def held(rows):
        c = lib.make_kv_cache(kind, 1, 16, H, D, k_amax=30.0, v_amax=60.0)
        q = _call(lib, c, rows.cuda(), torch.arange(T), Hq, q_norm=w, k_norm=w)
        return q, K.cache_values(c, "k")[0, :, :T], K.cache_values(c, "v")[0, :, :T]  # [H, T, D]
    clean = held(x)
    y = x.clone()
    h = y.view(T, Hq + 2 * H, D)
    for side in (Hq, Hq + H):
        h[1, side, 37] = float("nan")  # row 1's keys and values are zeros
        h[2, side + 1, 5] = float("nan")
        h[3, side] = float("nan")
    got = held(y)
    assert torch.equal(got[0], clean[0])
    for i, side in ((1, "k"), (2, "v")):
        want = np.zeros((H, T, D), bool)
        if side == "k" and norm:
            want[0, 1] = want[1, 2] = want[0, 3] = True
        else:
            want[0, 1, slice(32, 48) if kind == "nvfp4" else 37] = True
            want[1, 2, slice(0, 16) if kind == "nvfp4" else 5] = True
            want[0, 3] = True
        assert np.array_equal(np.isnan(got[i]), want), side
        for head, t in ((0, 0), (1, 0), (1, 1), (0, 2), (1, 3)):
            assert np.array_equal(got[i][head, t], clean[i][head, t])


@pytest.mark.parametrize("kind", K.KINDS)
def test_rows_of_a_wider_tensor(lib, kind):
    """The rows of a projection that computes more than q, k and v: strided rows give what contiguous ones give."""
    T, Hq, H, D = 9, 4, 2, 64
    x = _rows(1, T, Hq, H, D).cuda()
    wide = torch.full((T, x.shape[1] + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + x.shape[1]] = x
    slots = _slots(T, 3, 16, 2)
    a, b = (lib.make_kv_cache(kind, 3, 16, H, D, k_amax=30.0, v_amax=30.0) for _ in range(2))
    qa = _call(lib, a, x, slots, Hq, q_norm=_weight(1, D), k_norm=_weight(2, D))
    qb = _call(lib, b, wide[:, 16:16 + x.shape[1]], slots, Hq, q_norm=_weight(1, D), k_norm=_weight(2, D))
    assert torch.equal(qa, qb)
    for n in ("k", "v", "k_scale", "v_scale"):
        if getattr(a, n) is not None:
            assert torch.equal(getattr(a, n), getattr(b, n))


@pytest.mark.parametrize("kind", K.KINDS)
def test_bad_positions_and_slots(lib, kind):
    """A position outside the angles skips the row whole, a slot past the pools skips its cache rows; both report."""
    T, Hq, H, D, pages = 5, 2, 1, 64, 2
    x = _rows(1, T, Hq, H, D).cuda() + 1
    for pos, slot, skipped, uncached in (([0, 9, 10, 3, -1], [0, 1, 2, 3, 4], (2, 4), (2, 4)),
                                         ([0, 1, 2, 3, 4], [32, 1, -7, 31, 2 ** 62], (), (0, 2, 4))):
        c = lib.make_kv_cache(kind, pages, 16, H, D, k_amax=30.0, v_amax=30.0)
        ws = lib.make_kv_workspace(c)
        q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lib.kv_write(c, x, torch.tensor(slot).cuda(), Hq, positions=torch.tensor(pos, dtype=torch.int32).cuda(),
                     cos_sin=_angles(10, 64).cuda(), q_out=q, workspace=ws)
        torch.cuda.synchronize()
        assert lib.last_device_status(ws) == lib.HQ_ERR_INVALID_ARG
        for t in range(T):
            assert bool((q[t] == 7.0).all()) == (t in skipped)
        held = np.abs(K.cache_values(c, "v")).transpose(0, 2, 1, 3).reshape(pages * 16, -1).sum(1) > 0
        want = np.zeros(pages * 16, bool)
        want[[slot[t] for t in range(T) if t not in uncached]] = True
        assert np.array_equal(held, want)


def _starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int64)


@pytest.mark.parametrize("kind", K.KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,page,heads", [([1], 16, 1), ([0, 5, 0, 16, 33, 0], 16, 3), ([700, 1, 129], 48, 2),
                                             (list(range(1, 60)), 32, 1)])
def test_read(lib, kind, D, lens, page, heads):
    table, pages = K.tables(lens, page)
    c = lib.make_kv_cache(kind, pages, page, heads, D, k_amax=168.0, v_amax=168.0)
    K.fill(c, 3, poison=(0,))
    ws = lib.make_kv_workspace(c)
    k, v = lib.kv_read(c, table.cuda(), _starts(lens).cuda(), sum(lens), workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_OK
    for side, got in (("k", k), ("v", v)):
        vals = K.cache_values(c, side)
        want = np.concatenate([K.rows_of(vals, table[b].clamp(min=0).numpy(), page, 0, n) for b, n in enumerate(lens)])
        err = np.abs(K.f64(got) - want)
        # bf16: as it is; else the fp32 product (2^-24) and one rounding to bf16
        assert np.all(err <= (0 if kind == "bf16" else (2.0 ** -8 + 2.0 ** -22) * np.abs(want)))


@pytest.mark.parametrize("kind", K.KINDS)
def test_read_from_inside(lib, kind):
    """`first` starts inside the sequences, rows outside every sequence keep their values, bad pages are left out."""
    lens, page = [40, 100, 17], 16
    table, pages = K.tables(lens, page)
    c = lib.make_kv_cache(kind, pages, page, 2, 64, k_amax=168.0, v_amax=168.0)
    K.fill(c, 3)
    first, take = [5, 33, 16], [20, 60, 1]
    ws = lib.make_kv_workspace(c)
    starts = _starts(take) + 3  # rows 0 .. 2 belong to no sequence, nor do the last two
    out = tuple(torch.full((sum(take) + 5, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bad = table.clone()
    bad[1, 4] = pages  # tokens 64 .. 79 of sequence 1
    lib.kv_read(c, bad.cuda(), starts.cuda(), sum(take) + 5, first=torch.tensor(first, dtype=torch.int32).cuda(), out=out,
                workspace=ws)
    torch.cuda.synchronize()
    assert lib.last_device_status(ws) == lib.HQ_ERR_INVALID_ARG
    for side, got in (("k", out[0]), ("v", out[1])):
        vals = K.cache_values(c, side)
        want = np.full((sum(take) + 5, 2, 64), 9.0)
        for b in range(3):
            r = K.rows_of(vals, table[b].clamp(min=0).numpy(), page, first[b], first[b] + take[b])
            j = first[b] + np.arange(take[b])
            ok = (b != 1) | (j < 64) | (j >= 80)
            want[int(starts[b]) + np.arange(take[b])[ok]] = r[ok]
        assert np.all(np.abs(K.f64(got) - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want))
    # a sequence that ends past the rows, and one whose tokens lie past the table
    for s, n in ((torch.tensor([0, 30]), 20), (torch.tensor([0, 20]), 20)):
        t = table[:1].cuda() if n == 20 and int(s[1]) == 30 else table[:1, :1].contiguous().cuda()
        lib.kv_read(c, t, s.cuda(), n, workspace=ws)
        torch.cuda.synchronize()
        assert lib.last_device_status(ws) == lib.HQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", K.KINDS)
def test_written_then_read_then_written_again(lib, kind):
    """What is read back and written again without norm or rotation is held as the same values: quantisation settles."""
    T, H, D, page = 33, 2, 128, 16
    c, c2 = (lib.make_kv_cache(kind, 3, page, H, D, k_amax=30.0, v_amax=30.0) for _ in range(2))
    slots = torch.arange(T)
    _call(lib, c, _rows(1, T, H, H, D).cuda(), slots, H)
    table, starts = torch.arange(3, dtype=torch.int32)[None].cuda(), _starts([T]).cuda()
    k, v = lib.kv_read(c, table, starts, T)
    x = torch.cat((torch.zeros_like(k), k, v), dim=1).reshape(T, -1)
    _call(lib, c2, x, slots, H)
    k2, v2 = lib.kv_read(c2, table, starts, T)
    torch.cuda.synchronize()
    if kind == "bf16":
        assert torch.equal(k, k2) and torch.equal(v, v2)
    for a, b in ((k, k2), (v, v2)):  # one more rounding to bf16 (2^-8) can move a value by one step of its format
        a, b = K.f64(a), K.f64(b)
        assert np.all(np.abs(a - b) <= {"bf16": 0.0, "e4m3": 2.0 ** -3, "nvfp4": 0.5}[kind] * np.abs(a) + 1e-3)


def test_write_refuses(lib):
    c = lib.make_kv_cache("e4m3", 2, 16, 2, 64)
    x, s = torch.zeros((3, 8 * 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    cs, pos = _angles(4, 64).cuda(), torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = dict(qkv=x, slots=s, num_q_heads=4)
    bad = [dict(qkv=x.float()), dict(num_q_heads=5), dict(slots=s.int()), dict(slots=s[:2]), dict(qkv=x.t().contiguous().t()),
           dict(cos_sin=cs), dict(cos_sin=cs, positions=pos.long()), dict(cos_sin=cs.double(), positions=pos),
           dict(q_norm=torch.ones(32, dtype=torch.bfloat16, device="cuda")), dict(k_norm=torch.ones(64, device="cuda")),
           dict(qkv=x.cpu()), dict(cos_sin=cs[:, :0], positions=pos)]
    for over in bad:
        with pytest.raises(lib.HQArgError):
            lib.kv_write(c, **{**ok, **over})
    wide = torch.zeros((3, 8 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    for over, code in ((dict(eps=-1.0), lib.HQ_ERR_INVALID_ARG), (dict(eps=float("nan")), lib.HQ_ERR_INVALID_ARG),
                       (dict(cos_sin=_angles(4, 24).cuda(), positions=pos), lib.HQ_ERR_ALIGNMENT),
                       (dict(cos_sin=_angles(4, 80).cuda(), positions=pos), lib.HQ_ERR_INVALID_ARG),
                       (dict(qkv=wide[:, :8 * 64]), lib.HQ_ERR_ALIGNMENT),
                       (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), lib.HQ_ERR_WORKSPACE)):
        with pytest.raises(lib.HQError) as e:
            lib.kv_write(c, **{**ok, **over})
        assert e.value.code == code
    with pytest.raises(lib.HQArgError):
        lib.kv_read(c, torch.zeros((2, 1), dtype=torch.int32, device="cuda"), _starts([1]).cuda(), 1)
    with pytest.raises(lib.HQArgError):
        lib.kv_read(c, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), _starts([1]).int().cuda(), 1)
