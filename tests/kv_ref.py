"""Plain 64-bit forms of the paged key-value cache's operators, on the CPU, and the caches the tests fill.

Nothing here shares code with the kernels.  Tensors come in as the GPU holds them and are worked on as numpy float64.
"""
import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
KINDS = ("bf16", "e4m3", "nvfp4")


def _e4m3(code):
    code = np.asarray(code).astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code > 127, -v, v)


def f64(t):
    """float64 numpy of a tensor's values."""
    return t.detach().cpu().to(torch.float64).numpy()


def cache_values(cache, side):
    """float64 [pages, heads, page_size, head_dim]: the values one pool stands for."""
    codes, scale = getattr(cache, side), getattr(cache, side + "_scale")
    if cache.kind == "bf16":
        return f64(codes)
    c = codes.cpu().numpy()
    if cache.kind == "e4m3":
        return _e4m3(c) * f64(scale)[..., None]
    v = np.empty((*c.shape[:-1], cache.head_dim))
    v[..., 0::2], v[..., 1::2] = E2M1[c & 15], E2M1[c >> 4]
    g = float(getattr(cache, side + "_global").cpu()[0])
    return v * np.repeat(_e4m3(scale.cpu().numpy()) * g, 16, axis=-1)


def fill(cache, seed, poison=()):
    """Random pools: values from N(0, 1) with strong channels, in the cache's format (bf16: the values; else random
    codes with scales of a realistic spread).  Pages in `poison` hold NaN, infinities and the largest values."""
    g = torch.Generator().manual_seed(seed)
    for side in ("k", "v"):
        t, s = getattr(cache, side), getattr(cache, side + "_scale")
        if cache.kind == "bf16":
            t.copy_((torch.randn(t.shape, generator=g) * torch.exp(0.5 * torch.randn(t.shape[-1], generator=g))))
        elif cache.kind == "e4m3":
            x = torch.randn(t.shape, generator=g).clamp(-4, 4) * 100
            t.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
            s.copy_(torch.exp(0.7 * torch.randn(s.shape, generator=g)) / 100)
        else:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
            s.copy_(torch.randint(0x20, 0x58, s.shape, generator=g, dtype=torch.uint8))  # 2^-3 .. 15
        for p in poison:
            if cache.kind == "bf16":
                t[p] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38],
                                    dtype=torch.bfloat16).repeat(t.shape[-1] // 4).to(t.device)
            else:
                t[p] = 0x7F
                s[p] = float("nan") if cache.kind == "e4m3" else 0x7F


def poison_tail(cache, table, lens):
    """NaN into the places of each sequence's last page that lie past its length."""
    for b, n in enumerate(lens):
        if n % cache.page_size:
            p, o = int(table[b, n // cache.page_size]), n % cache.page_size
            for side in ("k", "v"):
                t, s = getattr(cache, side), getattr(cache, side + "_scale")
                t[p, :, o:] = float("nan") if cache.kind == "bf16" else 0x7F
                if s is not None:
                    s[p, :, o:] = float("nan") if cache.kind == "e4m3" else 0x7F


def tables(lens, page, seed=0, spare=1, columns=None):
    """(int32 page table on the CPU, number of pages): page 0 .. spare - 1 belong to no sequence, entries past a
    sequence's pages are -1."""
    need = [-(-n // page) for n in lens]
    t = torch.full((len(lens), columns or max(max(need, default=1), 1)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).to(torch.int32) + spare
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, max(sum(need) + spare, 1)


def rows_of(values, table_row, page, lo, hi):
    """float64 [hi - lo, heads, dim]: tokens lo .. hi - 1 of a sequence."""
    j = np.arange(lo, hi)
    return values[np.asarray(table_row)[j // page], :, j % page]


def attention(cache, q, table, lens, scale, window=0, softcap=0.0, drop=None):
    """(out, lse, bound on |out|'s error, bound on |lse|'s error), each float64 on the CPU.

    The bounds: with u the unit roundoff of the 16-bit type the weights are rounded to (bf16 2^-8, f16 2^-11), the
    scores' error ds from fp32 sums of D products (each add and product within 2^-24 of the sum of magnitudes; the
    matrix unit may truncate, so twice that), from the rotation of the cap (a few 2^-23 of the cap) and from exp2's
    argument (|s| 2^-22), every weight is off by at most (u + 2 ds + 2^-18) of itself, an f16 weight also by 2^-25 of
    the largest; the output is rounded once to bf16 (2^-8)."""
    K, V = cache_values(cache, "k"), cache_values(cache, "v")
    Q, tab = f64(q), table.cpu().numpy()
    B, Hq, D = Q.shape
    G = Hq // cache.num_heads
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    bo, bl = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    u, sub = (2.0 ** -8, 0.0) if cache.kind == "bf16" else (2.0 ** -11, 2.0 ** -25)
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        keep = np.ones(n - lo, bool)
        if drop is not None:
            keep = ~drop(b, np.arange(lo, n))
        if not keep.any():
            continue
        row = np.maximum(tab[b], 0)
        k, v = rows_of(K, row, cache.page_size, lo, n)[keep], rows_of(V, row, cache.page_size, lo, n)[keep]
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            s = kk @ Q[b, h] * scale
            ds = 2 * D * 2.0 ** -24 * np.max(np.abs(kk) @ np.abs(Q[b, h])) * abs(scale)
            if softcap:
                s = softcap * np.tanh(s / softcap)
                ds += softcap * 2.0 ** -20
            ds += np.max(np.abs(s)) * 2.0 ** -21
            m = s.max()
            e = np.exp(s - m)
            z = e.sum()
            out[b, h], lse[b, h] = e @ vv / z, m + np.log(z)
            bo[b, h] = (2.0 ** -8 * np.abs(out[b, h]) + (u + 2 * ds + 2.0 ** -18) * (e @ np.abs(vv)) / z
                        + sub * np.abs(vv).sum(0) / z)
            bl[b, h] = ds + 2.0 ** -18 + abs(lse[b, h]) * 2.0 ** -22
    return out, lse, bo, bl


def norm_rotate(x, w, eps, cos_sin, positions, interleaved):
    """float64 [T, heads, D]: RMS norm over D (w None: none), rotation of the leading dims (cos_sin None: none)."""
    x = f64(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w)
    y = x.copy()
    if cos_sin is not None:
        cs = f64(cos_sin)[positions.cpu().numpy()]
        r = cs.shape[1]
        c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
        i = np.arange(r // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y
