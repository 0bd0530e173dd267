"""Plain 64-bit forms of the operators of a layer in 8-bit floating point with block scales, on the CPU, and how far a
right kernel may be from them.

Bounds count roundings, each off by at most half a step: bf16 2^-8 relative, fp32 2^-24, e4m3 2^-4 (2^-10 absolute among
its subnormals).  FINE covers the fp32 arithmetic of a row's statistics, its normalised values and silu: a sum of squares
along chains of at most 16 terms and 10 tree levels (its root takes half of that: 13 roundings), at most 10 more for
division, root, products and the fast exponential and reciprocal (2 ulp each at most after their corrections), together
below 32 * 2^-24."""
import numpy as np
import torch

BF16, E4M3, FINE = 2.0 ** -8, 2.0 ** -4, 2.0 ** -19


def f64(t):
    return t.detach().cpu().double().numpy()


def e4m3_values():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if b & 127 == 127 else -x if b > 127 else x
    return v


VALUES = e4m3_values()


def decode(codes):
    return VALUES[codes.detach().cpu().view(torch.uint8).numpy()]


def swiglu(x):
    """fp64 silu(gate) * up of fp64 rows [gate | up]."""
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore", invalid="ignore"):
        e = np.exp(-np.abs(g))
        sig = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * sig * u


def norm(x, w, eps):
    with np.errstate(invalid="ignore", over="ignore"):
        return x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * w


def check_bf16(got, want, tiny=2.0 ** -133):
    got = f64(got)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got))
    err = np.abs(got - want)[fine]
    assert np.all(err <= (BF16 + FINE) * np.abs(want[fine]) + tiny), float(np.max(err / (np.abs(want[fine]) + tiny)))


def check_act(act, want, block, rows_of_zeros=()):
    """e4m3 codes and scales of an activation operand against the fp64 values that they stand for."""
    rows, width = want.shape
    size = 128 if block else width
    scale = f64(act["scale"]).reshape(rows, width // size)
    code = decode(act["data"]).reshape(rows, width // size, size)
    want = want.reshape(rows, width // size, size)
    top = np.max(np.abs(want), axis=-1)
    s = top / 448
    # a scale among fp32's subnormals is rounded to a multiple of 2^-149, and so is what it scales
    assert np.all(np.abs(scale - s) <= FINE * s + 2.0 ** -148), float(np.max(np.abs(scale - s) / np.maximum(s, 1e-300)))
    assert np.all(code[scale == 0] == 0)
    big = s > 2.0 ** -120
    z = np.where(big[..., None], want / np.where(big, s, 1.0)[..., None], 0.0)
    err = np.where(big[..., None], np.abs(code - z), 0.0)
    bound = np.maximum(E4M3 * np.abs(z), 2.0 ** -10) + 2 * FINE * np.abs(z)
    assert np.all(err <= bound), float(np.max(err / bound))
    for r in rows_of_zeros:
        assert np.all(scale[r] == 0) and np.all(code[r] == 0)


def product(a, a_scale, w, w_scale, bias=None):
    """(fp64 product, the sum of its terms' magnitudes) from codes [M, K], [N, K] and scales [M, K/128],
    [ceil(N/128), K/128]."""
    M, K = a.shape
    N = w.shape[0]
    A, W = (decode(t).reshape(t.shape[0], K // 128, 128) for t in (a, w))
    A = A * f64(a_scale).reshape(M, K // 128, 1)
    W = W * np.repeat(f64(w_scale), 128, axis=0)[:N, :, None]
    A, W = A.reshape(M, K), W.reshape(N, K)
    y, size = A @ W.T, np.abs(A) @ np.abs(W).T
    return (y if bias is None else y + f64(bias)), size


def check_product(got, want, size, blocks, bias=None):
    """bf16's rounding, and fp32 sums: 128 products in a block (the tensor cores' sums taken as twice as coarse as
    fp32's), one rounding per block of the sum over them and two of its scale."""
    got = f64(got)
    add = np.abs(f64(bias)) if bias is not None else 0.0
    bound = BF16 * np.abs(want) + (128 * 2.0 ** -23 + (blocks + 4) * 2.0 ** -24) * size + 2.0 ** -23 * add + 2.0 ** -133
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - want) / bound)))


def operands(seed, M, N, K, bias=False, device="cuda"):
    """Codes and scales as a quantiser leaves them: full-range codes, scales that differ from block to block."""
    g = torch.Generator().manual_seed(seed)
    B = K // 128
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = (150 * n(M, K)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    w = (150 * n(N, K)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    a_scale = 0.01 * torch.exp(n(M, B))
    w_scale = 1e-4 * torch.exp(n(-(-N // 128), B))
    b = n(N).to(torch.bfloat16) if bias else None
    return tuple(None if t is None else t.to(device) for t in (a, a_scale, w, w_scale, b))
