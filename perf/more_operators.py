"""The operators of a decoder layer in 8-bit floating point with block scales: what is measured, and their plain forms.

A layer's activations and weights are e4m3 codes.  A row of activations has one fp32 scale, or one for every 128 of its
elements ("block"); weights have one fp32 scale for every block of 128 outputs by 128 inputs.

  norm    a sublayer's output is added to the residual stream and the sum's RMS norm goes to the next product as
          8-bit activations: scale = absmax / 448, code = e4m3(value / scale), a row or block of zeros has scale 0
  swiglu  silu(gate) * up of the first product's rows [gate | up], as 8-bit activations for the second
  gemm    out[m, n] = sum over blocks b of a_scale[m, b] * w_scale[n / 128, b] * (the block's sum of code products)

A case is a dict of plain values.
"""
import math

import torch

own = False


# ----------------------------------------------------------------- cases
def _norm(name, tokens, hidden, out, residual=True, padded=False):
    return dict(name=name, op="norm", tokens=tokens, hidden=hidden, out=out, residual=residual, padded=padded)


def _swiglu(name, rows, inner, out):
    return dict(name=name, op="swiglu", rows=rows, inner=inner, out=out)


def _gemm(name, m, n, k, bias=False):
    return dict(name=name, op="gemm", m=m, n=n, k=k, bias=bias)


def listed():
    return [
        # one user's decoding step: the smallest call, latency alone
        _norm("norm one token", 1, 4096, "block"),
        # a server's decoding step: a row per user, one scale per row
        _norm("norm step token", 64, 7168, "token"),
        # a small model's odd prompt for products that take bf16, the first layer: no residual yet
        _norm("norm prompt bf16", 1531, 2048, "bf16", residual=False),
        # a long prompt's prefill, padded to the batch's size
        _norm("norm prompt block", 8192, 7168, "block", padded=True),
        # a decoding step between the two products of a layer
        _swiglu("swiglu step block", 16, 7168, "block"),
        # the rows that 4096 tokens send to 8 experts each: short rows, many of them
        _swiglu("swiglu experts token", 32768, 768, "token"),
        # a long prompt's prefill
        _swiglu("swiglu prompt block", 8192, 7168, "block"),
        # one user's decoding step: the weights are all there is to read
        _gemm("gemm one token", 1, 4096, 7168),
        # a server's decoding step through the wide projection
        _gemm("gemm step", 64, 14336, 4096),
        # a short odd prompt into a vocabulary slice: odd rows and columns, with a bias
        _gemm("gemm ragged", 333, 1001, 2048, bias=True),
        # a chunk of a prompt
        _gemm("gemm chunk", 1024, 4096, 7168),
        # the largest: a long prompt's prefill through the wide projection
        _gemm("gemm prompt", 8192, 14336, 4096),
    ]


def draw(rng):
    log = lambda a, b: min(b, int(a * math.exp(rng.random() * math.log((b + 1) / a))))  # noqa: E731
    most = {op: max(work(c)["bytes" if op != "gemm" else "flops"] for c in listed() if c["op"] == op)
            for op in ("norm", "swiglu", "gemm")}
    op = rng.choice(["norm", "swiglu", "gemm", "gemm"])
    out = rng.choice(["block", "block", "token", "bf16"])
    if op == "norm":  # one-scale rows and bf16 rows need no whole blocks
        width = 128 * log(1, 128) if out == "block" else 16 * log(4, 1024)
        c = _norm("", log(1, 16384), width, out, rng.random() < 0.7, rng.random() < 0.3)
    elif op == "swiglu":
        out = "token" if out == "bf16" else out
        c = _swiglu("", log(1, 32768), 128 * log(1, 112) if out == "block" else 16 * log(4, 896), out)
    else:
        c = _gemm("", log(1, 8192), log(16, 16384), 128 * log(1, 64), rng.random() < 0.3)
    rows = "m" if op == "gemm" else "tokens" if op == "norm" else "rows"
    while work(c)["bytes" if op != "gemm" else "flops"] > most[op]:  # none costs more than the largest listed one
        c[rows] //= 2
    del c["name"]
    return c


def _scales(c, width):
    """fp32 scales of a row of activations."""
    return {"block": width // 128, "token": 1, "bf16": 0}[c["out"]]


def work(c):
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        b = m * k + n * k + 2 * m * n + 4 * m * (k // 128) + 4 * -(-n // 128) * (k // 128) + (2 * n if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * m * n * k}
    if c["op"] == "swiglu":
        r, w = c["rows"], c["inner"]
        return {"bytes": r * (4 * w + w + 4 * _scales(c, w)), "flops": 8 * r * w}
    t, w = c["tokens"], c["hidden"]
    out = 2 * w if c["out"] == "bf16" else w + 4 * _scales(c, w)
    return {"bytes": t * ((6 if c["residual"] else 2) * w + out) + 2 * w, "flops": 8 * t * w}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        t, w = c["tokens"], c["hidden"]
        gain = torch.exp(0.5 * _normal(g, w))  # channels differ in strength, a few by far
        gain = torch.where(torch.rand(w, generator=g, device="cuda") < 0.002, 30 * gain, gain)
        x = 0.5 * _normal(g, t, w)
        r = 3 * _normal(g, t, w) * gain
        if c["padded"]:  # rows that pad the batch hold zeros
            x[t - t // 64:] = 0
            r[t - t // 64:] = 0
        if not c["residual"]:
            x = r
        s["x"] = x.to(torch.bfloat16)
        s["residual"] = r.to(torch.bfloat16) if c["residual"] else None
        s["weight"] = (1 + 0.3 * _normal(g, w)).to(torch.bfloat16)
    elif c["op"] == "swiglu":
        s["x"] = (1.5 * _normal(g, c["rows"], 2 * c["inner"])).to(torch.bfloat16)
    else:
        m, n, k = c["m"], c["n"], c["k"]
        # activations and weights as a quantiser leaves them: every block's largest code is near 448
        a = _normal(g, m, k // 128, 128) * torch.exp(0.7 * _normal(g, m, k // 128, 1))
        top = a.abs().amax(-1, keepdim=True).clamp(min=1e-6)
        s["a"] = (a * (448 / top)).to(torch.float8_e4m3fn).view(torch.uint8).view(m, k)
        s["a_scale"] = (top[..., 0] / 448).contiguous()
        blocks = -(-n // 128)
        s["w"] = (100 * _normal(g, n, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["w_scale"] = (0.02 / 100) * torch.exp(0.3 * _normal(g, blocks, k // 128))
        s["bias"] = _normal(g, n).to(torch.bfloat16) if c["bias"] else None
        if own:  # the weights as a program lays them out once, and its workspace
            import quantized_gemm_dequant_gb300 as hq
            s["fmt"] = hq.make_format("e4m3_block", n, k)
            s["packed"] = hq.pack_weights(s["fmt"], s["w"], s["w_scale"])
            s["workspace"] = hq.make_workspace(s["fmt"], m)
    return s


# ----------------------------------------------------------------- plain forms
def _quantise(y, out):
    """fp32 [rows, width] -> the activations: (bf16 rows,) or (e4m3 codes, fp32 scales)."""
    if out == "bf16":
        return (y.to(torch.bfloat16),)
    b = y.unflatten(1, (-1, 128 if out == "block" else y.shape[1]))
    scale = b.abs().amax(-1, keepdim=True) / y.new_full((), 448.0)
    q = torch.where(scale > 0, b / scale, torch.zeros_like(b)).clamp(-448, 448)
    scale = scale[..., 0] if out == "block" else scale[:, 0, 0]
    return q.flatten(1).to(torch.float8_e4m3fn), scale


def _norm_plain(s):
    c, x = s["case"], s["x"].float()
    if c["residual"]:
        x = x + s["residual"].float()
    y = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * s["weight"].float()
    return (*_quantise(y, c["out"]), *((x.to(torch.bfloat16),) if c["residual"] else ()))


def _swiglu_plain(s):
    c, x = s["case"], s["x"].float()
    gate, up = x[:, :c["inner"]], x[:, c["inner"]:]
    return _quantise(gate / (1 + torch.exp(-gate)) * up, c["out"])


def _gemm_plain(s):
    c = s["case"]
    a = s["a"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * s["a_scale"][..., None]
    rows = s["w_scale"].repeat_interleave(128, dim=0)[:c["n"]]
    w = s["w"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * rows[..., None]
    y = a.flatten(1) @ w.flatten(1).T
    if c["bias"]:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


def _act_out(act, out):
    """The framework's activations as the values they stand for."""
    return (act["data"],) if out == "bf16" else (act["data"].view(torch.float8_e4m3fn), act["scale"])


def run(s):
    c = s["case"]
    if not own:
        return {"norm": _norm_plain, "swiglu": _swiglu_plain, "gemm": _gemm_plain}[c["op"]](s)
    import quantized_gemm_dequant_gb300 as hq
    if c["op"] == "gemm":
        return hq.gemm(s["fmt"], {"data": s["a"], "scale": s["a_scale"]}, s["packed"], c["m"], bias=s["bias"],
                       workspace=s["workspace"])
    afmt = {"block": "e4m3_block", "token": "e4m3_tok", "bf16": "bf16"}[c["out"]]
    if c["op"] == "swiglu":
        return _act_out(hq.swiglu_quantize(afmt, s["x"]), c["out"])
    act, stream = hq.add_rms_norm(afmt, s["x"], s["weight"], residual=s["residual"], eps=1e-6)
    return (*_act_out(act, c["out"]), *((stream,) if c["residual"] else ()))


# ----------------------------------------------------------------- 64 bits
def _e4m3_table():
    """fp64 values of the 256 e4m3 codes, from sign, exponent and mantissa."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if b & 127 == 127 else -x if b > 127 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _codes64(y, out):
    """What _quantise gives, from fp64 values and in fp64."""
    if out == "bf16":
        return (y,)
    rows, width = y.shape
    size = 128 if out == "block" else width
    f = torch.linalg.vector_norm(y.view(rows, width // size, size), ord=math.inf, dim=-1) / 448
    z = y / torch.where(f > 0, f, 1.0).repeat_interleave(size, dim=1)
    step = torch.exp2(torch.clamp(torch.frexp(z).exponent.double() - 1, min=-6.0) - 3)
    return torch.clamp(torch.round(z / step) * step, -448.0, 448.0), (f if out == "block" else f.view(rows))


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "gemm":
        t = _e4m3_table()
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        of = torch.arange(c["n"], device="cuda") // 128
        for b in range(c["k"] // 128):
            at = slice(128 * b, 128 * b + 128)
            p = torch.mm(t[s["a"][:, at].long()], t[s["w"][:, at].long()].T)
            y += p.mul_(s["a_scale"][:, b, None].double()).mul_(s["w_scale"].double()[of, b])
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["x"].double()
    if c["op"] == "swiglu":
        gate, up = x.split(c["inner"], dim=1)
        return _codes64(gate * torch.sigmoid(gate) * up, c["out"])
    if c["residual"]:
        x = x + s["residual"].double()
    size = torch.linalg.vector_norm(x, dim=1, keepdim=True) / math.sqrt(c["hidden"])
    y = x * s["weight"].double() / torch.hypot(size, torch.full_like(size, 1e-3))
    return (*_codes64(y, c["out"]), *((x,) if c["residual"] else ()))
