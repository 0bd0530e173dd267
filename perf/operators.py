"""The key-value cache operators: what is measured, and their plain forms.

Three operators work on one paged cache of keys and values.  A page holds `page` tokens of every key-value head, laid
out [pages, kv heads, page, head dim]; a token's place is its slot, page id * page + offset.  The cache holds bf16
values, e4m3 codes with one fp32 scale per (token, head), or NVFP4 (e2m1 codes two per byte, low nibble = even dim, an
e4m3 scale per 16 dims, one fp32 global scale for the keys and one for the values).

  write   the fused projection's rows [q heads | k heads | v heads] -> RMS norm of every query and key head, rotation
          by position, queries out in bf16, keys and values quantised into their slots
  read    the cached tokens of every sequence, given its page table, back as contiguous bf16 rows
  attend  one new token per sequence attends to that sequence's cached tokens

A case is a dict of plain values.  Lengths follow from the case alone, values from the seed.
"""
import math

import torch

own = False

FINE = 2.0 ** -126  # smallest normal fp32: no sum of exponentials that holds a term is below it


# ----------------------------------------------------------------- cases
def _attend(name, kind, batch, longest, kv_heads, group, dim, page, ragged=True, window=0, softcap=0.0):
    return dict(name=name, op="attend", kind=kind, batch=batch, longest=longest, kv_heads=kv_heads, group=group,
                dim=dim, page=page, ragged=ragged, window=window, softcap=softcap)


def _write(name, kind, tokens, kv_heads, group, dim, page, rotary, norm=True, interleaved=False, prefill=True):
    return dict(name=name, op="write", kind=kind, tokens=tokens, kv_heads=kv_heads, group=group, dim=dim, page=page,
                rotary=rotary, norm=norm, interleaved=interleaved, prefill=prefill)


def _read(name, kind, batch, longest, kv_heads, dim, page, ragged=True):
    return dict(name=name, op="read", kind=kind, batch=batch, longest=longest, kv_heads=kv_heads, dim=dim, page=page,
                ragged=ragged)


def listed():
    return [
        # one user's short prompt: the smallest call, latency alone
        _attend("attend one short", "bf16", 1, 300, 8, 4, 128, 16),
        # a server's batch of conversations on an unquantised cache
        _attend("attend batch bf16", "bf16", 24, 5000, 8, 4, 128, 16),
        # one document of 128 Ki tokens: all of the GPU on one sequence
        _attend("attend long e4m3", "e4m3", 1, 131072, 8, 4, 128, 64, ragged=False),
        # the throughput case of an 8-bit cache: many ragged contexts, four kv heads
        _attend("attend batch e4m3", "e4m3", 64, 16384, 4, 8, 128, 32),
        # a local layer: window and capped scores, wide heads
        _attend("attend window bf16", "bf16", 33, 9001, 4, 2, 256, 16, window=1024, softcap=50.0),
        # the largest: a 4-bit cache under a full batch
        _attend("attend batch nvfp4", "nvfp4", 128, 8192, 8, 8, 128, 64),
        # a decoding step's append: one token per sequence
        _write("append step e4m3", "e4m3", 48, 8, 4, 128, 32, 128, prefill=False),
        # a long prompt's prefill into an 8-bit cache
        _write("append prompt e4m3", "e4m3", 8192, 8, 4, 128, 64, 128),
        # small heads, partial interleaved rotation, no norm, an odd number of tokens
        _write("append prompt bf16", "bf16", 1531, 2, 7, 64, 16, 32, norm=False, interleaved=True),
        # a chunk of a prompt into a 4-bit cache, read back at once for the chunk's own attention
        _write("append chunk nvfp4", "nvfp4", 2048, 8, 4, 128, 64, 128),
        # cached prefixes of a batch, read back for a prefill kernel that takes bf16
        _read("read prefixes e4m3", "e4m3", 9, 16000, 8, 128, 32),
        # one cached document in 4 bits
        _read("read document nvfp4", "nvfp4", 1, 50001, 8, 128, 64, ragged=False),
    ]


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    log = lambda a, b: min(b, int(a * math.exp(rng.random() * math.log((b + 1) / a))))  # noqa: E731
    op = rng.choice(["attend", "attend", "write", "read"])
    kind = rng.choice(["bf16", "e4m3", "nvfp4"])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 48, 64, 128])
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
    if op == "write":
        tokens = log(1, 16384)
        rotary = rng.choice([dim, dim, dim // 2, 0])
        c = _write("", kind, tokens, kv, group, dim, page, rotary, rng.random() < 0.7, rng.random() < 0.3,
                   tokens > 256 or rng.random() < 0.3)
    elif op == "read":
        c = _read("", kind, log(1, 64), log(1, 65536), kv, dim, page, rng.random() < 0.7)
    else:
        longest = log(1, 131072)
        window = log(1, longest) if rng.random() < 0.25 else 0
        c = _attend("", kind, log(1, 256), longest, kv, group, dim, page, rng.random() < 0.7, window,
                    rng.choice([0.0, 0.0, 0.0, 30.0]))
    if op != "write":  # no drawn case costs more than the largest listed one, padded to its longest sequence or not
        while work(c)["bytes"] > most or c["batch"] * c["longest"] * kv * dim > 1 << 30:
            c["batch"], c["longest"] = (c["batch"] // 2, c["longest"]) if c["batch"] > 1 else (1, c["longest"] // 2)
            if op == "attend":
                c["window"] = min(c["window"], c["longest"])
    del c["name"]
    return c


def _lengths(c):
    """Tokens cached of each sequence: all of the longest, or spread from 1 to it by the golden ratio."""
    if not c["ragged"]:
        return [c["longest"]] * c["batch"]
    return [1 + int((c["longest"] - 1) * ((1.0 - 0.6180339887498949 * b) % 1.0 if b else 1.0))
            for b in range(c["batch"])]


def _row_bytes(c):
    """Bytes of one (token, head)'s codes and scale in the cache."""
    return {"bf16": 2 * c["dim"], "e4m3": c["dim"] + 4, "nvfp4": c["dim"] // 2 + c["dim"] // 16}[c["kind"]]


def work(c):
    kv, dim = c["kv_heads"], c["dim"]
    if c["op"] == "write":
        t, hq = c["tokens"], c["kv_heads"] * c["group"]
        put = t - _padding(c)
        b = 2 * t * (hq + 2 * kv) * dim + 2 * t * hq * dim + 2 * put * kv * _row_bytes(c) + t * (8 + 4)
        b += 4 * t * c["rotary"]
        if c["kind"] == "nvfp4":
            b += 2 * put * kv * (_row_bytes(c) + 2 * dim)
        return {"bytes": b, "flops": t * (hq + 2 * kv) * dim * 8}
    lens = _lengths(c)
    pages = sum(-(-n // c["page"]) for n in lens)
    if c["op"] == "read":
        n = sum(lens)
        return {"bytes": 2 * n * kv * (_row_bytes(c) + 2 * dim) + 4 * pages + 8 * len(lens), "flops": 2 * n * kv * dim}
    n = sum(min(x, c["window"]) if c["window"] else x for x in lens)
    hq = kv * c["group"]
    return {"bytes": 2 * n * kv * _row_bytes(c) + 4 * pages + len(lens) * hq * (4 * dim + 4),
            "flops": 4 * n * hq * dim}


# ----------------------------------------------------------------- formats, plain
def _to_e2m1(x):
    """Codes of e2m1(x): magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6, ties to even, saturating; a zero code has no sign."""
    a = x.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return torch.where((x < 0) & (m > 0), m + 8, m)


def _from_e2m1(packed):
    """fp32 values of packed e2m1 codes: [..., n] bytes -> [..., 2n]."""
    c = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)
    e, m = ((c >> 1) & 3).float(), (c & 1).float()
    v = torch.where(e > 0, torch.exp2(e - 1) * (1 + 0.5 * m), 0.5 * m)
    return torch.where(c > 7, -v, v)


def _quantise(kind, x, g):
    """fp32 [..., dim] -> (codes, scales) of the cache format; both as bytes where they are 8 bits."""
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    if kind == "e4m3":
        s = x.abs().amax(-1) / x.new_full((), 448.0)  # a division: by a Python number torch multiplies by 1 / 448
        y = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s
    b = x.unflatten(-1, (-1, 16))
    sb = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448).to(torch.float8_e4m3fn)
    d = (sb.float() * g)[..., None]
    c = _to_e2m1(torch.where(d > 0, b / d, torch.zeros_like(b))).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), sb.view(torch.uint8)


def _values(kind, codes, scales, g):
    """fp32 values of cache rows."""
    if kind == "bf16":
        return codes.float()
    if kind == "e4m3":
        return codes.view(torch.float8_e4m3fn).float() * scales[..., None]
    d = scales.view(torch.float8_e4m3fn).float() * g
    return (_from_e2m1(codes).unflatten(-1, (-1, 16)) * d[..., None]).flatten(-2)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _empty_cache(c, pages):
    shape, dev = (pages, c["kv_heads"], c["page"]), "cuda"
    z = {}
    for side in ("k", "v"):
        if c["kind"] == "bf16":
            z[side] = torch.zeros(*shape, c["dim"], dtype=torch.bfloat16, device=dev)
        elif c["kind"] == "e4m3":
            z[side] = torch.zeros(*shape, c["dim"], dtype=torch.uint8, device=dev)
            z[side + "_scale"] = torch.zeros(*shape, dtype=torch.float32, device=dev)
        else:
            z[side] = torch.zeros(*shape, c["dim"] // 2, dtype=torch.uint8, device=dev)
            z[side + "_scale"] = torch.zeros(*shape, c["dim"] // 16, dtype=torch.uint8, device=dev)
            # calibrated largest magnitude / (6 * 448): keys carry a few strong channels
            z[side + "_global"] = torch.full((1,), (23.7 if side == "k" else 7.9) / 2688.0, device=dev)
    return z


def _tables(lens, page, g):
    """Page table [batch, most pages], the pages of all sequences in a random order; page 0 belongs to none, entries
    past a sequence's last page are -1."""
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(need), generator=g, device="cuda").cpu().to(torch.int32) + 1
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.cuda(), sum(need) + 1


def _padding(c):
    """Rows of a prefill step that pad it and are not cached (slot -1)."""
    return c["tokens"] // 32 if c["prefill"] else 0


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    kv, dim, page, kind = c["kv_heads"], c["dim"], c["page"], c["kind"]
    s = dict(case=c)
    if c["op"] == "write":
        t, hq = c["tokens"], kv * c["group"]
        put = t - _padding(c)
        if c["prefill"]:  # one prompt from its start
            lens = [max(put, 1)]
            table, pages = _tables(lens, page, g)
            i = torch.arange(t, device="cuda")
            slots = table[0].long()[(i // page).clamp(max=table.shape[1] - 1)] * page + i % page
            slots = torch.where(i < put, slots, torch.full_like(slots, -1))
            positions = i.to(torch.int32)
            s["starts"] = torch.tensor([0, put], dtype=torch.int64, device="cuda")
        else:  # one token of each of `tokens` sequences, each in a page of its own
            pages = t + 1
            positions = torch.randint(0, 8192, (t,), generator=g, device="cuda", dtype=torch.int32)
            table = torch.randperm(t, generator=g, device="cuda").to(torch.int32)[:, None] + 1
            off = torch.zeros_like(positions) if kind == "nvfp4" else positions % page
            slots = table[:, 0].long() * page + off
            s["starts"] = torch.arange(t + 1, dtype=torch.int64, device="cuda")
        s["table"] = table
        s["total"] = put if c["prefill"] else t
        gain = torch.exp(0.5 * _normal(g, (hq + 2 * kv) * dim))  # channels differ in strength
        s["qkv"] = (_normal(g, t, (hq + 2 * kv) * dim) * gain).to(torch.bfloat16)
        s["slots"], s["positions"] = slots, positions
        s["cos_sin"] = None
        if c["rotary"]:
            freq = 10000.0 ** (-torch.arange(0, c["rotary"], 2, device="cuda") / c["rotary"])
            a = torch.arange(max(8192, t), device="cuda")[:, None] * freq
            s["cos_sin"] = torch.cat((a.cos(), a.sin()), dim=1).contiguous()
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"] = (1 + 0.3 * _normal(g, dim)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.3 * _normal(g, dim)).to(torch.bfloat16)
        s["cache"] = _empty_cache(c, pages)
    else:
        lens = _lengths(c)
        s["table"], pages = _tables(lens, page, g)
        cache = _empty_cache(c, pages)
        for side in ("k", "v"):
            gain = torch.exp(0.5 * _normal(g, kv, 1, dim))
            for at in range(1, pages, max(1, (1 << 27) // (kv * page * dim))):  # a piece at a time: less memory
                to = min(pages, at + max(1, (1 << 27) // (kv * page * dim)))
                x = _normal(g, to - at, kv, page, dim) * gain
                codes, scales = _quantise(kind, x, cache.get(side + "_global"))
                cache[side][at:to] = codes
                if scales is not None:
                    cache[side + "_scale"][at:to] = scales
        s["cache"] = cache
        if c["op"] == "read":
            starts = [0]
            for n in lens:
                starts.append(starts[-1] + n)
            s["starts"] = torch.tensor(starts, dtype=torch.int64, device="cuda")
            s["total"] = starts[-1]
        else:
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            s["q"] = (1.5 * _normal(g, len(lens), kv * c["group"], dim)).to(torch.bfloat16)
    if own:  # the handle and the workspace that a server keeps
        import quantized_gemm_dequant_gb300 as hq
        s["handle"] = hq.KVCache(kind, **s["cache"])
        s["workspace"] = hq.make_kv_workspace(s["handle"], s["q"].shape[0] if c["op"] == "attend" else 0,
                                              kv * c.get("group", 1))
    return s


# ----------------------------------------------------------------- plain forms
def _norm_rotate(x, w, s, c):
    """fp32 [tokens, heads, dim] -> RMS norm with weight w over dim, then the rotation of the first `rotary` dims."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    r = c["rotary"]
    if not r:
        return x
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1)


def _put(cache, side, x, slots, kind, page):
    """Rows into their slots, in place; a negative slot writes page 0's first row, which no sequence owns, as it is."""
    codes, scales = _quantise(kind, x, cache.get(side + "_global"))
    keep, at = slots >= 0, slots.clamp(min=0)
    p, o = at // page, at % page
    old = cache[side][p, :, o]
    cache[side][p, :, o] = torch.where(keep[:, None, None], codes, old)
    if scales is not None:
        z = cache[side + "_scale"]
        z[p, :, o] = torch.where(keep.view(-1, *[1] * (scales.dim() - 1)), scales, z[p, :, o])


def _write_plain(s):
    c, cache = s["case"], s["cache"]
    kv, hq, dim = c["kv_heads"], c["kv_heads"] * c["group"], c["dim"]
    x = s["qkv"].float().unflatten(1, (hq + 2 * kv, dim))
    q = _norm_rotate(x[:, :hq], s["q_norm"], s, c)
    k = _norm_rotate(x[:, hq:hq + kv], s["k_norm"], s, c)
    _put(cache, "k", k, s["slots"], c["kind"], c["page"])
    _put(cache, "v", x[:, hq + kv:], s["slots"], c["kind"], c["page"])
    return q.to(torch.bfloat16)


def _read_plain(s):
    c, cache = s["case"], s["cache"]
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["starts"], row, right=True) - 1
    i = row - s["starts"][b]
    p, o = s["table"][b, i // c["page"]].long(), i % c["page"]
    got = [_values(c["kind"], cache[side][p, :, o], cache[side + "_scale"][p, :, o] if c["kind"] != "bf16" else None,
                   cache.get(side + "_global")).to(torch.bfloat16) for side in ("k", "v")]
    return got[0], got[1]


def _attend_plain(s):
    c, cache = s["case"], s["cache"]
    pages = s["table"].clamp(min=0).long()
    rows = []
    for side in ("k", "v"):
        scale = cache[side + "_scale"][pages] if c["kind"] != "bf16" else None
        x = _values(c["kind"], cache[side][pages], scale, cache.get(side + "_global"))  # [B, P, H, page, dim]
        rows.append(x.transpose(1, 2).flatten(2, 3))
    k, v = rows
    q = s["q"].float().unflatten(1, (c["kv_heads"], c["group"]))
    t = (q @ k.transpose(-1, -2)) * c["dim"] ** -0.5
    if c["softcap"]:
        t = c["softcap"] * torch.tanh(t / c["softcap"])
    pos, n = torch.arange(k.shape[2], device="cuda"), s["lens"][:, None]
    keep = pos < n
    if c["window"]:
        keep = keep & (pos >= n - c["window"])
    t = torch.where(keep[:, None, None], t, -torch.inf)
    top = t.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(t - top)
    z = e.sum(-1, keepdim=True)
    out = (e @ v) / z.clamp(min=FINE)
    return out.flatten(1, 2).to(torch.bfloat16), (top + torch.log(z)).flatten(1, 3)


def _cache_out(cache):
    """The cache's buffers as the values they hold."""
    return {n: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for n, t in cache.items()}


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "attend":
            return _attend_plain(s)
        if c["op"] == "read":
            return _read_plain(s)
        q = _write_plain(s)
        return (q, *_read_plain(s)) if c["kind"] == "nvfp4" else (q, _cache_out(s["cache"]))
    import quantized_gemm_dequant_gb300 as hq
    h, ws = s["handle"], s["workspace"]
    if c["op"] == "attend":
        return hq.paged_attention(h, s["q"], s["table"], s["lens"], window=c["window"], softcap=c["softcap"],
                                  workspace=ws)
    if c["op"] == "read":
        return hq.kv_read(h, s["table"], s["starts"], s["total"], workspace=ws)
    q = hq.kv_write(h, s["qkv"], s["slots"], c["kv_heads"] * c["group"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                    eps=1e-6, positions=s["positions"], cos_sin=s["cos_sin"], interleaved=c["interleaved"], workspace=ws)
    if c["kind"] == "nvfp4":
        return (q, *hq.kv_read(h, s["table"], s["starts"], s["total"], workspace=ws))
    return q, _cache_out(s["cache"])


# ----------------------------------------------------------------- 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _e4m3_table():
    """fp64 values of the 256 e4m3 codes, from sign, exponent and mantissa."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if b & 127 == 127 else -x if b > 127 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _rows64(c, cache, side, page_ids, n):
    """fp64 [kv heads, n, dim]: the first n tokens of a sequence with these pages."""
    ids = page_ids[:-(-n // c["page"])].long()
    x = cache[side].index_select(0, ids).movedim(1, 0).flatten(1, 2)[:, :n]
    if c["kind"] == "bf16":
        return x.double()
    f = cache[side + "_scale"].index_select(0, ids).movedim(1, 0).flatten(1, 2)[:, :n]
    if c["kind"] == "e4m3":
        return _e4m3_table()[x.long()] * f.double()[..., None]
    t = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    y = torch.empty(*x.shape[:-1], c["dim"], dtype=torch.float64, device="cuda")
    y[..., 0::2], y[..., 1::2] = t[(x % 16).long()], t[(x // 16).long()]
    return y * (_e4m3_table()[f.long()] * cache[side + "_global"].double()).repeat_interleave(16, dim=-1)


def _round64(x, mantissa, lowest, most):
    """fp64 x to the nearest value of `mantissa` fraction bits, exponents from `lowest`, at most `most`; ties to even."""
    e = torch.frexp(x).exponent.double() - 1
    step = torch.exp2(torch.clamp(e, min=lowest) - mantissa)
    return torch.clamp(torch.round(x / step) * step, -most, most)


def _write64(c, s):
    kv, hq, dim, r = c["kv_heads"], c["kv_heads"] * c["group"], c["dim"], c["rotary"]
    heads = s["qkv"].double().view(c["tokens"], hq + 2 * kv, dim)
    parts = []
    for x, w in ((heads[:, :hq], s["q_norm"]), (heads[:, hq:hq + kv], s["k_norm"])):
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / dim + 1e-6) * w.double()
        y = x.clone()
        if r:
            cs = s["cos_sin"].double()[s["positions"].long()]
            turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
            ia = torch.arange(r // 2, device="cuda")
            ia, ib = (2 * ia, 2 * ia + 1) if c["interleaved"] else (ia, ia + r // 2)
            z = torch.complex(x[..., ia], x[..., ib]) * turn
            y[..., ia], y[..., ib] = z.real, z.imag
        parts.append(y)
    q, k, v = parts[0], parts[1], heads[:, hq + kv:]
    if c["kind"] == "nvfp4":
        back = []
        for side, x in (("k", k), ("v", v)):
            g = s["cache"][side + "_global"].double()
            b = x[s["slots"] >= 0].unflatten(-1, (dim // 16, 16))
            d = _round64(b.abs().amax(-1, keepdim=True) / (6 * g), 3, -6, 448.0) * g
            y = torch.where(d > 0, _round64(b / torch.where(d > 0, d, 1.0), 1, 0, 6.0) * d, 0.0)
            back.append(y.flatten(-2))
        return q, back[0], back[1]
    out = {n: torch.zeros(t.shape, dtype=torch.float64, device="cuda") for n, t in s["cache"].items()}
    at = s["slots"][s["slots"] >= 0]
    for side, x in (("k", k), ("v", v)):
        x = x[s["slots"] >= 0]
        if c["kind"] == "e4m3":
            f = x.abs().amax(-1) / 448
            out[side + "_scale"][at // c["page"], :, at % c["page"]] = f
            x = torch.where(f[..., None] > 0, _round64(x / torch.where(f > 0, f, 1.0)[..., None], 3, -6, 448.0), 0.0)
        out[side][at // c["page"], :, at % c["page"]] = x
    return q, out


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "write":
        return _write64(c, s)
    cache, lens = s["cache"], _lengths(c)
    if c["op"] == "read":
        both = [torch.cat([_rows64(c, cache, side, s["table"][b], n).transpose(0, 1) for b, n in enumerate(lens)])
                for side in ("k", "v")]
        return both[0], both[1]
    outs, sums = [], []
    for b, n in enumerate(lens):
        first = max(0, n - c["window"]) if c["window"] else 0
        k, v = (_rows64(c, cache, side, s["table"][b], n)[:, first:] for side in ("k", "v"))
        q = s["q"][b].double().view(c["kv_heads"], c["group"], c["dim"])
        t = torch.bmm(q, k.mT) / math.sqrt(c["dim"])
        if c["softcap"]:
            t = torch.tanh(t / c["softcap"]) * c["softcap"]
        sums.append(torch.logsumexp(t, -1).flatten())
        outs.append(torch.bmm(torch.softmax(t, -1), v).flatten(0, 1))
    return torch.stack(outs), torch.stack(sums)
