"""Steps of a layer that reuse the same buffers, launched back to back, so that every kernel starts before the one ahead of
it has ended, give the bits of steps that wait for one another."""
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 16, 33, 100, 300])
def test_back_to_back(lib, T):
    H, I, steps = 1024, 1536, 40
    made = {}
    for name, n, k in (("wide", 2 * I, H), ("narrow", H, I)):
        _, _, w, sw, _ = B.operands(T, 1, n, k)
        fmt = lib.make_format("e4m3_block", n, k)
        made[name] = fmt, lib.pack_weights(fmt, w, 0.05 * sw), lib.make_workspace(fmt, T)
    g = torch.Generator().manual_seed(T)
    x0, r0 = ((s * torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda() for s in (0.5, 3.0))
    gain = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, up, gated = new(T, H), new(T, 2 * I), new(T, I)
    a, b = lib.quantize_act("e4m3_block", x0), lib.quantize_act("e4m3_block", torch.zeros_like(gated))

    def run(wait):
        x.copy_(x0)
        r, seen = r0.clone(), []

        def product(name, act, out):
            fmt, packed, ws = made[name]
            lib.gemm(fmt, act, packed, T, out=out, workspace=ws)

        for i in range(steps):
            for call in (lambda: lib.add_rms_norm("e4m3_block", x, gain, residual=r, residual_out=r, out=a),
                         lambda: product("wide", a, up),
                         lambda: lib.swiglu_quantize("e4m3_block", up, out=b),
                         lambda: product("narrow", b, x),
                         lambda: lib.quantize_act("e4m3_block", x, out=a),
                         lambda: product("wide", a, up),
                         lambda: lib.swiglu(up, out=gated),
                         lambda: lib.quantize_act("e4m3_block", gated, out=b),
                         lambda: product("narrow", b, x),
                         lambda: lib.add_rms_norm("bf16", x, gain, residual=r, residual_out=x, out={"data": up})):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen.append((x.clone(), r.clone()))
        torch.cuda.synchronize()
        return seen

    want = run(True)
    assert all(bool(torch.isfinite(t.float()).all()) for s in want for t in s)
    for _ in range(3):
        assert all(torch.equal(p, q) for s, t in zip(want, run(False)) for p, q in zip(s, t))
    assert all(lib.last_device_status(ws) == lib.HQ_OK for _, _, ws in made.values())
