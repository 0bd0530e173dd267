"""The operators with block scales together, as a layer's MLP uses them: residual and norm, the wide product, SwiGLU, the
narrow product, and the next norm.  Every step is held to the plain 64-bit form of what it was given."""
import numpy as np
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu


class Mlp:
    """Weights laid out once, workspaces and buffers of a layer."""

    def __init__(self, lib, H, I, most):
        g = torch.Generator().manual_seed(1)
        self.lib, self.norms = lib, [(1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.weights, self.packed = [], []
        for n, k in ((2 * I, H), (H, I)):
            w = 0.02 * torch.randn(n, k, generator=g)
            pad = torch.nn.functional.pad(w, (0, 0, 0, -n % 128)).unflatten(0, (-1, 128)).unflatten(2, (-1, 128))
            s = pad.abs().amax((1, 3)) / 448
            q = (pad / s[:, None, :, None]).flatten(2).flatten(0, 1)[:n].to(torch.float8_e4m3fn).view(torch.uint8)
            fmt = lib.make_format("e4m3_block", n, k)
            self.weights.append((q.cuda(), s.cuda()))
            self.packed.append((fmt, lib.pack_weights(fmt, q.cuda(), s.cuda()), lib.make_workspace(fmt, most)))

    def __call__(self, x, residual, afmt="e4m3_block"):
        """x: the attention's output; residual: the stream, updated in place.  Everything that was computed."""
        lib, T = self.lib, x.shape[0]
        a, _ = lib.add_rms_norm("e4m3_block", x, self.norms[0], residual=residual, residual_out=residual)
        r1 = residual.clone()
        up = lib.gemm(self.packed[0][0], a, self.packed[0][1], T, workspace=self.packed[0][2])
        b = lib.swiglu_quantize("e4m3_block", up)
        down = lib.gemm(self.packed[1][0], b, self.packed[1][1], T, workspace=self.packed[1][2])
        c, _ = lib.add_rms_norm(afmt, down, self.norms[1], residual=residual, residual_out=residual)
        return a, r1, up, b, down, c, residual


@pytest.mark.parametrize("T,H,I", [(1, 1024, 1536), (33, 640, 896), (150, 1024, 1152), (700, 896, 1280)])
def test_every_step(lib, T, H, I):
    layer = Mlp(lib, H, I, T)
    g = torch.Generator().manual_seed(T)
    x, r = ((s * torch.randn(T, H, generator=g)).to(torch.bfloat16) for s in (0.5, 3.0))
    a, r1, up, b, down, c, r2 = layer(x.cuda(), r.cuda())
    total = B.f64(x) + B.f64(r)
    B.check_bf16(r1, total)
    B.check_act(a, B.norm(total, B.f64(layer.norms[0])[None], 1e-6), True)
    (w1, s1), (w2, s2) = layer.weights
    B.check_product(up, *B.product(a["data"], a["scale"], w1, s1), H // 128)
    B.check_act(b, B.swiglu(B.f64(up)), True)
    B.check_product(down, *B.product(b["data"], b["scale"], w2, s2), I // 128)
    total = B.f64(down) + B.f64(r1)
    B.check_bf16(r2, total)
    B.check_act(c, B.norm(total, B.f64(layer.norms[1])[None], 1e-6), True)
    for fmt, _, ws in layer.packed:
        assert lib.last_device_status(ws) == lib.HQ_OK


def test_near_the_unquantised_layer(lib):
    """What 8 bits cost the layer: each e4m3 rounding is off by at most 2^-4 of its value, errors of many products
    average, so the layer's output stays within 5% of the unquantised one's norm."""
    T, H, I = 64, 1024, 1536
    layer = Mlp(lib, H, I, T)
    g = torch.Generator().manual_seed(5)
    x, r = ((s * torch.randn(T, H, generator=g)).to(torch.bfloat16) for s in (0.5, 3.0))
    _, _, _, _, down, _, _ = layer(x.cuda(), r.cuda())
    n = B.norm(B.f64(x) + B.f64(r), B.f64(layer.norms[0])[None], 1e-6)
    wide, narrow = (B.decode(q) * np.repeat(np.repeat(B.f64(s), 128, 0)[:q.shape[0]], 128, 1) for q, s in layer.weights)
    want = B.swiglu(n @ wide.T) @ narrow.T
    assert np.linalg.norm(B.f64(down) - want) < 0.05 * np.linalg.norm(want)


@pytest.mark.parametrize("afmt", ["bf16", "e4m3_tok", "e4m3_block"])
def test_captured_steps(lib, afmt):
    """A captured decoding step, replayed on new inputs, gives the bits of eager calls; the stream is updated in place by
    every replay.  Two graphs that share the layer's workspaces run at once: the products keep nothing there but their
    status."""
    T, H, I = 48, 1024, 1536
    layer = Mlp(lib, H, I, T)
    g = torch.Generator().manual_seed(9)
    new = lambda s: (s * torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
    xs, rs, graphs, outs = [new(0.5) for _ in range(2)], [new(3.0) for _ in range(2)], [], []
    for x, r in zip(xs, rs):
        layer(x, r.clone(), afmt)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(x, r, afmt))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        before = []
        for x, r in zip(xs, rs):
            x.copy_(new(0.5))
            before.append(r.clone())
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, r, b, out in zip(xs, rs, before, outs):
            want = layer(x, b, afmt)
            flat = lambda o: [t for v in o for t in (v.values() if isinstance(v, dict) else (v,))]  # noqa: E731
            assert all(torch.equal(p, q) for p, q in zip(flat(want), flat(out)))
            assert torch.equal(b, r)


def test_norm_feeds_the_other_formats(lib):
    """The norm's bf16 and per-token operands go into the products that take them, as hq_quantize_act's own would."""
    from workload import configs as W
    from workload import make_dense
    T, N, K = 20, 256, 512
    x, w = W.acts_fp32(3, T, K, device="cuda").to(torch.bfloat16), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    for cfg, afmt in (("w4a16_asym", "bf16"), ("moe_mxfp4", "e4m3_tok")):
        c = dict(W.CONFIGS[cfg], kind="dense")
        fmt, packed = lib.pack_inputs(make_dense(c, T, N=N, K=K), "cuda")
        act, _ = lib.add_rms_norm(afmt, x, w)
        y = lib.gemm(fmt, act, packed, T).float()
        plain, _ = lib.add_rms_norm("bf16", x, w)
        other = lib.gemm(fmt, plain if afmt == "bf16" else lib.quantize_act(afmt, plain["data"]), packed, T).float()
        # (codes of the two differ where bf16's rounding, 2^-8, moves a value across a border: by a step of 2^-3)
        assert float((y - other).norm() / other.norm()) <= (0.0 if afmt == "bf16" else 0.02)
