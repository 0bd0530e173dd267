"""Tensors that a call makes belong to the stream it runs on."""
import pytest
import torch

pytestmark = pytest.mark.gpu

M, N, K, T, E = 64, 512, 512, 16, 4


def _calls(lib):
    """name -> a function of `stream` that makes its outputs and workspaces itself and returns them."""
    from workload import make_dense, make_moe
    from workload import configs as W
    from tests import block_ref as B
    dense = make_dense(dict(W.CONFIGS["w4a16_asym"], kind="dense"), M, N=N, K=K)
    m = make_moe("moe_w4a16", T, E=E, N=N, K=K, topk=2)
    fmt, packed = lib.pack_inputs(dense, "cuda")
    mfmt, mpacked = lib.pack_inputs(m, "cuda")
    act, mact = ({k: v.cuda() for k, v in i["a"].items()} for i in (dense, m))
    ids, tw = m["ids"].cuda(), m["topk_w"].cuda()
    rows = torch.randn(T * 2, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    a, sa, w, sw, _ = B.operands(1, M, N, K)
    bfmt = lib.make_format("e4m3_block", N, K)
    bpacked = lib.pack_weights(bfmt, w, sw)
    x = torch.randn(M, 2 * N, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    return {
        "gemm": lambda s: lib.gemm(fmt, act, packed, M, stream=s),
        "gemm_block": lambda s: lib.gemm(bfmt, {"data": a, "scale": sa}, bpacked, M, stream=s),
        "gemm_static_scratch": lambda s: lib.gemm_static_scratch(fmt, act, packed, M, stream=s),
        "moe_gemm": lambda s: lib.moe_gemm(mfmt, mact, mpacked, ids, tw, stream=s),
        "moe_gemm_combine": lambda s: lib.moe_gemm_combine(mfmt, {"data": rows}, mpacked, ids, tw, stream=s),
        "pack_weights": lambda s: lib.pack_weights(bfmt, w, sw, stream=s),
        "swiglu": lambda s: lib.swiglu(x, stream=s),
        "swiglu_quantize": lambda s: lib.swiglu_quantize("e4m3_tok", x, stream=s),
        "add_rms_norm": lambda s: lib.add_rms_norm("e4m3_block", x, x[0].contiguous(), residual=x, stream=s),
        "quantize_act_tok": lambda s: lib.quantize_act("e4m3_tok", x, stream=s),
        "quantize_act_block": lambda s: lib.quantize_act("e4m3_block", x, stream=s),
        "quantize_act_nvfp4": lambda s: lib.quantize_act("nvfp4", x, stream=s),
        "workspace": lambda s: lib.make_workspace(fmt, M, stream=s),
        "combine_workspace": lambda s: lib.make_combine_workspace(mfmt, T, 2, stream=s),
    }


NAMES = ["gemm", "gemm_block", "gemm_static_scratch", "moe_gemm", "moe_gemm_combine", "pack_weights", "swiglu",
         "swiglu_quantize", "add_rms_norm", "quantize_act_tok", "quantize_act_block", "quantize_act_nvfp4", "workspace",
         "combine_workspace"]


@pytest.mark.parametrize("name", NAMES)
def test_new_tensors_belong_to_the_stream(lib, monkeypatch, name):
    """Every tensor that a call on another stream allocates comes from that stream's memory: what the current stream
    has freed but still works on is not written, and a workspace dropped at the call's end is not given to the current
    stream's work while the call still runs."""
    call = _calls(lib)[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = []

    def recorded(make):
        def f(*args, **kw):
            t = make(*args, **kw)
            if t.is_cuda:
                on.append(torch.cuda.current_stream().cuda_stream)
            return t
        return f

    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recorded(torch.empty_like))
    monkeypatch.setattr(lib, "_empty", recorded(lib._empty))
    call(side)
    torch.cuda.synchronize()
    assert on and all(s == side.cuda_stream for s in on)


@pytest.mark.parametrize("name", [n for n in NAMES if "workspace" not in n])
def test_results_on_another_stream(lib, name):
    call = _calls(lib)[name]
    flat = lambda o: [t for v in (o if isinstance(o, tuple) else (o,)) for t in  # noqa: E731
                      (v.values() if isinstance(v, dict) else (v,))]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.synchronize()
    for p, q in zip(flat(want), flat(got)):
        if name.startswith("moe"):
            # A row's place in its expert's list goes by atomics, and with it the order of its fp32 sums; the combine's
            # are atomic themselves.  K = 512 terms in any order: each sum is off by at most 512 * 2^-24 of the terms'
            # magnitudes, whose sum is below 32 times the largest output here (normal terms: sqrt(512) * 0.8 = 18), so two
            # differ by up to 2^-9 of that output, and by one bf16 rounding each, 2^-8 of the value.
            p, q = p.double(), q.double()
            assert bool(((p - q).abs() <= 2.0 ** -7 * p.abs() + 2.0 ** -9 * p.abs().max()).all())
        else:
            assert torch.equal(p, q)
