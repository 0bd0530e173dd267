"""The block-scaled operators at large offsets, with waits that run out, and in the debug build."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import block_ref as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_products_past_32_bits(lib):
    """An output of over 2^32 elements, activations and scales far from their start: the last rows are those of a call
    on these rows alone."""
    N, K, last = 16384, 256, 300
    M = (1 << 32) // N + 2 * last + 5
    a, sa, w, sw, b = B.operands(1, last, N, K, bias=True)
    fmt = lib.make_format("e4m3_block", N, K)
    packed = lib.pack_weights(fmt, w, sw)
    big = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(M, K // 128, device="cuda")
    big[-last:], scale[-last:] = a, sa
    got = lib.gemm(fmt, {"data": big, "scale": scale}, packed, M, bias=b)
    want, size = B.product(a, sa, w, sw, b)
    B.check_product(got[-last:], want, size, K // 128, b)
    assert torch.equal(got[0], b) and torch.equal(got[M - last - 1], b) and torch.equal(got[M // 2], b)


def test_weights_past_32_bits(lib):
    """Packed weights of over 2^32 bytes (more rows of 128 bytes than the CTA-pair kernel indexes): the last outputs."""
    N, K, M = 132000, 32768, 300
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 120, (N, K), generator=g, dtype=torch.uint8, device="cuda")
    sw = 1e-5 * (1 + torch.rand(-(-N // 128), K // 128, generator=g, device="cuda"))
    a, sa, *_ = B.operands(3, M, 128, K)
    fmt = lib.make_format("e4m3_block", N, K)
    packed = lib.pack_weights(fmt, w, sw)
    at = slice(N - 32 - 128, N)  # whole blocks of scales and the last, shorter one
    for m in (5, M):
        got = lib.gemm(fmt, {"data": a, "scale": sa}, packed, m)
        want, size = B.product(a[:m], sa[:m], w[at], sw[-2:])
        B.check_product(got[:, at], want, size, K // 128)


@pytest.mark.parametrize("afmt", ["bf16", "e4m3_tok", "e4m3_block"])
def test_rows_past_32_bits(lib, afmt):
    K, last = 8192, 40
    T = (1 << 32) // K + 2 * last
    g = torch.Generator().manual_seed(4)
    x, r = (torch.randn(last, K, generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    bx, br = (torch.zeros(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bx[-last:], br[-last:] = x.cuda(), r.cuda()
    act, res = lib.add_rms_norm(afmt, bx, w, residual=br, residual_out=br)
    # (sums of squares are added in an order that goes by the number of rows: no bits are compared)
    total = B.f64(x) + B.f64(r)
    B.check_bf16(res[-last:], total)
    want, end = B.norm(total, 1.0, 1e-6), {k: t[-last:] for k, t in act.items()}
    if afmt == "bf16":
        B.check_bf16(end["data"], want)
    else:
        B.check_act(end, want, afmt == "e4m3_block")
    assert not act["data"][T // 2].any() and not res[T // 2].any()
    if afmt != "bf16":
        sw = lib.swiglu_quantize(afmt, bx)
        B.check_act({k: t[-last:] for k, t in sw.items()}, B.swiglu(B.f64(x)), afmt == "e4m3_block")
        assert not sw["data"][T // 2].any()
    if afmt == "e4m3_block":
        q = lib.quantize_act(afmt, bx)
        B.check_act({k: t[-last:] for k, t in q.items()}, B.f64(x), True)
        assert not q["data"][T // 2].any()


def test_more_than_2_to_the_31_chunks(lib):
    """More chunks of 8 outputs than a 31-bit index holds, where a chunk's row comes from a plain division."""
    I, last = 32768, 3
    R = (1 << 31) // (I // 8) + last + 2
    x = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    end = torch.randn(last, 2 * I, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    x[-last:] = end.cuda()
    q = lib.swiglu_quantize("e4m3_block", x)
    B.check_act({k: t[-last:] for k, t in q.items()}, B.swiglu(B.f64(end)), True)
    assert not q["data"][R - last - 1].any() and not q["scale"][:-last].any()


@pytest.mark.parametrize("M,choice", [(5, "kernel=1,sk=2"), (30, "kernel=1,sk=4"), (60, "kernel=1,sk=2"),
                                      (100, "kernel=1,sk=8"), (600, "kernel=0,bt=256"), (600, "kernel=0,bt=128")])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lib, monkeypatch, M, choice):
    """With a bound of 1 ns the first wait that is not over at once runs out: the call returns, the status says so, and
    the same workspace serves the next call."""
    monkeypatch.setenv("HQ_TUNE", choice)
    N, K = 384, 2560
    a, sa, w, sw, b = B.operands(7, M, N, K, bias=True)
    fmt = lib.make_format("e4m3_block", N, K)
    packed, ws = lib.pack_weights(fmt, w, sw), lib.make_workspace(fmt, M)
    act = {"data": a, "scale": sa}
    torch.cuda.synchronize()
    seen = []
    try:
        lib.set_wait_limit_ns(1)
        for _ in range(5):
            lib.gemm(fmt, act, packed, M, bias=b, workspace=ws)
            torch.cuda.synchronize()
            seen.append(lib.last_device_status(ws))
            if seen[-1] == lib.HQ_ERR_TIMEOUT:
                break
    finally:
        lib.set_wait_limit_ns(0)
    assert lib.HQ_ERR_TIMEOUT in seen and all(s in (lib.HQ_OK, lib.HQ_ERR_TIMEOUT) for s in seen), seen
    got = lib.gemm(fmt, act, packed, M, bias=b, workspace=ws)
    assert lib.last_device_status(ws) == lib.HQ_OK
    want, size = B.product(a, sa, w, sw, b)
    B.check_product(got, want, size, K // 128, b)


DEBUG = """
import json, os, sys
import torch
sys.path.insert(0, {root!r})
import quantized_gemm_dequant_gb300 as hq
from tests import block_ref as B
assert hq.DEBUG
for choice in ("kernel=1,bt=16", "kernel=1,bt=32,sk=2", "kernel=1,bt=64", "kernel=1,bt=128,sk=2", "kernel=0,bt=128", "kernel=0,bt=256"):
    for N in (256, 201):
        os.environ["HQ_TUNE"] = choice
        M, K, limit = 70, 512, 37
        ops = B.operands(1, M, N, K, bias=True)
        fmt = hq.make_format("e4m3_block", N, K)
        packed, ws = hq.pack_weights(fmt, ops[2], ops[3]), hq.make_workspace(fmt, M)
        call = lambda out: hq.gemm(fmt, dict(data=ops[0], scale=ops[1]), packed, M, bias=ops[4], out=out, workspace=ws)
        os.environ.pop("HQ_DEBUG_ROW_LIMIT", None)
        whole = call(torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda"))
        ok = hq.last_device_status(ws)
        want, size = B.product(*ops)
        B.check_product(whole, want, size, K // 128, ops[4])
        os.environ["HQ_DEBUG_ROW_LIMIT"] = str(limit)
        cut = call(torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda"))
        print(json.dumps(dict(choice=choice, n=N, ok=ok, cut=hq.last_device_status(ws),
                              same=bool(torch.equal(cut[:limit], whole[:limit])), left=bool((cut[limit:] == 7).all()))))
"""


def test_debug_build_checks_output_rows(lib):
    """The debug build's index checks: clean calls report nothing; rows declared absent are caught and skipped."""
    r = subprocess.run([sys.executable, "-c", DEBUG.format(root=ROOT)], cwd=ROOT, env=dict(os.environ, HQ_LIBRARY="debug"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
    out = [json.loads(line) for line in r.stdout.splitlines() if line.startswith("{")]
    assert len(out) == 12
    for c in out:
        assert c["ok"] == lib.HQ_OK and c["cut"] == lib.HQ_ERR_BOUNDS and c["same"] and c["left"], c


def test_tables_of_values():
    """The reference's own decoding against torch's."""
    codes = torch.arange(256).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.decode(codes), want, equal_nan=True)
