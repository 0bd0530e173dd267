"""A decoder layer's attention block on quantised weights and a quantised paged cache, prompt and decoding.

    python examples/decode_attention.py [--cache e4m3] [--steps 32]

The block is  x -> QKV projection (UINT4 weights, group 128) -> per-head RMS norm, rotation and append to the cache ->
attention of each sequence's new token -> output projection (UINT4).  Ragged prompts are prefilled (their attention by
plain torch on rows that kv_read brings back), then the batch decodes step by step; one CUDA graph captures a step and
serves every length, because the kernels read lengths, page tables, positions and slots on the device.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_gemm_dequant_gb300 as hq  # noqa: E402
from workload import quant  # noqa: E402


class Attention:
    """The block's weights, its cache and what a server keeps for `batch` sequences of up to `longest` tokens."""

    def __init__(self, batch, longest, hidden=4096, q_heads=32, kv_heads=8, dim=128, kind="e4m3", page=64, seed=0):
        self.batch, self.q_heads, self.kv_heads, self.dim, self.page = batch, q_heads, kv_heads, dim, page
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (q_heads + 2 * kv_heads) * dim
        self.w_qkv = self._pack(g, rows, hidden)
        self.w_out = self._pack(g, hidden, q_heads * dim)
        self.q_norm, self.k_norm = (
            (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        a = torch.arange(longest, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, dim, 2, device="cuda") / dim)
        self.cos_sin = torch.cat((a.cos(), a.sin()), dim=1).contiguous()
        cols = -(-longest // page)
        self.cache = hq.make_kv_cache(kind, batch * cols, page, kv_heads, dim, k_amax=24.0, v_amax=8.0)
        # every sequence owns `cols` pages, in no order
        self.table = torch.randperm(batch * cols, generator=g, device="cuda").to(torch.int32).view(batch, cols)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.workspace = hq.make_kv_workspace(self.cache, batch, q_heads)
        self.gemm_ws = [hq.make_workspace(w[0], batch) for w in (self.w_qkv, self.w_out)]

    @staticmethod
    def _pack(g, n, k):
        codes, scales, zeros = quant.quant_uint4_zp(0.02 * torch.randn(n, k, generator=g, device="cuda"), 128)
        fmt = hq.make_format("uint4_zp", n, k)
        return fmt, hq.pack_weights(fmt, codes, scales.view(torch.uint8), zeros)

    def _slots(self, positions):
        """Slots of one token per sequence at `positions` (int32 [batch])."""
        p = positions.long()
        page = self.table.gather(1, (p // self.page)[:, None])[:, 0].long()
        return page * self.page + p % self.page

    def _append(self, x, positions, slots, workspace=None):
        qkv = hq.gemm(self.w_qkv[0], {"data": x}, self.w_qkv[1], x.shape[0], workspace=workspace)
        return hq.kv_write(self.cache, qkv, slots, self.q_heads, q_norm=self.q_norm, k_norm=self.k_norm,
                           positions=positions, cos_sin=self.cos_sin, workspace=self.workspace)

    def prefill(self, prompts):
        """prompts: one bf16 [n, hidden] per sequence.  Fills the cache; returns each prompt's last output row."""
        last = []
        for b, x in enumerate(prompts):
            n = x.shape[0]
            i = torch.arange(n, device="cuda")
            slots = self.table[b].long()[i // self.page] * self.page + i % self.page
            q = self._append(x, i.to(torch.int32), slots)
            starts = torch.tensor([0, n], device="cuda")
            k, v = hq.kv_read(self.cache, self.table[b:b + 1], starts, n, workspace=self.workspace)
            rep = self.q_heads // self.kv_heads
            q, k, v = (t.transpose(0, 1).float() for t in (q, k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)))
            s = (q @ k.transpose(1, 2)) * self.dim ** -0.5
            s = s.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), float("-inf"))
            o = (s.softmax(-1) @ v).transpose(0, 1).reshape(n, -1).to(torch.bfloat16)
            last.append(hq.gemm(self.w_out[0], {"data": o}, self.w_out[1], n)[-1])
            self.lens[b] = n
        return torch.stack(last)

    def step(self, x):
        """One new token per sequence, bf16 [batch, hidden], on the device alone (may be captured)."""
        q = self._append(x, self.lens, self._slots(self.lens), self.gemm_ws[0])
        self.lens += 1
        o, _ = hq.paged_attention(self.cache, q, self.table, self.lens, workspace=self.workspace)
        return hq.gemm(self.w_out[0], {"data": o.view(self.batch, -1)}, self.w_out[1], self.batch,
                       workspace=self.gemm_ws[1])


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("bf16", "e4m3", "nvfp4"), default="e4m3")
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    block = Attention(a.batch, a.prompt + a.steps + 1, kind=a.cache)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [max(1, a.prompt * (b + 1) // a.batch) for b in range(a.batch)]
    x = block.prefill([torch.randn(n, 4096, generator=g, device="cuda").to(torch.bfloat16) for n in lens])
    x = x / x.float().square().mean(-1, keepdim=True).sqrt().to(x.dtype)
    block.step(x)  # what a first call sets up is not captured
    block.lens -= 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x)
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(y / y.float().square().mean(-1, keepdim=True).sqrt().to(y.dtype))
    t1.record()
    torch.cuda.synchronize()
    print(f"{a.cache} cache, {a.batch} sequences of {min(lens)} to {max(lens)} tokens: {a.steps} steps, "
          f"{t0.elapsed_time(t1) / a.steps * 1e3:.1f} us a step, lengths now {block.lens.min()} to {block.lens.max()}")
    status = hq.last_device_status(block.workspace)
    if status != hq.HQ_OK:
        raise SystemExit(hq.status_string(status))


if __name__ == "__main__":
    main()
