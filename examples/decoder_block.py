"""One decoder block decoding tokens of several requests, on synthetic weights.

    python examples/decoder_block.py [--tokens 4] [--steps 16]

Every row of the batch is one request's next token, with an adapter of its own or none:

    qkv = linear_lora(norm(x))            4-bit projection, each request's low-rank adapter
    q, k = qk_norm_rope(qkv)              in place on the packed rows
    attention over the request's cache    plain torch (the library has none)
    x += linear_lora(attention)           4-bit projection, adapters again
    x += moe(norm(x))                     router, top experts, 4-bit experts

All buffers are made once; a step allocates nothing of the library's and is captured in a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_bit_q4_gb300 import q4lin  # noqa: E402

BF16 = torch.bfloat16


def q4_planes(gen, *shape):
    """Random Q4_G64_FP16 planes of shape [..., rows, K]: codes 1..15 (weights of mean zero) and scales."""
    *rows, K = shape
    Kp = (K + 127) // 128 * 128
    low, high = torch.randint(1, 16, (2, *rows, Kp // 2), dtype=torch.uint8, device="cuda", generator=gen)
    wq = low | high << 4
    scales = (torch.rand((*rows, Kp // 64), device="cuda", generator=gen) + 0.5) * (0.2 / K**0.5)
    return wq, scales.to(torch.float16)


class DecoderBlock:
    """Weights, cache and buffers of one block for up to ``batch`` requests of ``length`` tokens."""

    def __init__(self, batch, length, H=2048, Hq=32, Hk=4, D=128, F=768, E=64, top_k=8, L=4, R=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hk, self.D, self.top_k = Hq, Hk, D, top_k

        def bf16(*shape, std):
            return (torch.randn(shape, device="cuda", generator=gen) * std).to(BF16)

        n = (Hq + 2 * Hk) * D
        self.qkv, self.o = q4_planes(gen, n, H), q4_planes(gen, H, Hq * D)
        self.qkv_a, self.qkv_b = bf16(L, R, H, std=H**-0.5), bf16(L, n, R, std=0.1)
        self.o_a, self.o_b = bf16(L, R, Hq * D, std=(Hq * D) ** -0.5), bf16(L, H, R, std=0.1)
        self.adapter_scales = torch.full((L,), 2.0, device="cuda")
        self.gate_up, self.down = q4_planes(gen, E, 2 * F, H), q4_planes(gen, E, H, F)
        self.router = bf16(E, H, std=H**-0.5)
        self.norms = [1 + bf16(H, std=0.1) for _ in range(2)]
        self.q_weight, self.k_weight = 1 + bf16(D, std=0.1), 1 + bf16(D, std=0.1)
        angle = torch.arange(length, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
        self.cache = torch.zeros((2, batch, length, Hk, D), dtype=BF16, device="cuda")
        self.scratch = torch.empty(
            max(q4lin.lora_workspace_bytes(n, H, batch, L, R), q4lin.lora_workspace_bytes(H, Hq * D, batch, L, R),
                q4lin.moe_workspace_bytes(batch, H, F, E, top_k), 256), dtype=torch.uint8, device="cuda")

    def norm(self, x, i):
        f = x.float()
        return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6) * self.norms[i].float()).to(BF16)

    def attention(self, q, k, v, positions):
        """Row t appends its key and value to request t's cache and attends to that cache."""
        T, length = q.shape[0], self.cache.shape[2]
        rows = torch.arange(T, device="cuda")
        self.cache[0][rows, positions.long()] = k.view(T, self.Hk, self.D)
        self.cache[1][rows, positions.long()] = v.view(T, self.Hk, self.D)
        keys, values = self.cache[:, :T].float()
        grouped = q.float().view(T, self.Hk, self.Hq // self.Hk, self.D)
        s = torch.einsum("thgd,tlhd->thgl", grouped, keys) / self.D**0.5
        s = s.masked_fill(torch.arange(length, device="cuda") > positions[:, None, None, None], float("-inf"))
        return torch.einsum("thgl,tlhd->thgd", s.softmax(-1), values).reshape(T, -1).to(BF16)

    def step(self, x, adapters, positions):
        """The block's output for x [T, H], and what its operators took and gave on the way."""
        nq, nk = self.Hq * self.D, self.Hk * self.D
        xn = self.norm(x, 0)
        qkv = q4lin.linear_lora(*self.qkv, xn, self.qkv_a, self.qkv_b, adapters, self.adapter_scales, workspace=self.scratch)
        raw = qkv.clone()   # (only for the answer below: the heads are rotated in place)
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
        q4lin.qk_norm_rope(q, k, self.q_weight, self.k_weight, self.cos_sin, positions, q_out=q, k_out=k)
        a = self.attention(q, k, v, positions)
        o = q4lin.linear_lora(*self.o, a, self.o_a, self.o_b, adapters, self.adapter_scales, workspace=self.scratch)
        x1 = x + o
        hn = self.norm(x1, 1)
        y, ids, weights = q4lin.moe(hn, self.router, *self.gate_up, *self.down, self.top_k, workspace=self.scratch)
        return x1 + y, dict(xn=xn, raw=raw, qkv=qkv, a=a, o=o, hn=hn, y=y, ids=ids, weights=weights)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4, help="requests decoded together")
    ap.add_argument("--steps", type=int, default=16)
    args = ap.parse_args()
    q4lin.load()
    T = args.tokens
    block = DecoderBlock(T, 4 + args.steps)
    x = torch.randn((T, block.norms[0].shape[0]), device="cuda").to(BF16)
    adapters = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda") % 4
    adapters[0] = -1   # the first request has none
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # warm-up, as captures want it
        block.step(x, adapters, positions)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(x, adapters, positions)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.steps):
        graph.replay()
        x.copy_(out)      # the block's output is the next step's input, one position on
        positions += 1
    end.record()
    torch.cuda.synchronize()
    if q4lin.device_status() != q4lin.OK:
        raise SystemExit(f"device status: {q4lin.status_string(q4lin.device_status())}")
    if not torch.isfinite(out).all():
        raise SystemExit("the block's output is not finite")
    print(f"{args.steps} steps of {T} tokens: {start.elapsed_time(end) / args.steps * 1e3:.1f} us a step, "
          f"rms of the output {out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
