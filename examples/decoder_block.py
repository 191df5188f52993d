"""One decoder block answering several requests, on synthetic weights.

    python examples/decoder_block.py [--tokens 4] [--steps 16] [--prompt 100] [--kv-bits 4]

The requests' prompts go through the block together, packed (``prefill``), then every row of a batch is one
request's next token (``step``), with an adapter of its own or none:

    qkv = linear_lora(norm(x))            4-bit projection, each request's low-rank adapter
    q, k = qk_norm_rope(qkv)              in place on the packed rows
    kv4_append, kv4_attention             the request's paged 4-bit cache (prompts: prompt_attention on bf16)
    x += linear_lora(attention)           4-bit projection, adapters again
    x += moe(norm(x))                     router, top experts, 4-bit experts

``answer`` says what the head's logits hold for given tokens (a 4-bit projection, then token_logprobs).

Four bits cost a key or value up to a fourteenth of its group's largest magnitude (64 values of a head), about a
tenth of its size in norm for normally distributed ones; every decode step sees them so (with these weights and contexts of 20
to 500 tokens a step's attention is off by 15 % in norm, the block's output by 1 to 5 %).  With ``kv_bits`` 16
(``--kv-bits 16``) the cache holds bf16 and a step's attention over it is plain torch in FP32: the library attends over
4-bit caches only.  Heads of other than 64, 96 or 128 values need that too.

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
    """Weights, cache and buffers of one block for up to ``batch`` requests of ``length`` tokens.  ``kv_bits``: 4 (the
    library's paged cache) or 16 (bf16, attended to in plain torch)."""

    def __init__(self, batch, length, H=2048, Hq=32, Hk=4, D=128, F=768, E=64, top_k=8, L=4, R=16, V=8192, seed=0,
                 kv_bits=4):
        if kv_bits not in (4, 16):
            raise ValueError("kv_bits is 4 or 16")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hk, self.D, self.top_k, self.kv_bits = Hq, Hk, D, top_k, kv_bits

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
        # every request's pages lie anywhere in the pool
        pages = (length + q4lin.KV_PAGE - 1) // q4lin.KV_PAGE
        self.table = torch.randperm(batch * pages, device="cuda", generator=gen).int().view(batch, pages)
        if kv_bits == 4:
            self.cache = torch.zeros((batch * pages, Hk, q4lin.kv4_page_bytes(D)), dtype=torch.uint8, device="cuda")
        else:
            self.cache = torch.zeros((2, batch, length, Hk, D), dtype=BF16, device="cuda")
        self.head = q4_planes(gen, V, H)
        self.scratch = torch.empty(
            max(q4lin.lora_workspace_bytes(n, H, batch, L, R), q4lin.lora_workspace_bytes(H, Hq * D, batch, L, R),
                q4lin.moe_workspace_bytes(batch, H, F, E, top_k), q4lin.workspace_bytes(V, H, batch),
                q4lin.kv4_workspace_bytes(batch, 1, Hq, Hk, D, pages), 256), dtype=torch.uint8, device="cuda")

    def norm(self, x, i):
        f = x.float()
        return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6) * self.norms[i].float()).to(BF16)

    def heads(self, x):
        return x.unflatten(1, (-1, self.D))

    def attention(self, q, k, v, positions):
        """Row t appends its key and value to request t's cache and attends to that cache."""
        if self.kv_bits == 16:
            return self.attention16(q, k, v, positions)
        table = self.table[:q.shape[0]]
        q4lin.kv4_append(self.heads(k), self.heads(v), self.cache, table, positions)
        return q4lin.kv4_attention(self.heads(q), self.cache, table, positions + 1, workspace=self.scratch).flatten(1)

    def attention16(self, q, k, v, positions):
        """The same over a bf16 cache, in plain torch."""
        T, length = q.shape[0], self.cache.shape[2]
        rows = torch.arange(T, device="cuda")
        self.cache[0][rows, positions.long()] = self.heads(k)
        self.cache[1][rows, positions.long()] = self.heads(v)
        keys, values = self.cache[:, :T].float()
        grouped = q.float().view(T, self.Hk, self.Hq // self.Hk, self.D)
        s = torch.einsum("thgd,tlhd->thgl", grouped, keys) / self.D**0.5
        s = s.masked_fill(torch.arange(length, device="cuda") > positions[:, None, None, None], float("-inf"))
        return torch.einsum("thgl,tlhd->thgd", s.softmax(-1), values).reshape(T, -1).to(BF16)

    def prefill(self, x, adapters, cu_seqlens, rows, positions):
        """The block's output for whole packed prompts x [T, H]; their keys and values go to the cache.  Token t is token
        positions[t] of request rows[t]; request r's tokens are rows cu_seqlens[r] .. cu_seqlens[r + 1] - 1 of x and see
        one another only, nothing that the cache held before."""
        nq, nk = self.Hq * self.D, self.Hk * self.D
        qkv = q4lin.linear_lora(*self.qkv, self.norm(x, 0), self.qkv_a, self.qkv_b, adapters, self.adapter_scales)
        q, k, v = self.heads(qkv[:, :nq]), self.heads(qkv[:, nq:nq + nk]), self.heads(qkv[:, nq + nk:])
        q4lin.qk_norm_rope(q, k, self.q_weight, self.k_weight, self.cos_sin, positions, q_out=q, k_out=k)
        if self.kv_bits == 4:
            q4lin.kv4_append(k, v, self.cache, self.table, positions, rows=rows)
        else:
            self.cache[0][rows.long(), positions.long()] = k
            self.cache[1][rows.long(), positions.long()] = v
        a = q4lin.prompt_attention(q, k, v, cu_seqlens).flatten(1)
        x1 = x + q4lin.linear_lora(*self.o, a, self.o_a, self.o_b, adapters, self.adapter_scales)
        y, _, _ = q4lin.moe(self.norm(x1, 1), self.router, *self.gate_up, *self.down, self.top_k)
        return x1 + y

    def answer(self, x, tokens, top_k=5):
        """Log probabilities of given tokens (int32 [T, n]) after x [T, H], entropies, and the top tokens."""
        return q4lin.token_logprobs(q4lin.linear(*self.head, self.norm(x, 1), workspace=self.scratch), tokens, top_k)

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
    ap.add_argument("--prompt", type=int, default=100, help="tokens of the longest prompt")
    ap.add_argument("--kv-bits", type=int, default=4, choices=(4, 16), help="bits of the cache's keys and values")
    args = ap.parse_args()
    q4lin.load()
    T = args.tokens
    block = DecoderBlock(T, args.prompt + 4 + args.steps, kv_bits=args.kv_bits)
    H = block.norms[0].shape[0]
    adapters = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda") % 4
    adapters[0] = -1   # the first request has none
    # prompts of different lengths, one after the other
    lengths = torch.tensor([max(1, args.prompt * (T - r) // T) for r in range(T)], device="cuda")
    cu_seqlens = torch.nn.functional.pad(lengths.cumsum(0), (1, 0)).int()
    rows = torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(lengths)
    at = torch.arange(len(rows), dtype=torch.int32, device="cuda") - cu_seqlens[rows.long()]
    out = block.prefill(torch.randn((len(rows), H), device="cuda").to(BF16), adapters[rows.long()], cu_seqlens, rows, at)
    x = out[cu_seqlens[1:].long() - 1].clone()   # (each prompt's last row stands for its next token)
    positions = lengths.int()
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
    logprobs, entropy, ids, _ = block.answer(x, torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    print(f"token 0 after them: log probability {logprobs.mean().item():.2f}, entropy {entropy.mean().item():.2f}, "
          f"likeliest of the first request {ids[0].tolist()}")
    print(f"{args.steps} steps of {T} tokens: {start.elapsed_time(end) / args.steps * 1e3:.1f} us a step, "
          f"rms of the output {out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
