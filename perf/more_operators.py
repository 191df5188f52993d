"""Measured cases of a decoder's attention and of what its logits say.

Four operators, each in its plain form (elementary torch operations in 32 bits, rounded
once at the end) and as the call a user makes of the library (`own` true):

  prompt  attention over whole prompts: causal, grouped heads, sequences of different
          lengths packed after one another, rows behind the last one left as they were;
  append  keys and values of new tokens into a paged cache of 4-bit codes, and what the
          cache then holds for them;
  cache   attention of one or a few new tokens per sequence over that cache;
  logp    log probabilities of given tokens, the entropy and the top alternatives of
          rows of logits.

The cache is uint8 [pages, Hk, B]: for a page of 64 tokens and a head, K codes, V codes, K scales,
V scales.  A value is (q - 8) * s with one fp16 scale per 64 values of a head (the last group may
be shorter), s = fp16(largest magnitude / 7), q = x / s rounded to nearest even, plus 8, in [0, 15].
  K codes  [64 tokens][D / 2 bytes]: 8 values (block b) a 32-bit word, low nibble first; word
           c * (D / 32) + j of the row is block 4 j + c
  V codes  [D / 2 rows][64 bytes]: row i holds values 2 i (low nibble) and 2 i + 1 of every
           token; token o stands at byte 16 ((o % 8) / 2) + 4 (o / 16) + 2 (o % 2) + o % 16 / 8
  scales   [64 tokens][ceil(D / 64)]
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt: latency
        dict(name="prompt_t133_h32_8_d128", op="prompt", T=133, S=1, pad=0, Hq=32, Hk=8, D=128),
        # prompts of nine requests in a batch padded at its end, odd lengths, a head size that is no power of two
        dict(name="prompt_t2000_s9_h28_4_d96", op="prompt", T=2000, S=9, pad=48, Hq=28, Hk=4, D=96),
        # one long prompt
        dict(name="prompt_t8192_h32_8_d128", op="prompt", T=8192, S=1, pad=0, Hq=32, Hk=8, D=128),
        # a full prefill batch of prompts of very different lengths
        dict(name="prompt_t16384_s7_h32_4_d128", op="prompt", T=16384, S=7, pad=0, Hq=32, Hk=4, D=128),
        # a decode step's new tokens, one per request
        dict(name="append_t4_h8_d128", op="append", T=4, decode=True, Hk=8, D=128),
        # a long prompt's keys and values
        dict(name="append_t8192_h8_d128", op="append", T=8192, decode=False, Hk=8, D=128),
        # one request decoding
        dict(name="cache_s1_l1000_h32_8_d128", op="cache", S=1, L=1000, n=1, Hq=32, Hk=8, D=128),
        # a decode batch, contexts of different lengths (one of them empty)
        dict(name="cache_s64_l8192_h32_8_d128", op="cache", S=64, L=8192, n=1, Hq=32, Hk=8, D=128),
        # a few requests with long contexts, four tokens each (a draft being checked), an odd head size
        dict(name="cache_s5_l70001_n4_h28_4_d96", op="cache", S=5, L=70001, n=4, Hq=28, Hk=4, D=96),
        # the next token of one request
        dict(name="logp_t1_v131072", op="logp", T=1, V=131072, n=1, k=8, fp32=False, masked=False),
        # a batch over an odd vocabulary (rows start unaligned) of which a part is ruled out, 32-bit logits
        dict(name="logp_t75_v50001_fp32", op="logp", T=75, V=50001, n=3, k=5, fp32=True, masked=True),
        # scoring a prompt
        dict(name="logp_t1024_v131072", op="logp", T=1024, V=131072, n=1, k=0, fp32=False, masked=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["prompt", "append", "cache", "logp"])
    while True:
        hk = rng.randint(1, 8)
        d = rng.choice([64, 96, 128])
        hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
        if op == "prompt":
            T = _log(rng, 1, 16384)
            c = dict(op=op, T=T, S=min(T, _log(rng, 1, 32)), pad=rng.choice([0, 0, 1, 37, 200]), Hq=hq, Hk=hk,
                     D=rng.choice([64, 80, d, 128]))
            if sum(n * n for n in _lengths(c["T"], c["S"])) * hq * c["D"] > 8192 * 8192 * 32 * 128:
                continue
        elif op == "append":
            c = dict(op=op, T=_log(rng, 1, 8192), decode=rng.random() < 0.5, Hk=hk, D=d)
        elif op == "cache":
            c = dict(op=op, S=_log(rng, 1, 256), L=_log(rng, 1, 131072), n=rng.choice([1, 1, 1, 2, 3, 4, 8]), Hq=hq, Hk=hk, D=d)
            if c["S"] * c["L"] * hk * d > 64 * 8192 * 8 * 128 or c["S"] * c["L"] * hq * c["n"] * d > 64 * 8192 * 32 * 128:
                continue
        else:
            c = dict(op=op, T=_log(rng, 1, 1024), V=_log(rng, 1000, 131072), n=rng.randint(1, 4), k=rng.randint(0, 16),
                     fp32=rng.random() < 0.3, masked=rng.random() < 0.3)
            if c["T"] * c["V"] * (2 if c["fp32"] else 1) > 1024 * 131072:
                continue
        return c


def _lengths(total, parts):
    """`parts` lengths of very different size (at least 1 each) that add up to `total`."""
    rng = random.Random(total * 1009 + parts)
    w = [math.exp(rng.uniform(0.0, 3.0)) for _ in range(parts)]
    cut, acc = [0], 0.0
    for i, x in enumerate(w):
        acc += x
        cut.append(i + 1 + round((total - parts) * acc / sum(w)))
    return [b - a for a, b in zip(cut, cut[1:])]


def _contexts(c):
    """Tokens in the cache of each sequence: between a sixteenth of L and L, the first one L; the last of many none."""
    rng = random.Random(c["S"] * 7919 + c["L"])
    n = [c["L"]] + [_log(rng, max(1, c["L"] // 16), c["L"]) for _ in range(c["S"] - 1)]
    if c["S"] > 8:
        n[-1] = 0
    return n


# ------------------------------------------------------------------ inputs
def _bf(shape, g, std=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * std).bfloat16()


def _planes(cache, D):
    """Views of the cache: K codes [pages, Hk, 64, c, j, 4], V codes [pages, Hk, D / 2, 64], scales [pages, Hk, 64, groups]."""
    P, Hk, _ = cache.shape
    n, g = 32 * D, (D + 63) // 64
    kc = cache[..., :n].unflatten(-1, (64, 4, D // 32, 4))
    vc = cache[..., n:2 * n].unflatten(-1, (D // 2, 64))
    sc = cache.view(torch.float16)
    ks = sc[..., n:n + 64 * g].unflatten(-1, (64, g))
    vs = sc[..., n + 64 * g:n + 128 * g].unflatten(-1, (64, g))
    return kc, vc, ks, vs


def _page_bytes(D):
    return 64 * D + 256 * ((D + 63) // 64)


def _place(o):
    """Byte of token o in a row of V codes."""
    return 16 * ((o % 8) // 2) + 4 * (o // 16) + 2 * (o % 2) + o % 16 // 8


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(c=c)
    if c["op"] == "prompt":
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        lens = _lengths(T, c["S"])
        st["lens"] = lens
        st["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
        # the packed output of the q/k/v projection after its norms: the heads' rows are slices of it
        qkv = _bf((T + c["pad"], Hq + 2 * Hk, D), g)
        qkv[:, :Hq] *= 1.5
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        st["out"] = torch.zeros((T + c["pad"], Hq, D), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "append":
        T, Hk, D = c["T"], c["Hk"], c["D"]
        kv = _bf((T, 2 * Hk, D), g)
        kv *= 1.0 + 3.0 * (torch.rand((1, 2 * Hk, D), device=DEV, generator=g) < 0.03).to(kv.dtype)   # a few large channels
        st["k"], st["v"] = kv[:, :Hk], kv[:, Hk:]
        if c["decode"]:   # one token per sequence, each somewhere in its context
            m = 16
            st["rows"] = None
            pos = torch.randint(0, m * PAGE, (T,), device=DEV, generator=g)
            S = T
        else:             # prompts of up to four sequences, behind what their caches hold already
            S = min(T, 4)
            lens = _lengths(T, S)
            m = max(lens) // PAGE + 3
            st["rows"] = torch.tensor([s for s, n in enumerate(lens) for _ in range(n)], dtype=torch.int32, device=DEV)
            at = torch.randint(0, 2 * PAGE, (S,), device=DEV, generator=g)
            pos = torch.cat([at[s] + torch.arange(n, device=DEV) for s, n in enumerate(lens)])
        st["pos"] = pos.int()
        st["table"] = torch.randperm(S * m, device=DEV, generator=g).int().view(S, m)
        st["cache"] = torch.randint(0, 256, (S * m, Hk, _page_bytes(D)), dtype=torch.uint8, device=DEV, generator=g)
        st["ko"], st["vo"] = torch.empty((2, T, Hk, D), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "cache":
        S, n, Hq, Hk, D = c["S"], c["n"], c["Hq"], c["Hk"], c["D"]
        ctx = _contexts(c)
        st["ctx"] = ctx
        st["len"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        need = [(x + PAGE - 1) // PAGE for x in ctx]
        m, P = max(need), sum(need) + 3
        perm = torch.randperm(P, device=DEV, generator=g).int()
        table = torch.full((S, m), -1, dtype=torch.int32, device=DEV)
        at = 0
        for s, x in enumerate(need):
            table[s, :x] = perm[at:at + x]
            at += x
        st["table"] = table
        cache = torch.randint(0, 256, (P, Hk, _page_bytes(D)), dtype=torch.uint8, device=DEV, generator=g)
        _, _, ks, vs = _planes(cache, D)
        # values of about unit size, scales that differ from token to token
        ks.copy_(0.12 + 0.2 * torch.rand(ks.shape, device=DEV, generator=g))
        vs.copy_(0.12 + 0.2 * torch.rand(vs.shape, device=DEV, generator=g))
        st["cache"] = cache
        st["q"] = _bf((S * n, Hq, D), g, 1.5)
        st["out"] = torch.empty((S * n, Hq, D), dtype=torch.bfloat16, device=DEV)
        st["scratch"] = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    else:
        T, V = c["T"], c["V"]
        x = torch.randn((T, V), device=DEV, generator=g) * 2.5
        for i in range(4):   # the handful of tokens that a context makes likely
            x.scatter_add_(1, torch.randint(0, V, (T, 1), device=DEV, generator=g), 10.0 * torch.rand((T, 1), device=DEV, generator=g))
        st["tok"] = torch.randint(0, V, (T, c["n"]), device=DEV, generator=g).int()
        if c["masked"]:      # tokens that a grammar rules out; the given ones are not among them
            ban = torch.rand((T, V), device=DEV, generator=g) < 0.4
            ban.scatter_(1, st["tok"].long(), False)
            x.masked_fill_(ban, float("-inf"))
        st["x"] = x if c["fp32"] else x.bfloat16()
    return st


# ------------------------------------------------------------------ plain forms
def _plain_prompt(st):
    c = st["c"]
    Hk, G, D = c["Hk"], c["Hq"] // c["Hk"], c["D"]
    out = st["out"].clone()
    at = 0
    for n in st["lens"]:
        for h in range(Hk):
            k = st["k"][at:at + n, h].float()
            v = st["v"][at:at + n, h].float()
            for r in range(0, n, 2048):
                m = min(n, r + 2048)
                q = st["q"][at + r:at + m, h * G:(h + 1) * G].float().transpose(0, 1)
                s = (q @ k[:m].T) / math.sqrt(D)
                late = torch.arange(m, device=DEV) > torch.arange(r, m, device=DEV)[:, None]
                s = s.masked_fill(late, float("-inf"))
                p = torch.exp(s - s.amax(dim=-1, keepdim=True))
                o = (p @ v[:m]) / p.sum(dim=-1, keepdim=True)
                out[at + r:at + m, h * G:(h + 1) * G] = o.transpose(0, 1).bfloat16()
        at += n
    return out


def _slots(st):
    pos = st["pos"].long()
    row = torch.arange(len(pos), device=DEV) if st["rows"] is None else st["rows"].long()
    return st["table"][row, pos // PAGE].long(), pos % PAGE


def _pair(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8)


def _groups(x):
    """[..., D] -> [..., groups, 64], zeros behind a short last group."""
    pad = -x.shape[-1] % 64
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:-1] + (pad,))], dim=-1)
    return x.unflatten(-1, (-1, 64))


def _plain_append(st):
    c = st["c"]
    Hk, D = c["Hk"], c["D"]
    page, o = _slots(st)
    kc, vc, ks, vs = _planes(st["cache"], D)
    heads = torch.arange(Hk, device=DEV)
    where = (page[:, None], heads[None, :], o[:, None])
    got = {}
    for key, codes, scales in (("k", kc, ks), ("v", vc, vs)):
        x = _groups(st[key].float())
        s = (x.abs().amax(dim=-1) / 7.0).half()
        q = torch.where(s[..., None] > 0, torch.round(x / s.float()[..., None]), 0.0).clamp(-8.0, 7.0) + 8.0
        scales[where] = s
        b = _pair(q.flatten(-2)[..., :D].int())
        if key == "k":
            codes[where] = b.unflatten(-1, (D // 32, 4, 4)).transpose(-3, -2)
        else:
            codes[page[:, None, None], heads[None, :, None], torch.arange(D // 2, device=DEV), _place(o)[:, None, None]] = b
    for key in ("k", "v"):
        if key == "k":
            b = kc[where].transpose(-3, -2).flatten(-3)
            s = ks[where]
        else:
            b = vc[page[:, None, None], heads[None, :, None], torch.arange(D // 2, device=DEV), _place(o)[:, None, None]]
            s = vs[where]
        q = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2).float() - 8.0
        got[key] = (q * s.float().repeat_interleave(64, dim=-1)[..., :D]).bfloat16()
    return got


def _decode(st, s, n):
    """fp32 keys and values [n, Hk, D] of sequence s."""
    D = st["c"]["D"]
    pages = st["table"][s, :(n + PAGE - 1) // PAGE].long()
    kc, vc, ks, vs = _planes(st["cache"][pages], D)
    out = []
    kb = kc.transpose(-3, -2).flatten(-3)                                       # [pages, Hk, 64, D / 2]
    vb = vc[..., _place(torch.arange(PAGE, device=DEV))].transpose(-1, -2)      # the same order
    for b, sc in ((kb, ks), (vb, vs)):
        q = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2).float() - 8.0
        x = q * sc.float().repeat_interleave(64, dim=-1)[..., :D]
        out.append(x.transpose(1, 2).flatten(0, 1)[:n])
    return out


def _plain_cache(st):
    c = st["c"]
    n, Hk, G, D = c["n"], c["Hk"], c["Hq"] // c["Hk"], c["D"]
    out = torch.zeros_like(st["out"])
    for s, L in enumerate(st["ctx"]):
        if L == 0:
            continue
        k, v = _decode(st, s, L)
        q = st["q"][s * n:(s + 1) * n].float().view(n, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * n, D)
        x = torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(D)
        seen = torch.arange(L, device=DEV) < (L - n + 1 + torch.arange(n, device=DEV))[:, None]
        seen = seen.repeat(G, 1)
        x = x.masked_fill(~seen, float("-inf"))
        p = torch.where(seen, torch.exp(x - x.amax(dim=-1, keepdim=True)), 0.0)
        o = torch.bmm(p, v.transpose(0, 1)) / p.sum(dim=-1, keepdim=True)
        o = torch.where(seen.any(dim=1)[:, None], o, 0.0)
        out[s * n:(s + 1) * n] = o.view(Hk, G, n, D).permute(2, 0, 1, 3).reshape(n, Hk * G, D).bfloat16()
    return out


def _plain_logp(st):
    k = st["c"]["k"]
    x = st["x"].float()
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(dim=1, keepdim=True)
    d = torch.where(e > 0, x - m, 0.0)
    got = {"logp": st["x"].gather(1, st["tok"].long()).float() - m - torch.log(total),
           "entropy": (torch.log(total) - (e * d).sum(dim=1, keepdim=True) / total)[:, 0]}
    if k:
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)   # ties: the lowest token first
        got["top"] = top[:, :k] - m - torch.log(total)
        got["ids"] = ids[:, :k].int()
    return got


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["c"]
    if own:
        from weight_only_bit_q4_gb300 import q4lin
        if c["op"] == "prompt":
            return q4lin.prompt_attention(st["q"], st["k"], st["v"], st["cu"], out=st["out"])
        if c["op"] == "append":
            q4lin.kv4_append(st["k"], st["v"], st["cache"], st["table"], st["pos"], rows=st["rows"])
            k, v = q4lin.kv4_read(st["cache"], st["table"], st["pos"], c["D"], rows=st["rows"], k=st["ko"], v=st["vo"])
            return {"k": k, "v": v}
        if c["op"] == "cache":
            return q4lin.kv4_attention(st["q"], st["cache"], st["table"], st["len"], out=st["out"], workspace=st["scratch"])
        logp, entropy, ids, top = q4lin.token_logprobs(st["x"], st["tok"], c["k"])
        got = {"logp": logp, "entropy": entropy}
        if c["k"]:
            got["top"], got["ids"] = top, ids
        return got
    return {"prompt": _plain_prompt, "append": _plain_append, "cache": _plain_cache, "logp": _plain_logp}[c["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "prompt":
        pairs = sum(n * (n + 1) / 2 for n in _lengths(c["T"], c["S"]))
        return {"bytes": 4.0 * c["T"] * (c["Hq"] + c["Hk"]) * c["D"] + 4 * (c["S"] + 1), "flops": 4.0 * pairs * c["Hq"] * c["D"]}
    if c["op"] == "append":   # values in, codes and scales out; codes and scales in, values out
        held = c["D"] + 4 * ((c["D"] + 63) // 64)
        return {"bytes": 2.0 * c["T"] * c["Hk"] * (4 * c["D"] + held) + 8.0 * c["T"], "flops": 8.0 * c["T"] * c["Hk"] * c["D"]}
    if c["op"] == "cache":
        L = float(sum(_contexts(c)))
        held = c["D"] + 4 * ((c["D"] + 63) // 64)
        return {"bytes": L * c["Hk"] * held + 4.0 * c["S"] * c["n"] * c["Hq"] * c["D"] + L / 16,
                "flops": 4.0 * L * c["n"] * c["Hq"] * c["D"]}
    return {"bytes": c["T"] * (c["V"] * (4.0 if c["fp32"] else 2.0) + 8 * c["n"] + 8 * c["k"] + 4), "flops": 6.0 * c["T"] * c["V"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "prompt":
        out = st["out"].double()
        at = 0
        for n in st["lens"]:
            for h in range(c["Hq"]):
                g = h * c["Hk"] // c["Hq"]
                k, v = st["k"][at:at + n, g].double(), st["v"][at:at + n, g].double()
                for r in range(0, n, 4096):
                    m = min(n, r + 4096)
                    s = torch.mm(st["q"][at + r:at + m, h].double(), k[:m].t()) * c["D"] ** -0.5
                    keep = torch.ones_like(s, dtype=torch.bool).tril(diagonal=r)
                    out[at + r:at + m, h] = torch.mm(torch.softmax(torch.where(keep, s, -math.inf), dim=1), v[:m])
            at += n
        return out
    if c["op"] == "append":
        got = {}
        for key in ("k", "v"):
            x = st[key].double()
            parts = []
            for a in range(0, c["D"], 64):
                y = x[..., a:a + 64]
                s = torch.div(y.abs().max(dim=-1, keepdim=True).values, 7).half().double()
                q = torch.nan_to_num(torch.div(y, s)).round()
                parts.append(q.clamp(min=-8, max=7) * s)
            got[key] = torch.cat(parts, dim=-1)
        return got
    if c["op"] == "cache":
        n, D, G = c["n"], c["D"], c["Hq"] // c["Hk"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
        half = 32 * D
        sc = st["cache"].view(torch.float16).double()
        ng = (D + 63) // 64
        order = torch.tensor([_place(o) for o in range(PAGE)], device=DEV)
        words = torch.tensor([(b % 4) * (D // 32) + b // 4 for b in range(D // 8)], device=DEV)
        for s, L in enumerate(st["ctx"]):
            pages = st["table"][s, :-(-L // PAGE)].long()
            for h in range(c["Hk"] if L else 0):
                raw = st["cache"][pages, h]
                kb = raw[:, :half].reshape(-1, PAGE, D // 8, 4)[:, :, words].reshape(-1, D // 2)[:L]
                vb = raw[:, half:2 * half].reshape(-1, D // 2, PAGE)[:, :, order].transpose(1, 2).reshape(-1, D // 2)[:L]
                ks = sc[pages, h, half:half + PAGE * ng].reshape(-1, ng)[:L]
                vs = sc[pages, h, half + PAGE * ng:].reshape(-1, ng)[:L]
                kv = []
                for b, t in ((kb, ks), (vb, vs)):
                    x = torch.empty((L, D), dtype=torch.float64, device=DEV)
                    x[:, 0::2], x[:, 1::2] = (b % 16).double() - 8, torch.div(b, 16, rounding_mode="floor").double() - 8
                    for a in range(ng):
                        x[:, 64 * a:64 * a + 64] *= t[:, a:a + 1]
                    kv.append(x)
                for i in range(n):
                    m = L - n + 1 + i
                    if m > 0:
                        p = torch.softmax(torch.mm(st["q"][s * n + i, h * G:(h + 1) * G].double(), kv[0][:m].t()) * D ** -0.5, dim=1)
                        out[s * n + i, h * G:(h + 1) * G] = torch.mm(p, kv[1][:m])
        return out
    logs = torch.log_softmax(st["x"].double(), dim=1)
    p = logs.exp()
    got = {"logp": logs.gather(1, st["tok"].long()), "entropy": -torch.where(p > 0, p * logs, 0.0).sum(dim=1)}
    if c["k"]:
        got["top"] = torch.topk(logs, c["k"], dim=1).values
        got["ids"] = None
    return got
