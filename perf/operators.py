"""Measured cases of the operators around the 4-bit projections of a decoder block.

Three operators, each in its plain form (elementary torch operations in 32 bits, rounded
once at the end) and as the call a user makes of the library (`own` true):

  lora  Y = W X + scale_a B_a (A_a X): one shared Q4_G64_FP16 projection and, token by
        token, the low-rank adapter a of the request that the token belongs to (-1: none);
  moe   a mixture-of-experts layer: router logits, softmax, the top_k experts of each
        token, then sum_j p_j W_down,e_j (silu(W_gate,e_j x) * (W_up,e_j x)) with
        Q4_G64_FP16 expert weights;
  qkn   RMS norm of every query and key head of a packed projection output, then the
        position rotation, in one pass.

Weights are Q4_G64_FP16: w[n, k] = (q - 8) * s, codes [N, Kp/2] (low nibble: even k) and
fp16 scales [N, Kp/64], Kp = K rounded up to 128; the padded columns hold arbitrary codes.
"""
import math

import torch

own = False

DEV = "cuda"
SCRATCH_BYTES = 48 << 20   # the scratch buffer that a program keeps for all its calls


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request decoding one token through a packed q/k/v projection, its adapter chosen among 8
        dict(name="lora_6144x5120_t1_r16", op="lora", N=6144, K=5120, T=1, L=8, R=16, mix="mixed", several=False),
        # a small batch of requests, each with an adapter of its own or none, ranks that differ
        dict(name="lora_14336x5120_t13_r32", op="lora", N=14336, K=5120, T=13, L=24, R=32, mix="mixed", several=True),
        # a decode batch beyond the streaming routes, odd sizes (padded columns, ragged rows)
        dict(name="lora_5000x4104_t75_r64", op="lora", N=5000, K=4104, T=75, L=16, R=64, mix="mixed", several=False),
        # prefill: prompts of four requests after one another
        dict(name="lora_6144x5120_t1024_r16", op="lora", N=6144, K=5120, T=1024, L=4, R=16, mix="runs", several=False),
        # decode of one token through a layer of small experts
        dict(name="moe_t1_e64_k8", op="moe", T=1, H=2048, F=768, E=64, k=8, renorm=True),
        # few large experts, a few tokens
        dict(name="moe_t4_e8_k2", op="moe", T=4, H=5120, F=1408, E=8, k=2, renorm=True),
        # odd sizes: padded columns in both products, top 3 of 20, probabilities left as they are
        dict(name="moe_t19_e20_k3", op="moe", T=19, H=1992, F=1016, E=20, k=3, renorm=False),
        # a decode batch that touches nearly every expert
        dict(name="moe_t64_e128_k8", op="moe", T=64, H=2048, F=768, E=128, k=8, renorm=True),
        # one token: the heads of one packed row
        dict(name="qkn_t1_h32_8_d128", op="qkn", T=1, Hq=32, Hk=8, D=128, rot=128, inter=False, decode=True),
        # a decode batch, a head size that is no power of two, partial interleaved rotation
        dict(name="qkn_t133_h28_4_d96", op="qkn", T=133, Hq=28, Hk=4, D=96, rot=64, inter=True, decode=True),
        # prefill of a long prompt
        dict(name="qkn_t8192_h32_8_d128", op="qkn", T=8192, Hq=32, Hk=8, D=128, rot=128, inter=False, decode=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["lora", "moe", "qkn"])
    while True:
        if op == "lora":
            c = dict(op=op, N=_log(rng, 256, 14336), K=_log(rng, 256, 8192, 8), T=_log(rng, 1, 1024), L=_log(rng, 1, 64),
                     R=rng.choice([8, 16, 24, 32, 64]), mix=rng.choice(["mixed", "runs"]), several=rng.random() < 0.5)
            if c["N"] * c["K"] * c["T"] > 6144 * 5120 * 1024 or c["N"] * c["K"] > 14336 * 5120:
                continue
            if (c["N"] + c["K"]) * c["L"] * c["R"] > 64 << 20:
                continue
        elif op == "moe":
            c = dict(op=op, T=_log(rng, 1, 64), H=_log(rng, 512, 5120, 8), F=_log(rng, 256, 2048, 8), E=_log(rng, 8, 128),
                     k=rng.randint(1, 8), renorm=rng.random() < 0.5)
            if c["k"] > c["E"] or c["E"] * c["F"] * c["H"] > 128 * 768 * 2048:
                continue
        else:
            hk = rng.randint(1, 16)
            d = rng.choice([64, 80, 96, 128, 192, 256])
            rots = [d] + [r for r in (16, 32, 48, 64, 96, 128) if r < d]
            c = dict(op=op, T=_log(rng, 1, 8192), Hq=hk * rng.choice([1, 2, 4, 5, 8]), Hk=hk, D=d, rot=rng.choice(rots),
                     inter=rng.random() < 0.5, decode=rng.random() < 0.5)
            if c["T"] * (c["Hq"] + 2 * c["Hk"]) * c["D"] > 8192 * 6144:
                continue
        if 3072 in c.values():
            continue
        return c


# ------------------------------------------------------------------ inputs
def _pad(K):
    return (K + 127) // 128 * 128


def _q4(rows, K, g):
    """Codes and scales of `rows` weight rows: uniform codes, half-normal fp16 scales."""
    Kp = _pad(K)
    wq = torch.randint(0, 256, (rows, Kp // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = (torch.randn((rows, Kp // 64), device=DEV, generator=g).abs() * 0.02 + 1e-3).half()
    return wq, s


def _bf(shape, g, std=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * std).bfloat16()


def _router_inputs(c, g):
    """Activations and router weights.  Ids are compared one by one, so tokens whose chosen
    logits lie closer together than 32-bit sums of another order can tell apart are drawn again."""
    w = _bf((c["E"], c["H"]), g, 2.0 / math.sqrt(c["H"]))
    x = _bf((c["T"], c["H"]), g)
    for _ in range(16):
        top = torch.sort(x.double() @ w.double().T, dim=1, descending=True).values[:, :c["k"] + 1]
        near = (top[:, :-1] - top[:, 1:] < 2e-5).any(dim=1) if top.shape[1] > 1 else torch.zeros(c["T"], dtype=torch.bool, device=DEV)
        if not bool(near.any()):
            break
        x = torch.where(near[:, None], _bf((c["T"], c["H"]), g), x)
    return x, w


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(c=c, scratch=torch.empty(SCRATCH_BYTES, dtype=torch.uint8, device=DEV))
    if c["op"] == "lora":
        N, K, T, L, R = c["N"], c["K"], c["T"], c["L"], c["R"]
        st["wq"], st["s"] = _q4(N, K, g)
        st["x"] = _bf((T, K), g)
        st["a"] = _bf((L, R, K), g, 1.0 / math.sqrt(K))
        st["b"] = _bf((L, N, R), g, 0.5)
        st["scales"] = torch.rand(L, device=DEV, generator=g) * 1.5 + 0.5
        if c["several"]:   # adapters of rank R / 2 and R stored side by side; what is past a rank is not read
            st["ranks"] = (torch.randint(1, 3, (L,), device=DEV, generator=g) * R // 2).int()
        else:
            st["ranks"] = None
        if c["mix"] == "mixed":   # every token a request of its own; about one in eight without an adapter
            ids = torch.randint(0, L, (T,), device=DEV, generator=g)
            if T > 1:
                ids = torch.where(torch.rand(T, device=DEV, generator=g) < 0.125, -1, ids)
        else:                     # prompts after one another
            cut = torch.sort(torch.randint(0, T + 1, (L - 1,), device=DEV, generator=g)).values
            ids = torch.bucketize(torch.arange(T, device=DEV), cut, right=True)
        st["ids"] = ids.int()
        st["y"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "moe":
        T, H, F, E, k = c["T"], c["H"], c["F"], c["E"], c["k"]
        st["x"], st["router"] = _router_inputs(c, g)
        wq, s = _q4(E * 2 * F, H, g)
        st["gu"], st["gu_s"] = wq.view(E, 2 * F, -1), s.view(E, 2 * F, -1)
        wq, s = _q4(E * H, F, g)
        st["dn"], st["dn_s"] = wq.view(E, H, -1), s.view(E, H, -1)
        st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        st["p"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    else:
        T, Hq, Hk, D, rot = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"]
        P = 16384
        # the packed output of the q/k/v projection; the heads' rows are slices of it
        st["qkv"] = _bf((T, (Hq + 2 * Hk) * D), g, 4.0)
        st["q"], st["kk"] = st["qkv"][:, :Hq * D], st["qkv"][:, Hq * D:(Hq + Hk) * D]
        st["qw"], st["kw"] = (1.0 + 0.2 * torch.randn((2, D), device=DEV, generator=g)).bfloat16()
        f = torch.arange(rot // 2, device=DEV, dtype=torch.float64) * (-2.0 / rot)
        ang = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * (10000.0 ** f)[None, :]
        st["cs"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        if c["decode"]:
            pos = torch.randint(0, P, (T,), device=DEV, generator=g)
        else:
            pos = torch.arange(T, device=DEV) + torch.randint(0, P - T, (1,), device=DEV, generator=g)
        st["pos"] = pos.int()
        st["qo"] = torch.empty((T, Hq * D), dtype=torch.bfloat16, device=DEV)
        st["ko"] = torch.empty((T, Hk * D), dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms
def _weights(wq, s, K):
    """fp32 weights [..., K] of packed codes [..., Kp/2] and scales [..., Kp/64]."""
    q = torch.stack([wq & 15, wq >> 4], dim=-1).flatten(-2).float() - 8.0
    return (q.unflatten(-1, (-1, 64)) * s.float().unsqueeze(-1)).flatten(-2)[..., :K]


def _plain_lora(st):
    c = st["c"]
    L, R = c["L"], c["R"]
    x, ids = st["x"].float(), st["ids"].long()
    y = x @ _weights(st["wq"], st["s"], c["K"]).T
    on = ids >= 0
    safe = ids.clamp(min=0)
    factor = torch.where(on, st["scales"][safe], 0.0)
    if c["T"] <= L:   # every token's own adapter, gathered
        u = torch.bmm(st["a"][safe].float(), x.unsqueeze(2)).squeeze(2) * factor[:, None]
        if st["ranks"] is not None:
            u = torch.where(torch.arange(R, device=DEV) < st["ranks"][safe][:, None], u, 0.0)
        y = y + torch.bmm(st["b"][safe].float(), u.unsqueeze(2)).squeeze(2)
    else:             # all adapters, the others' columns set to zero
        u = (x @ st["a"].float().view(L * R, -1).T).view(-1, L, R) * factor[:, None, None]
        keep = (torch.arange(L, device=DEV) == ids[:, None])[:, :, None]
        if st["ranks"] is not None:
            keep = keep & (torch.arange(R, device=DEV) < st["ranks"][:, None])
        u = torch.where(keep, u, 0.0).reshape(-1, L * R)
        y = y + u @ st["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    return y.bfloat16()


def _plain_moe(st):
    c = st["c"]
    T, H, F, E, k = c["T"], c["H"], c["F"], c["E"], c["k"]
    x = st["x"].float()
    p = torch.softmax(x @ st["router"].float().T, dim=1)
    top, ids = torch.sort(p, dim=1, descending=True, stable=True)   # ties: the lowest expert first
    top, ids = top[:, :k], ids[:, :k]
    if c["renorm"]:
        top = top / top.sum(dim=1, keepdim=True)
    if T * k <= E:    # the chosen experts of every token, gathered
        flat = ids.reshape(-1)
        xs = x[:, None, :].expand(T, k, H).reshape(T * k, H, 1)
        gu = torch.bmm(_weights(st["gu"][flat], st["gu_s"][flat], H), xs).squeeze(2)
        h = gu[:, :F] / (1.0 + torch.exp(-gu[:, :F])) * gu[:, F:]
        o = torch.bmm(_weights(st["dn"][flat], st["dn_s"][flat], F), h.unsqueeze(2)).view(T, k, H)
        y = (top[:, :, None] * o).sum(dim=1)
    else:             # every expert on every token, weighted by zero where it was not chosen
        gu = torch.matmul(x, _weights(st["gu"], st["gu_s"], H).transpose(1, 2))
        h = gu[..., :F] / (1.0 + torch.exp(-gu[..., :F])) * gu[..., F:]
        share = torch.zeros((T, E), device=DEV).scatter_(1, ids, top)
        o = torch.matmul(h * share.T[:, :, None], _weights(st["dn"], st["dn_s"], F).transpose(1, 2))
        y = o.sum(dim=0)
    return {"y": y.bfloat16(), "ids": ids.int(), "p": top}


def _turn(v, cos, sin, inter):
    """Rotation of the leading columns of [T, heads, D] by the angles of [T, 1, rot / 2]."""
    half = cos.shape[-1]
    a, rest = v[..., :2 * half], v[..., 2 * half:]
    if inter:
        u, w = a[..., 0::2], a[..., 1::2]
        r = torch.stack([u * cos - w * sin, w * cos + u * sin], dim=-1).flatten(-2)
    else:
        u, w = a[..., :half], a[..., half:]
        r = torch.cat([u * cos - w * sin, w * cos + u * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_qkn(st, eps=1e-6):
    c = st["c"]
    cs = st["cs"][st["pos"].long()][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    q = st["q"].float().view(c["T"], -1, c["D"])
    k = st["kk"].float().view(c["T"], -1, c["D"])
    q = q * torch.rsqrt((q * q).mean(dim=-1, keepdim=True) + eps) * st["qw"].float()
    k = k * torch.rsqrt((k * k).mean(dim=-1, keepdim=True) + eps) * st["kw"].float()
    return {"q": _turn(q, cos, sin, c["inter"]).flatten(1).bfloat16(), "k": _turn(k, cos, sin, c["inter"]).flatten(1).bfloat16()}


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["c"]
    if own:
        from weight_only_bit_q4_gb300 import q4lin
        if c["op"] == "lora":
            return q4lin.linear_lora(st["wq"], st["s"], st["x"], st["a"], st["b"], st["ids"], st["scales"], st["ranks"],
                                     y=st["y"], workspace=st["scratch"])
        if c["op"] == "moe":
            y, ids, p = q4lin.moe(st["x"], st["router"], st["gu"], st["gu_s"], st["dn"], st["dn_s"], c["k"],
                                  renormalize=c["renorm"], y=st["y"], ids=st["ids"], weights=st["p"], workspace=st["scratch"])
            return {"y": y, "ids": ids, "p": p}
        q, k = q4lin.qk_norm_rope(st["q"], st["kk"], st["qw"], st["kw"], st["cs"], st["pos"], interleaved=c["inter"],
                                  q_out=st["qo"], k_out=st["ko"])
        return {"q": q, "k": k}
    if c["op"] == "lora":
        return _plain_lora(st)
    if c["op"] == "moe":
        return _plain_moe(st)
    return _plain_qkn(st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "lora":
        N, K, T, L, R = c["N"], c["K"], c["T"], c["L"], c["R"]
        # distinct adapters that T tokens are expected to use
        used = min(L, T) if c["mix"] == "runs" else L * (1.0 - (1.0 - 1.0 / L) ** T)
        r = 0.75 * R if c["several"] else R
        b = N * _pad(K) / 64 * 34 + 2 * T * (K + N) + used * r * (N + K) * 2
        return {"bytes": b, "flops": 2.0 * N * K * T + 2.0 * T * r * (N + K)}
    if c["op"] == "moe":
        T, H, F, E, k = c["T"], c["H"], c["F"], c["E"], c["k"]
        used = E * (1.0 - (1.0 - k / E) ** T)
        w = 2 * F * _pad(H) / 64 * 34 + H * _pad(F) / 64 * 34
        return {"bytes": used * w + 2 * E * H + 4 * T * H + 8 * T * k, "flops": 2.0 * T * (E * H + k * 3 * F * H)}
    n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
    return {"bytes": 4 * n + 4 * c["T"] * (c["rot"] + 1) + 4 * c["D"], "flops": 8.0 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def _codes64(wq, s, K):
    w = torch.empty(wq.shape[:-1] + (2 * wq.shape[-1],), dtype=torch.float64, device=wq.device)
    w[..., 0::2] = (wq % 16).double()
    w[..., 1::2] = torch.div(wq, 16, rounding_mode="floor").double()
    w -= 8.0
    w *= s.double().repeat_interleave(64, dim=-1)
    return w[..., :K]


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "lora":
        x, ids = st["x"].double(), st["ids"].tolist()
        ranks = [c["R"]] * c["L"] if st["ranks"] is None else st["ranks"].tolist()
        y = torch.matmul(x, _codes64(st["wq"], st["s"], c["K"]).t())
        for a in sorted(set(ids) - {-1}):
            rows = torch.tensor([t for t, i in enumerate(ids) if i == a], device=DEV)
            A, B = st["a"][a, :ranks[a]].double(), st["b"][a, :, :ranks[a]].double()
            y[rows] += float(st["scales"][a]) * torch.matmul(torch.matmul(x[rows], A.t()), B.t())
        return y
    if c["op"] == "moe":
        x = st["x"].double()
        logits = torch.matmul(x, st["router"].double().t())
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        prob = e / e.sum(dim=1, keepdim=True)
        p, ids = torch.topk(prob, c["k"], dim=1)
        if c["renorm"]:
            p = p / p.sum(dim=1, keepdim=True)
        y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
        for n in sorted(set(ids.flatten().tolist())):
            t, j = torch.nonzero(ids == n, as_tuple=True)
            gu = torch.matmul(x[t], _codes64(st["gu"][n], st["gu_s"][n], c["H"]).t())
            gate, up = gu[:, :c["F"]], gu[:, c["F"]:]
            o = torch.matmul(gate * torch.sigmoid(gate) * up, _codes64(st["dn"][n], st["dn_s"][n], c["F"]).t())
            y[t] += p[t, j][:, None] * o
        return {"y": y, "ids": None, "p": p}
    got = {}
    half = c["rot"] // 2
    cs = st["cs"].double()[st["pos"].long()]
    z = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]
    for key, src, w in (("q", st["q"], st["qw"]), ("k", st["kk"], st["kw"])):
        v = src.double().reshape(c["T"], -1, c["D"])
        v = v / torch.sqrt(v.pow(2).sum(dim=-1, keepdim=True) / c["D"] + 1e-6) * w.double()
        first = slice(0, c["rot"], 2) if c["inter"] else slice(0, half)
        second = slice(1, c["rot"], 2) if c["inter"] else slice(half, c["rot"])
        r = torch.complex(v[..., first], v[..., second]) * z
        v[..., first], v[..., second] = r.real, r.imag
        got[key] = v.reshape(c["T"], -1)
    return got
