"""The serving operators around the PTPC-FP8 linear layers, as a user calls them, and their plain forms.

Three operators make up the attention half of a transformer layer whose linears run in FP8 and whose KV cache is
FP8 (E4M3 codes with one scale a (token, KV head)):

* ``residual_norm`` / ``residual_norm_quantize``: a block's output is normalised (optional), gated (optional), scaled
  and added to the residual stream, and the sum is normalised for the next block, as bf16 or as the per-token FP8
  codes and scales that ``scaled_mm`` reads;
* ``rope_kv_cache_append``: queries and keys are rotated by their positions; keys and values are quantised and
  written to their slots of the paged cache;
* ``chunk_attention``: causal attention of each sequence's newest tokens over its paged cache.

``run`` makes the framework's calls where ``own`` is true and computes the plain form otherwise.  Codes are returned
as float8 views, that is, as the values they stand for.
"""
import math
import random

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
ROPE_BASE = 500000.0


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One token through a layer of the 70B shape: the call that a decode step makes twice a layer.
        dict(name="norm 70B one token", op="norm", T=1, C=8192, post=False, gate="none", scale=1.0, quant=True),
        # A prompt of 2048 tokens at the 8B width, pre-norm only.
        dict(name="norm 8B prompt", op="norm", T=2048, C=4096, post=False, gate="none", scale=1.0, quant=True),
        # The 70B prefill step, with the norm behind the block and a gate a channel.
        dict(name="norm 70B prefill", op="norm", T=8192, C=8192, post=True, gate="channel", scale=0.7, quant=True),
        # A ragged batch of an odd width, a gate of its own for every token, bf16 output.
        dict(name="norm ragged bf16", op="norm", T=3001, C=5136, post=True, gate="token", scale=1.0, quant=False),
        # A decode step of 32 sequences at the 70B shape.
        dict(name="append 70B decode", op="append", T=32, Hq=64, Hkv=8, D=128, rot=128, interleaved=False, bs=16),
        # The 70B prefill step: 8192 tokens of a fused QKV projection.
        dict(name="append 70B prefill", op="append", T=8192, Hq=64, Hkv=8, D=128, rot=128, interleaved=False, bs=16),
        # A ragged batch, heads of 64 of which 32 values turn, in neighbouring pairs.
        dict(name="append ragged D64", op="append", T=3001, Hq=12, Hkv=12, D=64, rot=32, interleaved=True, bs=24),
        # Five drafted tokens of eight sequences checked at once (70B shape): latency counts.
        dict(name="attn draft 70B", op="attn", B=8, q_lo=5, q_hi=5, one=0.0, c_lo=2000, c_hi=4096, Hq=64, Hkv=8,
             D=128, bs=16, lens=1),
        # One chunk of 2048 tokens at the end of a context of 32768 (70B shape).
        dict(name="attn chunk 70B", op="attn", B=1, q_lo=2048, q_hi=2048, one=0.0, c_lo=30720, c_hi=30720, Hq=64,
             Hkv=8, D=128, bs=16, lens=2),
        # Whole prompts of different lengths, packed (8B shape): the context is the chunk itself.
        dict(name="attn prompts 8B", op="attn", B=8, q_lo=300, q_hi=4000, one=0.0, c_lo=0, c_hi=0, Hq=32, Hkv=8,
             D=128, bs=16, lens=3),
        # A serving step that mixes chunks of prompts with single tokens (70B shape).
        dict(name="attn mixed 70B", op="attn", B=32, q_lo=16, q_hi=512, one=0.7, c_lo=500, c_hi=8000, Hq=64, Hkv=8,
             D=128, bs=16, lens=4),
        # Few tokens on long contexts, heads of 64 in groups of 16, blocks of 24.
        dict(name="attn long D64", op="attn", B=2, q_lo=20, q_hi=77, one=0.0, c_lo=40000, c_hi=60000, Hq=32, Hkv=2,
             D=64, bs=24, lens=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn"])
    if op == "norm":
        C = 16 * _log_int(rng, 64, 1024)
        T = _log_int(rng, 1, min(16384, 8192 * 8192 // C))
        return dict(op=op, T=T, C=C, post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                    scale=rng.choice([1.0, 0.5, 0.22]), quant=rng.random() < 0.7)
    D = rng.choice([64, 128])
    bs = rng.choice([8, 16, 24, 32, 48, 64])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "append":
        T = _log_int(rng, 1, 8192)
        return dict(op=op, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]),
                    interleaved=rng.random() < 0.4, bs=bs)
    B = _log_int(rng, 1, 24)
    Hq = G * Hkv
    q_hi = _log_int(rng, 1, 1024)
    # B * Hq * q * context stays below a quarter of the largest listed case's
    c_most = max(64, min(60000, (1 << 30) // (B * Hq * q_hi)))
    c_hi = _log_int(rng, 32, c_most)
    return dict(op=op, B=B, q_lo=max(1, q_hi // rng.choice([1, 4, 50])), q_hi=q_hi, one=rng.choice([0.0, 0.0, 0.5]),
                c_lo=c_hi // rng.choice([1, 2, 10]), c_hi=c_hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                lens=rng.randrange(1 << 20))


def _lens(case):
    """(new tokens, context length with them) of every sequence."""
    r = random.Random(case["lens"])
    q = [1 if r.random() < case["one"] else r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    return q, [n + r.randint(case["c_lo"], case["c_hi"]) for n in q]


def work(case):
    if case["op"] == "norm":
        T, C = case["T"], case["C"]
        rows = 2 + 2 + 2 + (1 if case["quant"] else 2) + (2 if case["gate"] == "token" else 0)
        once = 2 + (2 if case["post"] else 0) + (2 if case["gate"] == "channel" else 0)
        return {"bytes": T * C * rows + C * once + (4 * T if case["quant"] else 0), "flops": T * C * 10}
    if case["op"] == "append":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        per = Hq * D * 4 + Hkv * D * 4 + Hkv * (D + 4) * 2 + case["rot"] * 4 + 16
        return {"bytes": T * per, "flops": T * (Hq + 2 * Hkv) * D * 3}
    q, c = _lens(case)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    seen = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, c))
    return {"bytes": sum(q) * Hq * D * 4 + sum(c) * Hkv * 2 * (D + 4), "flops": 4 * D * Hq * seen}


# ------------------------------------------------------------------------------------------------- inputs

def _spread(g, shape, dev):
    """Normal values times a factor of each row's own, a few columns large: what activations look like."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.7 * torch.randn(shape[:-1] + (1,), generator=g, device=dev))
    x[..., torch.randint(0, shape[-1], (2,), generator=g, device=dev)] *= 10.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"] == "norm":
        T, C = case["T"], case["C"]
        s["y"], s["residual"] = _spread(g, (T, C), dev), _spread(g, (T, C), dev)
        weight = lambda: (1.0 + 0.1 * torch.randn((C,), generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
        s["pre"], s["post"] = weight(), weight() if case["post"] else None
        shape = {"none": None, "channel": (C,), "token": (T, C)}[case["gate"]]
        s["gate"] = torch.randn(shape, generator=g, device=dev).to(torch.bfloat16) if shape else None
        return s
    D, Hq, Hkv, bs = case["D"], case["Hq"], case["Hkv"], case["bs"]
    if case["op"] == "append":
        T, rot = case["T"], case["rot"]
        qkv = _spread(g, (T, Hq + 2 * Hkv, D), dev)  # the fused projection's output; q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        longest = 2 * T + 4096
        angle = torch.arange(longest, dtype=torch.float64, device=dev)[:, None] * \
            ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        first = int(torch.randint(0, T + 4096, (1,), generator=g, device=dev))
        s["positions"] = torch.arange(first, first + T, device=dev)
        blocks = (T + bs - 1) // bs + 3
        table = torch.randperm(blocks, generator=g, device=dev)
        at = torch.arange(T, device=dev)
        s["slots"] = table[at // bs] * bs + at % bs
        s["k_cache"] = torch.zeros((blocks, bs, Hkv, D), dtype=torch.uint8, device=dev)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["k_scale"] = torch.ones((blocks, bs, Hkv), device=dev)
        s["v_scale"] = torch.ones_like(s["k_scale"])
        return s
    q, c = _lens(case)
    need = [(m + bs - 1) // bs for m in c]
    blocks = sum(need) + 2
    most = max(need)
    perm = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    at = torch.arange(most, device=dev)
    s["block_tables"] = torch.where(at[None] < torch.tensor(need, device=dev)[:, None],
                                    perm[(first[:, None] + at[None]).clamp(max=blocks - 1)], -1).to(torch.int32)
    s["context_lens"] = torch.tensor(c, dtype=torch.int32, device=dev)
    s["cu_q"] = torch.tensor([0] + q, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    s["max_q"], s["max_context"] = max(q), max(c)
    s["q"] = torch.randn((sum(q), Hq, D), generator=g, device=dev).to(torch.bfloat16)
    for name in ("k", "v"):
        x = torch.randn((blocks * bs, Hkv, D), generator=g, device=dev)
        x *= torch.exp(0.4 * torch.randn((blocks * bs, Hkv, 1), generator=g, device=dev))
        code, scale = _quantise(x)
        s[name + "_cache"] = code.view(torch.uint8).view(blocks, bs, Hkv, D)
        s[name + "_scale"] = scale.view(blocks, bs, Hkv)
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _quantise(x):
    """E4M3 codes (as float8) and one fp32 scale for each vector along the last axis."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_norm(s):
    c = s["case"]
    u = s["y"].float()
    if s["post"] is not None:
        u = _norm(u, s["post"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["residual"].float() + c["scale"] * u
    x = _norm(h, s["pre"])
    if not c["quant"]:
        return {"h": h.to(torch.bfloat16), "x": x.to(torch.bfloat16)}
    code, scale = _quantise(x)
    return {"h": h.to(torch.bfloat16), "x": code, "x_scale": scale}


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] in 32 bits, its first `rot` values turned; cos and sin [T, rot / 2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, :c["rot"] // 2], table[:, c["rot"] // 2:]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
    k, k_scale = _quantise(_rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"]))
    v, v_scale = _quantise(s["v"].float())
    s["k_cache"].view(-1, c["Hkv"], c["D"])[s["slots"]] = k.view(torch.uint8)
    s["v_cache"].view(-1, c["Hkv"], c["D"])[s["slots"]] = v.view(torch.uint8)
    s["k_scale"].view(-1, c["Hkv"])[s["slots"]] = k_scale
    s["v_scale"].view(-1, c["Hkv"])[s["slots"]] = v_scale
    return _appended(s, q)


def _appended(s, q):
    return {"q": q, "k_cache": s["k_cache"].view(torch.float8_e4m3fn), "v_cache": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attention(s):
    c = s["case"]
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    dev, B, G, L, n = s["q"].device, c["B"], Hq // Hkv, s["max_context"], s["max_q"]
    at = torch.arange(L, device=dev)
    slots = s["block_tables"].long()[:, at // bs] * bs + at % bs  # [B, L]; behind a context's end: anything valid
    slots = slots.clamp(min=0)
    values = lambda m: (s[m + "_cache"].view(torch.float8_e4m3fn).view(-1, Hkv, D)[slots].float()  # noqa: E731
                        * s[m + "_scale"].view(-1, Hkv)[slots][..., None]).transpose(1, 2)  # [B, Hkv, L, D]
    cu, ctx = s["cu_q"].long(), s["context_lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = (q @ values("k").transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, n, G, L)
    sees = at[None, None] <= (ctx - new)[:, None, None] + i[None, :, None]  # [B, n, L]
    score.masked_fill_(~sees[:, None, :, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(B, Hkv, n * G, L) @ values("v")).view(B, Hkv, n, G, D) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(torch.bfloat16)
    row = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return {"out": out[b, row - cu[b]]}


# ------------------------------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        import fp8_quantized_gemm_ptpc_b200 as ptpc
        if c["op"] == "norm":
            more = dict(post_weight=s["post"], gate=s["gate"], residual_scale=c["scale"], eps=EPS)
            if not c["quant"]:
                h, x = ptpc.residual_norm(s["y"], s["residual"], s["pre"], **more)
                return {"h": h, "x": x}
            h, x, x_scale = ptpc.residual_norm_quantize(s["y"], s["residual"], s["pre"], **more)
            return {"h": h, "x": x.view(torch.float8_e4m3fn), "x_scale": x_scale}
        if c["op"] == "append":
            q = ptpc.rope_kv_cache_append(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"],
                                          s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                          interleaved=c["interleaved"])
            return _appended(s, q)
        return {"out": ptpc.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                            s["block_tables"], s["context_lens"], s["cu_q"], s["max_q"],
                                            s["max_context"], 1.0 / math.sqrt(c["D"]))}
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attention}[c["op"]](s)


# ------------------------------------------------------------------------------------------------- 64 bits

def _e4m3(x):
    """The nearest E4M3 value (ties to the even code) of |x| <= 448, in 64 bits."""
    exponent = torch.frexp(x)[1].to(torch.float64) - 1  # x = m * 2^e, 1 <= |m| < 2
    step = torch.exp2(exponent.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_codes(x):
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return _e4m3(x / scale[..., None]), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        y, r, w = s["y"].double(), s["residual"].double(), s["pre"].double()
        if case["post"]:
            y = y / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["post"].double()
        if s["gate"] is not None:
            y = y * s["gate"].double()
        h = r + case["scale"] * y
        x = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt() * w
        if not case["quant"]:
            return {"h": h, "x": x}
        code, scale = _exact_codes(x)
        return {"h": h, "x": code, "x_scale": scale}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        cos = s["cos_sin"][s["positions"], :half].double()[:, None]
        sin = s["cos_sin"][s["positions"], half:].double()[:, None]
        turned = []
        for x in (s["q"].double(), s["k"].double()):
            z = x.clone()
            z[..., first] = x[..., first] * cos - x[..., second] * sin
            z[..., second] = x[..., second] * cos + x[..., first] * sin
            turned.append(z)
        found = {"q": turned[0]}
        for name, x in (("k", turned[1]), ("v", s["v"].double())):
            code, scale = _exact_codes(x)
            cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda")
            scales = torch.ones(s[name + "_scale"].shape, dtype=torch.float64, device="cuda")
            cache.view(-1, Hkv, D)[s["slots"]] = code
            scales.view(-1, Hkv)[s["slots"]] = scale
            found[name + "_cache"], found[name + "_scale"] = cache, scales
        return found
    G, bs = Hq // Hkv, case["bs"]
    new, ctx = _lens(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, m) in enumerate(zip(new, ctx)):
        blocks = s["block_tables"][b, :(m + bs - 1) // bs].long()
        for h in range(Hkv):
            k, v = ((s[x + "_cache"][blocks, :, h].view(torch.float8_e4m3fn).double()
                     * s[x + "_scale"][blocks, :, h].double()[..., None]).reshape(-1, D)[:m] for x in "kv")
            for i in range(0, n, 512):  # bounds the scores held at once
                j = min(n, i + 512)
                q = s["q"][row + i:row + j, h * G:(h + 1) * G].double()
                z = torch.einsum("igd,ld->igl", q, k) / math.sqrt(D)
                hidden = torch.arange(m, device="cuda")[None] > torch.arange(m - n + i, m - n + j, device="cuda")[:, None]
                p = torch.softmax(z.masked_fill(hidden[:, None], float("-inf")), -1)
                out[row + i:row + j, h * G:(h + 1) * G] = torch.einsum("igl,ld->igd", p, v)
        row += n
    return {"out": out}
