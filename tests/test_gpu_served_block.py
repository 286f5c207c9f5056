"""The operators around a block as a served model runs them: norm to codes,
QKV projection on the codes, rotary append to the paged cache, attention of
the new tokens, output projection, norms and residual add; two layers, prompts
of different lengths in a padded batch, then a token for each sequence.

Tolerance against the same model in 64 bits (with the codes of weights and
scales as the library made them).  Every stage's output is rounded to bf16
(2^-9 of the value or less, rms).  An input that is off by that crosses the
border between two codes with a probability of 2^-8 / 2^-3 = 2^-5 or less and
is then off by a step of 2^-3: 2^-3 * 2^-2.5 = 2^-5.5 rms of each quantised
tensor.  A layer has three of those behind one another on the way to its
output (the block's input, keys or values, the attention's output), two layers
six: sqrt(6) 2^-5.5 plus the bf16 roundings, less than 2^-3.5; held to 2^-3 of
what the layers added to the residual."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS, LAYERS, EPS, ALPHA = 8, 2, 128, 16, 2, 1e-5, 0.5
C, QKV = Hq * D, (Hq + 2 * Hkv) * D


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


class Model:
    def __init__(self, ptpc, blocks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.layers = []
        for _ in range(LAYERS):
            wqkv = ptpc.quantize_weights((rand(C, QKV) / math.sqrt(C)).to(bf))
            wo = ptpc.quantize_weights((rand(C, C) / math.sqrt(C)).to(bf))
            norms = [(1 + 0.1 * rand(C)).to(bf) for _ in range(2)]
            cache = [torch.zeros(blocks, BS, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.ones(blocks, BS, Hkv, device="cuda") for _ in range(2)]
            self.layers.append((wqkv, wo, norms, cache + scales))
        self.last = (1 + 0.1 * rand(C)).to(bf)
        angle = torch.arange(512, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()

    def step(self, ptpc, h, positions, slots, tables, ctx, cu, max_q, max_context, dense=False):
        """(residual stream, normed output) of the new tokens' residual h [T, C]."""
        y, gate, post = None, None, None
        for wqkv, wo, (pre, behind), cache in self.layers:
            h, xq, xs = ptpc.residual_norm_quantize(y, h, pre, post_weight=post, residual_scale=ALPHA, eps=EPS)
            qkv = ptpc.scaled_mm(xq, xs, *wqkv)
            q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D))
                       for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
            if dense:
                q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
            q = ptpc.rope_kv_cache_append(q, k, v, self.cos_sin, positions, slots, *cache, q_out=q)
            o = ptpc.chunk_attention(q, *cache, tables, ctx, cu, max_q, max_context, 1 / math.sqrt(D),
                                     out=torch.zeros_like(h).view(-1, Hq, D))
            y, post = ptpc.linear(o.view(-1, C), *wo), behind
        return ptpc.residual_norm(y, h, self.last, post_weight=post, residual_scale=ALPHA, eps=EPS)

    def plain(self, h, n, m):
        """The same in 64 bits, whole contexts at once: h [sum m, C] residuals of
        all positions; the streams of the last n of each sequence."""
        dec = lambda w: (w[0].view(torch.float8_e4m3fn).double() * w[1].double()[:, None]).T  # noqa: E731
        norm = lambda x, w: x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()  # noqa: E731

        def codes(x):
            s = x.abs().amax(-1, keepdim=True) / 448
            s = torch.where(s == 0, torch.ones_like(s), s)
            return (x / s).float().to(torch.float8_e4m3fn).double() * s

        h = h.double()
        pos = torch.cat([torch.arange(x, device="cuda") for x in m])
        cs = self.cos_sin.double()[pos][:, None]
        c, s = cs[..., :D // 2], cs[..., D // 2:]

        def turn(x):
            a, b = x[..., :D // 2], x[..., D // 2:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        for wqkv, wo, (pre, behind), _ in self.layers:
            qkv = (codes(norm(h, pre)) @ dec(wqkv)).to(torch.bfloat16).double().view(-1, Hq + 2 * Hkv, D)
            q, k, v = turn(qkv[:, :Hq]), codes(turn(qkv[:, Hq:Hq + Hkv])), codes(qkv[:, Hq + Hkv:])
            o = torch.zeros_like(q)
            at = 0
            for x in m:
                r = slice(at, at + x)
                at += x
                kk, vv = (t[r].repeat_interleave(Hq // Hkv, 1) for t in (k, v))
                z = torch.einsum("ihd,jhd->hij", q[r], kk) / math.sqrt(D)
                z = z.masked_fill(torch.ones(x, x, device="cuda").triu(1).bool(), float("-inf"))
                o[r] = torch.einsum("hij,jhd->ihd", z.softmax(-1), vv)
            h = h + ALPHA * norm(codes(o.reshape(-1, C).to(torch.bfloat16).double()) @ dec(wo), behind)
        rows, at = [], 0
        for a, b in zip(n, m):
            rows += range(at + b - a, at + b)
            at += b
        return h[rows], norm(h, self.last)[rows]


def batch(n, m, pad=0):
    """Places of the last n of m positions of each sequence, with `pad` rows behind that write nothing."""
    per = 512 // BS
    tables = torch.randperm(len(m) * per, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(len(m), per)
    pos = torch.cat([torch.arange(b - a, b) for a, b in zip(n, m)])
    seq = torch.cat([torch.full((a,), i) for i, a in enumerate(n)])
    slots = tables[seq, pos // BS].long() * BS + pos % BS
    none = torch.full((pad,), -1)
    return [t.cuda() for t in (torch.cat([pos, torch.zeros(pad, dtype=torch.int64)]), torch.cat([slots, none]), tables,
                               torch.tensor(m, dtype=torch.int32),
                               torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32))]


def near(got, want, base):
    off, size = (got.double() - want).square().mean().sqrt(), (want - base).square().mean().sqrt()
    assert float(off) <= 2.0 ** -3 * float(size), (float(off), float(size))


def stream(rows, seed):
    return torch.randn(rows, C, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def test_prompts_then_tokens(ptpc):
    m = [100, 1, 257, 31]
    model = Model(ptpc, len(m) * (512 // BS))
    h0 = stream(sum(m) + len(m), 1)
    prompts, tokens = h0[:sum(m)], h0[sum(m):]
    pad = 11
    got, x = model.step(ptpc, torch.cat([prompts, stream(pad, 2)]), *batch(m, m, pad), max(m), max(m))
    want, wx = model.plain(prompts, m, m)
    near(got[:sum(m)], want, prompts.double())
    near(x[:sum(m)], wx, torch.zeros_like(wx))
    # a token more of each sequence
    more = [a + 1 for a in m]
    got, x = model.step(ptpc, tokens, *batch([1] * len(m), more), 1, max(more))
    at, rows = 0, []
    for i, a in enumerate(m):
        rows += [prompts[at:at + a], tokens[i:i + 1]]
        at += a
    want, wx = model.plain(torch.cat(rows), [1] * len(m), more)
    near(got, want, tokens.double())
    near(x, wx, torch.zeros_like(wx))
    for _, _, _, (kc, vc, ks, vs) in model.layers:
        assert int((ks != 1).sum()) <= sum(more) * Hkv          # padding wrote nothing


def test_views_and_dense_copies_give_the_same(ptpc):
    m = [70, 5]
    h0 = stream(sum(m), 4)
    out = []
    for dense in (False, True):
        model = Model(ptpc, len(m) * (512 // BS), seed=5)
        out.append(model.step(ptpc, h0, *batch(m, m), max(m), max(m), dense=dense))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_captured_steps_replay_what_runs_eagerly(ptpc):
    """Two steps captured into graphs on a stream of their own, replayed with
    new inputs beside eager calls on the current stream."""
    m = [40, 129, 7]
    B = len(m)
    eager, replayed = (Model(ptpc, B * (512 // BS), seed=6) for _ in range(2))
    prompt = stream(sum(m), 7)
    for model in (eager, replayed):
        model.step(ptpc, prompt, *batch(m, m), max(m), max(m))
    h = stream(B, 8)
    places = batch([1] * B, [a + 1 for a in m])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.step(ptpc, h, *places, 1, 300)                  # first use of each kernel, the same slots again later
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(replayed.step(ptpc, h, *places, 1, 300))
        graphs.append(g)
    for i in range(4):
        new = stream(B, 20 + i)
        for a, b in zip(places, batch([1] * B, [x + 1 + i for x in m])):
            a.copy_(b)
        h.copy_(new)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graphs[i % 2].replay()
        want = eager.step(ptpc, new, *batch([1] * B, [x + 1 + i for x in m]), 1, 300)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(outs[i % 2], want))


def test_wrappers_refuse_what_does_not_fit(ptpc):
    """Before anything is launched: other types, shapes, pitches and devices."""
    T, nb = 6, 4
    x, w = stream(T, 30), torch.ones(C, dtype=torch.bfloat16, device="cuda")
    fine = dict(y=x, residual=x, pre_weight=w, post_weight=w, gate=w)
    for call in (ptpc.residual_norm, ptpc.residual_norm_quantize):
        for name, bad, error in (
                ("y", x[:, :-16], ValueError), ("y", x.float(), TypeError), ("y", x.t(), ValueError),
                ("residual", x.cpu(), TypeError), ("residual", x[0], ValueError), ("pre_weight", w[:-16], ValueError),
                ("pre_weight", w.cpu(), TypeError), ("post_weight", w.float(), TypeError), ("gate", x[:-1], ValueError),
                ("gate", w[:16], ValueError), ("h_out", x[:, :-16], ValueError), ("y", None, ptpc.PtpcError),
                ("eps", 0.0, ptpc.PtpcError), ("residual_scale", math.inf, ptpc.PtpcError)):
            with pytest.raises(error):
                call(**{**fine, name: bad})
    with pytest.raises(ValueError):
        ptpc.residual_norm(x, x, w, out=torch.zeros(T, 2 * C, dtype=torch.bfloat16, device="cuda")[:, :C])
    with pytest.raises(ValueError):
        ptpc.residual_norm_quantize(x, x, w, Xq=torch.zeros(T, C + 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ptpc.residual_norm_quantize(x, x, w, x_scale=torch.zeros(T + 1, device="cuda"))

    q = stream(T, 31).view(T, Hq, D)
    k = q[:, :Hkv]
    cache = [torch.zeros(nb, BS, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(nb, BS, Hkv, device="cuda") for _ in range(2)]
    at = torch.arange(T, device="cuda")
    table = torch.zeros(16, D, device="cuda")
    fine = dict(q=q, k=k, v=k, cos_sin=table, positions=at, slots=at, k_cache=cache[0], v_cache=cache[1],
                k_scale=scales[0], v_scale=scales[1])
    for name, bad, error in (
            ("q", q.float(), TypeError), ("q", q.transpose(0, 1), ValueError), ("k", q, ValueError),
            ("v", k[:-1], ValueError), ("cos_sin", table.double(), TypeError), ("cos_sin", table[:, :24].contiguous(), ptpc.PtpcError),
            ("positions", at.int(), TypeError), ("slots", at[:-1], ValueError), ("slots", at.cpu(), TypeError),
            ("k_scale", scales[0][:, :8], ValueError), ("v_cache", cache[1][:2], ValueError), ("q_out", k, ValueError)):
        with pytest.raises(error):
            ptpc.rope_kv_cache_append(**{**fine, name: bad})

    i32 = dict(dtype=torch.int32, device="cuda")
    fine = dict(q=q, k_cache=cache[0], v_cache=cache[1], k_scale=scales[0], v_scale=scales[1],
                block_tables=torch.zeros(2, 4, **i32), context_lens=torch.ones(2, **i32), cu_q=torch.zeros(3, **i32),
                max_q=4, max_context=64, softmax_scale=0.1)
    for name, bad, error in (
            ("q", q[:, :3].contiguous(), ValueError), ("q", q[..., :64].contiguous(), ValueError),
            ("block_tables", torch.zeros(3, 4, **i32), ValueError), ("context_lens", at[:2], TypeError),
            ("cu_q", torch.zeros(2, **i32), ValueError), ("cu_q", torch.zeros(3, dtype=torch.int32), TypeError),
            ("max_q", -1, ptpc.PtpcError), ("softmax_scale", 0.0, ptpc.PtpcError), ("out", q[:-1], ValueError),
            ("ws", ptpc.Workspace(256, "cpu"), ValueError)):
        with pytest.raises(error):
            ptpc.chunk_attention(**{**fine, name: bad})
    for c in cache:
        assert int(c.sum()) == 0
