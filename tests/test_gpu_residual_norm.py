"""The residual add with the norms on either side of it, against the formula in
64 bits, at one token to more rows than the GPU holds at once, at widths that
fill a thread's vectors and that do not, with and without the norm behind the
block, gates and strides.

Tolerances.  An output of type t is rounded once: at most eps(t) / 2 of its
value.  Before that everything is fp32: a mean of squares is a sum of at most
8 + 8 + 5 + 5 levels (a thread's vector, its vectors, two reductions), each at
most 2^-24 off, and 1 / sqrt halves that; with the products around it a factor
is off by less than F = 24 * 2^-24.  h is a sum, so F counts on |residual| +
|a u|, and an error of h passes into x with the factor |w| * rstd.
A code is the nearest to x / s: off by half a step, 2^-4 of the value or 2^-10
among the subnormals, and by what x is off."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F = 24 * 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


def values(shape, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(torch.bfloat16)


def reference(y, residual, pre, post, gate, a, eps):
    """(h, x, what counts for the error of h, rstd) in 64 bits."""
    h, count = residual.double(), residual.double().abs()
    if y is not None:
        u = y.double()
        if post is not None:
            u = u * post.double() / (u.square().mean(-1, keepdim=True) + eps).sqrt()
        if gate is not None:
            u = u * gate.double()
        h = h + a * u
        count = count + (a * u).abs()
    rstd = 1.0 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, h * pre.double() * rstd, count, rstd


def inside(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, by up to {float((off / bound).max()):.3g} of the bound"


def check(ptpc, T, C, quant, post=False, gate=None, a=1.0, eps=1e-5, first=False, pad=0, inplace=False, zero_rows=(),
          tiny_rows=()):
    wide = values((T, C + pad), 1)
    y = None if first else wide[:, :C]
    residual = values((T, C + pad), 2)[:, :C].clone() if not pad else values((T, C + pad), 2)[:, :C]
    pre, post_w = values((C,), 3, 0.0), values((C,), 4, 0.0) if post else None
    g = {None: None, "channel": values((C,), 5, 0.0), "token": values((T, C + pad), 6)[:, :C]}[gate]
    for r in zero_rows:
        residual[r] = 0
        if y is not None:
            y[r] = 0
    for r in tiny_rows:
        residual[r] *= 2.0 ** -100
        if y is not None:
            y[r] *= 2.0 ** -100

    def dev(t, ld):
        if t is None:
            return None
        if t.dim() == 1 or not ld:
            return t.contiguous().cuda()
        full = torch.zeros((t.shape[0], t.shape[1] + ld), dtype=t.dtype, device="cuda")
        full[:, :t.shape[1]] = t.cuda()
        return full[:, :t.shape[1]]

    yd, rd, gd = dev(y, pad), dev(residual, pad), dev(g, pad)
    more = dict(post_weight=dev(post_w, 0), gate=gd, residual_scale=a, eps=eps, h_out=rd if inplace else None)
    h64, x64, count, rstd = reference(y, residual, pre, post_w, g, a, eps)
    x_off = F * (x64.abs() + count * pre.double().abs() * rstd)
    if quant:
        h, code, scale = ptpc.residual_norm_quantize(yd, rd, dev(pre, 0), **more)
        s = scale.double().cpu()
        amax = x64.abs().amax(-1)
        some = amax / 448 > 2.0 ** -126
        inside(s[some], (amax / 448)[some], (x_off.amax(-1) / 448 + 2 * F * amax / 448)[some], "scale")
        assert (s[amax == 0] == 1).all() and (code.cpu()[amax == 0] == 0).all()
        q = x64 / s[:, None]
        c = code.view(torch.float8_e4m3fn).cpu().double()
        inside(c[some], q[some], (torch.maximum(q.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
                                  + 2 * x_off / s[:, None])[some], "codes")
    else:
        h, x = ptpc.residual_norm(yd, rd, dev(pre, 0), **more)
        inside(x.cpu(), x64, BF16 * (x64.abs() + x_off) + x_off + 2.0 ** -133, "x")
    inside(h.cpu(), h64, BF16 * (h64.abs() + F * count) + F * count + 2.0 ** -133, "h")
    if inplace:
        assert h.data_ptr() == rd.data_ptr()


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("T,C", [(1, 16), (1, 4096), (1, 8192), (1, 16384), (7, 28672), (5, 57344), (3, 65552), (147, 4112),
                                 (148, 8192), (300, 1024), (301, 2064), (1000, 5136), (2048, 4096), (160, 16400),
                                 (150, 32768), (149, 33024)])
def test_norm_only(ptpc, T, C, quant):
    check(ptpc, T, C, quant)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("post,gate,a", [(True, None, 1.0), (False, "channel", 0.5), (True, "token", 0.22),
                                         (True, "channel", -1.5), (False, "token", 0.0)])
@pytest.mark.parametrize("T,C", [(1, 8192), (77, 1040), (300, 8192), (151, 20480), (4, 36880)])
def test_block_norm_and_gate(ptpc, T, C, post, gate, a, quant):
    check(ptpc, T, C, quant, post=post, gate=gate, a=a)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("T,C", [(9, 256), (333, 4112), (5, 33024)])
def test_strides_in_place_and_first_norm(ptpc, T, C, quant):
    check(ptpc, T, C, quant, post=True, gate="token", pad=24)
    check(ptpc, T, C, quant, post=True, gate="channel", pad=8, inplace=True)
    check(ptpc, T, C, quant, first=True)


@pytest.mark.parametrize("T,C,post,gate,a,more", [
    (1200, 8192, True, "channel", 0.7, {}), (2369, 4096, False, None, 1.0, dict(inplace=True)),
    (1185, 7200, True, "token", 0.5, dict(pad=16)), (600, 16384, True, None, -1.5, dict(inplace=True, pad=8)),
    (9500, 1024, False, "token", 1.0, {}), (2400, 4080, False, "channel", 0.25, dict(zero_rows=(0, 1111, 2399))),
    (2401, 3600, True, "token", 1.0, {}), (1184, 8208, False, None, 1.0, dict(first=True)),
    (1187, 8192, False, None, 1.0, dict(first=True, tiny_rows=(0, 1186)))])
@pytest.mark.parametrize("quant", [True, False])
def test_several_rows_a_cta(ptpc, T, C, post, gate, a, more, quant):
    check(ptpc, T, C, quant, post=post, gate=gate, a=a, **more)


@pytest.mark.parametrize("quant", [True, False])
def test_zero_and_tiny_rows(ptpc, quant):
    """Rows of zeros (the norm's eps alone: x = 0, scale 1, codes 0) and rows so
    small that eps outweighs them."""
    check(ptpc, 20, 512, quant, post=True, zero_rows=(0, 7, 19), tiny_rows=(3, 8))
    check(ptpc, 200, 4096, quant, zero_rows=(199,), tiny_rows=(0, 100), eps=1e-30)


def test_other_rows_and_inputs_stay(ptpc):
    """Nothing is written outside the outputs' own elements; inputs stay."""
    T, C = 37, 400
    y, r, w = (values(s, i).cuda() for i, s in enumerate([(T, C), (T, C), (C,)]))
    keep = [t.clone() for t in (y, r, w)]
    h = torch.full((T + 2, C + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((T + 2, C), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 2 + 8,), -3.0, device="cuda")
    ptpc.residual_norm_quantize(y, r, w, h_out=h[1:T + 1, :C], Xq=q[1:T + 1], x_scale=s[4:T + 4])
    for t, k in zip((y, r, w), keep):
        assert torch.equal(t, k)
    assert (h[0] == 7).all() and (h[T + 1] == 7).all() and (h[:, C:] == 7).all()
    assert (q[0] == 0xA5).all() and (q[T + 1] == 0xA5).all()
    assert (s[:4] == -3).all() and (s[T + 4:] == -3).all()


def test_no_rows_and_repeat(ptpc):
    w = values((64,), 1).cuda()
    h, x = ptpc.residual_norm(None, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w)
    assert h.shape == (0, 64) and x.shape == (0, 64)
    y, r = values((50, 64), 2).cuda(), values((50, 64), 3).cuda()
    a, b = ptpc.residual_norm_quantize(y, r, w), ptpc.residual_norm_quantize(y, r, w)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_non_finite_row_stays_in_its_row(ptpc):
    """A row with an infinity or NaN gives no other row anything."""
    y, r, w = values((6, 1024), 1).cuda(), values((6, 1024), 2).cuda(), values((1024,), 3).cuda()
    h0, q0, s0 = ptpc.residual_norm_quantize(y, r, w, post_weight=w)
    y[2, 5], r[4, 9] = float("inf"), float("nan")
    h1, q1, s1 = ptpc.residual_norm_quantize(y, r, w, post_weight=w)
    for i in (0, 1, 3, 5):
        assert torch.equal(h0[i], h1[i]) and torch.equal(q0[i], q1[i]) and s0[i] == s1[i]


def test_codes_feed_the_gemm(ptpc):
    """residual_norm_quantize, then scaled_mm: what linear gives on the norm's
    bf16 output, up to that output's rounding (2^-8 a value) and the codes'
    (2^-4), which both add up like independent errors over 1024 products."""
    T, C, Co = 33, 1024, 256
    y, r, w = values((T, C), 1, 0.3).cuda(), values((T, C), 2, 0.3).cuda(), values((C,), 3, 0.0).cuda()
    W = values((C, Co), 4, 0.0).cuda()
    Wq, ws = ptpc.quantize_weights(W)
    h, Xq, xs = ptpc.residual_norm_quantize(y, r, w)
    out = ptpc.scaled_mm(Xq, xs, Wq, ws)
    x = Xq.view(torch.float8_e4m3fn).double() * xs.double()[:, None]
    ref = x @ (Wq.view(torch.float8_e4m3fn).double() * ws.double()[:, None]).T
    assert ((out.double() - ref).abs() <= 1e-2 * ref.abs() + 1e-3 * ref.square().mean().sqrt()).all()


def test_captured(ptpc):
    """Captured and replayed on new inputs: what the same call gives eagerly."""
    T, C = 40, 2048
    y, r, w = values((T, C), 1).cuda(), values((T, C), 2).cuda(), values((C,), 3).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ptpc.residual_norm_quantize(y, r, w, post_weight=w, gate=y)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ptpc.residual_norm_quantize(y, r, w, post_weight=w, gate=y)
    for seed in (7, 8):
        y.copy_(values((T, C), seed).cuda())
        graph.replay()
        want = ptpc.residual_norm_quantize(y, r, w, post_weight=w, gate=y)
        assert all(torch.equal(i, j) for i, j in zip(got, want))
