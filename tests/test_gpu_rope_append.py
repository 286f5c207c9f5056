"""The rotation of queries and keys with the append to the FP8 cache, against
the formula bit for bit (each product and sum rounded to fp32, the codes those
of the fp32 quotient), and against 64 bits: a turned value is two products and
a sum, each at most 2^-24 off, and its bf16 rounding at most 2^-8."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


def table(n, rot):
    angle = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def rotate(x, cs, rot, interleaved):
    """x [T, H, D], cs [T, rot] of x's own type; separate products and sums."""
    x = x.clone()
    a = x[..., 0:rot:2].clone() if interleaved else x[..., :rot // 2].clone()
    b = x[..., 1:rot:2].clone() if interleaved else x[..., rot // 2:rot].clone()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = ac - bs, bc + as_
    else:
        x[..., :rot // 2], x[..., rot // 2:rot] = ac - bs, bc + as_
    return x


def quantise(x):
    """E4M3 codes and scales of fp32 vectors: the nearest code (ties to even)
    of the fp32 quotient, found in 64 bits."""
    amax = x.abs().amax(-1)
    s = amax / 448.0
    none = s == 0
    s = torch.where(none, torch.ones_like(s), s)
    q = (x / s[..., None]).double()
    step = torch.exp2((torch.frexp(q)[1].double() - 1).clamp(min=-6) - 3)
    v = (torch.round(q / step) * step).clamp(-448, 448)
    codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8)      # exact: v is an E4M3 value
    return torch.where(none[..., None], torch.zeros_like(codes), codes), s


def values(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[:-1] + (1,), generator=g))).to(torch.bfloat16)


def case(ptpc, T, Hq, Hkv, D, rot, interleaved, bs, seed=0, fused=True, pad=0, inplace=False, bad=True):
    g = torch.Generator().manual_seed(seed)
    n_pos, nb = 2 * T + 64, (T + bs - 1) // bs + 2
    cs = table(n_pos, rot)
    heads = Hq + 2 * Hkv
    qkv = values((T, heads * D + pad), seed + 1)
    positions = torch.randint(0, n_pos, (T,), generator=g)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if T > 4 and Hkv:
        qkv[3, Hq * D:] = 0                                  # zero keys and values: scale 1, codes 0
    if T > 8 and bad:
        slots[5], slots[6] = -1, nb * bs                     # skipped; the query still turns
        positions[7], positions[8] = -1, n_pos               # outside the table: nothing is written
    dev = qkv.cuda()
    views = [dev[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, heads))]
    if not fused:
        views = [v.contiguous() for v in views]
    kc = torch.full((nb, bs, Hkv, D), 0xAB, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.full((nb, bs, Hkv), -7.0, device="cuda")
    vs = ks.clone()
    q_out = views[0] if inplace else torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    got = ptpc.rope_kv_cache_append(*views, cs.cuda(), positions.cuda(), slots.cuda(), kc, vc, ks, vs, q_out=q_out,
                                    interleaved=interleaved)
    q, k, v = (qkv[:, a * D:b * D].reshape(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, heads)))
    told = (positions >= 0) & (positions < n_pos)
    at = cs[positions.clamp(0, n_pos - 1)]
    want = rotate(q.float(), at, rot, interleaved).to(torch.bfloat16)
    want[~told] = q[~told] if inplace else 9.0
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    q64 = rotate(q.double(), at.double(), rot, interleaved)
    size = rotate(q.double().abs(), torch.cat([at[:, :rot // 2].abs(), at[:, rot // 2:].abs()], 1).double(), rot, interleaved)
    size = torch.maximum(size.abs(), q64.abs()) + 2 * q.double().abs().amax(-1, keepdim=True)
    off = (got.cpu().double() - q64).abs()[told]
    assert (off <= (2.0 ** -8 * q64.abs() + 4 * 2.0 ** -24 * size)[told]).all()
    rk, rv = np.full((nb * bs, Hkv, D), 0xAB, np.uint8), np.full((nb * bs, Hkv, D), 0xAB, np.uint8)
    rks, rvs = np.full((nb * bs, Hkv), -7.0, np.float32), np.full((nb * bs, Hkv), -7.0, np.float32)
    kept = told & (slots >= 0) & (slots < nb * bs)
    for x, codes, scales in ((rotate(k.float(), at, rot, interleaved), rk, rks), (v.float(), rv, rvs)):
        c, s = quantise(x[kept])
        codes[slots[kept].numpy()], scales[slots[kept].numpy()] = c.numpy(), s.numpy()
    assert np.array_equal(kc.cpu().numpy().reshape(rk.shape), rk) and np.array_equal(vc.cpu().numpy().reshape(rv.shape), rv)
    assert np.array_equal(ks.cpu().numpy().reshape(rks.shape).view(np.uint32), rks.view(np.uint32))
    assert np.array_equal(vs.cpu().numpy().reshape(rvs.shape).view(np.uint32), rvs.view(np.uint32))
    if not inplace:
        assert torch.equal(dev.cpu().view(torch.int16), qkv.view(torch.int16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs", [
    (1, 64, 8, 128, 128, 16), (32, 64, 8, 128, 128, 16), (300, 32, 8, 128, 128, 32), (77, 12, 12, 64, 64, 24),
    (1000, 5, 1, 64, 32, 8), (9, 7, 7, 128, 16, 9), (33, 48, 3, 128, 96, 16), (2048, 64, 8, 128, 128, 64),
    (1500, 28, 4, 64, 48, 16), (3, 128, 8, 128, 64, 16), (1, 1, 1, 64, 16, 8), (5, 3, 1, 64, 64, 8),
])
def test_against_the_formula(ptpc, T, Hq, Hkv, D, rot, bs, interleaved):
    case(ptpc, T, Hq, Hkv, D, rot, interleaved, bs, seed=T)


@pytest.mark.parametrize("T", [6, 1200])
def test_dense_padded_and_in_place(ptpc, T):
    case(ptpc, T, 16, 2, 128, 128, False, 16, fused=False)
    case(ptpc, T, 16, 2, 128, 64, True, 16, pad=8)
    case(ptpc, T, 16, 2, 64, 64, False, 16, pad=40, inplace=True)
    case(ptpc, T, 16, 2, 64, 32, True, 16, inplace=True)


@pytest.mark.parametrize("T", [4, 900])
def test_keys_only(ptpc, T):
    """No query heads: the rotation and append of keys and values alone."""
    D, Hkv, bs = 128, 8, 16
    nb = T // bs + 1
    k, v = values((T, Hkv, D), 1), values((T, Hkv, D), 2)
    cs, pos = table(T, D), torch.arange(T)
    kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.uint8, device="cuda")
    vc, ks = torch.zeros_like(kc), torch.zeros((nb, bs, Hkv), device="cuda")
    vs = torch.zeros_like(ks)
    q = torch.empty((T, 0, D), dtype=torch.bfloat16, device="cuda")
    ptpc.rope_kv_cache_append(q, k.cuda(), v.cuda(), cs.cuda(), pos.cuda(), pos.cuda(), kc, vc, ks, vs)
    c, s = quantise(rotate(k.float(), cs, D, False))
    assert torch.equal(kc.cpu().view(-1, Hkv, D)[:T], c) and torch.equal(ks.cpu().view(-1, Hkv)[:T], s)


def test_values_as_the_plain_append_writes_them(ptpc):
    """With angles of zero (cosine 1, sine 0) nothing turns: the codes and scales
    are kv_cache_append's own, keys as well as values."""
    T, Hkv, D, bs = 500, 4, 128, 16
    nb = (T + bs - 1) // bs
    k, v = values((T, Hkv, D), 1).cuda(), values((T, Hkv, D), 2).cuda()
    k[0] *= 2.0 ** -110
    v[1] *= 2.0 ** -120
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(1))[:T].cuda()
    new = lambda: [torch.zeros((nb, bs, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((nb, bs, Hkv), device="cuda") for _ in range(2)]  # noqa: E731
    a, b = new(), new()
    cs = torch.cat([torch.ones(8, D // 2), torch.zeros(8, D // 2)], 1).cuda()
    ptpc.kv_cache_append(k, v, slots, *a)
    q = torch.empty((T, 0, D), dtype=torch.bfloat16, device="cuda")
    ptpc.rope_kv_cache_append(q, k, v, cs, torch.zeros(T, dtype=torch.int64, device="cuda"), slots, *b)
    # a negative zero turns into a positive one (0 + -0); its code stands for the same value
    for x, y in zip(a, b):
        if x.dtype == torch.uint8:
            x, y = (torch.where(t == 0x80, torch.zeros_like(t), t) for t in (x, y))
        assert torch.equal(x, y)


def test_non_finite_tokens_stay_in_their_slots(ptpc):
    T, Hq, Hkv, D, bs = 20, 8, 2, 64, 16
    qkv = values((T, (Hq + 2 * Hkv) * D), 3).cuda()
    cs, pos = table(T, D).cuda(), torch.arange(T, device="cuda")
    out = []
    for spoil in (False, True):
        x = qkv.clone()
        if spoil:
            x[4], x[9, ::3] = float("nan"), float("inf")
        kc = torch.zeros((2, bs, Hkv, D), dtype=torch.uint8, device="cuda")
        vc, ks = torch.zeros_like(kc), torch.zeros((2, bs, Hkv), device="cuda")
        vs = torch.zeros_like(ks)
        v = [x[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
        q = ptpc.rope_kv_cache_append(*v, cs, pos, pos, kc, vc, ks, vs)
        out.append([q] + [t.view(2 * bs, -1)[:T] for t in (kc, vc, ks, vs)])
    for a, b in zip(*out):
        for t in range(T):
            assert t in (4, 9) or torch.equal(a[t], b[t])


def test_captured(ptpc):
    T, Hq, Hkv, D, bs = 16, 16, 2, 128, 16
    qkv = values((T, (Hq + 2 * Hkv) * D), 3).cuda()
    v = [qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    cs, pos, slots = table(100, D).cuda(), torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    cache = [torch.zeros((2, bs, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((2, bs, Hkv), device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ptpc.rope_kv_cache_append(*v, cs, pos, slots, *cache)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = ptpc.rope_kv_cache_append(*v, cs, pos, slots, *cache)
    for seed in (5, 6):
        qkv.copy_(values(qkv.shape, seed).cuda())
        pos.add_(seed)
        slots.copy_(slots.flip(0))
        graph.replay()
        got = [q.clone()] + [t.clone() for t in cache]
        for t in cache:
            t.zero_()
        want = [ptpc.rope_kv_cache_append(*v, cs, pos, slots, *cache)] + cache
        assert all(torch.equal(a[:T] if a.shape[0] == T else a.flatten(0, 1)[:T],
                               b[:T] if b.shape[0] == T else b.flatten(0, 1)[:T]) for a, b in zip(got, want))
