"""Causal attention of new tokens over the FP8 paged cache, against the formula
in 64 bits (on the decoded cache), from one token to whole prompts, with
groups, head sizes and block sizes that fill tiles and that do not, rows that
see nothing, missing blocks, padded batches and split contexts.

Tolerance of an output, from the arithmetic that the header states.  With p
and V the exact weights and values, A = sum p |V|, N = the largest sum over d
of |q K| of a row in the exponent's units:
  - a key is off by 2^-12 of its value twice (two f16 roundings: the scale's
    remainder and the product), a score by at most N 2^-11, and a weight by
    that, numerator and denominator: 2 N 2^-11 A;
  - a weight is rounded to f16: 2^-11 A; a value twice: 2 * 2^-11 A;
  - f16's smallest step, 2^-24, is off by half of that for each position, where
    the largest weight is at least 1 and value scales lie within a factor of
    `spread`: L 2^-25 max|V| spread;
  - sums, exponentials and statistics in fp32: 2^-18 A;
  - the output's bf16 rounding: 2^-8 of the output."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


def quantise(x):
    amax = x.abs().amax(-1)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


class Case:
    """n: new tokens, m: contexts; the cache is filled with random keys and values."""

    def __init__(self, n, m, Hq, Hkv, D, bs, seed=0, q_size=1.0, v_spread=0.5, pad=0, before=0, behind=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.n, self.m, self.Hq, self.Hkv, self.D, self.bs = n, m, Hq, Hkv, D, bs
        B = len(n)
        self.max_blocks = max(1, max((x + bs - 1) // bs for x in m))
        nb = B * self.max_blocks + 2
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        self.tables = perm[:B * self.max_blocks].view(B, self.max_blocks).clone()
        for b in range(B):
            self.tables[b, (m[b] + bs - 1) // bs:] = -1
        k = rand(nb, bs, Hkv, D) * torch.exp(0.5 * rand(nb, bs, Hkv, 1))
        v = rand(nb, bs, Hkv, D) * torch.exp(v_spread * rand(nb, bs, Hkv, 1))
        (self.kc, self.ks), (self.vc, self.vs) = quantise(k), quantise(v)
        total = before + sum(n) + behind
        wide = (rand(total, Hq * D + pad) * q_size).to(torch.bfloat16)
        self.q = wide[:, :Hq * D].unflatten(1, (Hq, D))
        self.cu = torch.tensor([before] + n, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        self.ctx = torch.tensor(m, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(D)
        self.max_q, self.max_context = max(max(n), 1), max(max(m), 1)

    def run(self, ptpc, ws=None, out=None):
        if ws is None:
            ws = ptpc.Workspace(ptpc.lib.ptpc_chunk_attention_workspace_size(
                self.q.shape[0], len(self.n), self.Hq, self.Hkv, self.D, self.max_q, self.max_context), "cuda")
        out = ptpc.chunk_attention(self.q, self.kc, self.vc, self.ks, self.vs, self.tables, self.ctx, self.cu,
                                   self.max_q, self.max_context, self.scale, out=out, ws=ws)
        assert ptpc.device_status(ws) == 0
        return out

    def splits(self, ptpc):
        return ptpc.chunk_attention_splits(self.q.shape[0], len(self.n), self.Hq, self.Hkv, self.D, self.max_q,
                                           self.max_context)

    def reference(self):
        """(out, A, N, spread * L * max|V|) in 64 bits, rows of no sequence NaN."""
        G = self.Hq // self.Hkv
        out = torch.full(self.q.shape, float("nan"), dtype=torch.float64, device="cuda")
        size, reach, floor = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out)
        for b in range(len(self.n)):
            n, m, first = self.n[b], self.m[b], int(self.cu[b])
            if n == 0:
                continue
            pos = torch.arange(m, device="cuda")
            blk = self.tables[b].long()[pos // self.bs]
            there = blk >= 0
            dec = lambda c, s: (c[blk.clamp(min=0), pos % self.bs].view(torch.float8_e4m3fn).double()  # noqa: E731
                                * s[blk.clamp(min=0), pos % self.bs].double()[..., None])
            K, V = dec(self.kc, self.ks), dec(self.vc, self.vs)
            see = (pos[None] <= m - n + torch.arange(n, device="cuda")[:, None]) & there[None]
            rows = slice(first, first + n)
            for h in range(self.Hkv):
                q = self.q[rows, h * G:(h + 1) * G].double()
                sel = lambda t: torch.where(there[:, None], t[:, h], torch.zeros_like(t[:, h]))  # noqa: E731
                k, v = sel(K), sel(V)
                z = torch.einsum("igd,ld->igl", q, k) * self.scale
                z = z.masked_fill(~see[:, None], float("-inf"))
                p = torch.softmax(z, -1).nan_to_num(0.0)
                out[rows, h * G:(h + 1) * G] = torch.einsum("igl,ld->igd", p, v)
                size[rows, h * G:(h + 1) * G] = torch.einsum("igl,ld->igd", p, v.abs())
                near = torch.einsum("igd,ld->igl", q.abs(), k.abs()) * self.scale
                reach[rows, h * G:(h + 1) * G] = (near * see[:, None]).amax(-1, keepdim=True) if m else 0.0
                if m:
                    s = self.vs[blk.clamp(min=0), pos % self.bs][:, h][there]
                    spread = float(s.max() / s.min()) if s.numel() else 1.0
                    floor[rows, h * G:(h + 1) * G] = m * v.abs().amax() * spread
        return out, size, reach, floor

    def check(self, got):
        out, size, reach, floor = self.reference()
        real = ~out.isnan()
        bound = 2.0 ** -8 * out.abs() + (2 * reach * 2.0 ** -11 + 3 * 2.0 ** -11 + 2.0 ** -18) * size * (1 + 2.0 ** -8) \
            + floor * 2.0 ** -25 + 1e-30
        off = (got.double() - out).abs()
        bad = real & ~(off <= bound)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, by up to "
                               f"{float((off / bound)[real].nan_to_num(1e9).max()):.3g} of the bound")
        # and as a whole: rms error within 2^-9 of the outputs' (bf16's rounding has 2^-9 / sqrt(3) or less)
        if real.any() and float(out[real].square().sum()) > 0:
            assert float(off[real].square().mean().sqrt()) <= 2.0 ** -8 * float(out[real].square().mean().sqrt())


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 1, 128, 16), (2, 2, 64, 8), (64, 8, 128, 16), (12, 12, 64, 24), (7, 1, 128, 9),
                                         (32, 2, 64, 48), (5, 1, 128, 64), (48, 3, 128, 16)])
@pytest.mark.parametrize("n,m", [
    ([1], [1]), ([2], [2]), ([1], [300]), ([16], [16]), ([17], [129]), ([32], [256]), ([33], [257]), ([40], [1000]),
    ([128], [128]), ([129], [385]), ([300], [300]), ([1, 5, 130], [1, 128, 700]), ([257, 3], [1030, 64]),
])
def test_lengths(ptpc, n, m, Hq, Hkv, D, bs):
    c = Case(n, m, Hq, Hkv, D, bs, seed=sum(n) + sum(m) + Hq)
    c.check(c.run(ptpc))


def test_prompts_of_many_lengths(ptpc):
    n = [1, 700, 64, 3, 1500, 127, 129, 255, 500]
    c = Case(n, n, 32, 8, 128, 16, seed=5)
    assert c.splits(ptpc) == 1
    c.check(c.run(ptpc))


def test_many_sequences(ptpc):
    """More sequences than a warp's lanes, most of them one token."""
    g = torch.Generator().manual_seed(3)
    n = [1 if i % 3 else int(torch.randint(1, 90, (1,), generator=g)) for i in range(77)]
    m = [x + int(torch.randint(0, 300, (1,), generator=g)) for x in n]
    c = Case(n, m, 16, 2, 128, 16, seed=6)
    c.check(c.run(ptpc))


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(64, 8, 128, 16), (32, 2, 64, 24), (4, 4, 128, 8), (28, 4, 128, 32)])
@pytest.mark.parametrize("n,m", [([1], [5000]), ([7], [9000]), ([20], [4097]), ([5, 3, 1, 4], [3000, 777, 2, 2049])])
def test_split_contexts(ptpc, n, m, Hq, Hkv, D, bs):
    c = Case(n, m, Hq, Hkv, D, bs, seed=sum(m))
    assert c.splits(ptpc) > 1
    c.check(c.run(ptpc))


@pytest.mark.parametrize("n,m", [([5, 4, 3], [3, 0, 3]), ([40, 1], [7, 0]), ([300, 2], [100, 5000]), ([0, 6, 0], [50, 60, 0])])
def test_rows_that_see_nothing_and_empty_sequences(ptpc, n, m):
    """More new tokens than positions: the first ones see nothing and get 0;
    contexts of no position; sequences of no token."""
    c = Case(n, m, 16, 2, 128, 16, seed=9)
    got = c.run(ptpc)
    c.check(got)
    for b in range(len(n)):
        first = int(c.cu[b])
        none = max(0, n[b] - m[b])
        assert (got[first:first + none] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [([40], [300]), ([2], [4000])])
def test_missing_blocks(ptpc, n, m, D):
    """Entries that are negative or past the cache: their positions are left
    out; a table of nothing else gives 0."""
    c = Case(n, m, 8, 2, D, 16, seed=11)
    c.tables[0, 1] = -1
    c.tables[0, 3:9] = -7
    c.check(c.run(ptpc))
    far = c.tables.clone()
    far[far < 0] = c.kc.shape[0] + 5
    same = c.run(ptpc).clone()
    c.tables = far
    assert torch.equal(c.run(ptpc), same)
    c.tables = torch.full_like(far, 2 ** 31 - 1)
    assert (c.run(ptpc) == 0).all()


def test_table_shorter_than_the_context(ptpc):
    c = Case([20], [500], 8, 2, 128, 16, seed=12)
    whole = c.tables
    c.tables = whole.clone()
    c.tables[0, 20:] = -1
    want = c.run(ptpc).clone()
    c.tables = whole[:, :20].contiguous()
    assert torch.equal(c.run(ptpc), want)


@pytest.mark.parametrize("n,m", [([6, 50], [200, 90]), ([3, 2], [3000, 4000])])
def test_strided_queries_and_padded_rows(ptpc, n, m):
    """q as a slice of a wider projection; rows in front of the first sequence
    and behind the last are left as they were, whatever they hold."""
    c = Case(n, m, 16, 2, 128, 16, seed=13, pad=40, before=3, behind=70)
    with torch.no_grad():
        c.q[:3], c.q[-70:] = float("nan"), float("inf")
    out = torch.full(c.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(ptpc, out=out)
    assert (got[:3] == 5).all() and (got[-70:] == 5).all()
    c.check(got)


@pytest.mark.parametrize("q_size,v_spread", [(1e-20, 0.5), (30.0, 0.5), (1.0, 3.0), (4.0, 0.0)])
def test_sizes_of_queries_and_values(ptpc, q_size, v_spread):
    """Flat and peaked softmaxes; value scales far apart."""
    c = Case([33, 2], [700, 3000], 16, 2, 128, 16, seed=14, q_size=q_size, v_spread=v_spread)
    c.check(c.run(ptpc))


def test_query_range(ptpc):
    """Queries near bf16's largest and among its subnormals, with a softmax
    scale that keeps the scores in range."""
    for size in (1e-39, 1e-30, 1e20, 1e37):
        c = Case([9], [200], 8, 2, 128, 16, seed=15, q_size=size)
        c.scale = float(min(1.0, 1.0 / (size * math.sqrt(c.D))))
        c.check(c.run(ptpc))


def test_growing_scores(ptpc):
    """Keys that grow along the context: the running maximum moves in every tile."""
    c = Case([40, 2], [1500, 3000], 16, 2, 128, 16, seed=16)
    for b, m in enumerate(c.m):
        for i in range((m + 15) // 16):
            c.ks[c.tables[b, i].long()] *= 1.0 + i / 20.0
    c.check(c.run(ptpc))


def test_zero_values_beside_small_ones(ptpc):
    """Zero value vectors (scale 1, codes 0) among small ones: they weigh in the
    sum and must not push the small ones out of f16's range."""
    c = Case([20], [640], 8, 1, 128, 16, seed=17, v_spread=0.0)
    c.vs *= 1e-3
    blk = c.tables[0, ::5].long()
    c.vc[blk], c.vs[blk] = 0, 1.0
    out, size, reach, floor = c.reference()
    off = (c.run(ptpc).double() - out).abs()
    # the zero vectors' unit is 2^k >= 1 where the others' scale is near 2e-5: floor counts the spread (5e4)
    assert (off <= 2.0 ** -8 * out.abs() + (2 * reach + 4) * 2.0 ** -11 * size + 640 * 2.0 ** -25 * 1e-2).all()


def test_bad_values_in_places_that_a_row_does_not_see(ptpc):
    """NaN codes, infinite and NaN scales of a later token reach no earlier
    row; the rows that see them have NaN.  Behind the context anything goes."""
    for D, G in ((128, 4), (64, 1), (128, 16)):
        c = Case([150], [400], 2 * G, 2, D, 16, seed=18)
        clean = c.run(ptpc).clone()
        at = 300                                   # token 50 of the 150 is the first to see it
        blk, off = int(c.tables[0, at // 16]), at % 16
        for what in ("v code", "v scale inf", "v scale nan", "k scale nan", "k code"):
            kc, vc, ks, vs = c.kc.clone(), c.vc.clone(), c.ks.clone(), c.vs.clone()
            if what == "v code":
                c.vc[blk, off, :, 5] = 0x7F
            elif what == "k code":
                c.kc[blk, off, :, 7] = 0xFF
            elif what.startswith("v scale"):
                c.vs[blk, off] = float(what.split()[2])
            else:
                c.ks[blk, off] = float("nan")
            got = c.run(ptpc)
            if "code" in what:
                assert torch.equal(got[:50], clean[:50]), what
            else:    # the 32 positions' reference may be another one now: other roundings
                far = (got[:50].double() - clean[:50].double()).abs()
                assert (far <= 2.0 ** -7 * clean[:50].double().abs() + 2.0 ** -8 * clean.double().square().mean().sqrt()).all(), what
            if what in ("v code", "v scale nan", "k code", "k scale nan"):
                assert got[50:, :].isnan().any(-1).all(), what
            c.kc, c.vc, c.ks, c.vs = kc, vc, ks, vs
        last = int(c.tables[0, 24])                # positions 384..399 of 400 are its; it is full
        spare = [i for i in range(c.kc.shape[0]) if i not in c.tables[0].tolist()]
        c.vc[spare], c.kc[spare] = 0x7F, 0x7F
        c.m = [395]
        c.ctx.fill_(395)
        c.n, c.cu = [145], torch.tensor([0, 145], dtype=torch.int32, device="cuda")
        c.q, c.max_q = c.q[:145], 145
        want = c.run(ptpc).clone()
        c.vc[last, 11:], c.kc[last, 11:], c.vs[last, 11:], c.ks[last, 11:] = 0x7F, 0x7F, float("inf"), float("nan")
        assert torch.equal(c.run(ptpc), want)


def test_one_token_as_decode_attention_gives_it(ptpc):
    """Chunks of one token: what decode_attention computes, within both kernels' roundings."""
    c = Case([1, 1, 1, 1], [5, 130, 1000, 2500], 64, 8, 128, 16, seed=19)
    got = c.run(ptpc)
    c.check(got)
    dec = ptpc.decode_attention(c.q.contiguous(), c.kc, c.vc, c.ks, c.vs, c.tables, c.ctx, c.max_context, c.scale)
    rms = dec.double().square().mean().sqrt()
    assert ((got.double() - dec.double()).abs() <= 2e-2 * dec.double().abs() + 2e-3 * rms).all()


def test_chunks_of_a_prompt_as_the_prompt(ptpc):
    """A prompt in one call and in chunks: each row within the roundings (the
    tiles are the same; only the plan of the split may differ)."""
    whole = Case([600], [600], 32, 4, 128, 16, seed=20)
    want = whole.run(ptpc).clone()
    for a, b in ((0, 250), (250, 251), (251, 600)):
        part = Case([b - a], [b], 32, 4, 128, 16, seed=20)
        part.kc, part.vc, part.ks, part.vs, part.tables = whole.kc, whole.vc, whole.ks, whole.vs, whole.tables
        part.q = whole.q[a:b]
        got = part.run(ptpc)
        rms = want.double().square().mean().sqrt()
        assert ((got.double() - want[a:b].double()).abs() <= 2e-2 * want[a:b].double().abs() + 2e-3 * rms).all()


def test_same_call_twice_and_two_streams(ptpc):
    a = Case([100, 3], [900, 5000], 32, 4, 128, 16, seed=21)
    b = Case([5], [6000], 64, 8, 128, 16, seed=22)
    one, two = a.run(ptpc).clone(), b.run(ptpc).clone()
    assert torch.equal(a.run(ptpc), one)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((one, ptpc.chunk_attention(a.q, a.kc, a.vc, a.ks, a.vs, a.tables, a.ctx, a.cu, a.max_q,
                                                  a.max_context, a.scale)))
        with torch.cuda.stream(s2):
            got.append((two, ptpc.chunk_attention(b.q, b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx, b.cu, b.max_q,
                                                  b.max_context, b.scale)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


def test_two_captured_graphs(ptpc):
    """Two graphs captured on one stream, replayed at once on two others: each
    has a workspace of its own."""
    cases = [Case([4], [4000], 64, 8, 128, 16, seed=s) for s in (23, 24)]
    want = [c.run(ptpc).clone() for c in cases]
    assert all(c.splits(ptpc) > 1 for c in cases)
    graphs, outs = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ptpc.chunk_attention(c.q, c.kc, c.vc, c.ks, c.vs, c.tables, c.ctx, c.cu, c.max_q,
                                             c.max_context, c.scale))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a replay follows the contexts that the device holds then
    cases[0].ctx.fill_(1000)
    cases[0].m = [1000]
    graphs[0].replay()
    cases[0].check(outs[0])


def test_long_cache_offsets(ptpc):
    """Slots whose byte offsets pass 2^32: a cache of 4.5 GB, tables at its end."""
    Hkv, D, bs, nb = 8, 128, 16, 275000
    free = torch.cuda.mem_get_info()[0]
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    c = Case([17], [600], 64, Hkv, D, bs, seed=25)
    want = c.run(ptpc).clone()
    big = {}
    for name in ("kc", "vc"):
        t = torch.zeros((nb, bs, Hkv, D), dtype=torch.uint8, device="cuda")
        t[-c.kc.shape[0]:] = getattr(c, name)
        big[name] = t
    for name in ("ks", "vs"):
        t = torch.ones((nb, bs, Hkv), device="cuda")
        t[-c.kc.shape[0]:] = getattr(c, name)
        big[name] = t
    c.tables = torch.where(c.tables >= 0, c.tables + (nb - c.kc.shape[0]), c.tables)
    c.kc, c.vc, c.ks, c.vs = big["kc"], big["vc"], big["ks"], big["vs"]
    assert torch.equal(c.run(ptpc), want)
