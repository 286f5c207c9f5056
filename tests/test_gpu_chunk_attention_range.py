"""Causal attention of new tokens over the FP8 paged cache where the scales of
keys or values lie far apart: zero vectors (scale 1, codes 0) among small ones,
neighbours 2^24 or more apart, large vectors of later tokens that a row does not
see.  Against the formula in 64 bits, row by row.

Tolerance of an output, with p, V the exact weights and values, s the value
scales, c the codes' values, N_l = softmax_scale sum |q k_l|, sums over the
positions that the row sees:
  - a score is off by 2^-11 N_l (the key's rounding to f16) and D 2^-24 N_l, a
    weight by that relatively, in numerator and denominator:
    (2^-11 + D 2^-24) (sum p N |V| + |out| sum p N);
  - a weight is rounded to f16, a value too: 2 * 2^-11 sum p |V|;
  - a weight P' below f16's normal numbers, 2^-14, is off by half a step, 2^-25,
    of its reference 2^r.  A value is |c| * 64 or less in the products.  2^r is at
    most 2^7 max(p s 2^-6), or 2^-88 max p: scales share a reference where they lie
    within 2^6 of one another, it is less than twice the largest, and vectors
    without a scale count with 2^-88.  So only positions with p s < 2^-7 max(p s)
    can be below 2^-14, each off by 2^-25 2^r |c| 64;
  - exponentials and sums in fp32, their arguments below 2^7: 2^-16 sum p |V|;
  - the output's rounding to bf16: 2^-8 of it."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


class Cache:
    """One sequence of m positions and its n newest tokens' queries.  Keys are
    small and random, values of one sign, so that an output is of the size of
    its terms; scales are set by position."""

    def __init__(self, n, m, Hq=8, Hkv=2, D=128, bs=16, seed=0, q_noise=0.05):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.n, self.m, self.Hq, self.Hkv, self.D, self.bs = n, m, Hq, Hkv, D, bs
        # all queries point along one direction, so that a key along it scores the same for every row
        self.q = (1.0 + q_noise * rand(n, Hq, D)).to(torch.bfloat16)
        self.kv = (rand(m, Hkv, D) * 32).to(torch.float8_e4m3fn)                # codes' values
        self.vv = (rand(m, Hkv, D).abs() * 64 + 64).clamp(max=448).to(torch.float8_e4m3fn)
        self.ks = torch.full((m, Hkv), 2.0 ** -9, device="cuda")
        self.vs = torch.full((m, Hkv), 2.0 ** -8, device="cuda")
        self.scale = 1.0 / math.sqrt(D)
        self.blocks = (m + bs - 1) // bs
        self.table = torch.randperm(self.blocks + 3, generator=g, device="cuda")[:self.blocks].to(torch.int32)

    def at(self, *ranges):
        pick = torch.zeros(self.m, dtype=torch.bool, device="cuda")
        for a, b in ranges:
            pick[a:b] = True
        return pick

    def zero_values(self, pick):
        self.vv[pick], self.vs[pick] = torch.zeros((), device="cuda").to(torch.float8_e4m3fn), 1.0

    def zero_keys(self, pick):
        self.kv[pick], self.ks[pick] = torch.zeros((), device="cuda").to(torch.float8_e4m3fn), 1.0

    def score(self, pick, nats):
        """Keys along the queries: they score `nats` above the others' mean."""
        self.kv[pick] = torch.ones((), device="cuda").to(torch.float8_e4m3fn)
        self.ks[pick] = nats / math.sqrt(self.D)

    def run(self, ptpc):
        bs, slots = self.bs, self.blocks + 3
        at = torch.arange(self.m, device="cuda")
        where = self.table.long()[at // bs] * bs + at % bs
        tensors = []
        for x, fill in ((self.kv.view(torch.uint8), 0x7F), (self.vv.view(torch.uint8), 0x7F), (self.ks, float("nan")),
                        (self.vs, float("inf"))):
            t = torch.full((slots * bs,) + x.shape[1:], fill, dtype=x.dtype, device="cuda")
            t[where] = x
            tensors.append(t.view(slots, bs, *x.shape[1:]))
        ws = ptpc.Workspace(ptpc.lib.ptpc_chunk_attention_workspace_size(self.n, 1, self.Hq, self.Hkv, self.D, self.n,
                                                                         self.m), "cuda")
        out = ptpc.chunk_attention(self.q, *tensors, self.table[None], torch.tensor([self.m], dtype=torch.int32, device="cuda"),
                                   torch.tensor([0, self.n], dtype=torch.int32, device="cuda"), self.n, self.m, self.scale,
                                   ws=ws)
        assert ptpc.device_status(ws) == 0
        return out

    def splits(self, ptpc):
        return ptpc.chunk_attention_splits(self.n, 1, self.Hq, self.Hkv, self.D, self.n, self.m)

    def reference(self):
        """(out, bound), 64 bits."""
        n, m, G = self.n, self.m, self.Hq // self.Hkv
        out = torch.zeros(n, self.Hq, self.D, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        hidden = torch.arange(m, device="cuda")[None] > torch.arange(m - n, m, device="cuda")[:, None]
        for h in range(self.Hq):
            q, c, s = self.q[:, h].double(), self.vv[:, h // G].double(), self.vs[:, h // G].double()
            k = self.kv[:, h // G].double() * self.ks[:, h // G].double()[:, None]
            v = c * s[:, None]
            # hidden positions hold anything, large values too: they are left out of the sums, not multiplied by 0
            z = (q @ k.T * self.scale).masked_fill(hidden, float("-inf"))
            p = torch.softmax(z, -1)
            reach = (q.abs() @ k.abs().T * self.scale).masked_fill(hidden, 0.0)
            o, size = p @ v, p @ v.abs()
            key = (2.0 ** -11 + self.D * 2.0 ** -24) * ((p * reach) @ v.abs() + o.abs() * (p * reach).sum(-1, keepdim=True))
            ps = p * torch.where((c == 0).all(-1), torch.zeros_like(s), s)
            top = torch.maximum(2 * ps.amax(-1), 2.0 ** -88 * p.amax(-1))[:, None]
            floor = 2.0 ** -25 * top * 64 * ((ps < 2.0 ** -7 * ps.amax(-1, keepdim=True)) & ~hidden).double() @ c.abs()
            out[:, h] = o
            bound[:, h] = 2.0 ** -8 * o.abs() + (key + (2 * 2.0 ** -11 + 2.0 ** -16) * size + floor) * (1 + 2.0 ** -7)
        return out, bound

    def check(self, ptpc):
        got = self.run(ptpc).double()
        out, bound = self.reference()
        off = (got - out).abs()
        bad = ~(off <= bound)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, by up to "
                               f"{float((off / (bound + 1e-300)).nan_to_num(1e9).max()):.3g} of the bound")


SHAPES = [dict(n=20, m=640), dict(n=20, m=640, D=64, Hkv=1), dict(n=150, m=500, Hq=16), dict(n=2, m=4000),
          dict(n=2, m=4000, D=64, bs=24), dict(n=1, m=700, Hq=4, Hkv=4)]
IDS = ["20 on 640", "20 on 640, D 64", "two streams", "split", "split, D 64", "one token"]


def test_the_shapes_cover_split_and_whole_contexts(ptpc):
    got = [Cache(**s).splits(ptpc) for s in SHAPES]
    assert min(got) == 1 and max(got) > 1


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("size", [1.0, 0.03, 1e-3, 3e4])
@pytest.mark.parametrize("nats", [0.0, 5.0, 10.0, 20.0])
@pytest.mark.parametrize("where", ["first", "middle", "end", "odd"])
def test_zero_values_in_whole_groups(ptpc, where, nats, size, shape):
    """32 neighbouring positions, or 64, without a value: they weigh in the sum
    alone, whatever they score and however small the values beside them."""
    c = Cache(**shape, seed=1)
    m = c.m
    pick = c.at(*{"first": [(0, 64)], "middle": [(256, 288), (320, 384)], "end": [(m - m % 32 - 32, m)],
                  "odd": [(100, 180)]}[where])
    c.vs *= size
    c.zero_values(pick)
    if nats:
        c.score(pick, nats)
    c.check(ptpc)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("size", [1.0, 1e-3])
def test_zero_values_between_others(ptpc, size, shape):
    """Single zero vectors that score far above their neighbours, and all but one zero."""
    c = Cache(**shape, seed=2)
    pick = c.at((37, 38), (70, 71), (c.m // 2, c.m // 2 + 1))
    c.vs *= size
    c.zero_values(pick)
    c.score(pick, 12.0)
    c.check(ptpc)
    c.zero_values(~c.at((70, 71)))
    c.check(ptpc)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_no_value_at_all(ptpc, shape):
    c = Cache(**shape, seed=3)
    c.zero_values(c.at((0, c.m)))
    assert (c.run(ptpc) == 0).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("apart", [7, 8, 20, 24, 30, 60])
def test_value_scales_far_apart(ptpc, apart, shape):
    """One vector in 32 is 2^apart times the others and scores as much lower, so
    that large and small ones count alike in the outputs."""
    c = Cache(**shape, seed=4)
    big = c.at(*[(i, i + 1) for i in range(5, c.m, 32)])
    c.vs[big] *= 2.0 ** apart
    c.score(big, -apart * math.log(2.0))
    c.check(ptpc)


@pytest.mark.parametrize("shape", SHAPES[:5] + [dict(n=30, m=32), dict(n=64, m=64, D=64)], ids=IDS[:5] + ["32", "64, D 64"])
@pytest.mark.parametrize("what", ["values", "keys", "both"])
@pytest.mark.parametrize("apart", [24, 40])
def test_large_vectors_of_later_tokens(ptpc, apart, what, shape):
    """The newest token's vectors are 2^apart times the others': rows that do
    not see it have what they had without it."""
    c = Cache(**shape, seed=5, q_noise=0.5)
    if what != "keys":
        c.vs[-1] *= 2.0 ** apart
    if what != "values":
        c.ks[-1] *= 2.0 ** apart
    got = c.run(ptpc)[:-1].double()
    out, bound = c.reference()
    off = (got - out[:-1]).abs()
    assert (off <= bound[:-1]).all(), float((off / bound[:-1]).max())


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("size", [2.0 ** -8, 2.0 ** -14, 2.0 ** -24])
def test_zero_keys_beside_small_ones(ptpc, size, shape):
    """A zero key has scale 1; small keys beside it, with queries that make up for them, keep their bits."""
    c = Cache(**shape, seed=6, q_noise=0.5)
    c.ks *= size
    c.scale = float(c.scale / size)
    c.zero_keys(c.at((33, 35), (128, 160), (c.m - 3, c.m - 2)))
    c.check(ptpc)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_random_scales(ptpc, shape):
    """Scales of keys and of values over some 2^17 and 2^35, in every group of 32."""
    c = Cache(**shape, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda t: torch.randn(t.shape, generator=g, device="cuda")  # noqa: E731
    c.vs *= torch.exp(4.0 * rand(c.vs))
    c.ks *= torch.exp(2.0 * rand(c.ks))
    c.check(ptpc)
    c.vs = c.vs.sort(0).values                  # growing, and falling, along the context
    c.check(ptpc)
    c.vs = c.vs.flip(0).contiguous()
    c.check(ptpc)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("size", [2.0 ** -84, 2.0 ** -66, 2.0 ** 90])
def test_the_ends_of_the_range(ptpc, size, shape):
    """Value scales near 2^-92 and 2^82, zero vectors that score above them."""
    c = Cache(**shape, seed=9)
    c.vs *= size
    c.check(ptpc)
    pick = c.at((10, 12), (96, 130))
    c.zero_values(pick)
    c.score(pick, 3.0)
    c.check(ptpc)


def test_same_bits_again(ptpc):
    for shape in (SHAPES[2], SHAPES[3]):
        c = Cache(**shape, seed=10)
        c.zero_values(c.at((0, 64), (100, 101)))
        c.vs[200:230] *= 2.0 ** 20
        one = c.run(ptpc)
        assert torch.equal(c.run(ptpc), one)
