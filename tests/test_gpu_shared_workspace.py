"""Entry points that share a workspace on one stream, as the default workspace
of a serving step does: data that one keeps there (quantised activations,
partial results of attention) must not reach another's counters.  Outputs are
compared bit for bit with those of a workspace of the call's own."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, CI, CO = 2048, 16384, 8192     # its last wave of tiles is split along K


@pytest.fixture(scope="module")
def ptpc():
    import fp8_quantized_gemm_ptpc_b200 as p
    return p


@pytest.fixture(scope="module")
def layer(ptpc):
    assert ptpc.gemm_tail_split(T, CI, CO) >= 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, CI, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(CI, CO, generator=g, device="cuda") / CI ** 0.5).to(torch.bfloat16)
    return x, ptpc.quantize_weights(w)


def attention(ptpc):
    """A call whose contexts are split over CTAs, so that partial results are kept."""
    Hq, Hkv, D, bs, m = 8, 1, 128, 16, 8192
    assert ptpc.chunk_attention_splits(4, 1, Hq, Hkv, D, 4, m) > 1
    g = torch.Generator(device="cuda").manual_seed(2)
    cache = [torch.randint(0, 120, (m // bs, bs, Hkv, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand(m // bs, bs, Hkv, generator=g, device="cuda") + 0.5 for _ in range(2)]
    tables = torch.arange(m // bs, dtype=torch.int32, device="cuda").view(1, -1)
    ctx = torch.tensor([m], dtype=torch.int32, device="cuda")
    q = torch.randn(4, Hq, D, generator=g, device="cuda").to(torch.bfloat16)

    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")

    def chunk(ws):
        return ptpc.chunk_attention(q, *cache, *scales, tables, ctx, cu, 4, m, 0.01, ws=ws)

    def decode(ws):
        return ptpc.decode_attention(q[:1], *cache, *scales, tables, ctx, m, 0.01, ws=ws)

    return chunk, decode


def test_calls_of_a_serving_step_in_one_workspace(ptpc, layer):
    x, w = layer
    chunk, decode = attention(ptpc)
    calls = [lambda ws: ptpc.linear(x, *w, ws=ws), lambda ws: ptpc.linear(x[:8], *w, ws=ws), chunk, decode,
             lambda ws: ptpc.scaled_mm(*ptpc.quantize_activations(x), *w, ws=ws)]
    want = [c(ptpc.Workspace(256, "cuda")) for c in calls]
    one = ptpc.Workspace(ptpc.workspace_size(ptpc.OP_LINEAR, T, CI, CO), "cuda")
    for order in ((0, 1, 4), (2, 4, 0), (3, 0, 2), (1, 2, 3, 4, 0, 1)):
        for i in order:
            assert torch.equal(calls[i](one), want[i]), (order, i)
    for i in (0, 2, 4, 1, 0, 3, 4):                       # and in the stream's default one
        assert torch.equal(calls[i](None), want[i]), i
    assert ptpc.device_status(one) == 0


def test_split_tail_captured_behind_other_data(ptpc, layer):
    x, w = layer
    chunk, _ = attention(ptpc)
    want = ptpc.linear(x, *w, ws=ptpc.Workspace(256, "cuda"))
    ws = ptpc.Workspace(ptpc.workspace_size(ptpc.OP_LINEAR, T, CI, CO), "cuda")
    chunk(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ptpc.linear(x, *w, ws=ws)
        chunk(ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk(ws)
        got = ptpc.linear(x, *w, ws=ws)
        chunk(ws)
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)
    assert ptpc.device_status(ws) == 0


def test_nothing_but_the_status_word_need_be_zero(ptpc, layer):
    """Every entry point that takes a workspace, with all of it but the first
    256 bytes holding ones before each call."""
    x, w = layer
    chunk, decode = attention(ptpc)
    wide = x[:, :1024].contiguous()
    raw = (torch.arange(1024 * 512, device="cuda").view(1024, 512) % 251 / 64 - 1).to(torch.bfloat16)
    w4 = ptpc.quantize_weights_fmt(raw, "e2m1")
    calls = [lambda ws: ptpc.linear(x, *w, ws=ws), lambda ws: ptpc.linear(x[:8], *w, ws=ws), chunk, decode,
             lambda ws: ptpc.scaled_mm(*ptpc.quantize_activations(x), *w, ws=ws),
             lambda ws: torch.cat([t.flatten().float() for t in ptpc.quantize_weights(raw, ws=ws)]),
             lambda ws: torch.cat([t.flatten().float() for t in ptpc.quantize_weights_fmt(raw, "e2m1", ws=ws)]),
             lambda ws: ptpc.linear_fmt(wide, *w4, "e2m1", ws=ws)]
    want = [c(ptpc.Workspace(256, "cuda")) for c in calls]
    ws = ptpc.Workspace(ptpc.workspace_size(ptpc.OP_LINEAR, T, CI, CO), "cuda")
    for i, c in enumerate(calls):
        ws.buf[256:] = 255
        assert torch.equal(c(ws), want[i]), i
        assert ptpc.device_status(ws) == 0
