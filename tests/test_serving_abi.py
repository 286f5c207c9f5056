"""The C entry points around a block of a served model (the norms with the
residual add, the rotary append, attention of new tokens over the cache)
reject what they do not take before they touch the GPU, and their queries
answer without one (runs without a GPU)."""
import ctypes
import math

import pytest

from test_abi import FAKE, ptpc  # noqa: F401  (the fixture builds the library)

P = ctypes.c_void_p
INF, NAN = math.inf, math.nan


class Call:
    """An entry point with arguments it would take, to be changed one at a time."""

    def __init__(self, ptpc, name, **args):  # noqa: F811
        self.fn, self.args = getattr(ptpc.lib, name), args

    def __call__(self, **change):
        unknown = set(change) - set(self.args)
        assert not unknown, unknown
        return self.fn(*{**self.args, **change}.values())


def norm(ptpc, quant):  # noqa: F811
    out = dict(Xq=FAKE, x_scale=FAKE) if quant else dict(x=FAKE)
    return Call(ptpc, "ptpc_residual_norm_quantize" if quant else "ptpc_residual_norm", y=FAKE, ldy=64, residual=FAKE,
                ldr=64, gate=FAKE, ldg=0, post_w=FAKE, pre_w=FAKE, T=4, C=64, eps=1e-5, a=1.0, h=FAKE, ldh=64, **out,
                stream=None)


@pytest.mark.parametrize("quant", [False, True])
def test_norm_refusals(ptpc, quant):  # noqa: F811
    call = norm(ptpc, quant)
    bad, shape, misaligned = ptpc.ERR_INVALID_ARG, ptpc.ERR_UNSUPPORTED_SHAPE, ptpc.ERR_MISALIGNED
    assert call(T=-1) == bad and call(C=-16) == bad
    assert call(C=0) == shape and call(C=72) == shape and call(C=2 ** 40) == shape and call(T=2 ** 40) == shape
    for eps in (0.0, -1e-5, INF, NAN):
        assert call(eps=eps) == bad
    for a in (INF, -INF, NAN):
        assert call(a=a) == bad
    for name in ("residual", "pre_w") + (("Xq", "x_scale") if quant else ("x",)):
        assert call(**{name: None}) == bad, name
    assert call(y=None) == bad                                   # a norm and a gate of nothing
    assert call(y=None, gate=None) == bad and call(y=None, post_w=None) == bad
    for ld in ("ldy", "ldr", "ldh"):
        assert call(**{ld: 56}) == bad and call(**{ld: 68}) == misaligned, ld
    assert call(ldg=56) == bad and call(ldg=68) == misaligned
    assert call(ldh=128) == bad                                  # in place at another pitch
    for name in ("y", "residual", "gate", "post_w", "pre_w", "h") + (("Xq", "x_scale") if quant else ("x",)):
        assert call(**{name: FAKE + 8}) == misaligned, name
    assert call(T=0, residual=None) == ptpc.OK                   # nothing to do


def test_append_refusals(ptpc):  # noqa: F811
    call = Call(ptpc, "ptpc_rope_kv_cache_append", Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, cos_sin=FAKE,
                max_position=1000, rotary_dim=64, interleaved=0, positions=FAKE, slots=FAKE, T=5, Hq=4, Hkv=2, D=128,
                block_size=16, num_blocks=8, Q_out=FAKE + 0x100000, ldo=512, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE,
                v_scale=FAKE, stream=None)
    bad, shape, misaligned = ptpc.ERR_INVALID_ARG, ptpc.ERR_UNSUPPORTED_SHAPE, ptpc.ERR_MISALIGNED
    for change in (dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(D=0), dict(block_size=0), dict(num_blocks=0),
                   dict(max_position=0), dict(rotary_dim=0), dict(ldq=504), dict(ldk=248), dict(ldv=248), dict(ldo=504),
                   dict(Q_out=FAKE, ldo=520)):
        assert call(**change) == bad, change
    for change in (dict(D=96, rotary_dim=32), dict(D=256), dict(block_size=4), dict(block_size=131072), dict(Hkv=2048),
                   dict(Hq=32768), dict(rotary_dim=24), dict(rotary_dim=144), dict(T=2 ** 40), dict(max_position=2 ** 40),
                   dict(num_blocks=2 ** 40), dict(num_blocks=2 ** 30, block_size=64)):
        assert call(**change) == shape, change
    for name in ("Q", "K", "V", "cos_sin", "positions", "slots", "Q_out", "k_cache", "v_cache", "k_scale", "v_scale"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 2}) == misaligned, name
    for change in (dict(ldq=516), dict(ldk=260), dict(ldv=260), dict(ldo=516)):
        assert call(**change) == misaligned, change
    assert call(T=0, K=None) == ptpc.OK


def test_chunk_attention_refusals(ptpc):  # noqa: F811
    sizes = dict(total_q=100, B=3, Hq=32, Hkv=8, D=128, max_q=64, max_context=5000)
    need = ptpc.lib.ptpc_chunk_attention_workspace_size(*sizes.values())
    assert need >= 256 and need % 256 == 0
    call = Call(ptpc, "ptpc_chunk_attention", q=FAKE, ldq=4096, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE,
                block_tables=FAKE, context_lens=FAKE, cu_q=FAKE, total_q=100, B=3, max_q=64, Hq=32, Hkv=8, D=128,
                block_size=16, num_blocks=1000, max_blocks=320, max_context=5000, softmax_scale=0.09, out=FAKE, ws=FAKE,
                ws_bytes=need, stream=None)
    bad, shape, misaligned = ptpc.ERR_INVALID_ARG, ptpc.ERR_UNSUPPORTED_SHAPE, ptpc.ERR_MISALIGNED
    for change in (dict(total_q=-1), dict(B=-1), dict(max_q=-1), dict(max_context=-1), dict(Hq=0), dict(Hkv=0), dict(D=0),
                   dict(block_size=0), dict(num_blocks=0), dict(max_blocks=0), dict(softmax_scale=0.0),
                   dict(softmax_scale=-1.0), dict(softmax_scale=INF), dict(softmax_scale=NAN), dict(ldq=4088)):
        assert call(**change) == bad, change
    for change in (dict(D=96), dict(Hq=33), dict(Hkv=2048, Hq=4096), dict(Hq=32768), dict(block_size=4), dict(B=65536),
                   dict(total_q=2 ** 40), dict(max_q=2 ** 40), dict(max_context=2 ** 40), dict(num_blocks=2 ** 30),
                   dict(max_blocks=2 ** 30)):
        assert call(**change) == shape, change
    for name in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_tables", "context_lens", "cu_q", "out", "ws"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 2}) == misaligned, name
    assert call(ldq=4100) == misaligned
    assert call(ws_bytes=need - 1) == ptpc.ERR_WORKSPACE_TOO_SMALL
    for change in (dict(total_q=0), dict(B=0), dict(max_q=0)):
        assert call(**change, q=None) == ptpc.OK                # nothing to do


def test_chunk_attention_queries(ptpc):  # noqa: F811
    size, splits = ptpc.lib.ptpc_chunk_attention_workspace_size, ptpc.chunk_attention_splits
    assert size(0, 3, 32, 8, 128, 64, 5000) == 256 and size(100, 0, 32, 8, 128, 64, 5000) == 256
    for wrong in ((-1, 3, 32, 8, 128, 64, 5000), (100, 3, 33, 8, 128, 64, 5000), (100, 3, 32, 8, 96, 64, 5000),
                  (100, 3, 32, 8, 128, 64, -1), (100, 70000, 32, 8, 128, 64, 10)):
        assert size(*wrong) == 0 and splits(*wrong) == 0, wrong
    assert splits(0, 3, 32, 8, 128, 64, 5000) == 0
    # a context of a few tiles is never split, nor one whose rows fill the GPU
    assert splits(1, 1, 32, 8, 128, 1, 500) == 1 and splits(8192, 1, 64, 8, 128, 8192, 8192) == 1
    # one token on a long context is, and the partial results have room
    for D in (64, 128):
        s = splits(1, 1, 64, 8, D, 1, 100000)
        assert 1 < s <= 64
        assert size(1, 1, 64, 8, D, 1, 100000) >= 256 + s * 64 * (D + 2) * 4


def test_wrappers_refuse_tensors_of_the_cpu(ptpc):  # noqa: F811
    import torch
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ptpc.residual_norm(x, x, w)
    with pytest.raises(TypeError):
        ptpc.residual_norm_quantize(y=x, residual=x, pre_weight=w)
    h = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache, scale = torch.zeros(4, 16, 2, 64, dtype=torch.uint8), torch.zeros(4, 16, 2)
    i64, i32 = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        ptpc.rope_kv_cache_append(h, h[:, :2], h[:, :2], torch.zeros(8, 64), i64, i64, cache, cache, scale, scale)
    with pytest.raises(TypeError):
        ptpc.chunk_attention(h, cache, cache, scale, scale, i32[None], i32[:1], i32, 2, 16, 0.1)
