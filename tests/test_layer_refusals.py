"""What the 4-bit layer's calls refuse before anything is queued: wrong sizes and types in the binding, null
contexts in the library (CPU)."""
import pytest
import torch

from post_quantization_expert_b200 import clha as L


@pytest.fixture(scope="module", autouse=True)
def lib():
    from post_quantization_expert_b200 import build
    build.build()
    return L.load()


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


U8, I32, I64, BF16 = torch.uint8, torch.int32, torch.int64, torch.bfloat16


def test_scale_bytes():
    assert L.clha_fp4_scale_bytes(L.FP4_E8M0_32, 1, 128) == 512
    assert L.clha_fp4_scale_bytes(L.FP4_E4M3_16, 129, 256) == 2 * 4 * 512
    assert L.clha_fp4_scale_bytes(L.FP4_E4M3_16, 0, 256) == 0
    for bad in ((7, 1, 128), (L.FP4_E8M0_32, -1, 128), (L.FP4_E8M0_32, 1, 0), (L.FP4_E8M0_32, 1, 192)):
        assert L.clha_fp4_scale_bytes(*bad) == -1


def test_route_buffers():
    ok = dict(logits=t(4, 8), ids=t(4, 2, dtype=I32), weights=t(4, 2), counts=t(8, dtype=I32))

    def call(bias=None, **kw):
        a = {**ok, **kw}
        L.clha_route_gated(None, a["logits"], 4, 8, 2, a["ids"], a["weights"], a["counts"], bias=bias)
    for kw in (dict(logits=t(3, 8)), dict(ids=t(4, 1, dtype=I32)), dict(weights=t(4, 1)), dict(counts=t(7, dtype=I32)),
               dict(bias=t(7))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(**kw)
    for kw in (dict(ids=t(4, 2, dtype=I64)), dict(weights=t(4, 2, dtype=BF16)), dict(counts=t(8, dtype=I64)),
               dict(bias=t(8, dtype=BF16))):
        with pytest.raises(TypeError, match=next(iter(kw))):
            call(**kw)


def test_fp4_buffers():
    f = L.FP4_E8M0_32
    q, s = t(4, 64, dtype=U8), t(512, dtype=U8)
    for X, codes, scales in ((t(3, 128), q, s), (t(4, 128), q[:3], s), (t(4, 128), q, s[:511])):
        with pytest.raises(ValueError):
            L.clha_fp4_quantize(None, X, 4, 128, f, codes, scales)
    with pytest.raises(TypeError):
        L.clha_fp4_quantize(None, t(4, 128), 4, 128, f, q.to(torch.int8), s)
    with pytest.raises(TypeError):
        L.clha_fp4_quantize(None, t(4, 128), 4, 128, f, q, s, perm=t(4, dtype=I64))
    with pytest.raises(ValueError, match="X_hat"):
        L.clha_fp4_dequantize(None, q, s, 4, 128, f, t(4, 127))
    with pytest.raises(ValueError, match="Y"):
        L.clha_fp4_matmul(None, f, q, s, 4, 128, t(128, 64, dtype=U8), t(512, dtype=U8), 128, t(4, 127))
    with pytest.raises(ValueError, match="seg"):
        L.clha_fp4_matmul(None, f, q, s, 4, 128, t(256, 64, dtype=U8), t(1024, dtype=U8), 128, t(4, 128),
                          seg=t(4, dtype=I64), E=2)
    with pytest.raises(ValueError, match="w_scale"):
        L.clha_fp4_matmul(None, f, q, s, 4, 128, t(256, 64, dtype=U8), t(1024, dtype=U8), 128, t(4, 128),
                          seg=t(5, dtype=I64), E=2, w_scale=t(1))
    with pytest.raises(TypeError, match="h"):
        L.clha_fp4_expert_act(None, f, q, s, 4, 128, t(128, 64, dtype=U8), s, t(128, 64, dtype=U8), s, 128, t(4, 128))


def test_combine_buffers():
    ok = dict(Z=t(128, 128), ids=t(4, 1, dtype=I32), weights=t(4, 1), seg=t(3, dtype=I64), perm=t(128, dtype=I32),
              Y=t(4, 128), add=None)

    def call(**kw):
        a = {**ok, **kw}
        L.clha_combine(None, a["Z"], 128, 128, a["ids"], a["weights"], 4, 1, 1, a["seg"], a["perm"], a["Y"], add=a["add"])
    for kw in (dict(Z=t(127, 128)), dict(ids=t(3, 1, dtype=I32)), dict(weights=t(3)), dict(seg=t(2, dtype=I64)),
               dict(perm=t(127, dtype=I32)), dict(Y=t(4, 127)), dict(add=t(4, 127))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(**kw)
    with pytest.raises(TypeError, match="add"):
        call(add=t(4, 128, dtype=I32))


def test_null_context(lib):
    n = None
    assert lib.clha_route_gated(n, n, 0, 0, n, n, n, n, n) == L.ERR_INVALID_ARG
    assert lib.clha_fp4_tensor_scale(n, n, 0, 1, 0, 128, 0, n) == L.ERR_INVALID_ARG
    assert lib.clha_fp4_quantize(n, n, 0, 0, 128, n, 0, n, 1, 0, n, 0, n, n) == L.ERR_INVALID_ARG
    assert lib.clha_fp4_dequantize(n, n, n, 0, 128, 0, n, 0, n, 0) == L.ERR_INVALID_ARG
    assert lib.clha_fp4_matmul(n, 0, n, n, n, 0, 128, n, 1, n, n, n, 128, n, 0) == L.ERR_INVALID_ARG
    assert lib.clha_fp4_expert_act(n, 0, n, n, n, 0, 128, n, 1, n, n, n, n, n, n, 128, n) == L.ERR_INVALID_ARG
    assert lib.clha_combine(n, n, 0, 0, 128, n, n, 0, 1, 1, n, n, n, 0, n, 0) == L.ERR_INVALID_ARG


def test_gather_scratch():
    assert L.clha_gather_scratch_bytes(0, 8) == 8 * 4
    assert L.clha_gather_scratch_bytes(256, 64) == 64 * 4
    assert L.clha_gather_scratch_bytes(257, 64) == 2 * 64 * 4
    for bad in ((-1, 8), (1, 0), (1, 1025), (2 ** 31, 8)):
        assert L.clha_gather_scratch_bytes(*bad) == -1
    ok = dict(X=t(4, 128), ids=t(4, 1, dtype=I32), X_packed=None, seg=t(3, dtype=I64), perm=t(132, dtype=I32),
              scratch=t(4, dtype=U8))

    def call(**kw):
        a = {**ok, **kw}
        L.clha_gather_scratch(None, a["X"], 4, 128, a["ids"], 1, 1, a["X_packed"], 132, a["seg"], a["perm"], a["scratch"])
    for kw in (dict(X=t(4, 127)), dict(ids=t(3, 1, dtype=I32)), dict(X_packed=t(131, 128)), dict(seg=t(2, dtype=I64)),
               dict(perm=t(131, dtype=I32))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(**kw)
    for kw in (dict(scratch=t(4)), dict(X_packed=t(132, 128, dtype=BF16))):
        with pytest.raises(TypeError, match=next(iter(kw))):
            call(**kw)
    n = None
    assert L.load().clha_gather_scratch(n, n, 0, 0, 128, n, 1, 1, n, 128, n, n, n, 0) == L.ERR_INVALID_ARG


def test_layer_shapes():
    """Tensors of another shape than the layer's, although they hold enough elements."""
    from types import SimpleNamespace
    from post_quantization_expert_b200.pipeline import Fp4Layer, MoEWeights
    b = lambda *s: t(*s, dtype=BF16)
    ok = dict(Wgu=b(8, 128, 256), Wd=b(4, 256, 128), Sgu=b(4, 128, 256), Sd=b(2, 256, 128))
    ctx = SimpleNamespace(device=0)
    for kw, more in ((dict(Wgu=b(8, 256, 256)), {}), (dict(Wgu=b(8, 256, 128)), {}), (dict(Sgu=b(4, 128, 128)), {}),
                     (dict(Sd=b(2, 128, 256)), {}), (dict(Sd=None), {}), ({}, dict(bias=t(5))), ({}, dict(x_scale=t(2))),
                     ({}, dict(h_scale=torch.tensor(1.0)))):
        with pytest.raises(ValueError, match=next(iter(kw or more))):
            Fp4Layer(ctx, MoEWeights(**{**ok, **kw}), 2, 16, **more)
    layer = object.__new__(Fp4Layer)
    layer.ctx, layer.timer, layer.E, layer.k, layer.fmt, layer.d_model, layer.max_tokens = ctx, None, 4, 2, 0, 256, 16
    X, lg, Y = t(3, 256), t(3, 4), t(3, 256)
    for name, a in (("X", (t(3, 512), lg, Y)), ("logits", (X, t(3, 8), Y)), ("logits", (X, t(4, 4), Y)),
                    ("Y", (X, lg, t(4, 256))), ("tokens", (t(17, 256), lg, Y))):
        with pytest.raises(ValueError, match=name):
            layer.forward(*a)
