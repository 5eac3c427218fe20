"""Refusals of the calls of a layer of routed experts, on the CPU: every check
happens on the host, before a launch."""
import ctypes

import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from mxfp8_gemm_mailbox_gb300 import _lib
from mxfp8_gemm_mailbox_gb300 import build as build_mod

P = ctypes.c_void_p
A = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def text(lib):
    return lib.mxfp8_last_error().decode()


def route(lib, logits=A, type=0, stride=64, tokens=4, experts=64, k=8, weight=A, expert=A, slot=A,
          row=A, begin=A, workspace=None, nbytes=0):
    return lib.mxfp8_route(P(logits), type, stride, tokens, experts, k, 1, P(weight), P(expert),
                           P(slot), P(row), P(begin), P(workspace), nbytes, None)


def test_route_refusals(lib):
    for bad in (dict(type=3), dict(type=-1), dict(tokens=-1), dict(stride=63), dict(logits=0),
                dict(logits=A + 1), dict(type=2, logits=A + 2), dict(weight=A + 2), dict(expert=0),
                dict(slot=A + 1), dict(row=0), dict(begin=0), dict(tokens=33),
                dict(tokens=129, workspace=A, nbytes=1535)):
        assert route(lib, **bad) == mx.ERR_INVALID, bad
        assert text(lib)
    for bad in (dict(experts=0), dict(experts=513, stride=600), dict(k=0), dict(k=33),
                dict(experts=4, k=5), dict(tokens=2 ** 29)):
        assert route(lib, **bad) == mx.ERR_UNSUPPORTED, bad


def test_route_workspace(lib):
    size = lib.mxfp8_route_workspace_bytes
    assert size(0, 64) == size(32, 64) == size(-5, 64) == size(200, 0) == size(200, 513) == 0
    assert size(33, 63) == 3 * 63 * 4 and size(129, 64) == 6 * 64 * 4 and size(16384, 256) == 257 * 256 * 4
    assert size(1 << 20, 512) == 4097 * 512 * 4


def quantize(lib, x=A, type=0, stride=64, x_rows=4, k=64, rows=None, out_rows=4, format=1, codes=A,
             scales=A, flags=None):
    return lib.mxfp8_quantize(P(x), type, stride, x_rows, k, P(rows), out_rows, format, P(codes),
                              P(scales), P(flags), None)


def test_quantize_refusals(lib):
    for bad in (dict(type=3), dict(format=0), dict(format=3), dict(x_rows=-1, out_rows=-1),
                dict(out_rows=5), dict(x=A + 8), dict(x=0), dict(codes=A + 8), dict(scales=0),
                dict(rows=A + 2), dict(flags=A + 1)):
        assert quantize(lib, **bad) == mx.ERR_INVALID, bad
        assert text(lib)
    for bad in (dict(k=0), dict(k=48, stride=48), dict(stride=32), dict(stride=68),
                dict(type=2, stride=66), dict(rows=A, out_rows=2 ** 33)):
        assert quantize(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert quantize(lib, x_rows=0, out_rows=0, x=0) == mx.OK


def dequantize(lib, codes=A, scales=A, rows=4, k=64, format=1, type=0, out=A):
    return lib.mxfp8_dequantize(P(codes), P(scales), rows, k, format, type, P(out), None)


def test_dequantize_refusals(lib):
    for bad in (dict(codes=A + 8), dict(scales=0), dict(rows=-1), dict(format=0), dict(type=5),
                dict(out=A + 4)):
        assert dequantize(lib, **bad) == mx.ERR_INVALID, bad
    for bad in (dict(k=16), dict(rows=2 ** 40)):
        assert dequantize(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert dequantize(lib, rows=0, codes=0) == mx.OK


def desc(**kw):
    d = dict(experts=4, n=64, k=256, gated=0, w_format=2, x_format=1, out_format=0, rows=8)
    d.update(kw)
    return _lib.ExpertDesc(**d)


def product(lib, w=A, laid=A, x=A, x_scale=A, begin=A, out=A, out_scale=A, workspace=A, nbytes=None,
            flags=A, **kw):
    nbytes = lib.mxfp8_expert_workspace_bytes() if nbytes is None else nbytes
    return lib.mxfp8_expert_product(ctypes.byref(desc(**kw)), P(w), P(laid), P(x), P(x_scale),
                                    P(begin), P(out), P(out_scale), P(workspace), nbytes, P(flags),
                                    None)


def test_product_refusals(lib):
    for bad in (dict(w=A + 16), dict(laid=A + 8), dict(x=A + 16), dict(x_scale=A + 2), dict(begin=0),
                dict(begin=A + 2), dict(out=A + 8), dict(out_format=1, out_scale=0),
                dict(workspace=A + 8), dict(nbytes=1024), dict(flags=A + 2), dict(gated=2),
                dict(w_format=0), dict(x_format=3), dict(out_format=3), dict(rows=-1)):
        assert product(lib, **bad) == mx.ERR_INVALID, bad
        assert text(lib)
    for bad in (dict(experts=0), dict(experts=513), dict(n=0), dict(n=12), dict(gated=1, n=40),
                dict(out_format=2, n=40), dict(k=0), dict(k=64), dict(k=192),
                dict(rows=2 ** 31 - 1, n=1 << 20)):
        assert product(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert product(lib, rows=0, x=0, out=0) == mx.OK
    assert lib.mxfp8_expert_product(None, *[None] * 8, 0, None, None) == mx.ERR_INVALID


def test_product_most_rows(lib):
    """Rows whose count with a tile's or the experts' would pass 31 bits, in one tile of W (past
    the check of tiles); the largest count allowed reaches the pointers' checks."""
    for rows in (2 ** 31 - 1, 2 ** 31 - 1024):
        assert product(lib, rows=rows, n=8, k=128, experts=1) == mx.ERR_UNSUPPORTED, rows
        assert product(lib, rows=rows, n=8, k=128, experts=512) == mx.ERR_UNSUPPORTED, rows
        assert "rows must be at most" in text(lib)
    assert product(lib, rows=2 ** 31 - 1025, n=8, k=128, experts=1, x=A + 16) == mx.ERR_INVALID


def test_scales(lib):
    size = lambda **kw: lib.mxfp8_expert_scales_bytes(ctypes.byref(desc(**kw)))  # noqa: E731
    assert size() == 4 * 1 * 2 * 512
    assert size(n=136) == 4 * 2 * 2 * 512
    assert size(n=96, gated=1) == 4 * 2 * 2 * 512
    assert size(k=100) == size(n=4) == size(experts=-1) == size(w_format=0) == 0
    assert size(experts=512, n=1 << 20, k=1 << 20) == 0
    lay = lambda a, b: lib.mxfp8_expert_lay_scales(ctypes.byref(desc()), P(a), P(b), None)  # noqa: E731
    assert lay(A + 2, A) == lay(A, A + 8) == lay(0, A) == lay(A, 0) == mx.ERR_INVALID
    assert lib.mxfp8_expert_workspace_bytes() < 1 << 26


def combine(lib, y=A, stride=64, slots=8, weight=A, slot=A, tokens=4, k=2, n=64, add=None, out=A,
            flags=None):
    return lib.mxfp8_combine(P(y), stride, slots, P(weight), P(slot), tokens, k, n, P(add), P(out),
                             P(flags), None)


def test_combine_refusals(lib):
    for bad in (dict(y=A + 8), dict(weight=A + 2), dict(slot=0), dict(add=A + 8), dict(out=0),
                dict(tokens=-1), dict(slots=-1), dict(flags=A + 2)):
        assert combine(lib, **bad) == mx.ERR_INVALID, bad
    for bad in (dict(n=0), dict(n=60), dict(k=0), dict(k=33), dict(stride=56), dict(stride=68),
                dict(tokens=2 ** 30)):
        assert combine(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert combine(lib, tokens=0, y=0) == mx.OK


def test_tensors_that_the_binding_refuses(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mx.route(x, 2)
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        mx.route(x.double(), 2)
    with pytest.raises(TypeError, match="tensor"):
        mx.route([1.0], 2)
    with pytest.raises(ValueError, match="mxfp8"):
        mx.quantize(x, "fp4")
    with pytest.raises(ValueError, match="CUDA"):
        mx.quantize(x, "mxfp4")
    with pytest.raises(TypeError, match="dtype"):
        mx.dequantize(x, x, torch.float64)
    with pytest.raises(TypeError, match="bfloat16"):
        mx.combine(x, x, x)
    codes = torch.zeros(2, 64, 128, dtype=torch.uint8)
    scale = torch.zeros(2, 64, 4, dtype=torch.uint8)
    with pytest.raises(TypeError, match="one-byte"):
        mx.ExpertProduct(codes.float(), scale)
    with pytest.raises(ValueError, match="E2M1"):
        mx.ExpertProduct(codes, scale[..., :3])
    with pytest.raises(ValueError, match="even"):
        mx.ExpertProduct(codes[:, :63].contiguous(), scale[:, :63].contiguous(), gated=True)
    with pytest.raises(ValueError, match="CUDA"):
        mx.ExpertProduct(codes, scale)
