"""Refusals of the latent-attention and adapter calls, on the CPU: every check
happens on the host, before a launch."""
import ctypes

import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from mxfp8_gemm_mailbox_gb300 import _lib
from mxfp8_gemm_mailbox_gb300 import build as build_mod

P = ctypes.c_void_p
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def text(lib):
    return lib.mxfp8_last_error().decode()


def test_workspace_sizes(lib):
    for latent in (0, 64, 128, 384, 1024, -512):
        assert lib.mxfp8_latent_workspace_bytes(latent) == 0
    assert lib.mxfp8_latent_workspace_bytes(512) >= lib.mxfp8_latent_workspace_bytes(256) > 0
    assert lib.mxfp8_adapters_workspace_bytes(7168, 16384, 64) >= 8 * 7168 * 4
    for n, k, r in ((100, 512, 8), (0, 512, 8), (256, 33, 8), (256, 512, 0), (256, 512, 257),
                    (256, 32800, 8)):
        assert lib.mxfp8_adapters_workspace_bytes(n, k, r) == 0


def query(lib, rows=1, heads=4, nope=64, latent=512, a=0x1000, b=0x1000, w=0x1000, q=0x1000):
    return lib.mxfp8_latent_query(P(a), P(b), P(w), P(q), rows, heads, nope, latent, None)


def test_query_refusals(lib):
    for bad in (dict(rows=-1), dict(a=0), dict(b=0x1008), dict(w=None), dict(q=0x1004)):
        assert query(lib, **bad) == mx.ERR_INVALID, bad
    for bad in (dict(heads=0), dict(heads=257), dict(nope=0), dict(nope=48), dict(nope=544),
                dict(latent=128), dict(rows=65536)):
        assert query(lib, **bad) == mx.ERR_UNSUPPORTED, bad
        assert text(lib)
    assert query(lib, rows=0, a=0) == mx.OK  # nothing to do, nothing launched


def values(lib, rows=1, heads=4, latent=512, value=64, o=0x1000, w=0x1000, x=0x1000, s=0x1001):
    return lib.mxfp8_latent_values(P(o), P(w), P(x), P(s), rows, heads, latent, value, None)


def test_values_refusals(lib):
    for bad in (dict(rows=-1), dict(o=0), dict(w=0x1008), dict(x=None), dict(s=0)):
        assert values(lib, **bad) == mx.ERR_INVALID, bad
    for bad in (dict(heads=0), dict(value=16), dict(value=1024), dict(latent=500)):
        assert values(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert values(lib, rows=0, o=0) == mx.OK


def attend(lib, ws=None, flags=0, **change):
    fields = dict(heads=16, latent=512, rows=2, requests=1, page_size=64, pages=4, table_width=2,
                  scale=0.1, token_stride=576, page_stride=64 * 576)
    ptrs = dict(q=0x1000, cache=0x1000, table=0x1000, lengths=0x1000, begin=0x1000, tree=0,
                out=0x1000, workspace=0x1000)
    for k, v in change.items():
        (fields if k in fields else ptrs)[k] = v
    d = _lib.LatentDesc(*fields.values())
    size = lib.mxfp8_latent_workspace_bytes(512) if ws is None else ws
    return lib.mxfp8_latent_attend(ctypes.byref(d), *(P(v) for v in ptrs.values()), size,
                                   P(flags), None)


def test_attend_refusals(lib):
    assert lib.mxfp8_latent_attend(None, *[P(0x1000)] * 8, 1 << 30, None, None) == mx.ERR_INVALID
    for bad in (dict(q=0), dict(cache=0x1008), dict(table=0), dict(lengths=0x1002), dict(begin=0),
                dict(tree=0x1004), dict(out=0), dict(workspace=0x1010), dict(ws=0), dict(flags=2),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(pages=0), dict(table_width=0), dict(rows=-1),
                dict(requests=0)):
        assert attend(lib, **bad) == mx.ERR_INVALID, bad
        assert text(lib)
    for bad in (dict(heads=0), dict(heads=300), dict(latent=64), dict(page_size=0),
                dict(page_size=12), dict(page_size=4), dict(requests=257), dict(requests=-1),
                dict(token_stride=568), dict(token_stride=577), dict(page_stride=100),
                dict(page_stride=64), dict(table_width=1 << 26), dict(rows=1 << 17)):
        assert attend(lib, **bad) == mx.ERR_UNSUPPORTED, bad
    assert attend(lib, rows=0, q=0) == mx.OK


def test_attend_refuses_more_tiles_than_it_numbers(lib):
    # 65535 x 256 / 128 + 1 row tiles of 2^21 / 64 token tiles: past 2^31
    assert attend(lib, rows=65535, heads=256, table_width=1 << 15) == mx.ERR_UNSUPPORTED
    assert "tiles" in text(lib)


def test_run_adapted_needs_a_handle(lib):
    d = _lib.Adapters(0x1000, 0x1000, None, None, 1, 8)
    assert lib.mxfp8_publish_gemm_run_adapted(None, P(0x1000), P(0x1000), 1, None, ctypes.byref(d),
                                              P(0x1000), P(0x1000), 1 << 30, None,
                                              None) == mx.ERR_INVALID


def test_binding_refuses_wrong_tensors():
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(TypeError, match="bfloat16"):
        mx.latent_query(z(1, 4, 64), z(1, 4, 64), z(4, 512, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        mx.latent_query(z(1, 4, 64), z(1, 4, 64), z(4, 512, 64))
    with pytest.raises(ValueError, match="w must be"):
        mx.latent_values(z(1, 4, 512), z(4, 64))
    with pytest.raises(ValueError, match="latent must be"):
        mx.LatentAttention(4, 128, device="cpu")
    at = mx.LatentAttention(4, 256, device="cpu")
    with pytest.raises(ValueError, match="q must be"):
        at.run(z(1, 5, 320), z(2, 8, 320), z(1, 1), z(1), z(2), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        at.run(z(1, 4, 320), z(2, 8, 320), z(1, 1), z(1), z(2), 1.0)
    for args in ((1, z(1, 4, 64), z(4, 512, 64)), (z(1, 4, 64), None, z(4, 512, 64)),
                 (z(1, 4, 64), z(1, 4, 64), "w")):
        with pytest.raises((TypeError, ValueError)):
            mx.latent_query(*args)
    with pytest.raises(TypeError, match="must be a tensor"):
        mx.latent_values(z(1, 4, 512), [1.0])
    for a, b, error in ((z(2, 8, 64), z(2, 128, 7), ValueError),
                        (z(2, 8, 64), z(1, 128, 8), ValueError),
                        (z(2, 8, 64, dtype=torch.float32), z(2, 128, 8), TypeError),
                        (z(2, 300, 64), z(2, 128, 300), ValueError),
                        (z(0, 8, 64), z(0, 128, 8), ValueError),
                        (z(2, 8, 64), z(2, 100, 8), ValueError)):
        with pytest.raises(error):
            mx.Adapters(a, b)
