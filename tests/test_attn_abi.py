"""CPU checks of the attention calls' argument rejection: every refusal comes
from the host before a device call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from w4a4_rank_gemm_b200 import build
    build.build()
    from w4a4_rank_gemm_b200 import serq
    return serq


FAKE = ctypes.c_void_p(0x1000)


def rope_opts(lib, **kw):
    o = lib.RopeOpts()
    lib.lib.serq_rope_opts_init(ctypes.byref(o))
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def test_rope_defaults(lib):
    o = rope_opts(lib)
    assert (o.head_dim, o.rot_dim, o.layout, o.scaling) == (128, 128, lib.ROPE_HALF, lib.ROPE_PLAIN)
    assert (o.theta, o.factor, o.original_len, o.low, o.high, o.amplitude) == (1e4, 1.0, 8192.0, 1.0, 4.0, 1.0)


@pytest.mark.parametrize("kw,shape", [
    (dict(head_dim=96), True), (dict(rot_dim=24), True), (dict(rot_dim=0), True), (dict(rot_dim=144), True),
    (dict(head_dim=64), True), (dict(layout=2), False), (dict(scaling=3), False), (dict(scaling=-1), False),
    (dict(theta=1.0), False), (dict(theta=float("nan")), False), (dict(factor=0.5), False),
    (dict(factor=float("inf")), False), (dict(amplitude=0.0), False), (dict(scaling=2, low=4.0), False),
    (dict(scaling=2, original_len=0.0), False), (dict(scaling=2, low=-1.0), False),
    (dict(scaling=2, high=float("nan")), False)])
def test_rope_create_rejection(lib, kw, shape):
    out = ctypes.c_void_p()
    o = rope_opts(lib, **kw)
    want = lib.ERR_UNSUPPORTED_SHAPE if shape else lib.ERR_INVALID_ARG
    assert lib.lib.serq_rope_create(ctypes.byref(o), ctypes.byref(out)) == want
    assert out.value is None


def test_null_handles(lib):
    L = lib.lib
    out = ctypes.c_void_p()
    assert L.serq_rope_create(None, ctypes.byref(out)) == lib.ERR_INVALID_ARG
    L.serq_rope_destroy(None)
    L.serq_kv_cache_destroy(None)
    assert L.serq_rope_append(None, FAKE, FAKE, 256, FAKE, 256, FAKE, 256, 1, 2, None, None, 0.0, 1, FAKE, FAKE, FAKE, 1,
                              1, FAKE, 256, None) == lib.ERR_INVALID_ARG
    assert L.serq_attn_prefill(None, FAKE, 256, 1, 2, 1.0, 1, FAKE, FAKE, FAKE, 1, 1, 0, None, 0, FAKE, 256,
                               None) == lib.ERR_INVALID_ARG
    assert b"null cache" in L.serq_last_error_string()
    assert L.serq_attn_decode(None, FAKE, 256, 2, 1.0, 1, FAKE, FAKE, 1, 1, 0, 0, None, 0, FAKE, 256,
                              None) == lib.ERR_INVALID_ARG
    assert L.serq_attn_prefill_ws_bytes(None, 1, 1, 1, 1, 0) == 0
    assert L.serq_attn_decode_ws_bytes(None, 1, 1, 1, 0, 0) == 0


@pytest.mark.parametrize("args,shape", [
    ((FAKE, FAKE, 4, 24, 2, 128, 1 << 20), True), ((FAKE, FAKE, 4, 512, 2, 128, 1 << 20), True),
    ((FAKE, FAKE, 4, 8, 2, 128, 1 << 20), True), ((FAKE, FAKE, 4, 64, 2, 80, 1 << 20), True),
    ((None, FAKE, 4, 64, 2, 128, 1 << 20), False), ((FAKE, None, 4, 64, 2, 128, 1 << 20), False),
    ((FAKE, FAKE, 0, 64, 2, 128, 1 << 20), False), ((FAKE, FAKE, 4, 64, 0, 128, 1 << 20), False),
    ((FAKE, FAKE, 4, 64, 2, 128, 64 * 2 * 128 - 8), False), ((FAKE, FAKE, 4, 64, 2, 128, 64 * 2 * 128 + 4), False),
    ((ctypes.c_void_p(0x1008), FAKE, 4, 64, 2, 128, 1 << 20), False)])
def test_cache_create_rejection(lib, args, shape):
    out = ctypes.c_void_p()
    want = lib.ERR_UNSUPPORTED_SHAPE if shape else lib.ERR_INVALID_ARG
    assert lib.lib.serq_kv_cache_create(*args, ctypes.byref(out)) == want
    assert out.value is None
