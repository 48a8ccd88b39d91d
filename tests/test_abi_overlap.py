"""The GDN mixer's calls refuse outputs that lie on what the call reads or writes
besides (NVFP4_ERR_ALIAS), without a GPU.  The pointers are addresses that nothing
may dereference; what the calls allow is run in test_gpu_overlap.py."""
import ctypes

import pytest

from nvfp4_w4a4_quantized_05_amd import _lib

ALIAS = 8
MB = 1 << 20


def at(mb, more=0):
    return ctypes.c_void_p(mb * MB + more)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def prefill(lib, *, x=at(1), gates=at(2), cu=at(3), s_in=at(4), s_out=at(5), slots=at(6), o=at(7), ws=at(16), ldx=1024, q=0,
            k=128, v=256, ldg=8, ldo=256, T=8):
    # 2 sequences, heads 1/2, 2 slots: pools of 256 KiB, x rows of 2 KiB, gates rows of 32 bytes
    return lib.nvfp4_gdn_prefill(x, ldx, q, k, v, gates, 0, ldg, 0, 4, cu, 2, T, 1, 2, s_in, s_out, slots, 2, o, ldo, ws,
                                 1 << 40, None)


@pytest.mark.parametrize("kw", [
    dict(o=at(1)), dict(o=at(1, 512), ldo=1024), dict(o=at(1, 256), ldo=1024), dict(o=at(1, 7 * 2048)), dict(x=at(7, 7 * 512)),
    dict(o=at(1, 2 * 768), ldo=1016),                                # other columns, but another step from row to row
    dict(o=at(1, 2 * 896), ldo=1024),                                # runs into the next row's q
    dict(o=at(2)), dict(gates=at(7, 16), ldg=128), dict(o=at(3)), dict(o=at(4)), dict(o=at(5, 262144 - 16)), dict(o=at(6)),
    dict(s_out=at(4, 16)), dict(s_in=at(5, 262144 - 16)), dict(s_out=at(1, 1024)), dict(s_out=at(3)), dict(s_out=at(6)),
    dict(ws=at(1)), dict(x=at(16, 1024)), dict(o=at(16)), dict(s_in=at(16)), dict(s_out=at(16)), dict(cu=at(16)), dict(slots=at(16, 4))])
def test_gdn_prefill(lib, kw):
    assert prefill(lib, **kw) == ALIAS


def decode(lib, *, x=at(1), xt=1, gates=at(2), states=at(4), slots=at(6), o=at(7), ot=1, ldx=1024, ldg=8, ldo=256, B=2):
    return lib.nvfp4_gdn_decode(x, xt, ldx, 0, 128, 256, gates, 0, ldg, 0, 4, B, 1, 2, states, slots, 2, o, ot, ldo, None)


@pytest.mark.parametrize("kw", [
    dict(o=at(1)), dict(o=at(1, 512), ldo=1024), dict(o=at(1, 2048)), dict(x=at(7, 512)), dict(o=at(2)), dict(o=at(2, 32)),
    dict(o=at(4, 131072)), dict(o=at(6)), dict(states=at(1, 1024)), dict(states=at(2)), dict(states=at(6)), dict(B=1, o=at(1, 1008)),
    dict(xt=0, ot=0, o=at(1, 1024), ldo=1024)])
def test_gdn_decode(lib, kw):
    assert decode(lib, **kw) == ALIAS


def conv(lib, *, x=at(1), w=at(2), cu=at(3), state=at(4), slots=at(6), y=at(7), ldx=64, ldy=64, T=8):
    return lib.nvfp4_conv_silu(x, 1, ldx, 64, w, 4, cu, 2, T, state, slots, 2, y, ldy, None)


@pytest.mark.parametrize("kw", [
    dict(y=at(1)), dict(y=at(1, 128), ldx=128, ldy=120), dict(y=at(1, 64), ldx=128, ldy=128), dict(y=at(2, 64)), dict(y=at(3)),
    dict(y=at(4, 700)), dict(y=at(6)), dict(state=at(1, 2)), dict(state=at(2)), dict(state=at(3)), dict(state=at(6))])
def test_conv_silu(lib, kw):
    assert conv(lib, **kw) == ALIAS


def add(lib, *, x=at(1), xt=1, r=at(2), rt=1, w=at(3), t=at(4), y=at(5), yt=1, gs=at(6), codes=at(7), scales=at(8), ldx=64, ldr=64,
        ldt=64, ldy=64, rows=4):
    return lib.nvfp4_add_rmsnorm(x, xt, ldx, r, rt, ldr, 1.0, w, 1e-6, rows, 64, t, ldt, y, yt, ldy, gs, codes, scales, None)


@pytest.mark.parametrize("kw", [
    dict(y=at(1, 16)), dict(y=at(1, 128)), dict(y=at(1), ldy=72), dict(y=at(1), yt=0), dict(y=at(2, 32)), dict(t=at(2, 128)),
    dict(t=at(2), ldt=72), dict(t=at(1, 16)), dict(t=at(1), rt=0), dict(y=at(4)), dict(y=at(4, 128)), dict(y=at(3)), dict(t=at(3)),
    dict(y=at(3), yt=0, rows=1), dict(y=at(6)), dict(codes=at(1)), dict(codes=at(2, 64)), dict(codes=at(3)), dict(codes=at(4)),
    dict(codes=at(5)), dict(codes=at(6)), dict(scales=at(1, 511)), dict(scales=at(7)), dict(scales=at(7, 127)), dict(scales=at(5)),
    dict(scales=at(3, 255))])
def test_add_rmsnorm(lib, kw):
    assert add(lib, **kw) == ALIAS


def gated(lib, *, o=at(1), ot=1, z=at(2), w=at(3), y=at(5), yt=1, gs=at(6), codes=at(7), scales=at(8), ldo=64, ldz=64, ldy=64):
    return lib.nvfp4_rmsnorm_gated(o, ot, ldo, z, 1, ldz, w, 1e-6, 4, 64, 64, y, yt, ldy, gs, codes, scales, None)


@pytest.mark.parametrize("kw", [
    dict(y=at(1, 32)), dict(y=at(1, 128)), dict(y=at(1), ldy=72), dict(y=at(1), yt=0), dict(y=at(2, 128)), dict(y=at(3)),
    dict(y=at(6)), dict(codes=at(1)), dict(codes=at(2, 504)), dict(codes=at(3)), dict(codes=at(5)), dict(scales=at(2)),
    dict(scales=at(7, 64)), dict(scales=at(6, 3))])
def test_rmsnorm_gated(lib, kw):
    assert gated(lib, **kw) == ALIAS


def test_nothing_was_launched(lib):
    assert lib.nvfp4_last_hip_error() == 0
