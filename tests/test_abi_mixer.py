"""Refusals of the GDN mixer's entry points, without a GPU: every bad argument
returns its status before anything is launched.  The pointers are addresses
that nothing may dereference."""
import ctypes
import math

import numpy as np
import pytest

from nvfp4_w4a4_quantized_05_amd import _lib
from oracle import gdn_ref as G
from oracle import mixer_ref as M

OK, NULL, SHAPE, DTYPE, MODE, ALIGN, WORKSPACE, HIP, ALIAS, TOO_LARGE = range(10)
P = ctypes.c_void_p(0x10000)
P2, P4, P8, P16 = (ctypes.c_void_p(0x10000 + n) for n in (2, 4, 8, 16))
FAR = ctypes.c_void_p(0x10000000)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def prefill(lib, x=P, ldx=1024, q=0, k=128, v=256, gates=P, gt=0, ldg=8, g=0, b=4, cu=P, n=2, T=0, n_qk=1, n_v=2,
            s_in=None, s_out=None, slots=None, n_slots=2, o=P, ldo=256, ws=P, wsb=1 << 40):
    return lib.nvfp4_gdn_prefill(x, ldx, q, k, v, gates, gt, ldg, g, b, cu, n, T, n_qk, n_v, s_in, s_out, slots,
                                 n_slots, o, ldo, ws, wsb, None)


def test_gdn_prefill_rejects_bad_arguments(lib):
    def bad(**kw):
        return prefill(lib, **dict(dict(T=8), **kw))
    assert bad(gt=2) == DTYPE
    for kw in (dict(ldx=0), dict(ldx=1 << 23), dict(ldg=0), dict(ldg=1 << 23), dict(n_qk=0), dict(n_v=0), dict(n_v=3, n_qk=2),
               dict(n_v=65536), dict(q=-1), dict(q=1024 - 127), dict(k=1024 - 127), dict(v=1024 - 255), dict(v=-1),
               dict(g=7), dict(b=7), dict(b=-1), dict(q=1 << 62), dict(T=-1), dict(T=1 << 31), dict(n=0), dict(n=(1 << 20) + 1),
               dict(n=1 << 20, n_v=2, ldo=256), dict(n_slots=-1), dict(ldo=255), dict(ldo=1 << 61)):
        assert bad(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(gates=None), dict(o=None), dict(cu=None)):
        assert bad(**kw) == NULL, kw
    for kw in (dict(x=P8), dict(ldx=1028), dict(q=4), dict(k=132), dict(v=260), dict(gates=P2), dict(gates=ctypes.c_void_p(0x10001), gt=1),
               dict(cu=P2), dict(s_in=P8), dict(s_out=P4), dict(slots=P2), dict(o=P8), dict(ldo=260)):
        assert bad(**kw) == ALIGN, kw
    need = lib.nvfp4_gdn_prefill_workspace_size(8, 2, 1, 2)
    if need:
        assert bad(wsb=need - 1) == WORKSPACE
        assert bad(ws=None) == NULL and bad(ws=P16) == ALIGN
    assert lib.nvfp4_gdn_prefill_workspace_size(-1, 1, 1, 1) == 0
    assert lib.nvfp4_gdn_prefill_workspace_size(8, 1, 2, 3) == 0
    assert lib.nvfp4_last_hip_error() == 0


def decode(lib, x=P, xt=1, ldx=1024, q=0, k=128, v=256, gates=P, gt=0, ldg=8, g=0, b=4, B=2, n_qk=1, n_v=2, states=P,
           slots=None, n_slots=2, o=P, ot=1, ldo=256):
    return lib.nvfp4_gdn_decode(x, xt, ldx, q, k, v, gates, gt, ldg, g, b, B, n_qk, n_v, states, slots, n_slots, o, ot,
                                ldo, None)


def test_gdn_decode_rejects_bad_arguments(lib):
    for kw in (dict(xt=2), dict(gt=-1), dict(ot=7)):
        assert decode(lib, **kw) == DTYPE, kw
    for kw in (dict(ldx=0), dict(ldg=1 << 23), dict(n_v=3, n_qk=2), dict(q=1024), dict(g=7), dict(B=-1), dict(B=(1 << 20) + 1),
               dict(B=1 << 19, n_v=4, v=256, ldo=512), dict(n_slots=-1), dict(ldo=128)):
        assert decode(lib, **kw) == SHAPE, kw
    for kw in (dict(x=None), dict(gates=None), dict(states=None), dict(o=None)):
        assert decode(lib, **kw) == NULL, kw
    for kw in (dict(x=P8), dict(q=4), dict(xt=0, q=2), dict(ldx=1028), dict(xt=0, ldx=1026), dict(gates=P2), dict(states=P8),
               dict(slots=P2), dict(o=P8), dict(ldo=260), dict(ot=0, ldo=258)):
        assert decode(lib, **kw) == ALIGN, kw
    assert decode(lib, B=0, x=None, gates=None, states=None, o=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def conv(lib, x=P, dt=1, ldx=64, C=64, w=P, W=4, cu=P, n=2, T=8, state=None, slots=None, n_slots=2, y=FAR, ldy=64):
    return lib.nvfp4_conv_silu(x, dt, ldx, C, w, W, cu, n, T, state, slots, n_slots, y, ldy, None)


def test_conv_silu_rejects_bad_arguments(lib):
    assert conv(lib, dt=2) == DTYPE
    for kw in (dict(W=1), dict(W=5), dict(C=0, ldx=0), dict(C=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), dict(n_slots=-1), dict(T=-1),
               dict(T=1 << 31), dict(T=(1 << 22) + 1, cu=None), dict(n=0), dict(ldx=63), dict(ldy=63), dict(ldx=1 << 61)):
        assert conv(lib, **kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        assert conv(lib, **kw) == NULL, kw
    odd = ctypes.c_void_p(0x10001)
    for kw in (dict(x=odd), dict(dt=0, x=P2), dict(y=odd), dict(state=odd), dict(w=P2), dict(cu=P2), dict(slots=P2)):
        assert conv(lib, **kw) == ALIGN, kw
    assert conv(lib, y=P) == ALIAS
    assert conv(lib, y=ctypes.c_void_p(0x10000 + 7 * 128)) == ALIAS      # the last row of x
    assert conv(lib, x=ctypes.c_void_p(0x10000000 + 7 * 128)) == ALIAS   # the last row of y
    assert conv(lib, T=0, x=None, w=None, y=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def add(lib, x=P, xt=1, ldx=64, r=P, rt=1, ldr=64, scale=1.0, w=P, eps=1e-6, rows=4, cols=64, ro=P, ldro=64, y=P, yt=1,
        ldy=64, gs=None, codes=None, scales=None):
    return lib.nvfp4_add_rmsnorm(x, xt, ldx, r, rt, ldr, scale, w, eps, rows, cols, ro, ldro, y, yt, ldy, gs, codes,
                                 scales, None)


Q = dict(gs=P, codes=P, scales=P)


def test_add_rmsnorm_rejects_bad_arguments(lib):
    for kw in (dict(xt=2), dict(rt=3), dict(yt=-1)):
        assert add(lib, **kw) == DTYPE, kw
    for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(cols=0), dict(cols=16385, ldx=20000, ldr=20000, ldro=20000, ldy=20000),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(scale=math.inf), dict(scale=math.nan),
               dict(ldx=63), dict(ldr=63), dict(ldro=63), dict(ldy=63), dict(ldx=1 << 62), dict(cols=40, **Q)):
        assert add(lib, **kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(gs=P), dict(gs=P, codes=P), dict(codes=P, scales=P)):
        assert add(lib, **kw) == NULL, kw
    odd = ctypes.c_void_p(0x10001)
    for kw in (dict(x=odd), dict(xt=0, x=P2), dict(r=odd), dict(ro=odd), dict(w=P2), dict(y=odd), dict(yt=0, y=P2), dict(Q, codes=P4),
               dict(Q, gs=P2), dict(Q, x=P8), dict(Q, ldx=68), dict(Q, r=P8), dict(Q, ldro=68), dict(Q, y=P8), dict(Q, w=P4)):
        assert add(lib, **kw) == ALIGN, kw
    assert add(lib, rows=0, x=None, w=None, y=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def gated(lib, o=P, ot=1, ldo=256, z=P, zt=1, ldz=256, w=P, eps=1e-6, rows=4, cols=256, group=128, y=P, yt=1, ldy=256,
          gs=None, codes=None, scales=None):
    return lib.nvfp4_rmsnorm_gated(o, ot, ldo, z, zt, ldz, w, eps, rows, cols, group, y, yt, ldy, gs, codes, scales, None)


def test_rmsnorm_gated_rejects_bad_arguments(lib):
    for kw in (dict(ot=2), dict(zt=2), dict(yt=2)):
        assert gated(lib, **kw) == DTYPE, kw
    for kw in (dict(group=8), dict(group=2048, cols=2048, ldo=2048, ldz=2048, ldy=2048), dict(group=96), dict(group=0), dict(group=-128),
               dict(cols=192), dict(cols=0), dict(rows=-1), dict(rows=1 << 27), dict(ldo=128), dict(ldz=128), dict(ldy=128),
               dict(eps=0.0), dict(eps=math.nan)):
        assert gated(lib, **kw) == SHAPE, kw
    for kw in (dict(o=None), dict(z=None), dict(w=None), dict(y=None), dict(scales=P)):
        assert gated(lib, **kw) == NULL, kw
    for kw in (dict(o=P8), dict(ldo=260), dict(z=P8), dict(ldz=260), dict(w=P4), dict(y=P8), dict(ldy=260), dict(Q, codes=P4)):
        assert gated(lib, **kw) == ALIGN, kw
    assert gated(lib, rows=0, o=None, z=None, w=None, y=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def test_references_against_closed_forms():
    """The fp64 references on inputs whose results are known."""
    # packed sequences are the recurrence of each alone, from its own start
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((9, n, 8)) for n in (1, 1, 2))
    g, b = -rng.random((9, 2)), rng.random((9, 2))
    s0 = rng.standard_normal((2, 8, 8))
    o, S, _ = M.gdn_packed_ref(q, k, v, g, b, [0, 4, 4, 9], [None, s0, s0])
    o1, S1, _, _ = G.gdn_recurrence_ref(q[4:], k[4:], v[4:], g[4:], b[4:], s0=s0)
    assert np.array_equal(o[4:], o1) and np.array_equal(S[2], S1) and np.array_equal(S[1], s0)
    # a convolution with one tap is that row; with all ones it is a moving sum
    x = rng.standard_normal((5, 3))
    old = rng.standard_normal((1, 2, 3))
    one = np.array([[0.0, 0.0, 1.0]] * 3)
    y, _, new = M.conv_silu_ref(x, one, [0, 5], old)
    assert np.allclose(y, M.silu(x)) and np.array_equal(new[0], x[3:])
    y, _, _ = M.conv_silu_ref(x, np.ones((3, 3)), [0, 5], old)
    assert np.allclose(y[0], M.silu(old[0].sum(0) + x[0])) and np.allclose(y[4], M.silu(x[2:].sum(0)))
    # norms: unit rows, scale invariance, silu at zero
    t, y, _ = M.add_rmsnorm_ref(x, x, 2.0, np.ones(3), 1e-30)
    assert np.allclose(t, 3 * x) and np.allclose(np.mean(y * y, axis=1), 1)
    assert np.allclose(M.rmsnorm_gated_ref(x, x * 0, np.ones(3), 1e-6), 0)
    assert np.allclose(M.silu([0.0, 50.0, -800.0]), [0.0, 50.0, 0.0])
