"""Refusals of the attention layer's entry points, without a GPU: every bad argument
returns its status before anything is launched, and the binding refuses what it can
see.  The pointers are addresses that nothing may dereference."""
import ctypes
import math

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from nvfp4_w4a4_quantized_05_amd import _lib
from oracle import attn_ref as A

OK, NULL, SHAPE, DTYPE, MODE, ALIGN, WORKSPACE, HIP, ALIAS = range(9)
MB = 1 << 20


def at(mb, more=0):
    return mb * MB + more


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def cache(fmt=0, k=at(1), v=at(2), ks=at(3), vs=at(4), kg=at(5), vg=at(5, 64), pages=4, page=64, heads=2, d=128):
    # 4 pages of 2 heads x 64 x 128: 64 KiB each of K and V in E4M3
    return _lib._KvCacheStruct(k, v, ks, vs, kg, vg, fmt, pages, page, heads, d)


def rows_call(f, c=None, table=at(6), ldt=4, most=4, lens=at(7), cu=at(8), n=3, T=8, k=at(9), ldk=256, v=at(10), ldv=256, dt=1):
    c = cache() if c is None else c
    return f(ctypes.byref(c), table, ldt, most, lens, cu, n, T, k, ldk, v, ldv, dt, None)


def attn(lib, c=None, table=at(6), ldt=4, most=4, lens=at(7), cu=at(8), n=3, T=8, q=at(9), ldq=512, hq=4, scale=0.1, tree=None,
         o=at(10), ldo=512, ws=at(32), wsb=1 << 40):
    c = cache() if c is None else c
    return lib.nvfp4_attn_cached(ctypes.byref(c), table, ldt, most, lens, cu, n, T, q, ldq, hq, scale, tree, o, ldo, ws, wsb, None)


SHARED_SHAPE = [dict(ldt=3), dict(most=0, ldt=0), dict(n=0), dict(n=(1 << 20) + 1), dict(T=-1), dict(T=1 << 30), dict(cu=None),
                dict(ldt=1 << 61), dict(c=cache(pages=0)), dict(c=cache(page=8)), dict(c=cache(page=48)), dict(c=cache(page=2048)),
                dict(c=cache(heads=0)), dict(c=cache(d=96)), dict(c=cache(d=512)), dict(c=cache(d=0))]
SHARED_NULL = [dict(table=None), dict(lens=None), dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(kg=None)),
               dict(c=cache(vg=None)), dict(c=cache(fmt=1, ks=None)), dict(c=cache(fmt=1, vs=None))]
SHARED_ALIGN = [dict(table=at(6, 2)), dict(lens=at(7, 1)), dict(cu=at(8, 2)), dict(c=cache(k=at(1, 8))), dict(c=cache(v=at(2, 4))),
                dict(c=cache(kg=at(5, 2))), dict(c=cache(vg=at(5, 1))), dict(c=cache(fmt=1, ks=at(3, 8))),
                dict(c=cache(fmt=1, vs=at(4, 8)))]


@pytest.mark.parametrize("name", ["nvfp4_kv_cache_write", "nvfp4_kv_cache_read"])
def test_cache_calls_reject_bad_arguments(lib, name):
    f = getattr(lib, name)
    assert f(None, at(6), 4, 4, at(7), at(8), 3, 8, at(9), 256, at(10), 256, 1, None) == NULL
    assert rows_call(f, dt=2) == DTYPE and rows_call(f, dt=-1) == DTYPE
    assert rows_call(f, c=cache(fmt=2)) == MODE
    for kw in SHARED_SHAPE + [dict(ldk=255), dict(ldv=128), dict(ldk=1 << 61), dict(T=(1 << 30) - 1, c=cache(heads=4096, d=256), ldk=1 << 20, ldv=1 << 20)]:
        assert rows_call(f, **kw) == SHAPE, kw
    for kw in SHARED_NULL + [dict(k=None), dict(v=None)]:
        assert rows_call(f, **kw) == NULL, kw
    for kw in SHARED_ALIGN + [dict(k=at(9, 8)), dict(v=at(10, 2)), dict(ldk=260), dict(ldv=257), dict(dt=0, ldk=258)]:
        assert rows_call(f, **kw) == ALIGN, kw
    assert rows_call(f, T=0, k=None, v=None, table=None, lens=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def test_cache_calls_reject_overlaps(lib):
    w, r = lib.nvfp4_kv_cache_write, lib.nvfp4_kv_cache_read
    fp4 = dict(fmt=1)
    for kw in (dict(k=at(1)), dict(k=at(1, 65536 - 16)), dict(v=at(2, 16)), dict(k=at(2)), dict(v=at(1)), dict(table=at(1, 4)),
               dict(lens=at(2)), dict(cu=at(2, 64)), dict(c=cache(v=at(1, 32768))), dict(c=cache(kg=at(1))), dict(c=cache(vg=at(2, 4))),
               dict(c=cache(**fp4, ks=at(1, 16))), dict(c=cache(**fp4, vs=at(3))), dict(c=cache(**fp4), k=at(3)), dict(c=cache(**fp4), v=at(4))):
        assert rows_call(w, **kw) == ALIAS, kw
    for kw in (dict(k=at(1)), dict(v=at(2)), dict(k=at(10)), dict(k=at(9), v=at(9, 128)), dict(k=at(6)), dict(v=at(7)), dict(k=at(8)),
               dict(k=at(5)), dict(c=cache(**fp4), v=at(4, 16)), dict(c=cache(**fp4), k=at(3))):
        assert rows_call(r, **kw) == ALIAS, kw


def test_attn_rejects_bad_arguments(lib):
    assert lib.nvfp4_attn_cached(None, at(6), 4, 4, at(7), at(8), 3, 8, at(9), 512, 4, 0.1, None, at(10), 512, at(32), 1 << 40, None) == NULL
    assert attn(lib, c=cache(fmt=-1)) == MODE
    for kw in SHARED_SHAPE + [dict(ldq=511), dict(ldo=511), dict(ldq=1 << 61), dict(hq=3), dict(hq=0), dict(hq=-2), dict(hq=8192),
                              dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf)]:
        assert attn(lib, **kw) == SHAPE, kw
    for kw in SHARED_NULL + [dict(q=None), dict(o=None), dict(ws=None)]:
        assert attn(lib, **kw) == NULL, kw
    for kw in SHARED_ALIGN + [dict(q=at(9, 8)), dict(o=at(10, 8)), dict(ldq=516), dict(ldo=514), dict(tree=at(11, 4)), dict(ws=at(32, 128))]:
        assert attn(lib, **kw) == ALIGN, kw
    size = lib.nvfp4_attn_cached_workspace_size
    need = size(8, 3, 4, 2, 128)
    assert need > 0 and attn(lib, wsb=need - 1) == WORKSPACE
    for bad in ((0, 3, 4, 2, 128), (8, 0, 4, 2, 128), (8, 3, 3, 2, 128), (8, 3, 4, 0, 128), (8, 3, 4, 2, 96), (1 << 30, 3, 4, 2, 128)):
        assert size(*bad) == 0, bad
    for kw in (dict(o=at(9)), dict(o=at(9, 512)), dict(o=at(1)), dict(o=at(2, 32768)), dict(o=at(5)), dict(o=at(6)), dict(o=at(7)),
               dict(o=at(8)), dict(tree=at(10)), dict(ws=at(9)), dict(ws=at(1)), dict(ws=at(10)), dict(tree=at(32)),
               dict(c=cache(fmt=1), o=at(3)), dict(c=cache(fmt=1), o=at(4))):
        assert attn(lib, **kw) == ALIAS, kw
    assert attn(lib, T=0, q=None, o=None, ws=None, wsb=0) == OK
    assert lib.nvfp4_last_hip_error() == 0


def rope(lib, x=at(1), xt=1, ldx=768, qc=0, kc=512, T=8, hq=4, hk=2, d=128, qw=at(2), kw=at(3), eps=1e-6, table=at(4), n_pos=16, rot=64,
         pos=at(5), axes=1, pair=None, adj=0, q=at(6), ldq=512, k=at(7), ldk=256):
    return lib.nvfp4_qk_norm_rope(x, xt, ldx, qc, kc, T, hq, hk, d, qw, kw, eps, table, n_pos, rot, pos, axes, pair, adj, q, ldq, k, ldk, None)


def test_norm_rope_rejects_bad_arguments(lib):
    assert rope(lib, xt=2) == DTYPE
    assert rope(lib, adj=2) == MODE and rope(lib, adj=-1) == MODE
    for kw in (dict(d=96), dict(d=32), dict(hq=0), dict(hk=0), dict(hq=5000, ldx=1 << 20), dict(hk=-1), dict(T=-1), dict(T=(1 << 25) + 1),
               dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(rot=0), dict(rot=8), dict(rot=40), dict(rot=144), dict(n_pos=0),
               dict(axes=0), dict(axes=5), dict(ldx=0), dict(qc=-8), dict(qc=264), dict(kc=520), dict(kc=-8), dict(ldq=504), dict(ldk=248),
               dict(ldx=1 << 61, qc=0), dict(axes=2, pair=bytes([0] * 31 + [2])), dict(qc=1 << 62)):
        assert rope(lib, **kw) == SHAPE, kw
    for kw in (dict(x=None), dict(qw=None), dict(kw=None), dict(table=None), dict(pos=None), dict(q=None), dict(k=None), dict(axes=2)):
        assert rope(lib, **kw) == NULL, kw
    for kw in (dict(x=at(1, 8)), dict(ldx=772), dict(xt=0, ldx=772), dict(qc=4), dict(kc=508), dict(qw=at(2, 8)), dict(kw=at(3, 4)),
               dict(table=at(4, 8)), dict(pos=at(5, 2)), dict(q=at(6, 8)), dict(k=at(7, 2)), dict(ldq=516), dict(ldk=260)):
        assert rope(lib, **kw) == ALIGN, kw
    for kw in (dict(k=at(6)), dict(k=at(6, 512)), dict(q=at(2)), dict(k=at(3)), dict(q=at(4)), dict(q=at(5)), dict(q=at(1)),
               dict(q=at(1, 16), ldq=768), dict(k=at(1), ldk=768), dict(q=at(1, 512), ldq=768), dict(xt=0, q=at(1), ldq=768)):
        assert rope(lib, **kw) == ALIAS, kw
    assert rope(lib, T=0, x=None, q=None, k=None, qw=None, kw=None, table=None, pos=None) == OK
    assert lib.nvfp4_last_hip_error() == 0


def test_binding_refuses_what_it_sees():
    u8, f = torch.uint8, torch.float32
    k, v, g = torch.zeros((3, 2, 64, 128), dtype=u8), torch.zeros((3, 2, 128, 64), dtype=u8), torch.ones(1)
    for a in (dict(format="int4"), dict(format="nvfp4"), dict(v=k), dict(k=k.float()), dict(k=k[0]), dict(k_gs=g.double()),
              dict(k_scales=torch.zeros((3, 2, 64, 8), dtype=u8)), dict(k=k.transpose(0, 1)), dict()):  # the last: not on a GPU
        with pytest.raises(ValueError):
            nv.KvCache(**dict(dict(k=k, v=v, k_gs=g, v_gs=g, format="fp8"), **a))
    x = torch.zeros((4, 768), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.qk_norm_rope(x, torch.ones(128), torch.ones(128), torch.zeros((4, 64), dtype=f), torch.zeros(4, dtype=torch.int32),
                        q_col=0, k_col=512, n_q_heads=4, n_kv_heads=2)


def test_references_against_closed_forms():
    """The fp64 references on inputs whose results are known."""
    rng = np.random.default_rng(0)
    # a rotation by 0 is the norm; by a quarter turn (a, b) -> (-b, a); a head of ones times w is w
    x = rng.standard_normal((2, 3, 8))
    one, zero = np.ones((2, 2)), np.zeros((2, 2))
    n = A.norm_rope_ref(x, np.ones(8), 1e-30, one, zero, False)
    assert np.allclose(np.mean(n * n, -1), 1) and np.allclose(n / x, (n / x)[..., :1])
    t = A.norm_rope_ref(x, np.ones(8), 1e-30, zero, one, False)
    assert np.allclose(t[..., :2], -n[..., 2:4]) and np.allclose(t[..., 2:4], n[..., :2]) and np.allclose(t[..., 4:], n[..., 4:])
    t = A.norm_rope_ref(x, np.ones(8), 1e-30, zero, one, True)
    assert np.allclose(t[..., 0], -n[..., 1]) and np.allclose(t[..., 3], n[..., 2]) and np.allclose(t[..., 4:], n[..., 4:])
    # codes: every code's value is its own, ties go to even
    every = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(A.e4m3_codes(A.e4m3_values(every) * 0.3125, 0.3125), every)
    assert A.e4m3_codes(np.array([17 / 16, 19 / 16, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, np.inf, np.nan]), 1.0).tolist() == \
        [0x38, 0x3A, 0x00, 0x02, 0x7E, 0x7F, 0x7F]
    # equal scores: the mean of what is seen; one key: its value; nothing seen: zeros, whatever is hidden
    k, v = np.zeros((5, 1, 4)), rng.standard_normal((5, 1, 4))
    seen = np.array([[1, 1, 1, 1, 1], [0, 0, 1, 0, 0], [0, 0, 0, 0, 0]], bool)
    o, _, _, _ = A.attn_ref(rng.standard_normal((3, 2, 4)), k, v, seen, 1.0)
    assert np.allclose(o[0], v.mean(0)) and np.allclose(o[1], v[2]) and np.all(o[2] == 0)
    hidden = v.copy()
    hidden[[0, 1, 3, 4]] = np.nan
    assert np.array_equal(A.attn_ref(np.ones((1, 2, 4)), k, hidden, seen[1:2], 1.0)[0][0], np.broadcast_to(v[2], (2, 4)))
    # masks: causal rows, drafts behind a context
    assert A.seen_ref(2, 3, 4).tolist() == [[True, True, False, False], [True, True, True, False]]
    assert A.seen_ref(2, 3, 3, [1, -1]).tolist() == [[True, True, False], [True, True, True]]
