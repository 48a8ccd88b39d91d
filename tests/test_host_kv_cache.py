"""nvfp4_kv_cache_write and _read in a build for the host (tests/host_wave): accesses, bytes and values, as
tests/test_gpu_kv_cache.py checks them on the GPU."""
import numpy as np
import pytest

from oracle import attn_ref as A
from tests import host_wave as H
from tests.attn_util import Paged
from tests.test_gpu_kv_cache import CASES, want_codes


def rows_of(paged, T, bf16, seed):
    x = np.random.default_rng(seed).standard_normal((2, T, paged.hk * paged.d)).astype(np.float32)
    return (H.bf16(x), H.f32(H.bf16(x))) if bf16 else (x, x)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("hk,d,page", [(2, 256, 64), (2, 128, 16), (3, 64, 32), (1, 128, 1024)])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("at_end", [True, False])
def test_write(host_lib, fmt, bf16, hk, d, page, case, at_end):
    rows, kv = CASES[case]
    lead, tail = (2, 3) if case else (0, 0)
    T = lead + sum(rows) + tail
    paged = Paged(fmt, hk, d, page, kv, d + case)
    paged.table[0, 0] = -1
    given, x = rows_of(paged, T, bf16, case)
    _, _, left = H.kv_rows(host_lib, paged, rows, kv, *given, write=True, cu=case > 0, lead=lead, at_end=at_end)
    row = lead
    for i, (n, length) in enumerate(zip(rows, kv)):
        for name, t in zip("kv", x):
            c, s = want_codes(fmt, t[row:row + n].reshape(n, hk, d), paged.gs[name]) if n else (None, None)
            for j in range(n):
                p = length - n + j
                if 0 <= p < paged.max_pages * page and 0 <= paged.table[i, p // page] < paged.n_pages:
                    pg, at = paged.place(i, p)
                    paged.codes[name][pg, :, at] = c[j]
                    if s is not None:
                        paged.scales[name][pg, :, at] = s[j]
        row += n
    for name in "kv":
        assert np.array_equal(left[name, "codes"], paged.codes[name])
        assert np.array_equal(left[name, "scales"], paged.scales[name])


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("hk,d,page", [(2, 256, 64), (2, 128, 16), (3, 64, 32)])
@pytest.mark.parametrize("at_end", [True, False])
def test_read(host_lib, fmt, bf16, hk, d, page, at_end):
    rows, kv, lead, tail = [90, 0, 1, 33, 16, 200, 6], [90, 5, 40, 100, 16, 150, -3], 2, 3
    paged = Paged(fmt, hk, d, page, kv, d)
    paged.table[3, 80 // page] = -1
    T = lead + sum(rows) + tail
    fill = np.full((T, hk * d), 7.5, np.float32)
    k, v, _ = H.kv_rows(host_lib, paged, rows, kv, *[H.bf16(fill) if bf16 else fill] * 2, write=False, lead=lead, at_end=at_end)
    for name, got in (("k", k), ("v", v)):
        want, row = fill.astype(np.float64), lead
        for i, (n, length) in enumerate(zip(rows, kv)):
            for j in range(n):
                p = length - n + j
                want[row + j] = 0.0
                if 0 <= p < paged.max_pages * page and 0 <= paged.table[i, p // page] < paged.n_pages:
                    pg, at = paged.place(i, p)
                    want[row + j] = A.kv_values(fmt, paged.codes[name][pg, :, at], paged.scales[name][pg, :, at], paged.gs[name]).ravel()
            row += n
        once = want.astype(np.float32)
        assert np.array_equal(got, H.bf16(once) if bf16 else once)
