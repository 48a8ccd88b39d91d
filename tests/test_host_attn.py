"""nvfp4_attn_cached's kernels in a build for the host: the sources as they are,
lane by lane, on arrays that end at unmapped pages.  What is checked is that
no lane reads or writes past an array, that lanes which exchange values or meet
at a barrier all come there, and the results, against the fp64 formula within the
bound that tests/test_gpu_attn.py derives (products of 32 are summed in another
order here, which that bound covers).  Needs clang (skipped without it)."""
import numpy as np
import pytest

from oracle import attn_ref as A
from tests import host_wave as H
from tests.attn_util import Paged
from tests.test_gpu_attn import tolerance, tree_masks

FORMS = {"16 rows": (16, False), "32 rows": (32, False), "16 rows a wave": (16, True), "32 rows a wave": (32, True),
         "128 rows": (128, False)}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if H.clang() is None:
        pytest.skip("clang not available")
    return H.build(str(tmp_path_factory.mktemp("host")))


def run(lib, paged, rows, kv, hq, form, *, seed=0, tree=None, scale=None, spread=1.0, cu=True, lead=0, tail=0, at_end=True,
        q_edit=None):
    """One call; `form`: the kernel that it is meant for.  Checks every row and the rows around the sequences."""
    d, T = paged.d, lead + sum(rows) + tail
    got_form = H.plan(lib, T, len(rows), paged.hk, hq // paged.hk, d)
    assert (got_form[0], bool(got_form[2])) == FORMS[form], got_form
    q = (spread * np.random.default_rng(seed).standard_normal((T, hq * d))).astype(np.float32)
    if q_edit:
        q_edit(q)
    bits = H.bf16(q)
    got, starts = H.attn(lib, paged, rows, kv, hq, bits, tree=tree, scale=scale, cu=cu, lead=lead, tail=tail, at_end=at_end)
    assert np.all(got[:lead] == 7.5) and np.all(got[lead + sum(rows):] == 7.5)
    qh = H.f32(bits).astype(np.float64).reshape(T, hq, d)
    sc = float(np.float32(d ** -0.5 if scale is None else scale))
    for i, (n, length) in enumerate(zip(rows, kv)):
        if n == 0:
            continue
        have = min(max(length, 0), paged.max_pages * paged.page)
        at = slice(starts[i], starts[i] + n)
        mask = A.seen_ref(n, length, have, None if tree is None else tree[i])
        page = paged.table[i, np.arange(have) // paged.page]
        mask &= ((page >= 0) & (page < paged.n_pages))[None]
        O, mag, big, flat = A.attn_ref(qh[at], paged.values("k", i, have), paged.values("v", i, have), mask, sc)
        g = got[at].astype(np.float64).reshape(n, hq, d)
        nan = np.isnan(O)
        assert np.array_equal(np.isnan(g), nan), f"sequence {i}: NaN at {np.argwhere(np.isnan(g) != nan)[:3].tolist()}"
        err, tol = np.abs(g - O)[~nan], tolerance(O, mag, big, flat, d, have)[~nan]
        assert np.all(err <= tol), f"sequence {i}: worst {np.max(err / tol)} of the tolerance"
    return got


# query and key/value heads, head size, page; rows of each sequence, what each has before them
CASES = {
    "16 rows": ((6, 1, 256, 64), [1, 2, 0, 1], [300, 0, 40, 15]),
    "32 rows": ((4, 2, 128, 16), [12, 9, 0, 17], [900, 5, 0, 63]),
    "128 rows": ((6, 2, 64, 32), [40, 0, 130, 3], [70, 0, 5, 1000]),
}


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("form", list(CASES))
@pytest.mark.parametrize("at_end", [True, False])
def test_bounds_and_values(lib, fmt, form, at_end):
    (hq, hk, d, page), rows, ctx = CASES[form]
    kv = [a + b for a, b in zip(rows, ctx)]
    paged = Paged(fmt, hk, d, page, kv, 3)
    paged.set_nan("v", 0, kv[0] - 1, 0, 5)
    run(lib, paged, rows, kv, hq, form, lead=2, tail=3, at_end=at_end)
