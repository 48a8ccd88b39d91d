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
def lib(host_lib):
    return host_lib


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
    "16 rows a wave": ((8, 8, 64, 16), [1, 2, 0, 1] * 16, [700, 0, 40, 15] + [17, 5, 0, 64] * 15),
    "32 rows a wave": ((24, 8, 64, 32), [7, 13, 0, 9] * 4, [600, 0, 40, 15] + [17, 5, 0, 64] * 3),
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


def check_one_hot(got, q, paged, kv, rows, starts, hq, scale):
    """Rows whose largest score is ahead of the others by more than scores can be off by, and 40 beside: the other
    weights are below e^-40 in all, so o is that key's value, times and divided by its weight: three fp32 roundings and
    one to bf16.  (A row has one key that is ahead in nearly all of the random rows; how many is asserted.)"""
    d, checked, seen = paged.d, 0, 0
    for i, (n, length) in enumerate(zip(rows, kv)):
        k, v = paged.values("k", i, length), paged.values("v", i, length)
        for j in range(n):
            for h in range(hq):
                keys = k[:length - n + j + 1, h // (hq // paged.hk)]
                x = q[starts[i] + j].reshape(hq, d)[h]
                s = keys @ x * scale
                big = np.max(np.abs(keys) @ np.abs(x)) * scale
                order = np.argsort(s)
                seen += 1
                if len(s) > 1 and s[order[-1]] - s[order[-2]] < 4 * (d + 8) * 2.0 ** -24 * big + 40:
                    continue
                checked += 1
                want = v[order[-1], h // (hq // paged.hk)]
                g = got[starts[i] + j].reshape(hq, d)[h]
                tol = (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -50 * np.abs(v).max()
                assert np.all(np.abs(g - want) <= tol), (i, j, h, s[order[-1]], np.abs(g - want).max())
    assert checked > 0.9 * seen, (checked, seen)


# maxima of about 1e8 to 1e26 in scores, positive and (few keys) negative
FACTORS = [1e8, 3e8, 1e9, 1e10, 3e10, 1e13, 1e17, 1e25]


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("form,heads,rows,ctx", [("16 rows", (4, 2, 64, 16), [1, 2], [129, 2]), ("32 rows", (4, 1, 64, 32), [5, 6], [600, 1]),
                                                 ("128 rows", (4, 1, 64, 16), [20, 30], [60, 0])])
@pytest.mark.parametrize("factor", FACTORS)
def test_finite_queries_of_any_size(lib, fmt, form, heads, rows, ctx, factor):
    """One-hot softmaxes: scores up to 1e27 in both directions give the value of the largest."""
    hq, hk, d, page = heads
    kv = [a + b for a, b in zip(rows, ctx)]
    paged = Paged(fmt, hk, d, page, kv, 21)
    q = H.bf16(factor * np.random.default_rng(5).standard_normal((sum(rows), hq * d)).astype(np.float32))
    got, starts = H.attn(lib, paged, rows, kv, hq, q)
    check_one_hot(got, H.f32(q).astype(np.float64), paged, kv, rows, starts, hq, float(np.float32(d ** -0.5)))


def common_part(hk, d, page, kv, group, n_rows, seed):
    """Scores of about 10,450 that differ by up to 39, every sum of which is exact in fp32: dim 0 gives each key
    4080 * 256, dim 1 a product of whole numbers up to 255 * 15.  (cache, queries [n_rows, hq * d], scale)."""
    paged = Paged("fp8", hk, d, page, kv, seed)
    rng = np.random.default_rng(seed)
    live = paged.codes["k"] != 0x7F
    for dim, values in ((0, np.array([256.0])), (1, np.arange(1.0, 16.0))):
        codes = A.e4m3_codes(rng.choice(values, paged.codes["k"].shape[:3]), 1.0)
        paged.codes["k"][..., dim] = np.where(live[..., dim], codes, 0x7F)
    q = np.zeros((n_rows, hk * group, d), np.float32)
    q[..., 0], q[..., 1] = 4080.0, rng.integers(1, 256, q.shape[:2])
    return paged, q.reshape(n_rows, -1), float(np.float32(0.01 / paged.gs["k"]))


def check_common_part(got, q, paged, rows, kv, starts, hq, scale):
    """As tests/test_gpu_attn.py's bound, with scores that are exact: their factor's error counts for their distance from
    the maximum only (39 of them; 8 for the sum's d)."""
    for i, (n, length) in enumerate(zip(rows, kv)):
        mask = A.seen_ref(n, length, length)
        x = q[starts[i]:starts[i] + n].astype(np.float64).reshape(n, hq, paged.d)
        O, mag, _, flat = A.attn_ref(x, paged.values("k", i, length), paged.values("v", i, length), mask, scale)
        err = np.abs(got[starts[i]:starts[i] + n].astype(np.float64).reshape(O.shape) - O)
        assert np.all(err <= tolerance(O, mag, np.full((n, hq), 39.0), flat, 8, length))


@pytest.mark.parametrize("heads,rows,ctx", [((4, 2, 64, 16), [1, 2], [700, 2]), ((4, 1, 128, 32), [5, 6], [600, 1]),
                                            ((4, 1, 64, 16), [30, 30], [400, 0])])
def test_large_scores_that_differ_little(lib, heads, rows, ctx):
    """Weights of scores far from zero go by their differences, in every part of a cut row."""
    hq, hk, d, page = heads
    kv = [a + b for a, b in zip(rows, ctx)]
    paged, q, scale = common_part(hk, d, page, kv, hq // hk, sum(rows), 22)
    got, starts = H.attn(lib, paged, rows, kv, hq, H.bf16(q), scale=scale)
    check_common_part(got, q, paged, rows, kv, starts, hq, scale)


TOP = 2 ** 31 - 1
LENGTHS = [([1, 1, 1], [5, 70, 1000]), ([3, 3, 3], [TOP, 100, 3]), ([5, 2], [TOP - 200, TOP]), ([40, 1, 90], [90, TOP, 4000]),
           ([100, 60], [TOP - 128, 60]), ([2, 0, 3], [-5, TOP, 0]), ([1] * 70, [TOP] * 35 + [64] * 35)]


@pytest.mark.parametrize("rows,kv", LENGTHS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2)])
def test_ranges_take_every_step_once(lib, rows, kv, tree, hq, hk):
    """Each unit's steps are in one range or in neighbouring ones, none twice, none left out, for lengths up to int32's
    last; whole units have no slot, cut ones those of their cuts."""
    d, page, max_pages = 64, 1024, 1 << 21
    tile_rows = H.plan(lib, sum(rows), len(rows), hk, hq // hk, d)[0]
    tokens = tile_rows // (hq // hk)
    got = {}
    for r, seq, tile, minor, k0, k1, slot, steps in H.pieces(lib, rows, kv, hq, hk, d, page, max_pages, tree).tolist():
        got.setdefault((seq, tile, minor), []).append((r, k0, k1, slot, steps))
    units = {(i, t, h) for i, n in enumerate(rows) for t in range(-(-n // tokens)) for h in range(hk)}
    assert set(got) == units
    for (seq, tile, _), parts in got.items():
        last = kv[seq] if tree else min(kv[seq], kv[seq] - rows[seq] + min((tile + 1) * tokens, rows[seq]))
        steps = -(-max(0, min(last, TOP - 127)) // 64)
        assert {p[4] for p in parts} == {steps}
        assert [p[0] for p in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))
        assert parts[0][1] == 0 and parts[-1][2] >= steps and all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
        slots = [-1] if len(parts) == 1 else [2 * parts[0][0] + 1] + [2 * p[0] for p in parts[1:]]
        assert [p[3] for p in parts] == slots


# scale, tensor scale of the keys, size of the queries: scores of ordinary size whose factors' product is not
FACTORS_OF_SCORES = [(3.2e38, 1e-30, 1e-9), (1e30, 1e9, 3e-40), (1e-12, 2.0 ** -100, 6e37)]


@pytest.mark.parametrize("form", list(CASES))
@pytest.mark.parametrize("scale,k_gs,spread", FACTORS_OF_SCORES)
def test_factors_whose_product_is_no_fp32_number(lib, form, scale, k_gs, spread):
    (hq, hk, d, page), rows, ctx = CASES[form]
    kv = [a + b for a, b in zip(rows, ctx)]
    run(lib, Paged("fp8", hk, d, page, kv, 23, k_gs=k_gs), rows, kv, hq, form, scale=scale, spread=spread)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("at_end", [True, False])
@pytest.mark.parametrize("hq,hk,d,page,form", [(160, 1, 64, 32, "128 rows"), (40, 1, 128, 16, "128 rows"), (20, 1, 256, 64, "32 rows"),
                                               (7, 1, 64, 256, "16 rows"), (300, 1, 64, 16, "128 rows")])
def test_many_heads_of_one_key_value_head(lib, fmt, at_end, hq, hk, d, page, form):
    """Groups of heads that fill no tile, or take several; tiles whose last waves have no row."""
    kv = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 257]
    run(lib, Paged(fmt, hk, d, page, kv, hq + d), [1] * len(kv), kv, hq, form, cu=False, at_end=at_end)
