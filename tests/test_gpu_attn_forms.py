"""Every form of the attention kernels (rows at a time, a range for a workgroup or for a wave) with every head size and
cache format, against the fp64 formula.  A call's form is known by the workspace that it asks for, so a changed
rule cannot leave a form without a case unnoticed.  Bound: tests/test_gpu_attn.py."""
import numpy as np
import pytest

import nvfp4_w4a4_quantized_05_amd as nv
from tests.attn_util import Paged
from tests.test_gpu_attn import run, tree_masks

JOINT_BYTES = 32
FORMS = {"16 rows": (16, 1), "32 rows": (32, 1), "16 rows a wave": (16, 4), "32 rows a wave": (32, 4), "128 rows": (128, 1)}


def workspace(form, d):
    rows, waves = FORMS[form]
    ranges = waves * (512 if d < 256 else 256)
    return 2 * ranges * rows * (d + 3) * 4 + ranges * JOINT_BYTES


def batch(form, d):
    """(query heads, key/value heads, rows of each sequence, lengths) that the form is chosen for; one long cut sequence, empty ones,
    lengths of a step and beside it."""
    few = [1000, 1, 63, 64, 65]
    many = [3000] + [[80, 1, 40, 64, 65, 0, 129, 17, 200][i % 9] for i in range(1, 72)]
    if form == "16 rows":
        return 24 if d == 256 else 8, 4, [2, 1, 2, 0, 3], [n + 3 for n in few]
    if form == "32 rows":
        return 24, 4, [4, 5, 3, 4, 4], [n + 5 for n in few]
    if form == "128 rows":
        return 24, 4, [40, 7, 0, 90, 30], [n + 90 for n in few]
    heads = (8, 8) if form == "16 rows a wave" else (32, 8)
    rows = [(1, 2, 0, 1)[i % 4] if form == "16 rows a wave" else (6, 8, 5, 7, 0, 9)[i % 6] for i in range(72)]
    return *heads, rows, [k + n for k, n in zip(many, rows)]


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("d", [64, 128, 256])
def test_batches_choose_the_form(form, d):
    hq, hk, rows, _ = batch(form, d)
    need = nv.load().nvfp4_attn_cached_workspace_size(sum(rows), len(rows), hq, hk, d)
    assert need == workspace(form, d), [f for f in FORMS if need == workspace(f, d)]


@pytest.mark.gpu
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("tree", [False, True])
def test_every_form(form, d, fmt, tree):
    hq, hk, rows, kv = batch(form, d)
    print(f"[attn] {form} {fmt} {hq}/{hk}x{d} tree {tree}", flush=True)
    rng = np.random.default_rng(d)
    paged = Paged(fmt, hk, d, 32, kv, d + 2)
    paged.set_nan("v", 0, kv[0] - 1, hk - 1, 5)   # seen by the last row, or by one branch
    paged.set_nan("v", 0, 300, 1, 9)              # by all rows
    paged.set_nan("k", 1, 0, 2, 3)
    run(paged, rows, kv, hq, seed=15, tree=[tree_masks(rng, n) for n in rows] if tree else None, lead=1, tail=2)
