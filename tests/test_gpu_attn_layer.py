"""The mixer layer of examples/attn_layer.py: its calls in the order a model
makes them, each checked against the fp64 reference on what the call before
left (tolerances of tests/test_gpu_rope.py and tests/test_gpu_attn.py; codes and
values of the cache exactly), over prompts, a chunk, single tokens, a tree of
drafts and the accepted branch; and a captured step against the eager one."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from examples import attn_layer
from oracle import attn_ref as A
from tests.attn_util import i32
from tests.gpu_util import host_f32, need_gpu
from tests.test_gpu_attn import tolerance
from tests.test_gpu_kv_cache import want_codes

pytestmark = pytest.mark.gpu
HIDDEN, PAGE, ROT = 256, 16, 32


def check_heads(layer, t, positions):
    """q and k of a call from the projection's columns."""
    x = host_f32(t["rows"]).astype(np.float64)
    table = layer.cos_sin.cpu().numpy()[positions]
    cos, sin = table[:, :ROT // 2], table[:, ROT // 2:]
    col = 0
    for name, heads, w in (("q", layer.n_q, layer.q_w), ("k", layer.n_kv, layer.k_w)):
        xs = x[:, col:col + heads * layer.d].reshape(-1, heads, layer.d)
        col += heads * layer.d
        w = w.cpu().numpy()
        want = A.norm_rope_ref(xs, w, 1e-6, cos, sin, False)
        turn = np.abs(A.norm_rope_ref(xs, w, 1e-6, np.ones_like(cos), np.zeros_like(sin), False))
        both = turn[..., :ROT // 2] + turn[..., ROT // 2:ROT]
        turn[..., :ROT // 2] = turn[..., ROT // 2:ROT] = both
        tol = (layer.d / 32 + 12) * 2.0 ** -24 * turn + 2.0 ** -8 * np.abs(want) + 2.0 ** -126
        assert np.all(np.abs(host_f32(t[name]).reshape(want.shape) - want) <= tol), name


def check_call(layer, t, positions, rows, kv, table, tree=None):
    """One call's operators; the sequences' values are read back out of the cache."""
    hk, d, hq = layer.n_kv, layer.d, layer.n_q
    check_heads(layer, t, positions)
    cu = np.concatenate([[0], np.cumsum(rows)])
    all_of = np.concatenate([[0], np.cumsum(kv)])
    dev = t["q"].device
    values = nv.kv_cache_read(layer.cache, table, i32(kv, dev), i32(all_of, dev), rows=int(all_of[-1]), out_dtype=torch.float32)
    values = [host_f32(v).astype(np.float64).reshape(-1, hk, d) for v in values]
    new = [host_f32(t[n]).reshape(-1, hk, d) for n in "kv"]
    q, o = host_f32(t["q"]).astype(np.float64).reshape(-1, hq, d), host_f32(t["o"]).astype(np.float64).reshape(-1, hq, d)
    scale = float(np.float32(d ** -0.5))
    for i, (n, length) in enumerate(zip(rows, kv)):
        if n == 0:
            continue
        k, v = (x[all_of[i]:all_of[i + 1]] for x in values)
        at = slice(cu[i], cu[i + 1])
        for got, x, gs in ((k, new[0], layer.cache.k_gs), (v, new[1], layer.cache.v_gs)):
            gs = np.float32(gs.item())
            codes, scales = want_codes(layer.cache.format, x[at], gs)
            assert np.array_equal(got[length - n:], A.kv_values(layer.cache.format, codes, scales, gs).astype(np.float32))
        seen = A.seen_ref(n, length, length, None if tree is None else tree[i])
        O, mag, big, flat = A.attn_ref(q[at], k, v, seen, scale)
        err, tol = np.abs(o[at] - O), tolerance(O, mag, big, flat, d, length)
        assert np.all(err <= tol), f"sequence {i}: {np.max(err / tol)}"
    want = nv.quantize(t["o"], layer.out_gs, from_amax=False)
    assert torch.equal(t["out_codes"], want[0]) and torch.equal(t["out_scales"], want[1])


def make(fmt, d, n_seqs, room, dev, seed):
    pages = -(-room // PAGE)
    layer = attn_layer.AttnLayer(HIDDEN, 4, 2, d, ROT, n_seqs * pages, page_size=PAGE, n_pos=room, fmt=fmt, seed=seed, device=dev)
    order = np.random.default_rng(seed).permutation(n_seqs * pages).astype(np.int32)
    return layer, torch.from_numpy(order.reshape(n_seqs, pages)).to(dev)


def rows_of(n, dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn((n, HIDDEN), generator=g, device=dev).bfloat16() for _ in range(2))


@pytest.mark.parametrize("fmt,d", [("fp8", 128), ("nvfp4", 64)])
def test_layer_is_its_parts(fmt, d):
    dev = need_gpu()
    layer, table = make(fmt, d, 4, 300, dev, 1)
    kv = [0, 0, 0, 0]

    def call(rows, seed, positions=None, tree=None):
        for i in range(4):
            kv[i] += rows[i]
        if positions is None:
            positions = [p for n, length in zip(rows, kv) for p in range(length - n, length)]
        one = all(n == 1 for n in rows) and tree is None
        x, r = rows_of(sum(rows), dev, seed)
        before, t = r.clone(), {}
        y = layer.forward(x, r, i32(positions, dev), table, i32(kv, dev),
                          None if one else i32(np.concatenate([[0], np.cumsum(rows)]), dev),
                          None if tree is None else torch.from_numpy(np.concatenate(tree)).to(dev), trace=t)
        print(f"[layer] {fmt} rows {rows} lengths {kv}", flush=True)
        assert np.all(np.abs(host_f32(r) - (host_f32(x) + host_f32(before))) <= 2.0 ** -7 * np.abs(host_f32(r)))
        check_call(layer, t, np.array(positions), rows, kv, table, tree)
        assert y.shape == x.shape and bool(torch.isfinite(y).all())

    call([70, 1, 0, 33], 2)               # prompts
    call([40, 130, 17, 0], 3)             # chunks that go on, and new ones
    for step in range(3):
        call([1, 1, 1, 1], 4 + step)      # one token each
    # drafts: two guesses, one and two tokens behind them
    tree = [np.array([0b00001, 0b00010, 0b00101, 0b01010, 0b11010], dtype=np.int64)] * 4
    depth = [0, 0, 1, 1, 2]
    call([5] * 4, 8, [length + p for length in kv for p in depth], tree)
    # the second branch (drafts 1, 3, 4) is taken: its rows go where the drafts stood, then decoding goes on
    for i in range(4):
        kv[i] -= 5
    call([3] * 4, 9)
    call([1, 1, 1, 1], 10)


def test_step_under_graph_capture():
    """A decode step and a tree's captured; lengths, positions and pages change between the replays."""
    dev = need_gpu()
    layer, table = make("fp8", 128, 3, 200, dev, 2)
    rows = [20, 90, 3]
    x, r = rows_of(sum(rows), dev, 1)
    layer.forward(x, r, i32([p for n in rows for p in range(n)], dev), table, i32(rows, dev), i32([0, 20, 110, 113], dev))
    xs, rs0 = rows_of(3, dev, 2)
    rs, pos, lens = rs0.clone(), i32(rows, dev), i32([n + 1 for n in rows], dev)
    layer.forward(xs, rs, pos, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(xs, rs, pos, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(xs, rs, pos, table, lens)
    for step in range(4):
        print(f"[layer] replay {step}", flush=True)
        pos.copy_(i32([n + step for n in rows], dev))
        lens.copy_(i32([n + step + 1 for n in rows], dev))
        if step == 2:
            table.copy_(table.flip(0))  # other pages: what they hold is another request's
        rs.copy_(rs0)
        graph.replay()
        torch.cuda.synchronize()
        got, cache = y.clone(), [layer.cache.k.clone(), layer.cache.v.clone()]
        rs2 = rs0.clone()
        want = layer.forward(xs, rs2, pos, table, lens)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(rs, rs2)
        assert torch.equal(cache[0], layer.cache.k) and torch.equal(cache[1], layer.cache.v)


def test_example_runs(capsys):
    need_gpu()
    attn_layer.main()
    out = capsys.readouterr().out
    assert out.count("finite: True") == 4
