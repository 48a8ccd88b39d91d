"""nvfp4_gdn_prefill and nvfp4_gdn_decode against the fp64 recurrence.

State tolerance (u = 2^-24): a perturbation of a token's write is carried on by
alpha I - beta khat khat^T, of norm c_t = max(alpha_t, |alpha_t - beta_t|) <= 1.
Written token by token, a token adds at most (128 + 16) u M_t, M_t the running
maximum of |S_s|_F + beta_s |v_s|.  Written in chunks of up to 64 tokens, u_t
gathers besides the 128-term product with the chunk's start state two sums of
up to 64 earlier writes (the inverse's product and the one that forms it), and
the state's update one more: (128 + 16 + 4 * 64) u M_t per token.  So
e_t <= c_t e_{t-1} + 400 u M_t, and 160 u M_t for the token form of decode.

Output tolerance.  decode, fp32: both terms of o = (alpha S_{t-1}^T q + (k . q) w)
/ sqrt(128) are at most 2 M_t, each off by (128 + 16) u of itself, on a state off by
e_{t-1}; a bf16 o adds 2^-8 |o|.  prefill: o is a bf16 result of products whose
operands are rounded to bf16 once (2^-9 of each): the chunk's start state, the
scores and the writes, so with s the chunk's first token
|do_t| <= [e_t + 2^-9 |S_{s-1}|_F a_t + 2^-8 sum_{j = s..t} a_{t,j} |qhat_t . khat_j| |w_j|
+ 400 u M_t] / sqrt(128) + 2^-8 |o_t|, a the decays in between."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from oracle import gdn_ref as G
from oracle import mixer_ref as M
from tests.gpu_util import host_f32, need_gpu

pytestmark = pytest.mark.gpu
D, U, CHUNK = 128, 2.0 ** -24, 64
BF, F32 = torch.bfloat16, torch.float32


def _inputs(T, n_qk, n_v, seed, kind="mixed"):
    """q | k | v | g | beta as fp32 arrays, values exact in bf16 for q, k, v."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, D * (2 * n_qk + n_v))).astype(np.float32)
    g = -np.exp(rng.uniform(np.log(1e-4), np.log(2.0), (T, n_v))).astype(np.float32)
    beta = (1 / (1 + np.exp(-rng.standard_normal((T, n_v))))).astype(np.float32)
    k = x[:, n_qk * D:2 * n_qk * D]
    if kind == "hold":                 # nothing decays, keys point the same way: the inverse has no small entries
        g[:] = 0
        k[:] = np.abs(k) + 1
        beta[:] = np.where(rng.random(beta.shape) < 0.5, 1.0, beta)
    elif kind == "reset":              # alpha = 0 now and then, beta = 0 and 1
        g[rng.random(g.shape) < 0.1] = -np.inf
        g[rng.random(g.shape) < 0.05] = -500.0
        beta[rng.random(beta.shape) < 0.3] = 0.0
        beta[rng.random(beta.shape) < 0.3] = 1.0
    elif kind == "zero":               # keys and queries of length zero
        k[rng.random(T) < 0.3] = 0
        x[rng.random(T) < 0.2, :n_qk * D] = 0
    elif kind == "scales":             # rows of very different size, equal keys in a run
        x *= np.exp2(rng.integers(-20, 21, (T, 1))).astype(np.float32)
        k[T // 2:] = k[T // 2]
    return torch.from_numpy(x).to(BF).float().numpy(), g, beta   # what the kernels get


def _host(x, g, beta, n_qk, n_v):
    T = x.shape[0]
    q = x[:, :n_qk * D].reshape(T, n_qk, D)
    k = x[:, n_qk * D:2 * n_qk * D].reshape(T, n_qk, D)
    return q, k, x[:, 2 * n_qk * D:].reshape(T, n_v, D), g, beta


def _bounds(q, k, v, g, beta, cu, starts, per_token):
    """Per row and head: the state allowance e_t, M_t and (chunked) the bf16 allowance of o; and the exact results."""
    n_v, head = v.shape[1], np.arange(v.shape[1]) * q.shape[1] // v.shape[1]
    o, S, norms = M.gdn_packed_ref(q, k, v, g, beta, cu, starts)
    alpha = np.exp(g.astype(np.float64))
    c = np.maximum(alpha, np.abs(alpha - beta))
    e, Mt, half = np.zeros(norms.shape), np.zeros(norms.shape), np.zeros(norms.shape)
    final = np.zeros((len(cu) - 1, n_v))
    qh, kh = G.l2_normalize(q)[:, head], G.l2_normalize(k)[:, head]
    for i in range(len(cu) - 1):
        a, b = int(cu[i]), int(cu[i + 1])
        acc = np.zeros(n_v)
        run = np.zeros(n_v) if starts is None or starts[i] is None else np.linalg.norm(starts[i].reshape(n_v, -1), axis=1)
        prev = run.copy()                                        # |S_{t-1}|_F
        for t in range(a, b):
            w_max = beta[t] * (np.linalg.norm(v[t], axis=1) + prev)     # |w_t| at most
            run = np.maximum(run, np.maximum(norms[t], prev) + beta[t] * np.linalg.norm(v[t], axis=1))
            acc = c[t] * acc + per_token * U * run
            e[t], Mt[t] = acc, run
            if (t - a) % CHUNK == 0:
                s, base, wr, decays = t, prev.copy(), [], []
            wr.append(w_max)
            decays = [d * alpha[t] for d in decays] + [np.ones(n_v)]
            base = base * alpha[t]
            dots = [np.abs(np.sum(qh[t] * kh[s + j], axis=1)) for j in range(t - s + 1)]
            half[t] = 2.0 ** -9 * base + 2.0 ** -8 * sum(d * p * w for d, p, w in zip(decays, dots, wr))
            prev = norms[t]
        final[i] = acc
    return o, S, e, Mt, half, norms, final


def _prefill(lens, n_qk, n_v, *, kind="mixed", gates=F32, start=True, seed=0, pad=0, tail=0, skip=(), separate=False):
    dev = need_gpu()
    print(f"[prefill] lens {lens} heads {n_qk}/{n_v} {kind} gates {gates} start {start}", flush=True)
    n, T = len(lens), sum(lens) + tail
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, g, beta = _inputs(T, n_qk, n_v, seed, kind)
    gt = torch.from_numpy(np.concatenate([beta, g], 1)).to(gates)           # beta first, then g
    beta, g = gt.float().numpy()[:, :n_v], gt.float().numpy()[:, n_v:]
    xt = torch.full((T, x.shape[1] + 8 * pad), float("nan"), dtype=BF, device=dev)
    xt[:sum(lens), 8 * pad:] = torch.from_numpy(x[:sum(lens)]).to(dev).to(BF)
    gd = torch.full((T, 2 * n_v + pad), float("nan"), dtype=gates, device=dev)
    gd[:sum(lens), :2 * n_v] = gt[:sum(lens)].to(dev)
    rng = np.random.default_rng(seed + 1)
    slots = rng.permutation(n + 2)[:n].astype(np.int32)
    for i in skip:
        slots[i] = -5 if i % 2 else n + 2
    pool = torch.from_numpy((rng.standard_normal((n + 2, n_v, D, D)) * 0.3).astype(np.float32)).to(dev)
    before = pool.clone()
    out = torch.full_like(pool, 7.0) if separate else pool
    o = torch.full((T, n_v * D + 8 * pad), float("nan"), dtype=BF, device=dev)
    nv.gdn_prefill(xt, gd, torch.from_numpy(cu).to(dev), q_col=8 * pad, k_col=8 * pad + n_qk * D,
                   v_col=8 * pad + 2 * n_qk * D, g_col=n_v, beta_col=0, n_qk_heads=n_qk, n_v_heads=n_v,
                   state_in=pool if start else None, state_out=out, slots=torch.from_numpy(slots).to(dev), o=o)
    torch.cuda.synchronize()
    starts = [before[s].cpu().numpy() if start and i not in skip else None for i, s in enumerate(slots)]
    q, k, v, g, beta = _host(x, g, beta, n_qk, n_v)
    O, S, e, Mt, half, norms, final = _bounds(q, k, v, g, beta, cu, starts, 400)
    ov, sv = host_f32(o).astype(np.float64), out.cpu().numpy()
    worst = [0.0, 0.0]
    for i in range(n):
        a, b = cu[i], cu[i + 1]
        got = ov[a:b, :n_v * D].reshape(b - a, n_v, D)
        if i in skip:
            assert np.all(got == 0)
            continue
        tol = (e[a:b] + half[a:b] + 400 * U * Mt[a:b]) / np.sqrt(D) + 2.0 ** -8 * np.linalg.norm(O[a:b], axis=2) + 1e-30
        err = np.linalg.norm(got - O[a:b], axis=2)
        assert np.all(err <= tol), f"sequence {i}: o, worst error / tolerance {np.max(err / tol)}"
        es = np.linalg.norm((sv[slots[i]] - S[i]).reshape(n_v, -1), axis=1)
        assert np.all(es <= final[i] + 1e-30), f"sequence {i}: state, worst {np.max(es / (final[i] + 1e-30))}"
        worst = [max(worst[0], np.max(err / tol, initial=0.0)), max(worst[1], np.max(es / (final[i] + 1e-30)))]
    print(f"  worst error / tolerance: o {worst[0]:.3f}, state {worst[1]:.4f}", flush=True)
    assert np.all(np.isnan(ov[sum(lens):])) and np.all(np.isnan(ov[:, n_v * D:])), "o written where it must not be"
    free = [s for s in range(n + 2) if s not in [slots[i] for i in range(n) if i not in skip]]
    want = torch.full_like(pool, 7.0) if separate else before
    assert torch.equal(out[free], want[free]), "a slot of no sequence was written"
    if separate:
        assert torch.equal(pool, before), "state_in was written"


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [300]])
def test_prefill_lengths(lens):
    _prefill(lens, 2, 4, seed=lens[0])


@pytest.mark.parametrize("lens,n_qk,n_v,gates,start", [
    ([0, 1, 64, 0, 129, 5], 1, 1, BF, True), ([70, 3], 1, 3, F32, False), ([33, 64, 200], 4, 4, BF, True),
    ([5, 0, 0, 66], 2, 8, F32, True), ([130], 16, 32, BF, False), ([1] * 9, 2, 2, F32, True)])
def test_prefill_packed(lens, n_qk, n_v, gates, start):
    _prefill(lens, n_qk, n_v, gates=gates, start=start, seed=len(lens), pad=3, tail=2, separate=start)


@pytest.mark.parametrize("kind", ["hold", "reset", "zero", "scales"])
def test_prefill_hard_values(kind):
    _prefill([200, 64, 1, 77], 2, 4, kind=kind, seed=5)


@pytest.mark.parametrize("lens,n_qk,n_v,gates", [
    ([1, 70, 0, 64, 130, 3, 63, 65] * 8, 2, 8, BF),              # 64 sequences x 8 heads
    ([2, 66, 0, 1, 129] * 14, 1, 8, F32)])                       # 70 sequences x 8 heads
def test_prefill_many_sequences(lens, n_qk, n_v, gates):
    _prefill(lens, n_qk, n_v, gates=gates, seed=len(lens), pad=1, tail=3, skip=(4, 7, 23), separate=True)


@pytest.mark.parametrize("lens,n_qk,n_v,gates,kind", [
    ([1, 70, 0, 64, 130, 3, 63, 65] * 3, 2, 8, BF, "mixed"), ([200, 1, 0, 65] * 16, 1, 3, F32, "hold"),
    ([129] * 6, 16, 32, F32, "reset"), ([5, 64, 192] * 9, 4, 12, BF, "scales")])   # 192 to 324 sequences x heads
def test_prefill_some_sequences(lens, n_qk, n_v, gates, kind):
    _prefill(lens, n_qk, n_v, gates=gates, kind=kind, seed=len(lens) + n_v, pad=1, tail=3, skip=(2,), separate=True)


def test_prefill_many_sequences_hard_values():
    _prefill([64, 20, 70] * 22, 1, 8, kind="reset", seed=21)
    _prefill([30, 129] * 32, 2, 8, kind="scales", seed=22)
    _prefill([200] + [5] * 63, 1, 8, kind="hold", seed=23)


def test_prefill_of_a_sequence_does_not_depend_on_how_many_there_are():
    """Both walks over the chunks (few sequences, many) against each other: o within the rounding of its products."""
    x, gates, lay = _tensors(64 * 40, 2, 8, 24)
    one = torch.zeros((1, 8, D, D), device=x.device)
    many = torch.zeros((64, 8, D, D), device=x.device)
    o = nv.gdn_prefill(x, gates, torch.arange(0, 65 * 40, 40, dtype=torch.int32, device=x.device), **lay, state_out=many)
    for i in (0, 17, 63):
        r = slice(40 * i, 40 * i + 40)
        a = nv.gdn_prefill(x[r].contiguous(), gates[r].contiguous(), _cu(0, 40), **lay, state_out=one)
        assert torch.allclose(a.float(), o[r].float(), rtol=2.0 ** -6, atol=2.0 ** -8 * float(a.float().abs().max()))
        assert float((one[0] - many[i]).norm()) <= 40 * 400 * U * float(many[i].norm())


def test_prefill_long():
    _prefill([2500], 1, 2, seed=9)
    _prefill([1500], 1, 1, kind="hold", seed=10)


def test_prefill_skips_sequences_without_a_slot():
    _prefill([70, 5, 64, 0, 9], 1, 2, seed=11, skip=(0, 3, 4))


def _tensors(T, n_qk, n_v, seed, kind="mixed", gates=F32):
    dev = need_gpu()
    x, g, beta = _inputs(T, n_qk, n_v, seed, kind)
    lay = dict(q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v, n_qk_heads=n_qk, n_v_heads=n_v)
    return torch.from_numpy(x).to(dev).to(BF), torch.from_numpy(np.concatenate([g, beta], 1)).to(dev).to(gates), lay


def _cu(*c):
    return torch.tensor(c, dtype=torch.int32, device=need_gpu())


def test_prefill_of_no_tokens_and_without_states():
    dev = need_gpu()
    x, gates, lay = _tensors(70, 1, 2, 1)
    s0 = torch.randn((2, 2, D, D), device=dev)
    s1 = torch.full_like(s0, float("nan"))
    o = nv.gdn_prefill(x[:0], gates[:0], _cu(0, 0, 0), **lay, state_in=s0, state_out=s1)
    assert o.shape == (0, 2 * D) and torch.equal(s0, s1)
    nv.gdn_prefill(x[:0], gates[:0], _cu(0, 0, 0), **lay, state_out=s1)
    assert torch.equal(s1, torch.zeros_like(s1))
    want = nv.gdn_prefill(x, gates, _cu(0, 70), **lay, state_out=s1[:1])
    assert torch.equal(nv.gdn_prefill(x, gates, _cu(0, 70), **lay), want)


def test_prefill_gives_the_same_bits_and_keeps_sequences_apart():
    """The same call twice; a sequence alone or between others; a neighbour full of NaN."""
    x, gates, lay = _tensors(400, 2, 4, 2)
    s = torch.zeros((3, 4, D, D), device=x.device)
    o = nv.gdn_prefill(x, gates, _cu(0, 130, 250, 400), **lay, state_out=s)
    s2 = torch.zeros_like(s)
    assert torch.equal(nv.gdn_prefill(x, gates, _cu(0, 130, 250, 400), **lay, state_out=s2), o) and torch.equal(s, s2)
    one = torch.zeros((1, 4, D, D), device=x.device)
    alone = nv.gdn_prefill(x[130:250].contiguous(), gates[130:250].contiguous(), _cu(0, 120), **lay, state_out=one)
    assert torch.equal(alone, o[130:250]) and torch.equal(one[0], s[1])
    x[130:250] = float("nan")
    gates[130:250] = float("nan")
    o3 = nv.gdn_prefill(x, gates, _cu(0, 130, 250, 400), **lay, state_out=s2)
    assert torch.equal(o3[:130], o[:130]) and torch.equal(o3[250:], o[250:])
    assert torch.equal(s2[0], s[0]) and torch.equal(s2[2], s[2])


def test_prefill_row_numbers_outside_the_rows_are_cut_off():
    x, gates, lay = _tensors(100, 1, 1, 3)
    want = nv.gdn_prefill(x, gates, _cu(0, 100), **lay)
    got = nv.gdn_prefill(x, gates, _cu(0, 1000), **lay)
    assert torch.equal(got, want)


def _decode(B, n_qk, n_v, dtype, *, kind="mixed", seed=0, idle=(), pad=0, o_dtype=None):
    dev = need_gpu()
    print(f"[decode] B {B} heads {n_qk}/{n_v} {dtype} {kind} idle {idle}", flush=True)
    x, g, beta = _inputs(B, n_qk, n_v, seed, kind)
    gt = torch.from_numpy(np.concatenate([g, beta], 1)).to(dtype)
    g, beta = gt.float().numpy()[:, :n_v], gt.float().numpy()[:, n_v:]
    xt = torch.full((B, x.shape[1] + 8 * pad), float("nan"), dtype=dtype, device=dev)
    xt[:, :x.shape[1]] = torch.from_numpy(x).to(dev).to(dtype)
    gd = torch.full((B, 2 * n_v + pad), float("nan"), dtype=dtype, device=dev)
    gd[:, :2 * n_v] = gt.to(dev)
    rng = np.random.default_rng(seed + 1)
    slots = rng.permutation(B + 2)[:B].astype(np.int32)
    slots[list(idle)] = -1
    pool = torch.from_numpy((rng.standard_normal((B + 2, n_v, D, D)) * 0.3).astype(np.float32)).to(dev)
    before = pool.clone()
    od = o_dtype or dtype
    o = torch.full((B, n_v * D + 8 * pad), float("nan"), dtype=od, device=dev)
    nv.gdn_decode(xt, gd, pool, q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v, n_qk_heads=n_qk,
                  n_v_heads=n_v, slots=torch.from_numpy(slots).to(dev), o=o)
    torch.cuda.synchronize()
    cu = np.arange(B + 1)
    starts = [before[s].cpu().numpy() if s >= 0 else None for s in slots]
    q, k, v, g, beta = _host(x, g, beta, n_qk, n_v)
    O, S, e, Mt, _, _, _ = _bounds(q, k, v, g, beta, cu, starts, 160)
    ov, sv = host_f32(o).astype(np.float64), pool.cpu().numpy()
    for b in range(B):
        got = ov[b, :n_v * D].reshape(n_v, D)
        if slots[b] < 0:
            assert np.all(got == 0)
            continue
        tol = 4 * 144 * U * Mt[b] / np.sqrt(D) + 1e-30
        if od == BF:
            tol = tol + 2.0 ** -8 * np.linalg.norm(O[b], axis=1)
        err = np.linalg.norm(got - O[b], axis=1)
        assert np.all(err <= tol), f"request {b}: o, worst {np.max(err / tol)}"
        es = np.linalg.norm((sv[slots[b]] - S[b]).reshape(n_v, -1), axis=1)
        assert np.all(es <= e[b] + 1e-30), f"request {b}: state, worst {np.max(es / (e[b] + 1e-30))}"
    free = [s for s in range(B + 2) if s not in slots]
    assert torch.equal(pool[free], before[free]), "a slot of no request was written"
    assert np.all(np.isnan(ov[:, n_v * D:]))


@pytest.mark.parametrize("B,n_qk,n_v,dtype,o_dtype", [
    (1, 16, 32, BF, None), (1, 1, 1, F32, None), (5, 2, 4, F32, BF), (9, 1, 3, BF, F32), (33, 4, 4, BF, None),
    (64, 2, 8, F32, None)])
def test_decode(B, n_qk, n_v, dtype, o_dtype):
    _decode(B, n_qk, n_v, dtype, seed=B, o_dtype=o_dtype, pad=2, idle=(1, 3) if B > 4 else ())


@pytest.mark.parametrize("kind", ["hold", "reset", "zero", "scales"])
def test_decode_hard_values(kind):
    _decode(24, 2, 4, F32, kind=kind, seed=6)


def test_decode_continues_a_prompt():
    """A prompt, then tokens one by one, against the fp64 recurrence of all of them."""
    x, gates, lay = _tensors(150, 2, 4, 8)
    pool = torch.zeros((2, 4, D, D), device=x.device)
    slots = torch.tensor([1], dtype=torch.int32, device=x.device)
    nv.gdn_prefill(x, gates, _cu(0, 140), **lay, state_in=pool, state_out=pool, slots=slots)
    rows = [nv.gdn_decode(x[t:t + 1], gates[t:t + 1], pool, **lay, slots=slots, o=torch.empty((1, 4 * D), device=x.device))
            for t in range(140, 150)]
    q, k, v, g, beta = _host(host_f32(x), *host_f32(gates).reshape(150, 2, 4).transpose(1, 0, 2), 2, 4)
    O, S, e, Mt, _, _, final = _bounds(q, k, v, g, beta, [0, 150], None, 400)
    got = torch.cat(rows).double().cpu().numpy().reshape(10, 4, D)
    tol = (e[140:] + 4 * 144 * U * Mt[140:]) / np.sqrt(D)
    assert np.all(np.linalg.norm(got - O[140:], axis=2) <= tol)
    assert np.all(np.linalg.norm((pool[1].cpu().numpy() - S[0]).reshape(4, -1), axis=1) <= final[0])
    assert torch.equal(pool[0], torch.zeros_like(pool[0]))


def test_slots_past_32_bit_offsets():
    """A pool of more than 2^32 bytes (and 2^31 values): the last slots, by prefill and by decode."""
    dev = need_gpu()
    n_slots = (1 << 31) // (32 * D * D) + 3
    print(f"[gdn] pool of {n_slots} slots x 32 heads", flush=True)
    pool = torch.empty((n_slots, 32, D, D), device=dev)
    x, gates, lay = _tensors(70, 16, 32, 4)
    small = torch.randn((2, 32, D, D), device=dev) * 0.1
    last = torch.tensor([n_slots - 1, n_slots - 2], dtype=torch.int32, device=dev)
    pool[n_slots - 2:] = small.flip(0)
    a = nv.gdn_prefill(x, gates, _cu(0, 3, 70), **lay, state_in=small, state_out=small)
    b = nv.gdn_prefill(x, gates, _cu(0, 3, 70), **lay, state_in=pool, state_out=pool, slots=last)
    assert torch.equal(a, b) and torch.equal(pool[n_slots - 2:].flip(0), small)
    c = nv.gdn_decode(x[:2], gates[:2], small, **lay)
    d = nv.gdn_decode(x[:2], gates[:2], pool, **lay, slots=last)
    assert torch.equal(c, d) and torch.equal(pool[n_slots - 2:].flip(0), small)


def test_graph_replays_and_other_streams():
    """A decode step and a prompt captured once; lengths and slots change between replays."""
    x, gates, lay = _tensors(200, 2, 4, 12)
    dev = x.device
    cu, slots = _cu(0, 100, 200), torch.tensor([0, 1], dtype=torch.int32, device=dev)
    base = torch.randn((4, 4, D, D), device=dev) * 0.2
    pool, o = base.clone(), torch.zeros((200, 4 * D), dtype=BF, device=dev)
    od = torch.zeros((2, 4 * D), dtype=BF, device=dev)
    need = nv.load().nvfp4_gdn_prefill_workspace_size(200, 2, 2, 4)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)

    def step():
        nv.gdn_prefill(x, gates, cu, **lay, state_in=pool, state_out=pool, slots=slots, o=o, workspace=ws)
        nv.gdn_decode(x[:2], gates[:2], pool, **lay, slots=slots, o=od)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r, (c, s) in enumerate((((0, 100, 200), (0, 1)), ((0, 7, 200), (3, 2)), ((0, 0, 64), (1, 0)), ((0, 129, 130), (2, -1)))):
        cu.copy_(_cu(*c))
        slots.copy_(torch.tensor(s, dtype=torch.int32, device=dev))
        pool.copy_(base)
        o.zero_()
        step()
        want = [t.clone() for t in (pool, o, od)]
        pool.copy_(base)
        o.zero_()
        od.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((pool, o, od), want):
            assert torch.equal(got, w), f"replay {r}"


def test_refusals():
    x, gates, lay = _tensors(8, 1, 2, 1)
    dev, cu = x.device, _cu(0, 8)
    st = torch.zeros((1, 2, D, D), device=dev)
    st8 = torch.zeros((8, 2, D, D), device=dev)
    bad_lay = dict(lay, q_col=4)
    for bad in (lambda: nv.gdn_prefill(x.float(), gates, cu, **lay), lambda: nv.gdn_prefill(x, gates[:4], cu, **lay),
                lambda: nv.gdn_prefill(x, gates.half(), cu, **lay), lambda: nv.gdn_prefill(x, gates, cu.long(), **lay),
                lambda: nv.gdn_prefill(x, gates, cu[:1], **lay), lambda: nv.gdn_prefill(x, gates, cu, **lay, state_in=st[:, :1]),
                lambda: nv.gdn_prefill(x, gates, cu, **lay, state_out=st.double()),
                lambda: nv.gdn_prefill(x, gates, cu, **lay, slots=cu[:1]),
                lambda: nv.gdn_prefill(x, gates, cu, **lay, state_in=st, state_out=st8),
                lambda: nv.gdn_prefill(x, gates, cu, **lay, o=torch.empty((8, 256), device=dev)),
                lambda: nv.gdn_prefill(x.cpu(), gates, cu, **lay), lambda: nv.gdn_decode(x, gates, st[:, :1], **lay),
                lambda: nv.gdn_decode(x, gates[:3], st8, **lay), lambda: nv.gdn_decode(x, gates, st8, **lay, slots=cu),
                lambda: nv.gdn_decode(x, gates, st8.to(BF), **lay)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.gdn_prefill(x, gates, cu, **bad_lay), lambda: nv.gdn_decode(x, gates, st8, **bad_lay),
                lambda: nv.gdn_prefill(x, gates, cu, **dict(lay, v_col=3 * D)),
                lambda: nv.gdn_decode(x, gates, st8, **dict(lay, g_col=3)),
                lambda: nv.gdn_decode(x, gates, st8, **dict(lay, n_qk_heads=3))):
        with pytest.raises(nv.Nvfp4Error):
            bad()
    assert nv.gdn_decode(x[:0], gates[:0], st8, **lay).shape == (0, 2 * D)


@pytest.mark.parametrize("many", [0, 23, 90])
@pytest.mark.parametrize("part,value", [("q", np.nan), ("k", np.nan), ("k", -np.inf), ("v", np.nan), ("v", np.inf),
                                        ("g", np.nan), ("beta", np.inf)])
def test_prefill_what_is_not_finite_stays_where_it_belongs(many, part, value):
    """Bit for bit: a product with a zero of the inverse or the scores adds nothing, so what an infinity or NaN in
    one token cannot reach token by token (earlier tokens, other heads, columns, sequences) is as without it."""
    dev = need_gpu()
    lens = [7, 150, 3] + [1, 2] * many
    n, n_qk, n_v, T = len(lens), 2, 4, sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    x, g, beta = _inputs(T, n_qk, n_v, 31)
    head, col = 1, 37                     # of q and k: value heads 2 and 3; of v and the gates: value head 1
    for at in (0, 5, 38, 63, 64, 100, 127, 149):
        print(f"[not finite] {part} {value} many {many} token {at}", flush=True)
        res = []
        for planted in (False, True):
            xt, gt = torch.from_numpy(x).to(dev).to(BF), torch.from_numpy(np.concatenate([g, beta], 1)).to(dev)
            row = 7 + at
            if planted and part in "qkv":
                xt[row, {"q": head * D, "k": (n_qk + head) * D, "v": (2 * n_qk + head) * D}[part] + col] = value
            elif planted:
                gt[row, head + (n_v if part == "beta" else 0)] = value
            states = torch.ones((n, n_v, D, D), device=dev)
            o = nv.gdn_prefill(xt, gt, cu, q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v,
                               n_qk_heads=n_qk, n_v_heads=n_v, state_in=states, state_out=states)
            torch.cuda.synchronize()
            res.append((o.view(T, n_v, D).float(), states))
        (o0, s0), (o1, s1) = res
        hit_o, hit_s = torch.zeros_like(o0, dtype=torch.bool), torch.zeros_like(s0, dtype=torch.bool)
        if part == "q":
            hit_o[row, 2:] = True
        else:
            heads, cols = (slice(2, 4), slice(None)) if part == "k" else (slice(1, 2), slice(None))
            if part == "v":
                cols = slice(col, col + 1)
            hit_o[row:157, heads, cols] = True
            hit_s[1, heads, :, cols] = True
        assert torch.all(torch.isfinite(o0)) and torch.all(torch.isfinite(s0))
        assert not torch.any(torch.isfinite(o1[hit_o])) and not torch.any(torch.isfinite(s1[hit_s]))
        assert torch.equal(o1[~hit_o], o0[~hit_o]) and torch.equal(s1[~hit_s], s0[~hit_s])


def test_memory_a_call_makes_belongs_to_its_stream():
    """A call on a stream that is behind the current one: what the current stream takes and fills right after the call
    returns must not be the call's workspace, nor may the call's output be memory that the current stream still uses."""
    x, gates, lay = _tensors(600, 2, 4, 21)
    cu = _cu(0, 600)
    need = nv.load().nvfp4_gdn_prefill_workspace_size(600, 1, 2, 4)
    want, want_d = nv.gdn_prefill(x, gates, cu, **lay), nv.gdn_decode(x, gates, torch.zeros((600, 4, D, D), device=x.device), **lay)
    states = torch.zeros((600, 4, D, D), device=x.device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)     # cycles: about a millisecond, then it ends
    o = nv.gdn_prefill(x, gates, cu, **lay, stream=side)
    od = nv.gdn_decode(x, gates, states, **lay, stream=side)
    taken = [torch.full((need,), 255, dtype=torch.uint8, device=x.device) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(od, want_d)
    pools = {b["address"] + sum(c["size"] for c in b["blocks"][:i]): b["stream"] for b in torch.cuda.memory_snapshot()
             for i in range(len(b["blocks"]))}
    assert pools[o.data_ptr()] == pools[od.data_ptr()] == side.cuda_stream != pools[taken[0].data_ptr()]
