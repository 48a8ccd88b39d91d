"""The operators of a Gated DeltaNet mixer around its NVFP4 projections: their
cases, inputs, plain forms and 64-bit values.

  prefill     the gated delta rule over packed prompts (chunked form)
  decode      the same recurrence for one new token of many requests
  conv        the short causal convolution + SiLU over packed rows or requests
  add_norm    residual + scale * x, then RMSNorm with a weight
  gated_norm  RMSNorm per head of the mixer's output, times SiLU of its gate z

The shapes are those of the layer this repository measures: hidden 5120, one
in-projection row q 2048 | k 2048 | v 4096 | z 4096 | a 48 | b 48 (12384
columns), 16 q/k heads and 32 value heads of 128, prompts of up to 32,768
tokens.  ``own = False`` computes each operator with elementary torch
operations in fp32, rounded once at the end; ``own = True`` calls the
framework.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
D = 128            # head dimension
EPS = 1e-6         # RMSNorm epsilon, and the floor of |q|, |k|
CHUNK = 64         # tokens per step of the plain chunked form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one 32K-token prompt through one layer: the headline prefill
        {"name": "prefill_32k", "op": "prefill", "tokens": 32768, "seqs": 1, "lens_seed": 0, "n_qk": 16, "n_v": 32,
         "gates": "bf16", "start": False},
        # a batch of chat prompts of unequal lengths (an empty and a one-token one among them), each going on from
        # the state its slot holds, gates kept in fp32
        {"name": "prefill_ragged", "op": "prefill", "tokens": 8191, "seqs": 12, "lens_seed": 3, "n_qk": 16, "n_v": 32,
         "gates": "f32", "start": True},
        # a short prompt on the small head layout of the tests: latency of the whole chain
        {"name": "prefill_300", "op": "prefill", "tokens": 300, "seqs": 1, "lens_seed": 0, "n_qk": 2, "n_v": 4,
         "gates": "f32", "start": True},
        # one user decoding: launch latency
        {"name": "decode_1", "op": "decode", "batch": 1, "n_qk": 16, "n_v": 32, "dtype": "bf16", "idle": 0},
        # the decode batch of the GEMM workloads' largest M
        {"name": "decode_64", "op": "decode", "batch": 64, "n_qk": 16, "n_v": 32, "dtype": "bf16", "idle": 0},
        # a loaded server with unused rows of a captured batch, projections in fp32
        {"name": "decode_251", "op": "decode", "batch": 251, "n_qk": 16, "n_v": 32, "dtype": "f32", "idle": 5},
        # the qkv columns of the 32K-token in-projection
        {"name": "conv_32k", "op": "conv", "tokens": 32768, "seqs": 1, "lens_seed": 0, "channels": 8192, "width": 4,
         "dtype": "bf16", "step": False},
        # one token for each of 64 requests
        {"name": "conv_step_64", "op": "conv", "tokens": 64, "seqs": 64, "lens_seed": 0, "channels": 8192, "width": 4,
         "dtype": "bf16", "step": True},
        # the norm in front of the in-projection at 32K tokens
        {"name": "add_norm_32k", "op": "add_norm", "rows": 32768, "cols": 5120, "dtype": "bf16", "scale": 1.0},
        # the same for one decoded token, fp32 residual stream
        {"name": "add_norm_1", "op": "add_norm", "rows": 1, "cols": 5120, "dtype": "f32", "scale": 0.5},
        # the norm between recurrence and out-projection at 32K tokens
        {"name": "gated_norm_32k", "op": "gated_norm", "rows": 32768, "heads": 32, "group": 128, "dtype": "bf16"},
        # the same for a decode batch
        {"name": "gated_norm_64", "op": "gated_norm", "rows": 64, "heads": 32, "group": 128, "dtype": "bf16"},
    ]


def _size(n):
    return n + 16 if n == 3072 else n  # a width that no configuration here has


def _log_int(rng, lo, hi):
    return _size(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "decode", "conv", "add_norm", "gated_norm"))
    heads = rng.choice(((16, 32), (16, 32), (16, 16), (8, 32), (4, 12), (2, 4), (1, 3)))
    if op == "prefill":
        tokens = _log_int(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "seqs": _log_int(rng, 1, max(1, min(48, tokens))),
                "lens_seed": rng.randrange(1 << 30), "n_qk": heads[0], "n_v": heads[1],
                "gates": rng.choice(("bf16", "f32")), "start": rng.random() < 0.6}
    if op == "decode":
        batch = _log_int(rng, 1, 251)
        return {"op": op, "batch": batch, "n_qk": heads[0], "n_v": heads[1], "dtype": rng.choice(("bf16", "f32")),
                "idle": rng.randrange(0, 1 + batch // 4)}
    if op == "conv":
        step = rng.random() < 0.4
        tokens = _log_int(rng, 1, 512 if step else 32768)
        channels = D * (2 * heads[0] + heads[1])
        if rng.random() < 0.3:
            channels = _size(rng.randrange(64, channels + 1))  # odd channel counts
        return {"op": op, "tokens": tokens, "seqs": tokens if step else _log_int(rng, 1, max(1, min(48, tokens))),
                "lens_seed": rng.randrange(1 << 30), "channels": channels, "width": rng.choice((2, 3, 4, 4)),
                "dtype": rng.choice(("bf16", "bf16", "f32")) if tokens <= 16384 else "bf16", "step": step}
    if op == "add_norm":
        rows = _log_int(rng, 1, 32768)
        cols = _log_int(rng, 64, 5120)
        return {"op": op, "rows": rows, "cols": _size(cols // 16 * 16) if rng.random() < 0.7 else cols,
                "dtype": rng.choice(("bf16", "f32")) if rows <= 16384 else "bf16",
                "scale": round(rng.uniform(0.1, 2.0), 3)}
    group = rng.choice((64, 128, 128, 256))
    rows = _log_int(rng, 1, 32768)
    heads = rng.randrange(1, 4096 // group + 1)
    return {"op": op, "rows": rows, "heads": heads - (heads * group == 3072), "group": group,
            "dtype": rng.choice(("bf16", "f32")) if rows <= 16384 else "bf16"}


def lengths(case):
    """The packed sequences' lengths: they sum to the tokens; from four
    sequences on one is empty and one has a single token."""
    n, total = case["seqs"], case["tokens"]
    if n == 1:
        return [total]
    r = random.Random(case["lens_seed"])
    w = [r.uniform(0.1, 1.9) for _ in range(n)]
    ls = [int(total * x / sum(w)) for x in w]
    if n >= 4:
        ls[1], ls[2] = 0, min(1, total)
    ls[0] += total - sum(ls)
    return ls


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _qkv(g, rows, n_qk, n_v, dtype):
    """q | k | v rows as the convolution's SiLU leaves them: skewed, so that keys of a head are correlated."""
    return torch.nn.functional.silu(_randn(g, rows, D * (2 * n_qk + n_v))).to(dtype)


def _gate_rows(g, rows, n_v, dtype, wide):
    """Log-decay gates and write strengths.  Each head decays over a horizon
    drawn log-uniformly from 8 to 60,000 tokens, modulated per token; beta is
    a sigmoid.  ``wide``: columns of the in-projection's row, else compact."""
    horizon = torch.exp(math.log(8.0) + _rand(g, n_v) * math.log(7500.0))
    gate = -torch.exp(0.7 * _randn(g, rows, n_v)) / horizon
    beta = torch.sigmoid(_randn(g, rows, n_v))
    if not wide:
        return torch.cat([gate, beta], 1).to(dtype), 0, n_v
    buf = torch.zeros((rows, 12384), device=DEVICE, dtype=dtype)
    buf[:, 12288:12288 + n_v] = gate.to(dtype)
    buf[:, 12336:12336 + n_v] = beta.to(dtype)
    return buf, 12288, 12336


def _cu(case):
    c = [0]
    for n in lengths(case):
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEVICE)


def _slots(seed, n, pool):
    """n distinct slots of a pool, in no order."""
    return torch.tensor(random.Random(seed).sample(range(pool), n), dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op == "prefill":
        t, n_v = case["tokens"], case["n_v"]
        s["x"] = _qkv(g, t, case["n_qk"], n_v, torch.bfloat16)
        s["gates"], s["g_col"], s["beta_col"] = _gate_rows(g, t, n_v, DTYPES[case["gates"]],
                                                           case["gates"] == "bf16" and n_v <= 48)
        s["cu"] = _cu(case)
        pool = case["seqs"] + (3 if case["start"] else 0)
        s["states"] = _randn(g, pool, n_v, D, D) * (0.1 if case["start"] else 0.0)
        s["slots"] = _slots(seed, case["seqs"], pool)
        s["o"] = torch.empty((t, n_v * D), dtype=torch.bfloat16, device=DEVICE)
    elif op == "decode":
        b, n_v, dt = case["batch"], case["n_v"], DTYPES[case["dtype"]]
        s["x"] = _qkv(g, b, case["n_qk"], n_v, dt)
        s["gates"], s["g_col"], s["beta_col"] = _gate_rows(g, b, n_v, dt, case["dtype"] == "bf16" and n_v <= 48)
        s["states"] = _randn(g, b + 2, n_v, D, D) * 0.1
        idle = sorted(random.Random(seed + 1).sample(range(b), case["idle"]))  # unused rows of the batch
        s["live"] = torch.tensor([i for i in range(b) if i not in idle], dtype=torch.long, device=DEVICE)
        s["slots"] = torch.full((b,), -1, dtype=torch.int32, device=DEVICE)
        s["slots"][s["live"]] = _slots(seed, b, b + 2)[s["live"]]
        s["o"] = torch.empty((b, n_v * D), dtype=dt, device=DEVICE)
    elif op == "conv":
        t, c, w, dt = case["tokens"], case["channels"], case["width"], DTYPES[case["dtype"]]
        rows = torch.zeros((t, 12384 if c == 8192 else c), dtype=dt, device=DEVICE)  # qkv columns of the in-projection
        rows[:, :c] = _randn(g, t, c).to(dt)
        s["x"] = rows[:, :c]
        s["w"] = _randn(g, c, w) / math.sqrt(w)
        s["cu"] = None if case["step"] else _cu(case)
        pool = case["seqs"] + 2
        s["states"] = _randn(g, pool, w - 1, c).to(dt)
        s["slots"] = _slots(seed, case["seqs"], pool)
        s["y"] = torch.empty((t, c), dtype=dt, device=DEVICE)
    elif op == "add_norm":
        r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        spread = torch.exp(_randn(g, c))  # channels of unequal size, as in a residual stream
        s["x"] = _randn(g, r, c).mul_(0.3).to(dt)
        s["residual"] = (_randn(g, r, c) * spread).to(dt)
        s["w"] = 1.0 + 0.2 * _randn(g, c)
        s["sum"] = torch.empty((r, c), dtype=dt, device=DEVICE)
        s["y"] = torch.empty((r, c), dtype=torch.bfloat16, device=DEVICE)
    else:
        r, c, dt = case["rows"], case["heads"] * case["group"], DTYPES[case["dtype"]]
        rows = torch.zeros((r, 12384 if c == 4096 else c), dtype=dt, device=DEVICE)  # z columns of the in-projection
        at = 8192 if c == 4096 else 0
        rows[:, at:at + c] = _randn(g, r, c).to(dt)
        s["z"] = rows[:, at:at + c]
        s["o"] = (_randn(g, r, c) * torch.exp(_randn(g, r, 1))).mul_(0.1).to(dt)
        s["w"] = 1.0 + 0.2 * _randn(g, case["group"])
        s["y"] = torch.empty((r, c), dtype=torch.bfloat16, device=DEVICE)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)[case["op"]](s, case)


def _columns(s, case):
    n_qk = case["n_qk"]
    return dict(q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=s["g_col"], beta_col=s["beta_col"],
                n_qk_heads=n_qk, n_v_heads=case["n_v"])


def _own_prefill(s, case):
    import nvfp4_w4a4_quantized_05_amd as nv
    nv.gdn_prefill(s["x"], s["gates"], s["cu"], **_columns(s, case), state_in=s["states"] if case["start"] else None,
                   state_out=s["states"], slots=s["slots"], o=s["o"])
    return {"o": s["o"], "state": s["states"]}


def _own_decode(s, case):
    import nvfp4_w4a4_quantized_05_amd as nv
    nv.gdn_decode(s["x"], s["gates"], s["states"], **_columns(s, case), slots=s["slots"], o=s["o"])
    return {"o": s["o"], "state": s["states"]}


def _own_conv(s, case):
    import nvfp4_w4a4_quantized_05_amd as nv
    nv.conv_silu(s["x"], s["w"], cu_seqlens=s["cu"], state=s["states"], slots=s["slots"], out=s["y"])
    return {"y": s["y"], "state": s["states"]}


def _own_add_norm(s, case):
    import nvfp4_w4a4_quantized_05_amd as nv
    nv.add_rmsnorm(s["x"], s["w"], residual=s["residual"], scale=case["scale"], eps=EPS, residual_out=s["sum"],
                   out=s["y"])
    return {"sum": s["sum"], "y": s["y"]}


def _own_gated_norm(s, case):
    import nvfp4_w4a4_quantized_05_amd as nv
    nv.rmsnorm_gated(s["o"], s["z"], s["w"], eps=EPS, out=s["y"])
    return {"y": s["y"]}


# ---------------------------------------------------------------- the plain forms, fp32

def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp(min=EPS)


def _split(s, case, dtype):
    """q, k, v per value head and the gates: [rows, n_v, D] and [rows, n_v], q and k of unit length."""
    n_qk, n_v, rows = case["n_qk"], case["n_v"], s["x"].shape[0]
    x = s["x"].to(dtype)
    q = _unit(x[:, :n_qk * D].reshape(rows, n_qk, D)).repeat_interleave(n_v // n_qk, 1)
    k = _unit(x[:, n_qk * D:2 * n_qk * D].reshape(rows, n_qk, D)).repeat_interleave(n_v // n_qk, 1)
    v = x[:, 2 * n_qk * D:].reshape(rows, n_v, D)
    gate = s["gates"][:, s["g_col"]:s["g_col"] + n_v].to(dtype)
    beta = s["gates"][:, s["beta_col"]:s["beta_col"] + n_v].to(dtype)
    return q, k, v, gate, beta


def _padded(cu, longest, step):
    """Row numbers [seqs, longest rounded up to step] of the packed rows, and which of them exist."""
    at = torch.arange(-(-max(longest, 1) // step) * step, device=cu.device)
    real = at[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(real, cu[:-1, None] + at[None], 0).long(), real


def _plain_prefill(s, case):
    """The recurrence a chunk of 64 tokens at a time.  Inside a chunk, with G
    the running sum of g and S its start state:
        A_ij = beta_i (k_i . k_j) exp(G_{i-1} - G_j) for j < i,
        (I + A) U = beta (v - exp(G_{i-1}) k S),
        o_i = (exp(G_i) q_i S + sum_{j <= i} (q_i . k_j) exp(G_i - G_j) U_j) / sqrt(D),
        S' = exp(G_C) S + sum_j exp(G_C - G_j) k_j U_j^T.
    (I + A)^-1 comes from doubling the size of its inverted diagonal blocks.
    Chunks follow one another; everything else is batched."""
    n_v, lens = case["n_v"], lengths(case)
    rows, real = _padded(s["cu"], max(lens), CHUNK)
    q, k, v, gate, beta = _split(s, case, torch.float32)
    n, size = len(lens), rows.shape[1] // CHUNK

    def chunks(t):  # [tokens, n_v, ...] -> [chunk, seqs * n_v, 64, ...], zeros where there is no token
        t = t[rows] * real.reshape(*real.shape, *[1] * (t.dim() - 1))
        t = t.reshape(n, size, CHUNK, *t.shape[2:]).transpose(2, 3)
        return t.transpose(0, 1).reshape(size, n * n_v, CHUNK, *t.shape[4:]).contiguous()

    q, k, v, gate, beta = (chunks(t) for t in (q, k, v, gate, beta))
    total = gate.cumsum(-1)
    before = torch.nn.functional.pad(total[..., :-1], (1, 0))
    i = torch.arange(CHUNK, device=rows.device)
    lower, strict = i[:, None] >= i[None], i[:, None] > i[None]
    kt = k.transpose(-1, -2).contiguous()
    a = beta[..., None] * (k @ kt) * torch.exp(
        torch.where(strict, before[..., :, None] - total[..., None, :], -math.inf))
    inv = torch.eye(CHUNK, device=rows.device).expand_as(a)
    for size2 in (2, 4, 8, 16, 32, 64):  # the lower left quarter of each diagonal block of this size
        quarter = (i[:, None] // size2 == i[None] // size2) & (i[:, None] % size2 >= size2 // 2) & (i[None] % size2 < size2 // 2)
        inv = inv - inv @ (a * quarter) @ inv
    scores = (q @ kt) * torch.exp(torch.where(lower, total[..., :, None] - total[..., None, :], -math.inf))
    grown, seen, left = torch.exp(total), torch.exp(before), torch.exp(total[..., -1:] - total)
    slots = s["slots"].long()
    state = s["states"][slots] if case["start"] else torch.zeros_like(s["states"][slots])
    state = state.reshape(n * n_v, D, D)
    out = torch.empty_like(v)
    for c in range(size):
        u = inv[c] @ (beta[c][..., None] * (v[c] - seen[c][..., None] * (k[c] @ state)))
        out[c] = grown[c][..., None] * (q[c] @ state) + scores[c] @ u
        state = grown[c][:, -1, None, None] * state + kt[c] @ (left[c][..., None] * u)
    s["states"][slots] = state.reshape(n, n_v, D, D)
    out = out.reshape(size, n, n_v, CHUNK, D).permute(1, 0, 3, 2, 4).reshape(n * size * CHUNK, n_v * D)
    at = torch.arange(s["o"].shape[0], device=rows.device)
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    s["o"].copy_(out[seq * (size * CHUNK) + at - s["cu"][seq]] / math.sqrt(D))
    return {"o": s["o"], "state": s["states"]}


def _plain_decode(s, case):
    q, k, v, gate, beta = _split(s, case, torch.float32)
    at = s["slots"].clamp(min=0).long()
    old = s["states"][at]
    u = beta[..., None] * (v - (k[..., None] * old).sum(-2))
    new = torch.exp(gate)[..., None, None] * old + k[..., None] * u[..., None, :]
    o = (q[..., None] * new).sum(-2) / math.sqrt(D)
    s["states"][at[s["live"]]] = new[s["live"]]
    s["o"].copy_((o * (s["slots"] >= 0)[:, None, None]).reshape(s["o"].shape))
    return {"o": s["o"], "state": s["states"]}


def _conv_rows(s, case):
    """For each row and tap the row of [x; states] it reads, and the rows that each new state holds."""
    t, w, slots = case["tokens"], case["width"], s["slots"].long()
    if s["cu"] is None:
        start = torch.arange(t, device=slots.device)
        cu = torch.arange(t + 1, device=slots.device)
    else:
        cu = s["cu"].long()
        start = torch.repeat_interleave(cu[:-1], cu[1:] - cu[:-1], output_size=t)
    seq = torch.searchsorted(cu, torch.arange(t, device=cu.device), right=True) - 1
    tap = torch.arange(w, device=cu.device) - (w - 1)
    rows = torch.arange(t, device=cu.device)[:, None] + tap
    rows = torch.where(rows >= start[:, None], rows, t + slots[seq][:, None] * (w - 1) + rows - start[:, None] + w - 1)
    last = cu[1:, None] + torch.arange(-(w - 1), 0, device=cu.device)
    last = torch.where(last >= cu[:-1, None], last, t + slots[:, None] * (w - 1) + last - cu[:-1, None] + w - 1)
    return rows, last


def _plain_conv(s, case):
    rows, last = _conv_rows(s, case)
    pool = torch.cat([s["x"], s["states"].reshape(-1, case["channels"])])
    y = (pool.float()[rows] * s["w"].t()).sum(1)
    s["states"][s["slots"].long()] = pool[last]
    s["y"].copy_(y / (1 + torch.exp(-y)))
    return {"y": s["y"], "state": s["states"]}


def _plain_add_norm(s, case):
    t = s["residual"].float() + case["scale"] * s["x"].float()
    s["y"].copy_(t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"])
    s["sum"].copy_(t)
    return {"sum": s["sum"], "y": s["y"]}


def _plain_gated_norm(s, case):
    o, z = (s[n].float().reshape(case["rows"], -1, case["group"]) for n in ("o", "z"))
    y = o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"] * (z / (1 + torch.exp(-z)))
    s["y"].copy_(y.reshape(s["y"].shape))
    return {"y": s["y"]}


_run_plain = {"prefill": _plain_prefill, "decode": _plain_decode, "conv": _plain_conv, "add_norm": _plain_add_norm,
              "gated_norm": _plain_gated_norm}
_run_own = {"prefill": _own_prefill, "decode": _own_decode, "conv": _own_conv, "add_norm": _own_add_norm,
            "gated_norm": _own_gated_norm}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("prefill", "decode"):
        n_qk, n_v = case["n_qk"], case["n_v"]
        t = case["tokens"] if op == "prefill" else case["batch"] - case["idle"]
        n = case["seqs"] if op == "prefill" else t
        e = 2 if op == "prefill" or case["dtype"] == "bf16" else 4
        ge = 2 if case["gates" if op == "prefill" else "dtype"] == "bf16" else 4
        state = n * n_v * D * D * 4
        reads = 1 if op == "decode" or case["start"] else 0
        # a token and head: k S, the rank-one update and q S, 2 D^2 each
        return {"bytes": t * (e * D * (2 * n_qk + 2 * n_v) + ge * 2 * n_v) + state * (1 + reads),
                "flops": t * n_v * 6 * D * D}
    if op == "conv":
        e, c, w = (2 if case["dtype"] == "bf16" else 4), case["channels"], case["width"]
        return {"bytes": 2 * case["tokens"] * c * e + 4 * c * w + 2 * case["seqs"] * (w - 1) * c * e,
                "flops": case["tokens"] * c * (2 * w + 4)}
    n = case["rows"] * (case["cols"] if op == "add_norm" else case["heads"] * case["group"])
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "add_norm":
        return {"bytes": n * (3 * e + 2) + 4 * case["cols"], "flops": 7 * n}
    return {"bytes": n * (2 * e + 2) + 4 * case["group"], "flops": 9 * n}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_recurrence, "decode": _exact_recurrence, "conv": _exact_conv,
            "add_norm": _exact_add_norm, "gated_norm": _exact_gated_norm}[case["op"]](s, case)


def _exact_recurrence(s, case):
    """Token by token, S <- e^g S + beta k (v - S^T k)^T, o = S^T q / sqrt(D); decode is sequences of one token."""
    n_qk, n_v, x = case["n_qk"], case["n_v"], s["x"].double()
    if case["op"] == "prefill":
        lens, cu = lengths(case), s["cu"].tolist()
    else:
        lens, cu = [1] * case["batch"], list(range(case["batch"]))
    if max(lens) * (1e-4 + len(lens) * n_v * D * D * 8 * 8 / 3e12) > 12:
        return None
    slot = s["slots"].tolist()
    pool = s["states"].double()
    o = torch.zeros((x.shape[0], n_v, D), dtype=torch.float64, device=x.device)
    seqs = [i for i in range(len(lens)) if slot[i] >= 0]
    seqs.sort(key=lambda i: -lens[i])
    head = torch.arange(n_v, device=x.device) * n_qk // n_v
    live = torch.tensor([slot[i] for i in seqs], device=x.device)
    first = torch.tensor([cu[i] for i in seqs], device=x.device)
    keep = pool[live] if case["op"] == "decode" or case["start"] else torch.zeros_like(pool[live])
    q = x[:, :n_qk * D].reshape(-1, n_qk, D)
    k = x[:, n_qk * D:2 * n_qk * D].reshape(-1, n_qk, D)
    q = (q / torch.linalg.vector_norm(q, dim=-1, keepdim=True).clamp(min=EPS))[:, head]
    k = (k / torch.linalg.vector_norm(k, dim=-1, keepdim=True).clamp(min=EPS))[:, head]
    v = x[:, 2 * n_qk * D:].reshape(-1, n_v, D)
    alpha = s["gates"][:, s["g_col"]:s["g_col"] + n_v].double().exp()
    beta = s["gates"][:, s["beta_col"]:s["beta_col"] + n_v].double()
    for t in range(max(lens)):
        m = sum(lens[i] > t for i in seqs)  # the longest first: those that still have a token
        if m == 0:
            break
        r, state = first[:m] + t, keep[:m]
        seen = torch.matmul(k[r][:, :, None, :], state)[:, :, 0]
        state.mul_(alpha[r][..., None, None])
        state.add_(k[r][..., :, None] * (beta[r][..., None] * (v[r] - seen))[..., None, :])
        o[r] = torch.matmul(q[r][:, :, None, :], state)[:, :, 0] / math.sqrt(D)
    pool[live] = keep
    return {"o": o.reshape(o.shape[0], -1), "state": pool}


def _exact_conv(s, case):
    """Sequence by sequence on the rows its state and its tokens make together."""
    w, x, pool = case["width"], s["x"].double(), s["states"].double()
    weight, slot = s["w"].double(), s["slots"].long()
    if s["cu"] is None:
        both = torch.cat([pool[slot], x[:, None]], 1)  # [requests, w, channels]
        y = torch.einsum("bwc,cw->bc", both, weight)
        pool[slot] = both[:, 1:]
    else:
        y, cu, slot = torch.empty_like(x), s["cu"].tolist(), slot.tolist()
        for i, n in enumerate(lengths(case)):
            both = torch.cat([pool[slot[i]], x[cu[i]:cu[i] + n]])
            y[cu[i]:cu[i] + n] = sum(both[j:j + n] * weight[:, j] for j in range(w))
            pool[slot[i]] = both[n:]
    return {"y": y * torch.sigmoid(y), "state": pool}


def _exact_add_norm(s, case):
    t = torch.add(s["residual"].double(), s["x"].double(), alpha=case["scale"])
    length = torch.linalg.vector_norm(t, dim=-1, keepdim=True) / math.sqrt(case["cols"])
    return {"sum": t, "y": t * s["w"].double() * torch.rsqrt(length * length + EPS)}


def _exact_gated_norm(s, case):
    group = case["group"]
    o, z = s["o"].double().unflatten(-1, (-1, group)), s["z"].double().unflatten(-1, (-1, group))
    length = torch.linalg.vector_norm(o, dim=-1, keepdim=True) / math.sqrt(group)
    y = o * torch.rsqrt(length * length + EPS) * s["w"].double() * z * torch.sigmoid(z)
    return {"y": y.flatten(-2)}
