"""One attention mixer layer, serving from a paged cache in 8 or 4 bits: prompts,
chunks of prompts, one token at a time, and trees of drafted tokens.

    residual add + norm -> NVFP4 codes        add_rmsnorm
    in-projection q | k | v                   gemm_segmented
    norm and rotation of the heads            qk_norm_rope
    keys and values into the cache            kv_cache_write
    attention over the cache                  attn_cached
    out-projection                            quantize, gemm

Weights are random (the trained ones are not available), the activation and
cache scales are calibrated on the first batch, as a static recipe does.

    python examples/attn_layer.py            # needs an MI355X
"""
from __future__ import annotations

import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_quantized_05_amd as nv  # noqa: E402


class AttnLayer:
    def __init__(self, hidden: int, n_q: int, n_kv: int, d: int, rot: int, n_pages: int, *, page_size: int = 64,
                 n_pos: int = 4096, fmt: str = "fp8", seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device=device)

        self.hidden, self.n_q, self.n_kv, self.d = hidden, n_q, n_kv, d
        self.module_rows = [n_q * d, n_kv * d, n_kv * d]
        parts = [nv.quantize(randn(r, hidden) / hidden ** 0.5) for r in self.module_rows]
        self.in_codes = torch.cat([p[0] for p in parts])
        self.in_scales = torch.cat([p[1] for p in parts])
        self.module_gs = torch.cat([p[2] for p in parts])
        self.out_w = nv.quantize(randn(hidden, n_q * d) / (n_q * d) ** 0.5)
        self.norm_w = 1.0 + 0.1 * randn(hidden)
        self.q_w, self.k_w = 1.0 + 0.1 * randn(d), 1.0 + 0.1 * randn(d)
        angle = torch.arange(n_pos, dtype=torch.float64)[:, None] / 10000.0 ** (torch.arange(0, rot, 2) / rot)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.in_gs = self.out_gs = None
        self.calibrated = False
        self.cache = nv.KvCache.empty(n_pages, page_size, n_kv, d, torch.ones(1, device=device),
                                      torch.ones(1, device=device), format=fmt)

    def forward(self, x: torch.Tensor, residual: torch.Tensor, positions: torch.Tensor, page_table: torch.Tensor,
                kv_lens: torch.Tensor, cu_seqlens: torch.Tensor | None = None, tree: torch.Tensor | None = None,
                trace: dict | None = None) -> torch.Tensor:
        """x [T, hidden] bf16, the block before's output; residual [T, hidden]
        is updated in place.  kv_lens counts the new rows; with cu_seqlens they are
        packed prompts (or with tree drafts), without there is one for each
        request."""
        total = torch.empty_like(residual)
        norm = dict(residual=residual, residual_out=total)
        if self.in_gs is None:
            _, _, self.in_gs = nv.quantize(nv.add_rmsnorm(x, self.norm_w, out_dtype=torch.float32, **norm))
        _, codes, scales = nv.add_rmsnorm(x, self.norm_w, y_gs=self.in_gs, **norm)
        residual.copy_(total)
        rows = nv.gemm_segmented(codes, scales, self.in_gs, self.in_codes, self.in_scales, self.module_gs,
                                 self.module_rows, out_dtype=torch.bfloat16)
        k_col = self.n_q * self.d
        q, k = nv.qk_norm_rope(rows, self.q_w, self.k_w, self.cos_sin, positions, q_col=0, k_col=k_col,
                               n_q_heads=self.n_q, n_kv_heads=self.n_kv)
        v = rows[:, k_col + self.n_kv * self.d:]
        if not self.calibrated:
            top = 448.0 if self.cache.format == "fp8" else 448.0 * 6.0
            self.cache.k_gs.copy_(k.abs().max().float() / top)
            self.cache.v_gs.copy_(v.abs().max().float() / top)
            self.calibrated = True
        nv.kv_cache_write(k, v, self.cache, page_table, kv_lens, cu_seqlens)
        o = nv.attn_cached(q, self.cache, page_table, kv_lens, cu_seqlens, n_q_heads=self.n_q, tree=tree)
        out_codes, out_scales, self.out_gs = nv.quantize(o, self.out_gs)
        if trace is not None:
            trace.update(rows=rows, q=q, k=k, v=v, o=o, out_codes=out_codes, out_scales=out_scales)
        return nv.gemm(out_codes, out_scales, self.out_gs, *self.out_w, out_dtype=torch.bfloat16)


def main() -> None:
    torch.manual_seed(0)
    lens = [900, 1, 130, 2048, 64, 777, 300, 1500]
    pages = [-(-(n + 64) // 64) for n in lens]
    dev = "cuda"

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    order, at = torch.randperm(sum(pages)).tolist(), 0
    table = []
    for n in pages:
        table.append(order[at:at + n] + [-1] * (max(pages) - n))
        at += n
    table = i32(table)
    x = torch.randn((sum(lens), 5120), device=dev).bfloat16()

    def timed(f, n):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    for fmt in ("fp8", "nvfp4"):
        layer = AttnLayer(5120, 24, 4, 256, 64, sum(pages), fmt=fmt)
        cu = i32([0, *torch.tensor(lens).cumsum(0).tolist()])
        pos = i32([p for n in lens for p in range(n)])
        residual, args = torch.zeros_like(x), (pos, table, i32(lens), cu)
        y = layer.forward(x, residual, *args)
        print(f"{fmt} prompts: {len(lens)} of {sum(lens)} tokens in all, output {tuple(y.shape)}, "
              f"{timed(lambda: layer.forward(x, residual, *args), 5):.3f} ms")
        token = x[cu[1:].long() - 1].contiguous()
        res1, args = torch.zeros_like(token), (i32(lens), table, i32([n + 1 for n in lens]))
        y = layer.forward(token, res1, *args)
        print(f"{fmt} decode: {len(lens)} requests, output {tuple(y.shape)}, "
              f"{timed(lambda: layer.forward(token, res1, *args), 50):.3f} ms; finite: {bool(torch.isfinite(y).all())}")
        # four drafts of each request: two guesses for the next token, one after each
        drafts = x[:4 * len(lens)].contiguous()
        tree = torch.tensor([0b0001, 0b0010, 0b0101, 0b1010] * len(lens), device=dev)
        pos = i32([n + p for n in lens for p in (0, 0, 1, 1)])
        res2, args = torch.zeros_like(drafts), (pos, table, i32([n + 4 for n in lens]), i32(range(0, 4 * len(lens) + 1, 4)))
        y = layer.forward(drafts, res2, *args, tree=tree)
        print(f"{fmt} trees of 4: {timed(lambda: layer.forward(drafts, res2, *args, tree=tree), 50):.3f} ms; "
              f"finite: {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
