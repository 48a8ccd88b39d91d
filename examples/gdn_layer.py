"""One Gated DeltaNet mixer layer, serving: a batch of prompts, then one token
at a time for each of them.

    residual add + norm -> NVFP4 codes        add_rmsnorm
    in-projection q|k|v | z | a | b           gemm_segmented_gates
    short convolution of q|k|v                conv_silu
    recurrence                                gdn_prefill / gdn_decode
    norm, gate z -> NVFP4 codes               rmsnorm_gated
    out-projection                            gemm

Weights are random (the trained ones are not available), the activation
scales are calibrated on the first batch, as a static recipe does.  Every
request keeps its convolution inputs and its recurrent state in one slot.

    python examples/gdn_layer.py            # needs an MI355X
"""
from __future__ import annotations

import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_quantized_05_amd as nv  # noqa: E402

D = 128  # head dimension


class GdnLayer:
    def __init__(self, hidden: int, n_qk: int, n_v: int, n_slots: int, *, width: int = 4, seed: int = 0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device=device)

        self.hidden, self.n_qk, self.n_v = hidden, n_qk, n_v
        self.qkv, self.z = D * (2 * n_qk + n_v), D * n_v
        self.module_rows = [self.qkv, self.z, n_v, n_v]
        self.rows = sum(self.module_rows)
        parts = [nv.quantize(randn(r, hidden) / hidden ** 0.5) for r in self.module_rows]
        self.in_codes = torch.cat([p[0] for p in parts])
        self.in_scales = torch.cat([p[1] for p in parts])
        self.module_gs = torch.cat([p[2] for p in parts])
        self.out_w = nv.quantize(randn(hidden, self.z) / self.z ** 0.5)
        self.conv_w = randn(self.qkv, width) / width ** 0.5
        self.a_log = torch.rand(n_v, generator=g, device=device)
        self.dt_bias = -4.0 + randn(n_v)
        self.norm_w = 1.0 + 0.1 * randn(hidden)
        self.head_w = 1.0 + 0.1 * randn(D)
        self.in_gs = self.out_gs = None
        # what a request carries from call to call; zero for a new request
        self.conv_state = torch.zeros((n_slots, width - 1, self.qkv), dtype=torch.bfloat16, device=device)
        self.state = torch.zeros((n_slots, n_v, D, D), device=device)

    def free(self, slots: torch.Tensor) -> None:
        """Make slots ready for new requests."""
        self.conv_state[slots.long()] = 0
        self.state[slots.long()] = 0

    def _codes(self, norm, gs):
        """Codes of a norm's output under its calibrated scale (taken from this batch the first time)."""
        if gs is None:
            _, _, gs = nv.quantize(norm(out_dtype=torch.float32))
        _, codes, scales = norm(y_gs=gs)
        return codes, scales, gs

    def forward(self, x: torch.Tensor, residual: torch.Tensor, slots: torch.Tensor,
                cu_seqlens: torch.Tensor | None = None, trace: dict | None = None) -> torch.Tensor:
        """x [T, hidden] bf16, the block before's output; residual [T, hidden]
        is updated in place.  With cu_seqlens: packed prompts (each goes on
        from what its slot holds); without: one token per request."""
        T = x.shape[0]
        total = torch.empty_like(residual)
        codes, scales, self.in_gs = self._codes(
            lambda **k: nv.add_rmsnorm(x, self.norm_w, residual=residual, residual_out=total, **k), self.in_gs)
        residual.copy_(total)
        # rows of a multiple of 8 columns, so that every part of them starts 16-byte aligned
        rows = torch.empty((T, -(-self.rows // 8) * 8), dtype=torch.bfloat16, device=x.device)
        nv.gemm_segmented_gates(codes, scales, self.in_gs, self.in_codes, self.in_scales, self.module_gs,
                                self.module_rows, decay_module=2, a_log=self.a_log, dt_bias=self.dt_bias,
                                write_module=3, out_dtype=torch.bfloat16, out=rows)
        qkv = nv.conv_silu(rows[:, :self.qkv], self.conv_w, cu_seqlens=cu_seqlens, state=self.conv_state, slots=slots)
        lay = dict(q_col=0, k_col=D * self.n_qk, v_col=2 * D * self.n_qk, g_col=self.qkv + self.z,
                   beta_col=self.qkv + self.z + self.n_v, n_qk_heads=self.n_qk, n_v_heads=self.n_v, slots=slots)
        if cu_seqlens is None:
            o = nv.gdn_decode(qkv, rows, self.state, **lay)
        else:
            o = nv.gdn_prefill(qkv, rows, cu_seqlens, state_in=self.state, state_out=self.state, **lay)
        z = rows[:, self.qkv:self.qkv + self.z]
        codes, scales, self.out_gs = self._codes(lambda **k: nv.rmsnorm_gated(o, z, self.head_w, **k), self.out_gs)
        if trace is not None:
            trace.update(rows=rows, qkv=qkv, o=o, out_codes=codes, out_scales=scales)
        return nv.gemm(codes, scales, self.out_gs, *self.out_w, out_dtype=torch.bfloat16)


def main() -> None:
    torch.manual_seed(0)
    lens = [900, 1, 130, 2048, 64, 777, 300, 1500]
    layer = GdnLayer(5120, 16, 32, n_slots=len(lens))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    x = torch.randn((sum(lens), 5120), device="cuda").bfloat16()

    def timed(f, n=5):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    residual = torch.zeros_like(x)
    y = layer.forward(x, residual, slots, cu)
    print(f"prompts: {len(lens)} of {sum(lens)} tokens in all, output {tuple(y.shape)}, "
          f"{timed(lambda: layer.forward(x, residual, slots, cu)):.3f} ms")
    token, res1 = x[cu[1:].long() - 1].contiguous(), residual[cu[1:].long() - 1].contiguous()
    y = layer.forward(token, res1, slots)
    print(f"decode: {len(lens)} requests, output {tuple(y.shape)}, "
          f"{timed(lambda: layer.forward(token, res1, slots), 50):.3f} ms; finite: {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
