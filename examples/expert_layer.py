"""An expert layer in 8-bit integers, put together from the library's calls.

Tokens are routed to k of E experts, quantised, multiplied with their experts'
first matrices, gated (SwiGLU), quantised again, multiplied with the second
matrices and summed with the router's weights. Every size that depends on the
routing stays on the GPU: no call waits for another's result on the host.

``python examples/expert_layer.py`` runs a small layer and prints how far it is
from the same layer in fp32 torch operations; with a training step's gradient of
the output, ``router_gradient`` gives that of the router's logits.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import smem_swizzle_layouts_gb300 as g  # noqa: E402


def expect(name: str, t: torch.Tensor, dtype: torch.dtype, *shape: int) -> None:
    """The library reads bare pointers: another type, size or order of a tensor's elements is refused here."""
    if t.dtype != dtype or tuple(t.shape) != shape or (t.shape[-1] > 1 and t.numel() > 0 and t.stride(-1) != 1):
        raise ValueError(f"{name}: {dtype} {list(shape)} with neighbouring elements in a row, not "
                         f"{t.dtype} {list(t.shape)} with strides {list(t.stride())}")


def quantize_weights(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(int8 values, scale per channel) of weights [E, N, K]; K is a multiple of 16."""
    E, N, K = w.shape
    q = torch.empty(E, N, K, dtype=torch.int8, device=w.device)
    scale = torch.empty(E, N, device=w.device)
    flat = w.float().reshape(E * N, K).contiguous()
    g.gemm_quantize_int8(E * N, K, flat, g.OUT_F32, E * N, K, None, g.QUANT_PLAIN, q, K, scale)
    return q, scale


class ExpertLayer:
    """Weights and buffers of one layer for up to ``tokens`` tokens.

    ``w1`` [E, 2F, H] holds each expert's gate and up projections (F rows each), ``w2`` [E, H, F] its down
    projection. ``rule`` is the dict of gemm_route's options. The buffers are reused: one call at a time.
    """

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, k: int, rule: dict, tokens: int):
        dev = w1.device
        self.E, two_f, self.H = w1.shape
        self.F, self.k, self.rule, self.tokens = two_f // 2, k, rule, tokens
        self.T = 0  # of the last call
        if two_f % 2 or tuple(w2.shape) != (self.E, self.H, self.F):
            raise ValueError(f"w1 [E, 2F, H] {list(w1.shape)} and w2 [E, H, F] {list(w2.shape)} do not fit")
        self.q1, self.s1 = quantize_weights(w1)
        self.q2, self.s2 = quantize_weights(w2)
        rows = tokens * k
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids, self.slots = torch.empty(tokens, k, **i32), torch.empty(tokens, k, **i32)
        self.row_tokens, self.offsets = torch.empty(rows, **i32), torch.empty(self.E + 1, **i32)
        self.weights = torch.empty(tokens, k, device=dev)
        self.workspace = torch.empty(max(g.gemm_route_plan_workspace_size(tokens, self.E, k), 4), dtype=torch.uint8,
                                     device=dev)
        self.a1, self.sa1 = torch.empty(rows, self.H, dtype=torch.int8, device=dev), torch.empty(rows, device=dev)
        self.a2, self.sa2 = torch.empty(rows, self.F, dtype=torch.int8, device=dev), torch.empty(rows, device=dev)
        self.y1 = torch.empty(rows, two_f, device=dev)
        self.y2 = torch.empty(rows, self.H, device=dev)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
        """x [T, H] bf16 and the router's logits [T, E] fp32 to the layer's output [T, H] bf16."""
        T, (E, k, H, F) = x.shape[0], (self.E, self.k, self.H, self.F)
        if T > self.tokens:
            raise ValueError(f"{T} tokens in a layer of {self.tokens}")
        expect("x", x, torch.bfloat16, T, H)
        expect("logits", logits, torch.float32, T, E)
        if bias is not None:
            expect("bias", bias, torch.float32, E)
        self.T = T
        rows = T * k
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        g.gemm_route(T, E, logits, g.OUT_F32, logits.stride(0), bias, k, self.rule, self.weights, self.ids)
        g.gemm_route_plan(T, E, k, self.ids, self.offsets, self.slots, self.row_tokens, self.workspace,
                          self.workspace.numel())
        # each row of the sorted order is its token's row of x
        g.gemm_quantize_int8(rows, H, x, g.OUT_BF16, T, x.stride(0), self.row_tokens, g.QUANT_PLAIN, self.a1, H, self.sa1)
        g.gemm_int8_grouped(rows, 2 * F, H, E, self.offsets, self.a1, H, self.sa1, self.q1, H, 2 * F * H, self.s1,
                            self.y1, 2 * F, g.OUT_F32)
        # rows past offsets[E] (padded tokens) hold what was there before; no slot names them
        g.gemm_quantize_int8(rows, F, self.y1, g.OUT_F32, rows, 2 * F, None, g.QUANT_GATED, self.a2, F, self.sa2)
        g.gemm_int8_grouped(rows, H, F, E, self.offsets, self.a2, F, self.sa2, self.q2, F, H * F, self.s2,
                            self.y2, H, g.OUT_F32)
        g.gemm_route_combine(T, H, k, self.y2, g.OUT_F32, rows, H, self.slots, self.weights, out, g.OUT_BF16, H)
        return out

    def router_gradient(self, logits: torch.Tensor, d_out: torch.Tensor) -> torch.Tensor:
        """The gradient of the logits of the last call, from that of its output ([T, H] bf16)."""
        T, k, H, rows = self.T, self.k, self.H, self.T * self.k
        expect("logits", logits, torch.float32, T, self.E)
        expect("d_out", d_out, torch.bfloat16, T, H)
        d_rows, d_weights = torch.empty_like(self.y2), torch.empty(T, k, device=logits.device)
        g.gemm_route_combine_backward(T, H, k, d_out, g.OUT_BF16, d_out.stride(0), self.y2, g.OUT_F32, rows, H,
                                      self.slots, self.weights, d_rows, H, d_weights)
        d_logits = torch.empty_like(logits)
        g.gemm_route_backward(T, self.E, logits, g.OUT_F32, logits.stride(0), k, self.rule, self.ids, d_weights, d_logits,
                              d_logits.stride(0))
        return d_logits


def plain_layer(x, logits, w1, w2, k):
    """The same layer in torch operations: softmax over the chosen logits, unquantised fp32 weights."""
    top, ids = logits.topk(k, -1)
    weights = torch.softmax(top, -1)
    out = torch.zeros(x.shape, device=x.device)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = x[t].float() @ w1[e].float().t()
        gate, up = h.chunk(2, -1)
        out.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().t()))
    return out


def main(T: int = 200, E: int = 16, k: int = 4, H: int = 256, F: int = 128) -> float:
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    w1, w2 = rand(E, 2 * F, H) * H ** -0.5, rand(E, H, F) * F ** -0.5
    x, logits = rand(T, H).to(torch.bfloat16), rand(T, E)
    layer = ExpertLayer(w1, w2, k, dict(score=g.ROUTE_SOFTMAX, renormalize=1), tokens=T)
    y = layer(x, logits)
    ref = plain_layer(x, logits, w1, w2, k)
    err = float((y.float() - ref).norm() / ref.norm())
    grad = layer.router_gradient(logits, torch.ones_like(y))
    print(f"{T} tokens, {E} experts, {k} each: relative error of 8-bit layer {err:.4f}; "
          f"|d logits| {float(grad.norm()):.3f}; kernels launched {g.gemm_launch_count()}")
    return err


if __name__ == "__main__":
    main()
