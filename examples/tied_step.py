"""The ends of a training step of an expert model with a tied token table, put together from the library's calls.

Token ids become rows of the table; an expert layer's router chooses experts and has a balance loss; the table, as the
head's weights, gives the loss of the next tokens. The backward pass goes the same way back: the head's gradient of the
table is written first and the rows' gradient added to it. What lies between the ends is left to the caller: here a
residual whose weights are the router's, so that the step has a gradient through every call.

``python examples/tied_step.py`` takes a few steps on synthetic tokens and prints the losses.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import smem_swizzle_layouts_gb300 as g  # noqa: E402


def expect(name: str, t: torch.Tensor, dtype: torch.dtype, *shape: int) -> None:
    """The library reads bare pointers: another type, size or order of a tensor's elements is refused here."""
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: {dtype} {list(shape)}, contiguous, not {t.dtype} {list(t.shape)} with strides {list(t.stride())}")


class TiedEnds:
    """Buffers of both ends for up to ``tokens`` tokens of width ``H`` (a multiple of 8), in as many sequences at most, and a
    table of ``V`` rows.

    The calls forward keep what those backward need; the buffers are reused: one step at a time. The workspace has room for
    the most tokens, and the library's calls never ask for more for fewer.
    """

    def __init__(self, V: int, H: int, E: int, k: int, tokens: int, balance: float = 0.01, z: float = 1e-4, device="cuda"):
        if H % 8:
            raise ValueError(f"rows of {H} elements do not start on 16-byte words")
        self.V, self.H, self.E, self.k, self.tokens, self.balance, self.z = V, H, E, k, tokens, balance, z
        self.scale = math.sqrt(H)
        f32, i32 = dict(device=device), dict(dtype=torch.int32, device=device)
        self.weights, self.ids = torch.empty(tokens, k, **f32), torch.empty(tokens, k, **i32)
        self.losses, self.lse = torch.empty(tokens, **f32), torch.empty(tokens, **f32)
        room = max(g.gemm_cross_entropy_workspace_size(tokens, V), g.gemm_cross_entropy_backward_workspace_size(tokens, V, H),
                   g.gemm_embed_backward_workspace_size(tokens, H, V), g.gemm_route_balance_workspace_size(tokens, E, tokens))
        self.workspace = torch.empty(room, dtype=torch.uint8, device=device)  # one call uses it at a time

    def fits(self, T: int, S: int = 0) -> None:
        if T > self.tokens or S > self.tokens:
            raise ValueError(f"{T} tokens in {S} sequences, with buffers for {self.tokens} of each")

    def rows(self, table: torch.Tensor, words: torch.Tensor) -> torch.Tensor:
        """The scaled rows [T, H] of ``words`` [T] int32."""
        T = words.numel()
        self.fits(T)
        expect("table", table, torch.bfloat16, self.V, self.H)
        expect("words", words, torch.int32, T)
        out = torch.empty(T, self.H, dtype=torch.bfloat16, device=table.device)
        g.gemm_embed(T, self.H, self.V, words, table, g.OUT_BF16, self.H, self.scale, out, g.OUT_BF16, self.H)
        return out

    def route(self, logits: torch.Tensor, offsets: torch.Tensor):
        """Weights [T, k] and ids of the chosen experts, and the balance loss of each sequence (offsets [S + 1] int32)."""
        T, S = logits.shape[0], offsets.numel() - 1
        self.fits(T, S)
        expect("logits", logits, torch.float32, T, self.E)
        expect("offsets", offsets, torch.int32, S + 1)
        dev = logits.device
        self.counts, self.live = torch.empty(S, self.E, dtype=torch.int32, device=dev), torch.empty(S, dtype=torch.int32, device=dev)
        self.means, balance = torch.empty(S, self.E, device=dev), torch.empty(S, device=dev)
        g.gemm_route(T, self.E, logits, g.OUT_F32, self.E, None, self.k, None, self.weights, self.ids)
        g.gemm_route_balance(T, self.E, logits, g.OUT_F32, self.E, self.k, None, self.ids, S, offsets, self.counts, self.live, self.means,
                             balance, self.workspace, self.workspace.numel())
        return self.weights[:T], self.ids[:T], balance

    def head_inputs(self, table, hidden, targets) -> int:
        T = hidden.shape[0]
        self.fits(T)
        expect("table", table, torch.bfloat16, self.V, self.H)
        expect("hidden", hidden, torch.bfloat16, T, self.H)
        expect("targets", targets, torch.int32, T)
        return T

    def loss(self, table: torch.Tensor, hidden: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Each token's loss [T]; targets outside the table (padding) have none."""
        T = self.head_inputs(table, hidden, targets)
        g.gemm_cross_entropy(1, T, self.V, self.H, hidden, self.H, table, self.H, targets, self.losses, self.lse, self.workspace,
                             self.workspace.numel())
        return self.losses[:T]

    def loss_backward(self, table, hidden, targets, d_losses):
        """Gradients of hidden [T, H] and of the table [V, H], with that of a penalty z * lse^2 on the normalisers."""
        T = self.head_inputs(table, hidden, targets)
        expect("d_losses", d_losses, torch.float32, T)
        d_hidden, d_table = torch.empty_like(hidden), torch.empty_like(table)
        d_lse = 2.0 * self.z * self.lse[:T] * d_losses
        g.gemm_cross_entropy_backward(1, T, self.V, self.H, hidden, self.H, table, self.H, targets, self.lse, d_losses, d_lse, d_hidden,
                                      g.OUT_BF16, self.H, d_table, g.OUT_BF16, self.H, 0, self.workspace, self.workspace.numel())
        return d_hidden, d_table

    def route_backward(self, logits, offsets, d_weights):
        """The logits' gradient: through the weights, and of balance * mean over sequences of their losses."""
        T, S = logits.shape[0], offsets.numel() - 1
        self.fits(T, S)
        expect("logits", logits, torch.float32, T, self.E)
        expect("offsets", offsets, torch.int32, S + 1)
        expect("d_weights", d_weights, torch.float32, T, self.k)
        d_logits = torch.empty_like(logits)
        d_balance = torch.full((S,), self.balance / S, device=logits.device)
        g.gemm_route_backward(T, self.E, logits, g.OUT_F32, self.E, self.k, None, self.ids, d_weights, d_logits, self.E)
        g.gemm_route_balance_backward(T, self.E, logits, g.OUT_F32, self.E, self.k, None, self.ids, S, offsets, self.counts, self.live,
                                      d_balance, d_logits, self.E, 1)
        return d_logits

    def rows_backward(self, d_table: torch.Tensor, words: torch.Tensor, d_rows: torch.Tensor) -> None:
        """Adds the rows' gradient to the table's."""
        T = words.numel()
        self.fits(T)
        expect("d_table", d_table, torch.bfloat16, self.V, self.H)
        expect("words", words, torch.int32, T)
        expect("d_rows", d_rows, torch.bfloat16, T, self.H)
        g.gemm_embed_backward(T, self.H, self.V, words, d_rows, g.OUT_BF16, self.H, self.scale, d_table, g.OUT_BF16, self.H, 1,
                              self.workspace, self.workspace.numel())


def step(ends: TiedEnds, table, router, directions, words, targets, offsets):
    """One forward and backward pass: (loss, table's, router's and directions' gradients).

    The layer between the ends is hidden = rows + sum of the chosen directions [E, H] by their weights, with the router's
    logits rows @ router [H, E], in torch operations.
    """
    rows = ends.rows(table, words)
    logits = (rows.float() @ router).contiguous()
    weights, ids, balance = ends.route(logits, offsets)
    at = ids.clamp(min=0).long()
    hidden = (rows.float() + (weights[..., None] * directions[at]).sum(1)).to(torch.bfloat16)
    losses = ends.loss(table, hidden, targets)
    live = ((targets >= 0) & (targets < ends.V)).float()
    n = live.sum().clamp(min=1.0)
    lse = ends.lse[:words.numel()]
    total = (losses.sum() + ends.z * (lse * lse * live).sum()) / n + ends.balance * balance.mean()
    d_hidden, d_table = ends.loss_backward(table, hidden, targets, (live / n).contiguous())
    d = d_hidden.float()
    d_weights = (d[:, None] * directions[at]).sum(-1)
    d_directions = torch.zeros_like(directions).index_put_((at,), weights[..., None] * d[:, None], accumulate=True)
    d_logits = ends.route_backward(logits, offsets, d_weights)
    d_router = rows.float().t() @ d_logits
    ends.rows_backward(d_table, words, (d + d_logits @ router.t()).to(torch.bfloat16))
    return total, d_table, d_router, d_directions


def main(V: int = 2000, H: int = 128, E: int = 16, k: int = 4, T: int = 512, steps: int = 5) -> list:
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    table = (rand(V, H) * H ** -0.5).to(torch.bfloat16)
    router, directions = rand(H, E) * 0.1, rand(E, H) * 0.5
    words = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    targets = words.roll(-1).contiguous()
    targets[-1] = -1
    offsets = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    ends = TiedEnds(V, H, E, k, T)
    out = []
    for _ in range(steps):
        loss, d_table, d_router, d_directions = step(ends, table, router, directions, words, targets, offsets)
        for p, d in ((table, d_table), (router, d_router), (directions, d_directions)):
            p -= (0.5 * d.float()).to(p.dtype)
        out.append(float(loss))
    print(f"{T} tokens, {V} words, {E} experts: losses {', '.join(f'{v:.4f}' for v in out)}; kernels launched {g.gemm_launch_count()}")
    return out


if __name__ == "__main__":
    main()
