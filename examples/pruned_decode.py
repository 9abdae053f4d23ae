"""The operators around a pruned layer, together, as a program uses them.

``DecodeBlock`` is the end of a language model with pruned weights: a norm, a
pruned projection with the low-rank adapters of many requests beside it, a
residual sum, a norm, a pruned output head, and the penalties, biases and
grammar masks on its logits. ``step`` takes the residual stream of one token
of each request to the logits that the next tokens are picked from.

``recovery_step`` is one step of the training that follows pruning: the pruned
weights stay as they are, the norm's weight and bias learn. The product's own
gradient is the product with the transposed matrix, a plan of its own.

    python examples/pruned_decode.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_matrix_vector_gb300 as S  # noqa: E402
import workloads  # noqa: E402


def transposed(m) -> tuple:
    """CSR arrays of a matrix's transpose."""
    rows = np.repeat(np.arange(m.n_rows), np.diff(m.row_ptr))
    order = np.lexsort((rows, m.col_idx))
    row_ptr = np.concatenate([[0], np.cumsum(np.bincount(m.col_idx, minlength=m.n_cols))])
    return row_ptr.astype(np.int32), rows[order].astype(np.int32), m.values[order]


@dataclass
class DecodeBlock:
    width: int
    vocab: int
    slots: int
    rank: int
    seed: int = 1

    def __post_init__(self):
        dev, d = "cuda", self.width
        g = torch.Generator(device=dev).manual_seed(self.seed)
        self.matrix = workloads.llm(0.5, n=d, seed=self.seed)
        rng = np.random.default_rng(self.seed)
        kept = [np.sort(rng.choice(d, d // 4, replace=False)) for _ in range(self.vocab)]
        self.head_cols = np.concatenate(kept).astype(np.int32)
        self.head_ptr = (np.arange(self.vocab + 1) * (d // 4)).astype(np.int32)
        self.head_values = rng.normal(0, 0.05, self.head_cols.size).astype(np.float16)
        m = self.matrix
        self.projection = S.spmv_plan_create(m.row_ptr, m.col_idx, m.values, d, format="delta4")
        self.head = S.spmv_plan_create(self.head_ptr, self.head_cols, self.head_values, d,
                                       format="delta")
        def normal(*size, std=1.0, mean=0.0):
            return torch.randn(*size, generator=g, device=dev) * std + mean
        self.norms = [(normal(d, std=0.1, mean=1.0), normal(d, std=0.05)) for _ in range(2)]
        self.a = normal(self.slots, self.rank, d, std=d ** -0.5).half()
        self.b = normal(self.slots, d, self.rank, std=0.1).half()
        self.scales = torch.full((self.slots,), 2.0, device=dev)

    def product(self, plan, x, y):
        """The shared projection: one product per token."""
        for xt, yt in zip(x, y):
            S.spmv_run(plan, xt, yt)

    def step(self, residual, slot_ids, **constraints):
        """Logits (fp32) of one token per request; the residual stream (fp32)
        is updated. `constraints`: what spmv_logits_process takes."""
        n = residual.shape[0]
        x = torch.empty(n, self.width, dtype=torch.float16, device=residual.device)
        y = torch.empty(n, self.width, device=residual.device)
        S.spmv_layernorm(residual, *self.norms[0], x)
        self.product(self.projection, x, y)
        S.spmv_adapters_run(x, self.a, self.b, slot_ids, y, base=y, scales=self.scales)
        residual += y
        S.spmv_layernorm(residual, *self.norms[1], x)
        logits = torch.empty(n, self.vocab, device=residual.device)
        self.product(self.head, x, logits)
        S.spmv_logits_process(logits, logits, **constraints)
        return logits

    def recovery_step(self, x, target, lr: float = 0.1):
        """One step on the first norm for sum (W norm(x) - target)^2 / 2 over
        a few rows x. Returns the loss before it and the gradients (dx,
        dweight, dbias)."""
        if not hasattr(self, "projection_t"):
            self.projection_t = S.spmv_plan_create(*transposed(self.matrix), self.width,
                                                   format="delta4")
        weight, bias = self.norms[0]
        n = x.shape[0]
        mean, rstd = torch.empty(n, device=x.device), torch.empty(n, device=x.device)
        h = torch.empty(n, self.width, dtype=torch.float16, device=x.device)
        y, dh = torch.empty_like(x), torch.empty_like(x)
        S.spmv_layernorm(x, weight, bias, h, mean=mean, rstd=rstd)
        self.product(self.projection, h, y)
        error = y - target
        self.product(self.projection_t, error.half(), dh)
        dx, dweight, dbias = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(bias)
        S.spmv_layernorm_backward(dh, x, weight, mean, rstd, dx, dweight, dbias)
        loss = float((error * error).sum()) / 2
        weight -= lr * dweight / n
        bias -= lr * dbias / n
        return loss, dx, dweight, dbias


def main() -> None:
    torch.manual_seed(0)
    block = DecodeBlock(width=2048, vocab=4096, slots=4, rank=16)
    dev, n = "cuda", 6
    residual = torch.randn(n, block.width, device=dev)
    slot_ids = torch.tensor([0, 1, -1, 1, 3, 0], dtype=torch.int32, device=dev)
    history = torch.randint(0, block.vocab, (n * 20,), dtype=torch.int32, device=dev)
    offsets = torch.arange(n + 1, device=dev) * 20
    mask = torch.full((1, block.vocab // 32), -1, dtype=torch.int32, device=dev)
    mask[0, 64:] = 0  # a grammar that allows the first 2048 tokens
    mask_rows = torch.tensor([-1, 0, -1, -1, 0, -1], dtype=torch.int32, device=dev)
    tokens = []
    for _ in range(4):
        logits = block.step(residual, slot_ids, output=(history, offsets),
                            repetition=torch.full((n,), 1.2, device=dev),
                            frequency=torch.full((n,), 0.2, device=dev),
                            mask=mask, mask_rows=mask_rows)
        tokens.append(logits.argmax(1).tolist())
    print("tokens of", n, "requests, step by step:", tokens)
    x, target = torch.randn(n, block.width, device=dev), torch.randn(n, block.width, device=dev) * 0.1
    print("recovery loss:", [round(block.recovery_step(x, target)[0], 3) for _ in range(5)])


if __name__ == "__main__":
    main()
