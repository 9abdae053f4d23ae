"""A pruned model beside the dense one that it came from, as a program uses them.

``DenseTarget`` is the dense model with its two layers held in 4 bits
(``quantized`` packs them); the drafter is the ``DecodeBlock`` of
pruned_decode.py. ``speculate`` lets the drafter propose a few tokens for each
request, has the target look at all of them at once and keeps those that
``spmv_verify_drafts`` accepts, so that the tokens are distributed as the
target's own. ``distill_step`` is one step of the training that makes the
drafter agree with the target more often: the gradient of the distillation
from the target's top logits, through the pruned head, to the weight and bias
of the norm before it.

    python examples/draft_and_verify.py
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [p for p in (ROOT, os.path.join(ROOT, "examples")) if p not in sys.path]

import sparse_matrix_vector_gb300 as S  # noqa: E402
from pruned_decode import DecodeBlock, transposed  # noqa: E402


def quantized(w, group: int):
    """(weights, scales, zeros) of a matrix in 4 bits: each group's range in
    15 steps, with its zero on one of them."""
    rows, cols = w.shape
    groups = -(-cols // group)
    padded = torch.zeros(rows, groups * group, device=w.device)
    padded[:, :cols] = w.float()
    blocks = padded.view(rows, groups, group)
    low, high = blocks.amin(2).clamp(max=0), blocks.amax(2).clamp(min=0)
    scales = ((high - low) / 15).clamp(min=1e-8).half()
    zeros = (-low / scales.float()).round().clamp(0, 15)
    q = (blocks / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8)
    q = q.view(rows, -1)[:, : cols + cols % 2]
    return (q[:, ::2] | (q[:, 1::2] << 4)).contiguous(), scales, zeros.to(torch.uint8)


class DenseTarget:
    def __init__(self, block: DecodeBlock, group: int = 64, seed: int = 5):
        """The model that `block` was pruned from: its weights, and small ones
        where pruning left nothing."""
        self.block, self.group = block, group
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = block.width

        def dense(ptr, cols, values, rows):
            w = torch.randn(rows, d, generator=g, device="cuda") * 0.004
            at = torch.repeat_interleave(torch.arange(rows), torch.from_numpy(ptr).diff())
            w[at.cuda(), torch.from_numpy(cols).long().cuda()] = torch.from_numpy(values).cuda().float()
            return w
        m = block.matrix
        self.layer = dense(m.row_ptr, m.col_idx, m.values, m.n_rows)
        self.head = dense(block.head_ptr, block.head_cols, block.head_values, block.vocab)
        self.layer4, self.head4 = quantized(self.layer, group), quantized(self.head, group)

    def logits(self, residual):
        """Logits (fp32) of rows of the residual stream (fp32), all at once."""
        n, d = residual.shape
        x = torch.empty(n, d, dtype=torch.float16, device=residual.device)
        h, out = torch.empty_like(residual), torch.empty(n, self.block.vocab, device=residual.device)
        S.spmv_layernorm(residual, *self.block.norms[0], x)
        w, scales, zeros = self.layer4
        S.spmv_int4_run(x, w, scales, h, self.group, zeros=zeros, base=residual)
        S.spmv_layernorm(h, *self.block.norms[1], x)
        w, scales, zeros = self.head4
        S.spmv_int4_run(x, w, scales, out, self.group, zeros=zeros)
        return out


def pick(logits, uniforms, temperature):
    """A token of each row: a request without drafts takes one from its target."""
    n = logits.shape[0]
    tokens = torch.empty(n, dtype=torch.int32, device=logits.device)
    none = torch.empty(0, device=logits.device)
    S.spmv_verify_drafts(logits, None, none.int(), torch.zeros(n + 1, dtype=torch.int64, device=logits.device), none,
                         uniforms, tokens, torch.empty_like(tokens), temperature=temperature)
    return tokens


def speculate(block, target, embedding, last, drafts: int, temperature, generator):
    """Tokens of one round for requests whose last tokens are `last`: (tokens,
    accepted, and what they were decided from)."""
    n, dev = last.numel(), last.device

    def uniform(*size):
        return torch.rand(*size, generator=generator, device=dev)
    no_adapter = torch.full((n,), -1, dtype=torch.int32, device=dev)
    tokens, logits, drafted = last, [], []
    for _ in range(drafts):
        logits.append(block.step(embedding[tokens.long()].clone(), no_adapter))
        tokens = pick(logits[-1], uniform(n), temperature)
        drafted.append(tokens)
    # request by request: its drafts, and one row more of the target
    draft_logits = torch.stack(logits, 1).view(n * drafts, -1)
    draft_tokens = torch.stack(drafted, 1)
    seen = torch.cat([last[:, None], draft_tokens], 1).view(-1)
    target_logits = target.logits(embedding[seen.long()])
    offsets = torch.arange(n + 1, device=dev) * drafts
    out = torch.empty(n * (drafts + 1), dtype=torch.int32, device=dev)
    accepted = torch.empty(n, dtype=torch.int32, device=dev)
    given = (target_logits, draft_logits, draft_tokens.view(-1), offsets, uniform(n * drafts), uniform(n))
    S.spmv_verify_drafts(*given, out, accepted, temperature=temperature)
    return out.view(n, drafts + 1), accepted, given


def distill_step(block, target, hidden, top: int = 16, temperature: float = 1.0, lr: float = 0.0):
    """The mean distillation loss over rows of the drafter's last hidden state
    (fp32), from the target's logits for the same rows, and the gradients of
    the last norm's weight and bias."""
    if not hasattr(block, "head_t"):
        from types import SimpleNamespace
        head = SimpleNamespace(row_ptr=block.head_ptr, col_idx=block.head_cols, values=block.head_values,
                               n_rows=block.vocab, n_cols=block.width)
        block.head_t = S.spmv_plan_create(*transposed(head), block.vocab, format="csr")
    n, d, dev = hidden.shape[0], block.width, hidden.device
    weight, bias = block.norms[1]
    mean, rstd = torch.empty(n, device=dev), torch.empty(n, device=dev)
    x = torch.empty(n, d, dtype=torch.float16, device=dev)
    S.spmv_layernorm(hidden, weight, bias, x, mean=mean, rstd=rstd)
    logits = torch.empty(n, block.vocab, device=dev)
    block.product(block.head, x, logits)
    w, scales, zeros = target.head4
    teacher = torch.empty_like(logits)
    S.spmv_int4_run(x, w, scales, teacher, target.group, zeros=zeros)
    listed = teacher.topk(top, dim=1)
    log_sums = torch.logsumexp(teacher / temperature, 1)
    loss, stats = torch.empty(n, device=dev), torch.empty(n, 3, device=dev)
    tokens = listed.indices.int()
    S.spmv_distill(logits, tokens, listed.values, loss, temperature=temperature, log_sums=log_sums, stats=stats)
    # the gradient in place of the logits; x 1024 as the head's product takes fp16
    scale = torch.full((1,), 1024.0 / n, device=dev).expand(n)
    S.spmv_distill_backward(scale, logits, tokens, listed.values, stats, logits, temperature=temperature,
                            log_sums=log_sums)
    dx = torch.empty(n, d, device=dev)
    block.product(block.head_t, logits.half(), dx)
    dweight, dbias = torch.empty_like(weight), torch.empty_like(bias)
    S.spmv_layernorm_backward(dx / 1024, hidden, weight, mean, rstd, None, dweight, dbias)
    if lr:
        weight -= lr * dweight
        bias -= lr * dbias
    return float(loss.mean()), dweight, dbias, teacher


def main() -> None:
    g = torch.Generator(device="cuda").manual_seed(0)
    block = DecodeBlock(width=1024, vocab=4096, slots=1, rank=8)
    target = DenseTarget(block)
    n = 8
    embedding = torch.randn(block.vocab, block.width, generator=g, device="cuda")
    last = torch.randint(0, block.vocab, (n,), generator=g, device="cuda").int()
    temperature = torch.tensor([0.7] * 6 + [0.0] * 2, device="cuda")
    kept = 0
    for _ in range(4):
        tokens, accepted, _ = speculate(block, target, embedding, last, 4, temperature, g)
        last = tokens.gather(1, accepted.long()[:, None])[:, 0]
        kept += int(accepted.sum())
    print(f"accepted {kept} of {4 * 4 * n} drafted tokens; last tokens {last.tolist()}")
    hidden = torch.randn(64, block.width, generator=g, device="cuda")
    print("distillation loss:", [round(distill_step(block, target, hidden, lr=0.5)[0], 4) for _ in range(5)])


if __name__ == "__main__":
    main()
