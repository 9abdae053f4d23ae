"""The decode and recovery example against plain fp64 torch on the CPU: the
operators and the pruned products together."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def dense(ptr, cols, values, n_cols):
    w = torch.zeros(len(ptr) - 1, n_cols, dtype=torch.float64)
    rows = np.repeat(np.arange(len(ptr) - 1), np.diff(ptr))
    w[torch.from_numpy(rows), torch.from_numpy(cols.astype(np.int64))] = torch.from_numpy(values.astype(np.float64))
    return w


def norm(x, w, b, half=True):
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-5) * w + b
    return y.half().double() if half else y


@pytest.fixture(scope="module")
def block(spmv_lib):
    import pruned_decode
    return pruned_decode.DecodeBlock(width=512, vocab=600, slots=3, rank=8)


def test_decode_step(block):
    """Relative error of the logits: every x is rounded to fp16 (2^-11 of
    each element, independent in sign, on both sides of a 512-term product),
    and a value on the other side of a rounding moves one element by 2^-10;
    2^-9 of the row's norm covers both."""
    g = torch.Generator().manual_seed(3)
    residual = torch.randn(5, 512, generator=g)
    ids = torch.tensor([2, -1, 0, 2, 1], dtype=torch.int32)
    out = torch.tensor([1, 1, 5, 7, 9, 9, 9, 2, 3, 4], dtype=torch.int32)
    off = torch.arange(6) * 2
    freq = torch.full((5,), 0.5)
    mask = torch.full((5, 19), -1, dtype=torch.int32)
    mask[3] = 0
    m = block.matrix
    W = dense(m.row_ptr, m.col_idx, m.values, 512)
    H = dense(block.head_ptr, block.head_cols, block.head_values, 512)
    (w0, b0), (w1, b1) = [[t.cpu().double() for t in p] for p in block.norms]
    r = residual.double()
    x = norm(r, w0, b0)
    y = x @ W.T
    for t, s in enumerate(ids.tolist()):
        if s >= 0:
            y[t] += 2.0 * (block.b[s].cpu().double() @ (block.a[s].cpu().double() @ x[t]))
    r = r + y
    ref = norm(r, w1, b1) @ H.T
    for t in range(5):
        for v in out[2 * t:2 * t + 2].tolist():
            ref[t, v] -= 0.5
    dev = residual.cuda()
    logits = block.step(dev, ids.cuda(), output=(out.cuda(), off.cuda()), frequency=freq.cuda(), mask=mask.cuda()).cpu().double()
    assert (logits[3] == -float("inf")).all()
    for t in (0, 1, 2, 4):
        assert (logits[t] - ref[t]).norm() <= 2.0 ** -9 * ref[t].norm()
        assert (dev[t].cpu().double() - r[t]).norm() <= 2.0 ** -9 * r[t].norm()


def test_recovery_step(block):
    """The gradients against autograd in fp64 (the same roundings to fp16 of
    the norm's output and of the error as above), and a falling loss."""
    g = torch.Generator().manual_seed(4)
    x, target = torch.randn(6, 512, generator=g), torch.randn(6, 512, generator=g)
    m = block.matrix
    W = dense(m.row_ptr, m.col_idx, m.values, 512)
    w, b = [t.cpu().double().requires_grad_() for t in block.norms[0]]
    xd = x.double().requires_grad_()
    loss_ref = ((norm(xd, w, b, half=False) @ W.T - target.double()) ** 2).sum() / 2
    loss_ref.backward()
    loss, dx, dw, db = block.recovery_step(x.cuda(), target.cuda(), lr=0.05)
    assert abs(loss - float(loss_ref.detach())) <= 2.0 ** -8 * float(loss_ref.detach())
    for got, ref in ((dx, xd.grad), (dw, w.grad), (db, b.grad)):
        assert (got.cpu().double() - ref).norm() <= 2.0 ** -8 * ref.norm()
    assert block.recovery_step(x.cuda(), target.cuda(), lr=0.05)[0] < loss


def test_example_runs(block, capsys):
    import pruned_decode
    pruned_decode.main()
    assert "recovery loss" in capsys.readouterr().out
