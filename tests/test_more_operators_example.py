"""The example of a pruned model beside the dense one it came from, against
plain fp64 torch on the CPU: 4-bit products, verification and distillation
together with the norms and the pruned products."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [os.path.join(ROOT, "examples"), os.path.join(ROOT, "tests")]

pytestmark = pytest.mark.gpu


def norm(x, w, b, half=True):
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-5) * w + b
    return y.half().double() if half else y


def unpacked(packed, group, cols):
    w, scales, zeros = (t.cpu() for t in packed)
    q = torch.stack([w & 15, w >> 4], 2).view(w.shape[0], -1)[:, :cols].double()
    at = torch.arange(cols) // group
    return (q - zeros.double()[:, at]) * scales.double()[:, at]


@pytest.fixture(scope="module")
def pair(spmv_lib):
    import draft_and_verify
    from pruned_decode import DecodeBlock
    block = DecodeBlock(width=512, vocab=700, slots=1, rank=8)
    return block, draft_and_verify.DenseTarget(block, group=64)


def test_quantized_is_near(pair):
    """Half a step of a group's 15, and fp16's rounding of the step, 2^-11 of
    up to 15 steps."""
    _, target = pair
    for dense, packed in ((target.layer, target.layer4), (target.head, target.head4)):
        step = packed[1].cpu().double()[:, torch.arange(512) // 64]
        assert ((unpacked(packed, 64, 512) - dense.cpu().double()).abs() <= step * (1.0 + 2.0 ** -6)).all()


def test_target_logits(pair):
    """Every x is rounded to fp16 on both sides of a 512-term product, and a
    value on the other side of a rounding moves one element by 2^-10: 2^-9 of
    a row's norm covers both."""
    block, target = pair
    r = torch.randn(21, 512, generator=torch.Generator().manual_seed(1))
    (w0, b0), (w1, b1) = [[t.cpu().double() for t in p] for p in block.norms]
    h = r.double() + norm(r.double(), w0, b0) @ unpacked(target.layer4, 64, 512).T
    ref = norm(h, w1, b1) @ unpacked(target.head4, 64, 512).T
    got = target.logits(r.cuda()).cpu().double()
    assert ((got - ref).norm(dim=1) <= 2.0 ** -9 * ref.norm(dim=1)).all()


def test_speculate(pair):
    """The round's tokens by the rules in 64 bits, from the logits that the calls left."""
    import draft_and_verify
    from test_more_operators_gpu import verify_ref
    block, target = pair
    g = torch.Generator(device="cuda").manual_seed(2)
    embedding = torch.randn(700, 512, generator=g, device="cuda")
    last = torch.randint(0, 700, (9,), generator=g, device="cuda").int()
    temperature = torch.tensor([0.5, 1.0, 0.0] * 3, device="cuda")
    for _ in range(3):
        tokens, accepted, given = draft_and_verify.speculate(block, target, embedding, last, 3, temperature, g)
        t, q, x, offsets, au, su = (v.cpu() for v in given)
        out, acc = verify_ref(t, q, x, offsets.tolist(), au, su, temperature.cpu())
        assert accepted.tolist() == acc and tokens.view(-1).tolist() == [out[k] for k in range(36)]
        assert ((tokens >= 0).sum(1) == accepted + 1).all()
        last = tokens.gather(1, accepted.long()[:, None])[:, 0]


def test_distill_step(pair):
    """Loss and gradients against autograd in fp64. The gradient is made of the
    differences of two models' logits, 0.09 in the mean (0.004 sqrt(512)); the
    norm's output is rounded to fp16, which moves the student's by 2^-11 / sqrt(3)
    x 0.05 sqrt(128) = 1.6e-4, 0.0018 of that: 2^-7 is four times as much."""
    import draft_and_verify
    block, target = pair
    hidden = torch.randn(13, 512, generator=torch.Generator().manual_seed(3))
    w, b = [t.cpu().double().requires_grad_() for t in block.norms[1]]
    head = torch.zeros(700, 512, dtype=torch.float64)
    rows = np.repeat(np.arange(700), np.diff(block.head_ptr))
    head[torch.from_numpy(rows), torch.from_numpy(block.head_cols.astype(np.int64))] = torch.from_numpy(block.head_values.astype(np.float64))
    loss, dw, db, teacher = draft_and_verify.distill_step(block, target, hidden.cuda(), top=12, temperature=1.5)
    a = teacher.cpu().double() / 1.5
    lp, at = a.log_softmax(1).topk(12, 1)
    lq = (norm(hidden.double(), w, b, half=False) @ head.T / 1.5).log_softmax(1)
    rest = torch.ones_like(lq, dtype=torch.bool).scatter(1, at, False)
    r = 1 - lp.exp().sum(1)
    rq = torch.where(rest, lq.exp(), 0.0).sum(1)
    ref = ((lp.exp() * (lp - lq.gather(1, at))).sum(1) + r * (r.log() - rq.log())).mean()
    ref.backward()
    assert abs(loss - float(ref.detach())) <= 2.0 ** -8 * float(ref.detach()) + 2.0 ** -12
    for got, want in ((dw, w.grad), (db, b.grad)):
        assert (got.cpu().double() - want).norm() <= 2.0 ** -7 * want.norm()


def test_example_runs(pair, capsys):
    import draft_and_verify
    draft_and_verify.main()
    out = capsys.readouterr().out
    assert "accepted" in out and "distillation loss" in out
