"""GPU tests of the operators around a pruned layer, beside those in
test_operators_gpu.py (whose references and tolerances they use): paths that
only larger calls, other streams, several threads or unusual arguments reach."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_gb300")

import test_operators_gpu as ops  # noqa: E402
from test_operators_gpu import DEV, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- logits

@pytest.mark.parametrize("v", [40, 129, 5003])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32")], ids=lambda p: "-".join(p))
def test_logits_requests_with_and_without_lists_in_turn(spmv_lib, v, types):
    """Several requests per block, those without any listed token (empty
    lists, neutral parameters, lists outside the vocabulary) between those
    with some: each keeps to its own lists, every time."""
    g = gen(70 + v)
    n, each = 1400, 24
    kind = torch.arange(n) % 5                      # 0: empty, 1: neutral, 2: padding only, 3 and 4: listed
    lengths = torch.where(kind == 0, 0, torch.randint(1, each + 1, (n,), generator=g))
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    tok = torch.randint(0, v, (int(off[-1]),), generator=g).int()
    tok[torch.repeat_interleave(kind, lengths) == 2] = -1
    on = (kind != 1).float()
    kw = dict(output=(tok, off), repetition=1 + on * torch.rand(n, generator=g), frequency=on * torch.rand(n, generator=g),
              presence=on * 0.25)
    x = randn(g, n, v, dtype=types[0], std=3.0)
    ops.check_logits(x, types[1], **kw)
    dev = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV) for k, a in kw.items()}
    xd = x.to(DEV)
    first = None
    for _ in range(20):
        out = torch.empty(n, v, dtype=ops.TYPES[types[1]], device=DEV)
        S.spmv_logits_process(xd, out, **dev)
        first = out if first is None else first
        assert torch.equal(out, first)
