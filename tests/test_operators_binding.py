"""CPU tests of the binding of the operators around a pruned layer, with the
CUDA parts of torch that it uses replaced by records of what it asks of them."""
import contextlib
import threading

import pytest

torch = pytest.importorskip("torch")

import sparse_matrix_vector_gb300 as S  # noqa: E402
from sparse_matrix_vector_gb300 import operators as ops  # noqa: E402


@pytest.fixture
def pools(monkeypatch):
    """Streams without a GPU: `pools.current` is the current stream's handle,
    `pools.taken` lists (pool, bytes) of each block taken."""
    class Pools:
        current, taken = 0, []
    pools = Pools()
    pools.taken = []

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def use(stream):
        before, pools.current = pools.current, stream.cuda_stream
        yield
        pools.current = before

    empty = torch.empty

    def take(n, dtype=None, device=None):
        pools.taken.append((pools.current, n))
        return empty(n, dtype=dtype)

    monkeypatch.setattr(ops, "_raw_stream", lambda dev: pools.current)
    monkeypatch.setattr(ops, "_kept", threading.local())
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: Stream(0))
    monkeypatch.setattr(torch, "empty", take)
    return pools


@pytest.mark.parametrize("current", [0, 64, 128])
@pytest.mark.parametrize("handle", [0, 64, 128])
def test_a_workspace_comes_from_the_pool_of_the_stream_that_uses_it(pools, current, handle):
    pools.current = current
    address, n, owner = ops._workspace(None, 1000, handle=handle, dev=0)
    assert pools.taken == [(handle, 1000)]
    assert pools.current == current
    assert address == owner.data_ptr() and n == 1000


def test_the_default_stream_keeps_its_workspace_in_its_own_pool(pools):
    pools.current = 64
    first = ops._workspace(None, 1000, handle=0, dev=0)[0]
    assert ops._workspace(None, 500, handle=0, dev=0)[0] == first
    ops._workspace(None, 2000, handle=0, dev=0)          # the smaller one is dropped
    assert pools.taken == [(0, 1000), (0, 2000)]
    assert pools.current == 64


def _meta(*size, dtype=torch.float16):
    return torch.empty(*size, dtype=dtype, device="meta")


FAR = 2 ** 32 + 8  # (cut to 8 by a 32-bit argument)


@pytest.mark.parametrize("call", [
    lambda: S.spmv_layernorm(_meta(2, FAR), None, None, _meta(2, FAR)),
    lambda: S.spmv_layernorm(_meta(FAR), None, None, _meta(FAR)),
    lambda: S.spmv_layernorm_backward(_meta(2, FAR), _meta(2, FAR), None, _meta(2), _meta(2), _meta(2, FAR), None, None),
    lambda: S.spmv_adapters_run(_meta(FAR, 4), _meta(2, 3, 4), _meta(2, 5, 3), _meta(FAR), _meta(FAR, 5)),
    lambda: S.spmv_adapters_run(_meta(2, FAR), _meta(2, 3, FAR), _meta(2, 5, 3), _meta(2), _meta(2, 5)),
    lambda: S.spmv_adapters_run(_meta(2, 4), _meta(2, 3, 4), _meta(2, FAR, 3), _meta(2), _meta(2, FAR)),
    lambda: S.spmv_adapters_run(_meta(2, 4), _meta(2, FAR, 4), _meta(2, 5, FAR), _meta(2), _meta(2, 5)),
    lambda: S.spmv_adapters_run(_meta(2, 4), _meta(FAR, 3, 4), _meta(FAR, 5, 3), _meta(2), _meta(2, 5)),
    lambda: S.spmv_logits_process(_meta(2, FAR), _meta(2, FAR)),
    lambda: S.spmv_logits_process(_meta(FAR, 2), _meta(FAR, 2)),
    lambda: S.spmv_logits_process(_meta(2, 40), _meta(2, 40), mask=_meta(FAR, 2, dtype=torch.int32)),
])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(S.SpmvError) as e:
        call()
    assert e.value.status == 8  # too large


def test_workspaces_of_sizes_past_32_bits(spmv_lib):
    assert S.spmv_layernorm_backward_workspace(5000, FAR) == 0
    assert S.spmv_layernorm_backward_workspace(5000, 8 - 2 ** 32) == 0
    assert S.spmv_adapters_workspace(FAR + 5000, 2, 8) == 0
    assert S.spmv_adapters_workspace(5000, FAR, 8) == 0
    assert S.spmv_adapters_workspace(5000, 2, FAR) == 0
    assert S.spmv_adapters_workspace(5000 - 2 ** 32, 2, 8) == 0


def test_a_large_workspace_is_not_kept(pools):
    """A call with a large workspace on the default stream leaves nothing
    behind, and the smaller one that is kept stays."""
    first = ops._workspace(None, 1000, handle=0, dev=0)[0]
    n = (64 << 20) + 1
    for k in range(2):
        owner = ops._workspace(None, n, handle=0, dev=0)[2]
        assert owner.numel() == n and pools.taken == [(0, 1000)] + (k + 1) * [(0, n)]
    assert [t.numel() for t in ops._kept.by_device.values()] == [1000]
    assert ops._workspace(None, 1000, handle=0, dev=0)[0] == first
