"""CPU tests of the binding of the operators around a pruned layer, with the
CUDA parts of torch that it uses replaced by records of what it asks of them."""
import contextlib
import threading

import pytest

torch = pytest.importorskip("torch")

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
