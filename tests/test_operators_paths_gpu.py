"""GPU tests of the operators around a pruned layer, beside those in
test_operators_gpu.py (whose references and tolerances they use): paths that
only larger calls, other streams, several threads or unusual arguments reach."""
import ctypes
import threading

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


# ---------------------------------------------------------------- streams

class Gradient:
    """A gradient call that needs a workspace, and what it should give."""

    def __init__(self, g, n, d):
        self.x, self.dy, self.w = (randn(g, *size).to(DEV) for size in ((n, d), (n, d), (d,)))
        self.m, self.r = self.x.mean(1), torch.rand(n, generator=g).to(DEV) + 0.5
        self.need = S.spmv_layernorm_backward_workspace(n, d)
        assert self.need > 0
        self.ref = self.run()

    def outputs(self):
        return [torch.empty_like(t) for t in (self.x, self.w, self.w)]

    def run(self, out=None, stream=None):
        out = self.outputs() if out is None else out
        S.spmv_layernorm_backward(self.dy, self.x, self.w, self.m, self.r, *out, stream=stream)
        return out

    def check(self, out):
        assert all(torch.equal(a, b) for a, b in zip(out, self.ref))


def busy(times=20):
    """Work that keeps the current stream busy for some milliseconds."""
    a = torch.ones(8192, 8192, device=DEV)
    for _ in range(times):
        a = (a @ a) * 0.0 + 1.0
    return a


@pytest.mark.parametrize("as_int", [False, True])
def test_a_given_stream_leaves_the_current_streams_freed_blocks_alone(spmv_lib, as_int):
    """The current stream has work queued on a block that is free again; the
    call's own stream is idle and starts at once."""
    call = Gradient(gen(80), 5000, 1000)
    out = call.outputs()
    current, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        victim = torch.full((call.need,), 3, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        keep = busy()
        copy = victim.clone()
        del victim
        call.run(out, stream=other.cuda_stream if as_int else other)
        other.synchronize()
    torch.cuda.synchronize()
    call.check(out)
    assert (copy == 3).all() and keep.isfinite().all()


def test_the_default_streams_workspace_grows_under_another_current_stream(spmv_lib):
    """A thread whose current stream is another one calls on the default
    stream, which is busy: first a small call, then a larger one that replaces
    the kept workspace, then other work of the current stream on new memory."""
    small, large = Gradient(gen(81), 2000, 64), Gradient(gen(82), 5000, 1000)
    side = torch.cuda.Stream()
    outs = [c.outputs() for c in (small, large)]
    failed = []

    def work():
        try:
            keep = busy()
            with torch.cuda.stream(side):
                for c, out in zip((small, large), outs):
                    c.run(out, stream=0)
                    torch.full((c.need,), 255, dtype=torch.uint8, device=DEV)
                torch.full((small.need,), 255, dtype=torch.uint8, device=DEV)
            torch.cuda.synchronize()
            del keep
        except Exception as e:  # (shown by the test's thread)
            failed.append(e)

    torch.cuda.synchronize()
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    assert not failed
    small.check(outs[0])
    large.check(outs[1])


# --------------------------------------------------------------- adapters

@pytest.mark.parametrize("types", ops.ADAPTER_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("rank", [16, 32, 40, 64, 129, 256])
@pytest.mark.parametrize("n_in", [1536, 1544, 1531])
def test_adapters_bits_do_not_depend_on_the_tiles(spmv_lib, types, rank, n_in):
    """Prompts whose slots end in tiles of few and of many tokens: a token's
    result has the same bits wherever it stands, and every time. (Inner sums
    long enough that every warp takes several steps.)"""
    g = gen(91 + rank + n_in)
    sizes = [80, 100, 1, 65, 129, 200, 9]
    t = sum(sizes)
    ids = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(sizes))[torch.randperm(t, generator=g)]
    x, a, b, ids, base, scales = (v.to(DEV) for v in ops.adapter_case(g, t, n_in, 136, rank, len(sizes), *types, ids))

    def run(order):
        y = torch.empty_like(base)
        S.spmv_adapters_run(x[order], a, b, ids[order], y, base=base[order], scales=scales)
        back = torch.empty_like(y)
        back[order] = y
        return back

    first = run(torch.arange(t, device=DEV))
    for _ in range(4):
        assert torch.equal(run(torch.arange(t, device=DEV)), first)
        assert torch.equal(run(torch.randperm(t, generator=g).to(DEV)), first)


# ---------------------------------------------------------------- threads

def test_threads_with_calls_of_different_sizes(spmv_lib):
    """Threads on streams of their own, whose calls take more and less shared
    memory of the same kernels: none is refused, each is right."""
    g = gen(90)
    lists = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV)
             for k, a in ops.everything(g, 300, 40000, 20, 4).items()}

    def norm(d):
        x = randn(g, 4, d).to(DEV)
        return lambda out: S.spmv_layernorm(x, None, None, out), lambda: torch.empty_like(x)

    def adapters(rank):
        args = [t.to(DEV) for t in ops.adapter_case(g, 300, 128, 72, rank, 3, "f16", "f32")]
        return (lambda out: S.spmv_adapters_run(*args[:4], out, base=args[4], scales=args[5]),
                lambda: torch.empty_like(args[4]))

    def logits(v):
        x = randn(g, 300, v).to(DEV)
        kw = {k: lists[k] for k in ("output", "frequency", "presence")}
        return lambda out: S.spmv_logits_process(x, out, **kw), lambda: torch.empty_like(x)

    # (call, outputs, repeats) of each thread
    plans = [[(*norm(d), 3000) for d in sizes] + [(*adapters(r), 300) for r in ranks] + [(*logits(v), 300) for v in vocabs]
             for sizes, ranks, vocabs in (((12288, 10240), (256, 96), (20480 * 2, 16000)),
                                          ((10240, 12288), (64, 160), (18000, 20480 * 2)))]
    refs = []
    for plan in plans:
        refs.append([])
        for call, make, _ in plan:
            out = make()
            call(out)
            refs[-1].append(out)
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(plans))

    def work(plan, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for (call, make, times), right in zip(plan, ref):
                    out = make()
                    for _ in range(times):
                        call(out)
                    torch.cuda.current_stream().synchronize()
                    assert torch.equal(out, right)
        except Exception as e:  # (shown by the test's thread)
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(plans, refs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("t", [1, 40, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_adapters_infinite_weights_leave_infinities(spmv_lib, t, dtype):
    """One element of A x is infinite and the others are finite, far above
    fp16's range and of the opposite effect: y is that infinity, not NaN."""
    g = gen(92)
    n_in, n_out, rank = 64, 24, 8
    x = torch.full((t, n_in), 200.0).to(ops.TYPES[dtype])
    a = torch.full((2, rank, n_in), 200.0).to(ops.TYPES[dtype])     # A x = 2,560,000
    a[0, 3, 5] = float("inf")
    b = -torch.ones(2, n_out, rank).to(ops.TYPES[dtype])
    b[:, ::2, 3] = 1.0                                              # y = inf in even columns, -inf in odd ones
    b[:, ::2, 4:] = -3.0
    ids = torch.arange(t).int() % 2
    y = torch.empty(t, n_out, device=DEV)
    S.spmv_adapters_run(x.to(DEV), a.to(DEV), b.to(DEV), ids.to(DEV), y, base=randn(g, t, n_out).to(DEV))
    got = y.cpu()
    assert (got[::2, ::2] == float("inf")).all() and (got[::2, 1::2] == -float("inf")).all()
    assert got[1::2].isfinite().all()


@pytest.mark.parametrize("stride", [2 ** 31, 2 ** 31 - 1])
def test_logits_of_the_largest_vocabulary(spmv_lib, stride):
    """Token numbers up to the last that int32 holds, in several requests (8.6
    GB in place): the row's end, and a step past it, are above 2^31."""
    v = 2 ** 31 - 1
    buf = torch.zeros(stride + v + 8, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((2, v), (stride, 1))
    tokens = [torch.tensor([0, 77, 2 ** 30 + 1, v - 9_000_000, v - 20000, v - 2, v - 1]), torch.tensor([5, 2 ** 30, v - 3, v - 1])]
    off = torch.tensor([0, len(tokens[0]), len(tokens[0]) + len(tokens[1])], device=DEV)
    mask = torch.full((1, (v + 31) // 32), -1, dtype=torch.int32, device=DEV)
    mask[0, -1] = 0                                # the last 31 tokens
    S.spmv_logits_process(x, x, output=(torch.cat(tokens).int().to(DEV), off), presence=torch.ones(2, device=DEV),
                          mask=mask, mask_rows=torch.tensor([-1, 0], dtype=torch.int32, device=DEV))
    assert (x[0, tokens[0].to(DEV)] == -1).all()
    assert int((x[0] != 0).sum()) == len(tokens[0])
    assert (x[1, tokens[1][:2].to(DEV)] == -1).all()
    assert (x[1, v - 31:] == -float("inf")).all()
    assert int((x[1] != 0).sum()) == 2 + 31
    assert not buf[stride + v:].any() and not buf[v:stride].any()


def test_an_earlier_calls_error_is_not_reported_again(spmv_lib):
    """A call that the driver refuses (one that waits for the device, while a
    graph is captured) says so itself; the next calls are as good as ever."""
    import numpy as np
    plan = S.spmv_plan_create(np.array([0, 1], np.int32), np.zeros(1, np.int32), np.ones(1, np.float32), 4)
    g = gen(93)
    x, out = randn(g, 3, 200).to(DEV), torch.empty(3, 200, device=DEV)
    args = [v.to(DEV) for v in ops.adapter_case(g, 300, 64, 40, 16, 3, "f16", "f32")]
    none = [v.to(DEV) for v in ops.adapter_case(g, 5, 64, 40, 0, 0, "f16", "f32")]

    # (the driver's own capture: torch's would leave its random numbers in it)
    driver, side = ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream()

    def refused():
        graph = ctypes.c_void_p()
        torch.cuda.synchronize()
        assert driver.cuStreamBeginCapture_v2(ctypes.c_void_p(side.cuda_stream), 0) == 0
        try:
            with pytest.raises(S.SpmvError):
                S.spmv_plan_check(plan)
        finally:
            driver.cuStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
        torch.cuda.synchronize()

    refused()
    S.spmv_layernorm(x, None, None, out)
    assert out.isfinite().all()
    for a in (args, none):
        refused()
        y = torch.empty_like(a[4])
        S.spmv_adapters_run(*a[:4], y, base=a[4])
        assert y.isfinite().all()
    S.spmv_plan_destroy(plan)


def test_the_readmes_calls_run(spmv_lib):
    """The operators' calls as README.md prints them."""
    import os
    import re

    import numpy as np
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code, = [c for c in blocks if "spmv_logits_process" in c]
    g = gen(94)
    n, d = 3, 64
    plan = S.spmv_plan_create(np.arange(d + 1, dtype=np.int32), np.arange(d, dtype=np.int32), np.ones(d, np.float16), d)
    residual, x, y = randn(g, n, d).to(DEV), torch.empty(n, d, dtype=torch.float16, device=DEV), torch.empty(n, d, device=DEV)
    names = dict(S=S, plan=plan, residual=residual, x=x, y=y, weight=randn(g, d).to(DEV), bias=randn(g, d).to(DEV),
                 mean=torch.empty(n, device=DEV), rstd=torch.empty(n, device=DEV), a=randn(g, 2, 4, d, dtype="f16").to(DEV),
                 b=randn(g, 2, d, 4, dtype="f16").to(DEV), slot_ids=torch.zeros(n, dtype=torch.int32, device=DEV),
                 ranks=torch.full((2,), 4, dtype=torch.int32, device=DEV), scales=torch.ones(2, device=DEV),
                 logits=randn(g, n, d).to(DEV), tokens=torch.arange(n, dtype=torch.int32, device=DEV),
                 offsets=torch.arange(n + 1, device=DEV), values=torch.ones(n, device=DEV), rep=torch.ones(n, device=DEV),
                 freq=torch.ones(n, device=DEV), pres=torch.ones(n, device=DEV),
                 mask=torch.full((n, d // 32), -1, dtype=torch.int32, device=DEV),
                 mask_rows=torch.arange(n, dtype=torch.int32, device=DEV), dy=randn(g, n, d, dtype="f16").to(DEV),
                 dx=torch.empty(n, d, device=DEV), dweight=torch.empty(d, device=DEV), dbias=torch.empty(d, device=DEV))
    before = names["logits"].clone()
    exec(code, names)
    ref = before.clone()
    ref[torch.arange(n), torch.arange(n)] += 1.0 - 1.0 - 1.0  # bias, frequency, presence
    assert torch.allclose(names["logits"], ref, atol=1e-6)
    S.spmv_plan_destroy(plan)


# ------------------------------------- adapters: prompts and long inner sums
#
# The tolerance of test_operators_gpu.py with K = 256: a matrix instruction
# adds with an error of at most 2 u of what it has summed; the longest chains
# here are 12 of them and 16 partial sums in the first product (12288 inputs
# over 8 blocks of 8 warps at least) and 48 in the second (256 columns of B
# times three terms): 2 (12 + 48) + 16 + 2 < 256.

def check_prompts(case, ranks=None, in_place=False, y_layout=(None, 0)):
    """spmv_adapters_run against products per slot in 64 bits."""
    x, a, b, ids, base, scales = (v.to(DEV) for v in case)
    t, n_out = base.shape
    _, y = ops.out_like(t, n_out, base.dtype, *y_layout)
    given = base
    if in_place:
        y.copy_(base)
        given = y
    S.spmv_adapters_run(x, a, b, ids, y, base=given, scales=scales, ranks=ranks)
    k = 256 * ops.U
    ref, slack = base.double().clone(), k * base.double().abs()
    for s in range(a.shape[0]):
        at = (ids == s).nonzero()[:, 0]
        r = a.shape[1] if ranks is None else min(max(int(ranks[s]), 0), a.shape[1])
        A, B, xs = a[s, :r].double(), b[s, :, :r].double(), x[at].double()
        ref[at] += float(scales[s]) * (xs @ A.T @ B.T)
        slack[at] += k * abs(float(scales[s])) * (xs.abs() @ A.abs().T @ B.abs().T)
    v = base.dtype
    ops.close(y, ref.cpu(), (ops.ROUND[v] * ref.abs() + slack + ops.TINY[v]).cpu(), "y")


@pytest.mark.parametrize("types", [("f16", "f32"), ("bf16", "bf16")], ids=lambda p: "-".join(p))
@pytest.mark.parametrize("n_in,n_out", [(12288, 200), (12296, 136), (8195, 131)])
@pytest.mark.parametrize("rank", [16, 32, 64, 65, 128, 256])
@pytest.mark.parametrize("t", [1, 48, 256, 300, 600])
def test_adapters_long_inner_sums(spmv_lib, t, rank, n_in, n_out, types):
    """Rows of whole 32 bytes, of whole 16 bytes and of any alignment, long
    enough for the main loops of both products, one block of ranks and more."""
    g = gen(100 + t + rank + n_in)
    check_prompts(ops.adapter_case(g, t, n_in, n_out, rank, 4, *types))


@pytest.mark.parametrize("t", [300, 700])
@pytest.mark.parametrize("ids", ["none", "outside", "one", "runs", "alternating"])
def test_adapters_prompts_slot_ids(spmv_lib, t, ids):
    g = gen(141)
    slots = 6
    i = {"none": torch.full((t,), -1), "outside": torch.tensor([-7, slots, 2 ** 31 - 1, -2 ** 31, 3])[torch.arange(t) % 5],
         "one": torch.full((t,), 4), "runs": torch.arange(t) * slots // t, "alternating": torch.arange(t) % 2}[ids]
    ops.check_adapters(*ops.adapter_case(g, t, 160, 96, 16, slots, "f16", "f32", i))


@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("types", ops.ADAPTER_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("layout", [dict(x_layout=(161, 0)), dict(x_layout=(None, 1)), dict(y_layout=(131, 0)),
                                    dict(y_layout=(None, 3)), dict(base_layout=(133, 1)), dict(w_offset=1),
                                    dict(w_offset=8, x_layout=(176, 8), y_layout=(136, 8), base_layout=(144, 8))], ids=str)
def test_adapters_prompts_layouts(spmv_lib, types, layout, rank):
    g = gen(142)
    ops.check_adapters(*ops.adapter_case(g, 300, 160, 128, rank, 3, *types), **layout)


@pytest.mark.parametrize("layout", [(None, 0), (141, 0), (140, 3)], ids=str)
@pytest.mark.parametrize("t", [5, 300])
def test_adapters_in_place_layouts(spmv_lib, t, layout):
    g = gen(143)
    check_prompts(ops.adapter_case(g, t, 264, 136, 40, 3, "f16", "f32"), in_place=True, y_layout=layout)


def test_adapters_prompts_without_base_scales_or_sizes(spmv_lib):
    g = gen(144)
    t = 300
    x, a, b, ids, base, scales = ops.adapter_case(g, t, 100, 60, 16, 3, "f16", "f32")
    ops.check_adapters(x, a, b, ids, base, None, with_base=False)
    ops.check_adapters(*ops.adapter_case(g, t, 128, 61, 40, 3, "bf16", "bf16"), with_base=False)
    for n_in, rank, slots in ((100, 16, 0), (100, 0, 3), (0, 16, 3)):
        x, a, b, _, base, _ = ops.adapter_case(g, t, n_in, 60, rank, slots, "f16", "f32", ids)
        ops.check_adapters(x, a, b, ids, base, None)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-4, 1.0, 300.0])
def test_adapters_prompts_sizes_of_the_inner_product(spmv_lib, dtype, size):
    g = gen(145)
    x, a, b, ids, base, scales = ops.adapter_case(g, 300, 512, 40, 16, 2, dtype, "f32", torch.zeros(300))
    x, a = (x.float() * size).to(x.dtype), (a.float() * 22 * size).to(a.dtype)
    ops.check_adapters(x, a, b, ids, base * 0, scales)


def test_adapters_prompts_a_token_does_not_depend_on_its_tile(spmv_lib):
    """NaN and infinities of one token, or of one slot's weights, stay with
    the tokens that use them; so do those in ranks that a slot does not use."""
    g = gen(146)
    t = 400
    x, a, b, ids, base, scales = ops.adapter_case(g, t, 200, 72, 40, 4, "f16", "f32", torch.arange(t) % 4)
    x[7, 3], x[22, 0] = float("nan"), float("inf")
    a[3, 2, 5] = float("nan")
    ranks = torch.tensor([40, 17, 32, 40])
    a[1, 17:], b[1, :, 17:], a[2, 32:], b[2, :, 32:] = (float("nan"),) * 4
    y = torch.empty(t, 72, device=DEV)
    S.spmv_adapters_run(x.to(DEV), a.to(DEV), b.to(DEV), ids.to(DEV), y, base=base.to(DEV), scales=scales.to(DEV),
                        ranks=ranks.int().to(DEV))
    ref, slack = ops.adapters_ref(x, a, b, ids, base, ranks, scales)
    clean = [k for k in range(t) if k not in (7, 22) and k % 4 != 3]
    ops.close(y[clean], ref[clean], ops.U * ref[clean].abs() + slack[clean])
    assert y[7].isnan().all() and y[3].isnan().all() and not y[22].isfinite().any()


def test_adapters_most_slots_and_many_tokens(spmv_lib):
    g = gen(147)
    # (a reference per slot met: a dense one of 16384 slots would take long)
    x, a, b, ids, base, scales = ops.adapter_case(g, 300, 16, 8, 4, 16384, "f16", "f32")
    ids[:2] = torch.tensor([16383, 0])
    ops.check_adapters(x, a, b, ids, base, scales)
    check_prompts(ops.adapter_case(g, 30000, 32, 24, 8, 3, "f16", "f16"))


# --------------------------------------------------------- norm: long rows

@pytest.mark.parametrize("types", ops.PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("d", [13320, 16384, 16392, 20001])
def test_norm_and_gradient_of_long_rows(spmv_lib, types, d):
    """Both sides of where a row stops fitting one block, rows enough for
    several per block and for partial sums; the gradient in place of dy."""
    g = gen(150 + d)
    n = 70
    x = randn(g, n, d, dtype=types[0], std=1.5, mean=0.25)
    w = randn(g, d, mean=1.0, std=0.3)
    ops.check_norm(x, w, randn(g, d), types[1])
    dy = randn(g, n, d, dtype=types[1], std=0.5)
    ops.check_grad(dy, x, w)
    if types[0] == types[1]:
        m, r = x.float().mean(1).to(DEV), (torch.rand(n, generator=g) + 0.5).to(DEV)
        outs = []
        for in_place in (False, True):
            dyd = dy.to(DEV)
            dx, dw, db = dyd if in_place else torch.empty_like(dyd), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
            S.spmv_layernorm_backward(dyd, x.to(DEV), w.to(DEV), m, r, dx, dw, db)
            outs.append((dx, dw, db))
        assert all(torch.equal(p, q) for p, q in zip(*outs))


# ----------------------------------------------- columns side by side, rows in turn

def side_by_side(rows, widths, dtype):
    """Column ranges of one matrix."""
    buf = torch.zeros(rows, sum(widths), dtype=dtype, device=DEV)
    at = [sum(widths[:i]) for i in range(len(widths))]
    return [buf[:, a:a + w] for a, w in zip(at, widths)]


def rows_in_turn(rows, n, cols, dtype):
    buf = torch.zeros(rows * n, cols, dtype=dtype, device=DEV)
    return [buf[i::n] for i in range(n)]


@pytest.mark.parametrize("d", [64, 263])
@pytest.mark.parametrize("rows", [2, 300])
def test_inputs_and_outputs_of_one_matrix(spmv_lib, rows, d):
    """Column ranges of one matrix, and rows of it in turn, share no element."""
    g = gen(160 + d + rows)
    x = randn(g, rows, d).to(DEV)
    for xs, ys in (side_by_side(rows, (d, d), x.dtype), side_by_side(rows, (d, d), x.dtype)[::-1], rows_in_turn(rows, 2, d, x.dtype)):
        xs.copy_(x)
        y = torch.empty_like(x)
        S.spmv_layernorm(x, None, None, y)
        S.spmv_layernorm(xs, None, None, ys)
        assert torch.equal(y, ys) and torch.equal(x, xs)
        m, r = x.mean(1), torch.ones(rows, device=DEV)
        dy = randn(g, rows, d, dtype="f16").to(DEV)
        S.spmv_layernorm_backward(dy, x, None, m, r, y, None, None)
        S.spmv_layernorm_backward(dy, xs, None, m, r, ys, None, None)
        assert torch.equal(y, ys) and torch.equal(x, xs)
        p = torch.ones(rows, device=DEV)
        lists = (torch.zeros(rows, dtype=torch.int32, device=DEV), torch.arange(rows + 1, device=DEV))
        S.spmv_logits_process(x, y, output=lists, presence=p)
        S.spmv_logits_process(xs, ys, output=lists, presence=p)
        assert torch.equal(y, ys) and torch.equal(x, xs)
    case = [v.to(DEV) for v in ops.adapter_case(g, rows, d, d + 9, 16, 3, "f16", "f16")]
    # (the same strides and boundaries, in three matrices and in one)
    apart = [side_by_side(rows, (d, d + 9, d + 9), torch.float16)[i] for i in range(3)]
    one = side_by_side(rows, (d, d + 9, d + 9), torch.float16)
    for xs, bases, ys in (apart, one):
        xs.copy_(case[0])
        bases.copy_(case[4])
        S.spmv_adapters_run(xs, *case[1:4], ys, base=bases, scales=case[5])
    assert all(torch.equal(p, q) for p, q in zip(apart, one))
    assert torch.equal(one[0], case[0]) and torch.equal(one[1], case[4])


def test_shared_elements_are_refused(spmv_lib):
    buf = torch.zeros(9, 40, device=DEV)
    for x, y in ((buf[:, :16], buf[:, 15:31]), (buf[:, 8:24], buf[:, :16]), (buf[:, :30], buf[:, 10:40]), (buf[:8], buf[1:]),
                 (buf[::2, :16], buf[::2, 8:24]), (buf[:5, :8], buf.view(-1)[4:4 + 5 * 8].view(5, 8)), (buf[0, :8], buf[0, 7:15])):
        with pytest.raises(S.SpmvError):
            S.spmv_layernorm(x, None, None, y)
        with pytest.raises(S.SpmvError):
            S.spmv_logits_process(x, y)


# --------------------------------------------------- logits: many biases

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("size", [(1, 32000, 32000), (2, 50257, 40000), (3, 20480, 3000), (5, 128000, 9000), (470, 2100, 900)],
                         ids=lambda s: "x".join(map(str, s)))
def test_logits_many_biases_keep_list_order(spmv_lib, size, in_place):
    """More biases in a share than a block keeps, many of them repeated, some
    in padding: each token's are added in list order in fp32, bit for bit."""
    import numpy as np
    n, v, k = size
    g = gen(170 + v)
    tok = torch.randint(0, v, (n, k), generator=g)
    tok[:, ::9] = tok[:, 0:1]                       # one token in every piece of the list
    tok[:, 1::50] = -1
    tok[:, 2::50] = v
    val = torch.randn(n, k, generator=g) * 10.0 ** torch.randint(-3, 4, (n, k), generator=g)
    x = randn(g, n, v, std=3.0)
    inside = ((tok >= 0) & (tok < v)).numpy()
    sums = np.zeros((n, v), np.float32)
    np.add.at(sums, (np.nonzero(inside)[0], tok.numpy()[inside]), val.numpy()[inside])
    xd = x.to(DEV)
    out = xd if in_place else torch.full_like(xd, float("nan"))
    S.spmv_logits_process(xd, out, bias=(tok.reshape(-1).int().to(DEV), val.reshape(-1).to(DEV),
                                         torch.arange(n + 1, device=DEV) * k))
    met = torch.from_numpy(sums != 0)
    ref = torch.where(met, x + torch.from_numpy(sums), x)
    assert torch.equal(out.cpu(), ref)


@pytest.mark.parametrize("types", ops.LOGIT_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("size", [(2, 700, 600), (3, 5003, 2500)], ids=lambda s: "x".join(map(str, s)))
def test_logits_many_biases_with_all_the_rest(spmv_lib, size, types):
    """With penalties, masks, padding, and tokens whose counts pass the
    table's bits, biased and not."""
    n, v, k = size
    g = gen(180 + v)
    kw = ops.everything(g, n, v, 40, k, pad=True)
    tok = torch.randint(0, v, (20000,), generator=g).int()
    tok[:9000], tok[10000:19000] = 5, 77
    kw["output"] = (tok, torch.tensor([0] * n + [20000]))
    kw["frequency"] = kw["frequency"] * 0.01
    bias = [t.clone() for t in kw["bias"]]
    bias[2] = torch.cat([torch.zeros(1, dtype=torch.int64), torch.full((n,), k).cumsum(0)])
    bias[0] = torch.randint(-1, v + 1, (n * k,), generator=g).int()
    bias[0][-3] = 5
    bias[0][bias[0] == 77] = 78
    bias[1] = torch.randn(n * k, generator=g)
    kw["bias"] = tuple(bias)
    ops.check_logits(randn(g, n, v, dtype=types[0], std=3.0), types[1], **kw)
