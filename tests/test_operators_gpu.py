"""GPU tests of the operators around a pruned layer (include/spmv.h, last
section) against plain implementations in 64 bits on the CPU.

Tolerances, with u = 2^-24 (fp32's unit roundoff), v the unit roundoff of an
output's type and K a bound on the fp32 roundings that a sum goes through one
after another (a thread's share of a row plus the tree that joins the
shares; K = 128 covers the rows used here):
  norm:      |y - ref| <= v |ref| + K u (|w| (rstd mean|x| + 2 |xhat|) + |b|)
  gradient:  |dx - ref| <= v |ref| + K u rstd (|g| + mean|g| + |xhat| mean|g xhat|)
             |dw - ref| <= v |ref| + (n + 8) u sum|dy xhat|   (n rows in a chain)
  adapters:  |y - ref| <= v |ref| + K u |base| + K u s sum_j |B_j| sum_k |A_jk x_k|
             (A x is held in fp32, or in terms that keep 2^-22 of its largest)
  logits:    |y - ref| <= v |ref| + 8 u (|l| max(rep, 1/rep) + freq n + |pres|
             + (biases of the token) sum|bias|)
A type's smallest subnormal is added everywhere (its spacing below the
normal range)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_gb300")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 128
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
PAIRS = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *size, dtype="f32", std=1.0, mean=0.0):
    return (torch.randn(*size, generator=g) * std + mean).to(TYPES[dtype])


def to_dev(t, stride=None, offset=0):
    """A copy on the GPU, its rows `stride` elements apart and starting
    `offset` elements after a 256-byte boundary."""
    if t is None:
        return None
    if stride is None and offset == 0:
        return t.to(DEV)
    rows, cols = (1, t.shape[0]) if t.dim() == 1 else t.shape
    stride = cols if stride is None else stride
    buf = torch.full((offset + rows * stride + 8,), 7, dtype=t.dtype, device=DEV)
    view = buf[offset:].as_strided((rows, cols), (stride, 1))
    view.copy_(t.view(rows, cols))
    return view if t.dim() == 2 else view[0]


def out_like(rows, cols, dtype, stride=None, offset=0):
    stride = cols if stride is None else stride
    buf = torch.full((offset + rows * stride + 8,), float("nan"), dtype=dtype, device=DEV)
    return buf, buf[offset:].as_strided((rows, cols), (stride, 1))


def close(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape
    bad = torch.isfinite(ref) & ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} values out of tolerance, worst "
                           f"{((got - ref).abs() / tol)[bad].max():.3g} of it, first at "
                           f"{bad.nonzero()[0].tolist()}")
    odd = ~torch.isfinite(ref)
    assert torch.equal(got[odd].isnan(), ref[odd].isnan()), what
    keep = odd & ~ref.isnan()
    assert torch.equal(got[keep], ref[keep]), what


# ------------------------------------------------------------------- norm

def norm_ref(x, w, b, eps):
    x = x.double()
    d = x.shape[1]
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(d, dtype=torch.float64) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xhat = (x - mean) * rstd
    y = xhat * w + b
    slack = K * U * (w.abs() * (rstd * x.abs().mean(1, keepdim=True) + 2 * xhat.abs()) + b.abs())
    return y, mean[:, 0], rstd[:, 0], slack


def check_norm(x, w, b, y_type, eps=1e-5, stats=True, x_layout=(None, 0), y_layout=(None, 0)):
    n, d = x.shape
    buf, y = out_like(n, d, TYPES[y_type], *y_layout)
    mean = torch.full((n,), float("nan"), device=DEV) if stats else None
    rstd = torch.full((n,), float("nan"), device=DEV) if stats else None
    S.spmv_layernorm(to_dev(x, *x_layout), to_dev(w), to_dev(b), y, eps=eps, mean=mean, rstd=rstd)
    ref, m, r, slack = norm_ref(x, w, b, eps)
    v = TYPES[y_type]
    close(y, ref.to(torch.float64), ROUND[v] * ref.abs() + slack + TINY[v], "y")
    if stats:
        ax = x.double().abs().mean(1)
        close(mean, m, K * U * ax, "mean")
        close(rstd, r, K * U * r * (1 + r * ax), "rstd")
    # nothing outside the rows was written
    inside = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    stride = d if y_layout[0] is None else y_layout[0]
    inside[y_layout[1]:].as_strided((n, d), (stride, 1)).fill_(True)
    assert buf[~inside].isnan().all()


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (5, 7), (2, 31), (7, 64), (33, 255), (4, 257), (9, 1000),
                                   (3, 1024), (2, 4099), (3, 8192), (2, 12288), (2, 20001), (1, 70003)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_norm(spmv_lib, shape, types):
    g = gen(shape[0] * 100003 + shape[1])
    n, d = shape
    x = randn(g, n, d, dtype=types[0], std=2.0, mean=0.5)
    params = "f32" if n % 2 else types[1]
    w, b = randn(g, d, dtype=params, mean=1.0, std=0.3), randn(g, d, dtype=params)
    check_norm(x, w if d % 3 else None, b if d % 5 else None, types[1], stats=d % 7 != 0)


@pytest.mark.parametrize("rows", [2, 300, 5000])
@pytest.mark.parametrize("cols", [96, 1536])
def test_norm_many_rows(spmv_lib, rows, cols):
    g = gen(rows + cols)
    check_norm(randn(g, rows, cols), randn(g, cols, mean=1.0), randn(g, cols), "f16")


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("x_layout,y_layout", [((601, 0), (None, 0)), ((None, 1), (None, 1)), ((608, 0), (616, 8)),
                                               ((603, 3), (605, 5)), ((None, 0), (None, 3))], ids=str)
def test_norm_layouts(spmv_lib, types, x_layout, y_layout):
    g = gen(11)
    x = randn(g, 6, 600, dtype=types[0])
    check_norm(x, randn(g, 600), randn(g, 600), types[1], x_layout=x_layout, y_layout=y_layout)


def test_norm_difficult_rows(spmv_lib):
    """Constant rows, a mean far above the spread, huge and tiny values."""
    g = gen(5)
    x = randn(g, 6, 513)
    x[0] = 3.25
    x[1] += 4096.0
    x[2] *= 1e15
    x[3] *= 1e-18
    x[4] = 0.0
    check_norm(x, randn(g, 513), randn(g, 513), "f32")
    check_norm(x, None, None, "f32", eps=1e-3)


def test_norm_rows_with_inf_and_nan_stay_alone(spmv_lib):
    g = gen(6)
    x = randn(g, 5, 300)
    x[1, 7], x[3, 2] = float("nan"), float("inf")
    y = torch.empty(5, 300, device=DEV)
    S.spmv_layernorm(x.to(DEV), None, None, y)
    got = y.cpu()
    ref, _, _, slack = norm_ref(x, None, None, 1e-5)
    for r in (0, 2, 4):
        assert ((got[r].double() - ref[r]).abs() <= slack[r] + U * ref[r].abs()).all()
    assert got[1].isnan().all() and got[3].isnan().all()


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16")], ids=lambda p: "-".join(p))
@pytest.mark.parametrize("cols", [40, 999, 9216])
def test_norm_in_place_and_repeatable(spmv_lib, types, cols):
    g = gen(7)
    x = randn(g, 40, cols, dtype=types[0]).to(DEV)
    w, b = randn(g, cols).to(DEV), randn(g, cols).to(DEV)
    y = torch.empty_like(x)
    S.spmv_layernorm(x, w, b, y)
    z = torch.empty_like(x)
    S.spmv_layernorm(x, w, b, z)
    assert torch.equal(y, z)
    S.spmv_layernorm(x, w, b, x)
    assert torch.equal(x, y)


def test_norm_vector_and_broadcast_row(spmv_lib):
    g = gen(8)
    x = randn(g, 700)
    y = torch.empty(700, dtype=torch.float16, device=DEV)
    S.spmv_layernorm(x.to(DEV), None, None, y)
    ref, _, _, slack = norm_ref(x[None], None, None, 1e-5)
    close(y[None], ref, 2.0 ** -11 * ref.abs() + slack + 2.0 ** -24)
    rows = torch.empty(5, 700, dtype=torch.float16, device=DEV)
    S.spmv_layernorm(x.to(DEV).expand(5, 700), None, None, rows)
    assert torch.equal(rows, y.expand(5, 700))


def test_norm_offsets_past_32_bits(spmv_lib):
    """Rows more than 2^31 elements apart."""
    stride, d = 2 ** 31 + 64, 260
    buf = torch.empty(stride + d, dtype=torch.float16, device=DEV)
    x = buf.as_strided((2, d), (stride, 1))
    g = gen(9)
    h = randn(g, 2, d, dtype="f16")
    x.copy_(h)
    y = torch.empty(2, d, dtype=torch.float16, device=DEV)
    S.spmv_layernorm(x, None, None, y)
    ref, _, _, slack = norm_ref(h, None, None, 1e-5)
    close(y, ref, 2.0 ** -11 * ref.abs() + slack + 2.0 ** -24)
    S.spmv_layernorm(y, None, None, x)
    assert x.isfinite().all()


# --------------------------------------------------------------- gradient

def grad_ref(dy, x, w, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    xhat = (x - mean) * rstd
    g = dy * w
    a, c = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd * (g - a - xhat * c)
    dx_slack = K * U * rstd * (g.abs() + g.abs().mean(1, keepdim=True)
                               + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    n = x.shape[0]
    return (dx, dx_slack, (dy * xhat).sum(0), (n + 8) * U * (dy * xhat).abs().sum(0), dy.sum(0),
            (n + 8) * U * dy.abs().sum(0))


def check_grad(dy, x, w, param_type="f32", dy_layout=(None, 0), x_layout=(None, 0), dx_layout=(None, 0), want="xwb"):
    n, d = x.shape
    _, m, r, _ = norm_ref(x, None, None, 1e-5)
    m, r = m.float(), r.float()
    buf, dx = out_like(n, d, x.dtype, *dx_layout)
    p = TYPES[param_type]
    dw, db = (torch.full((d,), float("nan"), dtype=p, device=DEV) for _ in range(2))
    S.spmv_layernorm_backward(to_dev(dy, *dy_layout), to_dev(x, *x_layout), to_dev(w), m.to(DEV), r.to(DEV),
                              dx if "x" in want else None, dw if "w" in want else None,
                              db if "b" in want else None)
    rdx, sdx, rdw, sdw, rdb, sdb = grad_ref(dy, x, w, m, r)
    if "x" in want:
        close(dx, rdx, ROUND[x.dtype] * rdx.abs() + sdx + TINY[x.dtype], "dx")
    if "w" in want:
        close(dw, rdw, ROUND[p] * rdw.abs() + sdw + TINY[p], "dweight")
    else:
        assert dw.isnan().all()
    if "b" in want:
        close(db, rdb, ROUND[p] * rdb.abs() + sdb + TINY[p], "dbias")
    else:
        assert db.isnan().all()
    inside = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    stride = d if dx_layout[0] is None else dx_layout[0]
    inside[dx_layout[1]:].as_strided((n, d), (stride, 1)).fill_("x" in want)
    assert buf[~inside].isnan().all()


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (5, 7), (64, 31), (7, 64), (33, 255), (400, 257), (9, 1000),
                                   (3, 1024), (700, 64), (2, 4099), (65, 2048), (11, 8192), (310, 12288),
                                   (2, 20001), (1, 70003), (1025, 64), (1500, 300), (2000, 513), (1100, 1027), (1030, 2048),
                                   (1200, 2051), (900, 5003), (1026, 4096), (600, 8195), (300, 16384)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_gradient(spmv_lib, shape, types):
    n, d = shape
    g = gen(n * 7 + d)
    x = randn(g, n, d, dtype=types[0], std=1.5, mean=0.25)
    dy = randn(g, n, d, dtype=types[1], std=0.5)
    param = "f32" if d % 2 else types[0]
    w = randn(g, d, dtype=param, mean=1.0, std=0.3) if d % 3 else None
    check_grad(dy, x, w, param if w is not None else "f32")


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("shape", [
    # narrow unaligned rows; widths on both sides of each change of the columns per thread
    (1027, 1), (1500, 31), (3000, 101), (1300, 255), (1300, 257), (1100, 511), (1030, 513), (1100, 2056), (1030, 4101),
    (500, 6144), (400, 6160), (330, 8192), (310, 8200)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_norm_and_gradient_at_every_shape(spmv_lib, shape, types):
    n, d = shape
    g = gen(n * 5 + d)
    x = randn(g, n, d, dtype=types[0], std=1.5, mean=0.25)
    w = randn(g, d, mean=1.0, std=0.3)
    check_norm(x, w, randn(g, d), types[1])
    check_grad(randn(g, n, d, dtype=types[1], std=0.5), x, w)


@pytest.mark.parametrize("want", ["x", "w", "b", "wb", "xw", "xb", ""])
def test_gradient_parts(spmv_lib, want):
    g = gen(21)
    check_grad(randn(g, 37, 515, dtype="f16"), randn(g, 37, 515), randn(g, 515), want=want)


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("layouts", [((601, 0), (None, 0), (None, 0)), ((None, 1), (None, 3), (None, 5)),
                                     ((608, 0), (616, 8), (624, 0)), ((None, 0), (None, 0), (607, 3)),
                                     ((0, 0), (None, 0), (None, 0))], ids=str)
def test_gradient_layouts(spmv_lib, types, layouts):
    g = gen(22)
    x = randn(g, 19, 600, dtype=types[0])
    dy = randn(g, 19, 600, dtype=types[1])
    if layouts[0][0] == 0:   # one row of dy for all
        dy = dy[:1].expand(19, 600)
        _, m, r, _ = norm_ref(x, None, None, 1e-5)
        m, r = m.float(), r.float()
        dx, dw, db = torch.empty(19, 600, dtype=x.dtype, device=DEV), torch.empty(600, device=DEV), torch.empty(600, device=DEV)
        S.spmv_layernorm_backward(dy[:1].to(DEV).expand(19, 600), x.to(DEV), None, m.to(DEV), r.to(DEV), dx, dw, db)
        rdx, sdx, rdw, sdw, rdb, sdb = grad_ref(dy, x, None, m, r)
        close(dx, rdx, ROUND[x.dtype] * rdx.abs() + sdx + TINY[x.dtype])
        close(dw, rdw, U * rdw.abs() + sdw)
        close(db, rdb, U * rdb.abs() + sdb)
        return
    check_grad(dy, x, randn(g, 600), dy_layout=layouts[0], x_layout=layouts[1], dx_layout=layouts[2])


def test_gradient_in_place_repeatable_and_empty(spmv_lib):
    g = gen(23)
    x, dy = randn(g, 200, 1000).to(DEV), randn(g, 200, 1000).to(DEV)
    m, r = x.mean(1), torch.rand(200, device=DEV) + 0.5
    w = randn(g, 1000).to(DEV)
    outs = []
    for _ in range(2):
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        S.spmv_layernorm_backward(dy, x, w, m, r, dx, dw, db)
        outs.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    S.spmv_layernorm_backward(dy, x, w, m, r, dy, dw, db)
    assert torch.equal(dy, outs[0][0]) and torch.equal(dw, outs[0][1])
    dw.fill_(7), db.fill_(7)
    S.spmv_layernorm_backward(dy[:0], x[:0], w, m[:0], r[:0], dx[:0], dw, db)
    assert not dw.any() and not db.any()


def test_gradient_against_differences(spmv_lib):
    """Central differences of the forward formula in 64 bits: for a smooth f
    their error is of the order h^2 f''' (h = 1e-5: below 1e-8 here)."""
    g = gen(24)
    n, d, h = 4, 37, 1e-5
    x, w, b = randn(g, n, d).double(), randn(g, d).double(), randn(g, d).double()
    x, w, b = x.float().double(), w.float().double(), b.float().double()
    dy = randn(g, n, d)

    def f(x, w, b):
        return float((norm_ref(x, w, b, 1e-5)[0] * dy.double()).sum())

    def numeric(t, k):
        grad = torch.empty(t.numel(), dtype=torch.float64)
        for i in range(t.numel()):
            args = []
            for sign in (1, -1):
                moved = t.clone()
                moved.view(-1)[i] += sign * h
                args.append(f(*[moved if j == k else a for j, a in enumerate((x, w, b))]))
            grad[i] = (args[0] - args[1]) / (2 * h)
        return grad.view_as(t)

    _, m, r, _ = norm_ref(x, w, b, 1e-5)
    dx, dw, db = torch.empty(n, d, device=DEV), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    S.spmv_layernorm_backward(dy.to(DEV), x.float().to(DEV), w.float().to(DEV), m.float().to(DEV),
                              r.float().to(DEV), dx, dw, db)
    # 1e-8 of the differences, and fp32 (mean and rstd among it) beside it
    for got, t, k in ((dx, x, 0), (dw, w, 1), (db, b, 2)):
        ref = numeric(t, k)
        close(got, ref, 1e-7 + K * U * (ref.abs().max() + 1))


# --------------------------------------------------------------- adapters

def adapters_ref(x, a, b, ids, base, ranks, scales):
    n_slots, rank = a.shape[:2]
    ref, slack = base.double().clone(), K * U * base.double().abs()
    for t, s in enumerate(ids.tolist()):
        if not 0 <= s < n_slots:
            slack[t] = 0
            continue
        r = rank if ranks is None else min(max(int(ranks[s]), 0), rank)
        sc = 1.0 if scales is None else float(scales[s])
        A, B, xt = a[s, :r].double(), b[s, :, :r].double(), x[t].double()
        ref[t] += sc * (B @ (A @ xt))
        absh = A.abs() @ xt.abs()
        slack[t] += K * U * abs(sc) * (B.abs() @ absh)
    return ref, slack


def adapter_case(g, t, n_in, n_out, rank, slots, dtype, y_type, ids=None):
    x = randn(g, t, n_in, dtype=dtype)
    a = randn(g, slots, rank, n_in, dtype=dtype, std=max(n_in, 1) ** -0.5)
    b = randn(g, slots, n_out, rank, dtype=dtype, std=0.3)
    base = randn(g, t, n_out, dtype=y_type)
    if ids is None:
        ids = torch.randint(-1, slots, (t,), generator=g)
    scales = torch.rand(slots, generator=g) * 2 - 0.5
    return x, a, b, ids.int(), base, scales


def check_adapters(x, a, b, ids, base, scales, ranks=None, x_layout=(None, 0), y_layout=(None, 0),
                   base_layout=(None, 0), w_offset=0, with_base=True):
    t, n_out = base.shape
    buf, y = out_like(t, n_out, base.dtype, *y_layout)
    shift = lambda w: to_dev(w.reshape(-1), offset=w_offset).view(w.shape) if w_offset and w.numel() else w.to(DEV)  # noqa: E731
    S.spmv_adapters_run(to_dev(x, *x_layout), shift(a), shift(b), ids.to(DEV), y,
                        base=to_dev(base, *base_layout) if with_base else None,
                        ranks=None if ranks is None else ranks.int().to(DEV),
                        scales=None if scales is None else scales.to(DEV))
    ref, slack = adapters_ref(x, a, b, ids, base if with_base else torch.zeros_like(base), ranks, scales)
    close(y, ref, ROUND[base.dtype] * ref.abs() + slack + TINY[base.dtype], "y")
    inside = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    stride = n_out if y_layout[0] is None else y_layout[0]
    inside[y_layout[1]:].as_strided((t, n_out), (stride, 1)).fill_(True)
    assert buf[~inside].isnan().all()


ADAPTER_TYPES = [("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("types", ADAPTER_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("size", [
    # tokens, n_in, n_out, rank, slots
    (1, 1, 1, 1, 1), (1, 64, 48, 8, 2), (1, 1000, 777, 16, 3), (2, 65, 33, 5, 2), (3, 512, 512, 64, 1), (5, 130, 257, 3, 4),
    (8, 300, 200, 20, 3), (17, 256, 129, 33, 5), (33, 512, 96, 128, 2), (40, 72, 640, 256, 2), (64, 200, 72, 16, 64),
    (100, 333, 101, 12, 3), (150, 96, 64, 32, 2), (257, 64, 40, 16, 9), (300, 129, 65, 24, 300), (1030, 40, 24, 8, 4),
    (5000, 16, 8, 4, 7)], ids=lambda s: "x".join(map(str, s)))
def test_adapters(spmv_lib, size, types):
    t, n_in, n_out, rank, slots = size
    g = gen(sum(size))
    check_adapters(*adapter_case(g, t, n_in, n_out, rank, slots, *types))


@pytest.mark.parametrize("t", [1, 4, 31, 70, 260])
@pytest.mark.parametrize("types", [("f16", "f32"), ("bf16", "bf16")], ids=lambda p: "-".join(p))
def test_adapters_mixed_ranks(spmv_lib, t, types):
    """Ranks from nothing to all (one given beyond both ends); the rows and
    columns that a slot does not use hold NaN."""
    g = gen(31 + t)
    slots, rank = 9, 40
    x, a, b, ids, base, scales = adapter_case(g, t, 264, 88, rank, slots, *types)
    ranks = torch.tensor([0, 1, 7, 8, 16, 17, 39, 40, 99])
    ranks[0] = -3 if t % 2 else 0
    for s in range(slots):
        r = min(max(int(ranks[s]), 0), rank)
        a[s, r:] = float("nan")
        b[s, :, r:] = float("nan")
    check_adapters(x, a, b, ids, base, scales, ranks=ranks)


@pytest.mark.parametrize("t", [3, 90])
@pytest.mark.parametrize("ids", ["none", "outside", "one", "runs", "alternating"])
def test_adapters_slot_ids(spmv_lib, t, ids):
    g = gen(41)
    slots = 6
    i = {"none": torch.full((t,), -1), "outside": torch.tensor([-7, slots, 2 ** 31 - 1, -2 ** 31, 3])[torch.arange(t) % 5],
         "one": torch.full((t,), 4), "runs": torch.arange(t) * slots // t, "alternating": torch.arange(t) % 2}[ids]
    check_adapters(*adapter_case(g, t, 160, 96, 16, slots, "f16", "f32", i))


@pytest.mark.parametrize("t", [2, 80])
@pytest.mark.parametrize("types", ADAPTER_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("layout", [dict(x_layout=(161, 0)), dict(x_layout=(None, 1)), dict(y_layout=(131, 0)),
                                    dict(y_layout=(None, 3)), dict(base_layout=(133, 1)), dict(w_offset=1),
                                    dict(w_offset=8, x_layout=(176, 8), y_layout=(136, 8), base_layout=(144, 8))], ids=str)
def test_adapters_layouts(spmv_lib, t, types, layout):
    g = gen(42)
    check_adapters(*adapter_case(g, t, 160, 128, 16, 3, *types), **layout)


@pytest.mark.parametrize("t", [2, 80])
def test_adapters_without_base_scales_or_sizes(spmv_lib, t):
    g = gen(43)
    x, a, b, ids, base, scales = adapter_case(g, t, 100, 60, 16, 3, "f16", "f32")
    check_adapters(x, a, b, ids, base, None, with_base=False)
    # nothing to add: no slots, rank 0, no inputs
    for n_in, rank, slots in ((100, 16, 0), (100, 0, 3), (0, 16, 3)):
        x, a, b, _, base, _ = adapter_case(g, t, n_in, 60, rank, slots, "f16", "f32", ids)
        check_adapters(x, a, b, ids, base, None)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t", [2, 80])
@pytest.mark.parametrize("size", [1e-4, 1.0, 300.0])
def test_adapters_sizes_of_the_inner_product(spmv_lib, t, dtype, size):
    """A x far below and above what 16 bits hold: it is kept in 32."""
    g = gen(44)
    x, a, b, ids, base, scales = adapter_case(g, t, 512, 40, 16, 2, dtype, "f32", torch.zeros(t))
    x, a = (x.float() * size).to(x.dtype), (a.float() * 22 * size).to(a.dtype)
    check_adapters(x, a, b, ids, base * 0, scales)


@pytest.mark.parametrize("t", [1, 5, 80, 400])
def test_adapters_in_place_and_repeatable(spmv_lib, t):
    g = gen(45)
    x, a, b, ids, base, scales = adapter_case(g, t, 520, 264, 24, 5, "f16", "f32")
    x, a, b, ids, base, scales = (v.to(DEV) for v in (x, a, b, ids, base, scales))
    ys = [torch.empty_like(base) for _ in range(2)]
    for y in ys:
        S.spmv_adapters_run(x, a, b, ids, y, base=base, scales=scales)
    assert torch.equal(*ys)
    ws = torch.full((S.spmv_adapters_workspace(t, 5, 24) + 16,), 255, dtype=torch.uint8, device=DEV)
    S.spmv_adapters_run(x, a, b, ids, base, base=base, scales=scales, workspace=ws)
    assert torch.equal(base, ys[0])


def test_adapters_a_token_does_not_depend_on_its_batch(spmv_lib):
    """NaN and infinities of one token, or of one slot's weights, stay with
    the tokens that use them."""
    g = gen(46)
    x, a, b, ids, base, scales = adapter_case(g, 50, 200, 72, 16, 4, "f16", "f32", torch.arange(50) % 4)
    x[7, 3], x[22, 0] = float("nan"), float("inf")
    a[3, 2, 5] = float("nan")
    y = torch.empty(50, 72, device=DEV)
    S.spmv_adapters_run(x.to(DEV), a.to(DEV), b.to(DEV), ids.to(DEV), y, base=base.to(DEV), scales=scales.to(DEV))
    ref, slack = adapters_ref(x, a, b, ids, base, None, scales)
    clean = [t for t in range(50) if t not in (7, 22) and t % 4 != 3]
    close(y[clean], ref[clean], U * ref[clean].abs() + slack[clean])
    assert y[7].isnan().all() and y[3].isnan().all() and not y[22].isfinite().any()


# ----------------------------------------------------------------- logits

def logits_ref(x, prompt, output, rep, freq, pres, bias, mask, rows):
    n, v = x.shape
    ref, slack = x.double().clone(), torch.zeros(n, v, dtype=torch.float64)
    for i in range(n):
        lists = []
        for pair in (prompt, output):
            t = np.zeros(0, np.int64) if pair is None else pair[0].numpy()[int(pair[1][i]):int(pair[1][i + 1])].astype(np.int64)
            lists.append(torch.from_numpy(t[(t >= 0) & (t < v)]))
        count = torch.bincount(lists[1], minlength=v).double()
        seen = (torch.bincount(lists[0], minlength=v) > 0) | (count > 0)
        r = 1.0 if rep is None else float(rep[i])
        f = 0.0 if freq is None else float(freq[i])
        p = 0.0 if pres is None else float(pres[i])
        l = ref[i]
        slack[i] = 8 * U * (l.abs() * max(r, 1 / r) + abs(f) * count + abs(p))
        l = torch.where(seen, torch.where(l > 0, l / r, l * r), l)
        l = l - f * count - p * (count > 0)
        if bias is not None:
            lo, hi = int(bias[2][i]), int(bias[2][i + 1])
            per = torch.bincount(bias[0][lo:hi][(bias[0][lo:hi] >= 0) & (bias[0][lo:hi] < v)].long(), minlength=v)
            size = torch.zeros(v, dtype=torch.float64)
            for k in range(lo, hi):
                tok = int(bias[0][k])
                if 0 <= tok < v:
                    l[tok] += float(bias[1][k])
                    size[tok] += abs(float(bias[1][k]))
            finite = torch.where(size.isfinite(), size, 0.0)
            slack[i] += 8 * U * per * finite
        row = (i if rows is None else int(rows[i])) if mask is not None else -1
        if mask is not None and 0 <= row < mask.shape[0]:
            bits = (mask[row].numpy().astype(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
            l = torch.where(torch.from_numpy(bits.reshape(-1)[:v].astype(bool)), l, -math.inf)
        ref[i] = l
    return ref, slack


def ragged(g, n, longest, v, pad=False):
    lengths = torch.randint(0, longest + 1, (n,), generator=g)
    lengths[0] = longest
    if n > 1:
        lengths[1] = 0
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    tok = (torch.rand(int(off[-1]), generator=g) ** 3 * v).int().clamp(max=v - 1)
    if pad and tok.numel():
        tok[::5] = -1
        tok[1::7] = v
        tok[2::11] = 2 ** 31 - 1
        tok[3::13] = -2 ** 31
    return tok, off


def check_logits(x, out_type, x_layout=(None, 0), out_layout=(None, 0), **kw):
    n, v = x.shape
    buf, out = out_like(n, v, TYPES[out_type], *out_layout)
    dev = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV) for k, a in kw.items() if a is not None}
    S.spmv_logits_process(to_dev(x, *x_layout), out, **dev)
    ref, slack = logits_ref(x, kw.get("prompt"), kw.get("output"), kw.get("repetition"), kw.get("frequency"),
                            kw.get("presence"), kw.get("bias"), kw.get("mask"), kw.get("mask_rows"))
    v_t = TYPES[out_type]
    close(out, ref, ROUND[v_t] * ref.abs() + slack + TINY[v_t], "logits")
    inside = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    stride = v if out_layout[0] is None else out_layout[0]
    inside[out_layout[1]:].as_strided((n, v), (stride, 1)).fill_(True)
    assert buf[~inside].isnan().all()


def everything(g, n, v, history, biases, pad=False):
    masks = max(1, n // 2)
    rows = torch.randint(-1, masks, (n,), generator=g)
    return dict(prompt=ragged(g, n, history, v, pad), output=ragged(g, n, max(1, history // 2), v, pad),
                repetition=torch.rand(n, generator=g) + 0.7, frequency=torch.rand(n, generator=g),
                presence=torch.rand(n, generator=g) - 0.3,
                bias=(lambda p: (p[0], torch.randn(p[0].numel(), generator=g), p[1]))(ragged(g, n, biases, v, pad)),
                mask=torch.randint(-2 ** 31, 2 ** 31, (masks, (v + 31) // 32), generator=g).int(), mask_rows=rows.int())


LOGIT_TYPES = [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("types", LOGIT_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("size", [
    # requests, vocabulary, history, biases
    (1, 1, 3, 2), (1, 31, 5, 3), (3, 33, 40, 9), (2, 1000, 300, 20), (5, 4096, 50, 0), (4, 4097, 700, 64), (2, 8191, 9, 40),
    (3, 16385, 2000, 1500), (1, 50257, 5000, 33), (2, 128000, 300, 300), (300, 129, 20, 4)],
    ids=lambda s: "x".join(map(str, s)))
def test_logits(spmv_lib, size, types):
    n, v, history, biases = size
    g = gen(sum(size))
    check_logits(randn(g, n, v, dtype=types[0], std=3.0), types[1], **everything(g, n, v, history, biases))


@pytest.mark.parametrize("only", [["prompt", "repetition"], ["output", "frequency"], ["output", "presence"],
                                  ["output", "repetition"], ["bias"], ["mask"], ["mask", "mask_rows"], [],
                                  ["prompt", "output"], ["repetition", "frequency"]], ids=lambda o: "+".join(o) or "nothing")
def test_logits_parts(spmv_lib, only):
    g = gen(51)
    n, v = 6, 5000
    kw = everything(g, n, v, 400, 60)
    if "mask_rows" not in only:
        kw["mask"] = kw["mask"][torch.arange(n) % kw["mask"].shape[0]].contiguous()
    check_logits(randn(g, n, v, std=3.0), "f32", **{k: a for k, a in kw.items() if k in only})


def test_logits_padded_lists(spmv_lib):
    g = gen(52)
    check_logits(randn(g, 4, 3001), "f32", **everything(g, 4, 3001, 500, 80, pad=True))


@pytest.mark.parametrize("types", LOGIT_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("layouts", [((1001, 0), (None, 0)), ((None, 1), (None, 3)), ((1008, 8), (1016, 8)), ((1003, 0), (1005, 1))],
                         ids=str)
def test_logits_layouts(spmv_lib, types, layouts):
    g = gen(53)
    check_logits(randn(g, 3, 1000, dtype=types[0]), types[1], x_layout=layouts[0], out_layout=layouts[1],
                 **everything(g, 3, 1000, 90, 20))


@pytest.mark.parametrize("types", LOGIT_TYPES, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("size", [(9, 3, 6, 2), (9, 13, 20, 3), (9, 45, 40, 9), (9, 1003, 90, 20), (5, 16387, 9000, 30)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("layouts", [((1, 0), (1, 0)), ((3, 5), (3, 5)), ((6, 2), (6, 10)), ((2, 3), (10, 11)), ((7, 1), (3, 4)), ((5, 0), (5, 1))],
                         ids=str)
def test_logits_row_boundaries(spmv_lib, types, size, layouts):
    """Rows that start anywhere: vectors from the first boundary that x and
    out share, if they share one. (layouts: elements between rows, offset)"""
    n, v, history, biases = size
    g = gen(57 + v)
    check_logits(randn(g, n, v, dtype=types[0], std=3.0), types[1], *[(v + more, offset) for more, offset in layouts],
                 **everything(g, n, v, history, biases))


def test_logits_masks_and_special_values(spmv_lib):
    """A mask that leaves nothing; infinities, NaN and the type's lowest
    value in allowed and in masked places; a bias of -inf."""
    g = gen(54)
    n, v = 4, 200
    x = randn(g, n, v)
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min
    x[:, 40], x[:, 41], x[:, 42] = float("nan"), float("inf"), -float("inf")
    mask = torch.full((n, 7), -1, dtype=torch.int32)
    mask[0] = 0                       # nothing allowed
    mask[1, 1] = 0                    # tokens 32..63 masked
    kw = dict(repetition=torch.tensor([1.2, 1.2, 0.8, 1.0]), frequency=torch.full((n,), 0.5), presence=torch.full((n,), 0.1),
              output=(torch.tensor([0, 1, 2, 5, 5, 40, 41] * n).int(), torch.arange(n + 1) * 7),
              bias=(torch.tensor([7, 9, 9, 40] * n).int(), torch.tensor([-math.inf, 1.0, 2.0, math.inf] * n), torch.arange(n + 1) * 4),
              mask=mask)
    check_logits(x, "f32", **kw)
    out = torch.empty(n, v, device=DEV)
    S.spmv_logits_process(x.to(DEV), out, mask=mask.to(DEV))
    assert (out[0] == -math.inf).all() and (out[1, 32:64] == -math.inf).all()


def test_logits_repeated_biases_keep_list_order(spmv_lib):
    """Repeated biases are added in list order in fp32: the same bits always."""
    n, v = 2, 4096
    tokens = torch.tensor([5, 4000, 5, 5, 77] * 40 + [5]).int()
    g = gen(55)
    values = torch.randn(tokens.numel(), generator=g) * 10.0 ** torch.randint(-3, 4, (tokens.numel(),), generator=g)
    off = torch.tensor([0, 0, tokens.numel()])
    x = torch.zeros(n, v)
    out = torch.empty(n, v, device=DEV)
    S.spmv_logits_process(x.to(DEV), out, bias=(tokens.to(DEV), values.to(DEV), off.to(DEV)))
    ref = np.zeros(v, np.float32)
    for t, b in zip(tokens.tolist(), values.numpy()):
        ref[t] += b
    assert np.array_equal(out[1].cpu().numpy(), ref) and not out[0].any()


@pytest.mark.parametrize("v", [100, 5001, 70000])
def test_logits_in_place_repeatable_and_counts(spmv_lib, v):
    g = gen(56)
    kw = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV)
          for k, a in everything(g, 5, v, 3000, 200).items()}
    x = randn(g, 5, v).to(DEV)
    outs = [torch.empty_like(x) for _ in range(2)]
    for o in outs:
        S.spmv_logits_process(x, o, **kw)
    assert torch.equal(*outs)
    S.spmv_logits_process(x, x, **kw)
    assert torch.equal(x, outs[0])
    # one token many times, more than 16 bits count
    many = torch.full((70000,), v - 1, dtype=torch.int32, device=DEV)
    x = torch.zeros(1, v, device=DEV)
    o = torch.empty_like(x)
    S.spmv_logits_process(x, o, output=(many, torch.tensor([0, 70000], device=DEV)), frequency=torch.ones(1, device=DEV))
    assert float(o[0, v - 1]) == -70000.0 and not o[0, :v - 1].any()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16")], ids=lambda p: "-".join(p))
def test_logits_many_requests_long_lists(spmv_lib, types, in_place):
    """Enough requests that a block has a large share of the vocabulary, with
    more tokens and biases in it than it keeps as lists, and a token whose
    count passes 16 bits among them."""
    g = gen(57)
    n, v = 460, 7003
    x = randn(g, n, v, dtype=types[0], std=3.0)
    lengths = torch.zeros(n, dtype=torch.int64)
    lengths[3], lengths[4], lengths[200], lengths[459] = 30000, 2500, 100000, 9000
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    tok = torch.randint(0, v, (int(off[-1]),), generator=g).int()
    tok[off[200] + 5000:off[200] + 95000] = 6999          # 90000 times one token
    tok[off[459]:off[460]] = 17                           # one token only
    blen = torch.zeros(n, dtype=torch.int64)
    blen[3], blen[7], blen[200] = 1500, 700, 900
    boff = torch.cat([torch.zeros(1, dtype=torch.int64), blen.cumsum(0)])
    btok = torch.randint(0, v, (int(boff[-1]),), generator=g).int()
    kw = dict(prompt=(tok.flip(0).contiguous(), off), output=(tok, off), repetition=torch.rand(n, generator=g) + 0.7,
              frequency=torch.rand(n, generator=g) * 0.01, presence=torch.rand(n, generator=g),
              bias=(btok, torch.randn(btok.numel(), generator=g), boff),
              mask=torch.randint(-2 ** 31, 2 ** 31, (2, (v + 31) // 32), generator=g).int(),
              mask_rows=(torch.arange(n) % 3 - 1).int())
    dev = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV) for k, a in kw.items()}
    xd = x.to(DEV)
    out = xd if in_place else torch.full((n, v), float("nan"), dtype=TYPES[types[1]], device=DEV)
    S.spmv_logits_process(xd, out, **dev)
    ref, slack = logits_ref(x, kw["prompt"], kw["output"], kw["repetition"], kw["frequency"], kw["presence"],
                            kw["bias"], kw["mask"], kw["mask_rows"])
    t = TYPES[types[1]]
    close(out, ref, ROUND[t] * ref.abs() + slack + TINY[t], "logits")


# -------------------------------------------------------- streams and graphs

def _calls(g, big):
    n, d = (400, 4096) if big else (3, 200)
    x, dy = randn(g, n, d).to(DEV), randn(g, n, d, dtype="f16").to(DEV)
    w, b = randn(g, d).to(DEV), randn(g, d).to(DEV)
    m, r = x.mean(1), torch.rand(n, device=DEV) + 0.5
    ad = [v.to(DEV) for v in adapter_case(g, n, 512, 264, 16, 4, "f16", "f32")]
    lg = {k: tuple(t.to(DEV) for t in a) if isinstance(a, tuple) else a.to(DEV) for k, a in everything(g, n, 2000, 100, 20).items()}
    logits = randn(g, n, 2000).to(DEV)

    def outputs():
        return [torch.zeros(n, d, dtype=torch.float16, device=DEV), torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b),
                torch.zeros(n, 264, device=DEV), torch.zeros_like(logits)]

    def run(o, stream=None):
        S.spmv_layernorm(x, w, b, o[0], stream=stream)
        S.spmv_layernorm_backward(dy, x, w, m, r, o[1], o[2], o[3], stream=stream)
        S.spmv_adapters_run(ad[0], ad[1], ad[2], ad[3], o[4], base=ad[4], scales=ad[5], stream=stream)
        S.spmv_logits_process(logits, o[5], stream=stream, **lg)

    return outputs, run


@pytest.mark.parametrize("big", [False, True])
def test_other_streams_and_graphs(spmv_lib, big):
    outputs, run = _calls(gen(61), big)
    ref = outputs()
    run(ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream, make in ((side, lambda: side), (side.cuda_stream, lambda: side)):
        o = outputs()
        torch.cuda.synchronize()
        run(o, stream=stream)
        # the workspaces that the calls took are free again for this stream,
        # while the other one may still be at work on them
        torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
        make().synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, ref))
    o = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(o)
    for t in o:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_wrong_tensors_are_refused(spmv_lib):
    x = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError):
        S.spmv_layernorm(x, torch.zeros(8), None, x)                     # weight on the CPU
    with pytest.raises(ValueError):
        S.spmv_layernorm(x, torch.zeros(9, device=DEV), None, x)
    with pytest.raises(TypeError):
        S.spmv_layernorm(x, None, None, torch.zeros(4, 8, dtype=torch.float64, device=DEV))
    with pytest.raises(S.SpmvError):
        S.spmv_layernorm(x.half(), None, None, x)
    with pytest.raises(TypeError):
        S.spmv_layernorm(x, None, None, x, mean=torch.zeros(4, dtype=torch.float16, device=DEV))
    many = torch.zeros(5000, 8, device=DEV)
    with pytest.raises(S.SpmvError):
        S.spmv_layernorm_backward(many, many, None, many[:, 0].contiguous(), many[:, 0].contiguous(), torch.zeros_like(many),
                                  torch.zeros(8, device=DEV), None, workspace=torch.zeros(0, dtype=torch.uint8, device=DEV))
    with pytest.raises(S.SpmvError):
        S.spmv_adapters_run(x, torch.zeros(2, 4, 8, device=DEV), torch.zeros(2, 8, 4, device=DEV),
                            torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, 8, device=DEV))
    with pytest.raises(TypeError):
        S.spmv_adapters_run(x.half(), torch.zeros(2, 4, 8, device=DEV).half(), torch.zeros(2, 8, 4, device=DEV).half(),
                            torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 8, device=DEV))
    with pytest.raises(ValueError):
        S.spmv_logits_process(x, torch.zeros(4, 8, device=DEV), repetition=torch.ones(3, device=DEV))
