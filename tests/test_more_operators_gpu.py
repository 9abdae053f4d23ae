"""GPU tests of the operators that put a pruned model beside the dense one it
came from (include/spmv.h, last section) against plain implementations in 64
bits on the CPU.

Tolerances, with u = 2^-24 (fp32's unit roundoff), v the unit roundoff of an
output's type and K = 128 a bound on the fp32 roundings that a sum goes
through one after another:
  int4:     |y - ref| <= v |ref| + K u (|base| + sum_i |W_i x_i|)
            (weights less their zero points, and the products of 16-bit
            numbers, are exact)
  distill:  an exponential 2^d is off by E = (4 + 3 |d|) u of itself (4 u of
            the instruction, three roundings of its argument), so a row's sum
            S by dS = sum_v e_v (E_v + K u); the logarithms of p and q by K u
            of themselves and one, the latter by dS / S more.
  verify:   whole numbers, equal."""
import math

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_gb300")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 128
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
INF = float("inf")
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
    buf = torch.full((offset + rows * stride + cols + 8,), 7, dtype=t.dtype, device=DEV)
    view = buf[offset:].as_strided((rows, cols), (stride, 1))
    (view if stride else view[:1]).copy_(t.view(rows, cols) if stride else t.view(rows, cols)[:1])
    return view if t.dim() == 2 else view[0]


def out_like(rows, cols, dtype, stride=None, offset=0):
    stride = cols if stride is None else stride
    buf = torch.full((offset + rows * stride + 8,), float("nan"), dtype=dtype, device=DEV)
    return buf, buf[offset:].as_strided((rows, cols), (stride, 1))


def untouched(buf, rows, cols, stride, offset):
    """Whether everything but the rows still holds NaN."""
    keep = torch.ones(buf.numel(), dtype=torch.bool)
    keep[offset:].as_strided((rows, cols), (stride, 1)).fill_(False)
    return bool(buf.cpu()[keep].isnan().all())


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


# ------------------------------------------------------------------- int4

def int4_case(seed, t, n_in, n_out, group, x="f16", scales="f32", zeros=True, base=None):
    g = gen(seed)
    groups = -(-n_in // group) if n_in else 0
    w = torch.randint(0, 256, (n_out, (n_in + 1) // 2), generator=g, dtype=torch.uint8)
    sc = randn(g, n_out, groups, dtype=scales)
    z = torch.randint(0, 256, (n_out, groups), generator=g, dtype=torch.uint8) if zeros else None
    return randn(g, t, n_in, dtype=x), w, sc, z, None if base is None else randn(g, t, n_out, dtype=base, std=3.0)


def int4_ref(x, w, sc, z, base, group):
    n_out, n_in = w.shape[0], x.shape[1]
    q = torch.stack([w & 15, w >> 4], 2).view(n_out, -1)[:, :n_in].double()
    at = torch.arange(n_in) // group
    wd = (q - (8.0 if z is None else (z & 15).double()[:, at])) * sc.double()[:, at]
    y, slack = x.double() @ wd.T, x.double().abs() @ wd.abs().T
    if base is not None:
        y, slack = y + base.double(), slack + base.double().abs()
    return y, K * U * slack


def int4_check(t, n_in, n_out, group, x="f16", y="f32", scales="f32", zeros=True, base=False, seed=0, in_place=False,
               x_at=(None, 0), w_at=(None, 0), y_at=(None, 0)):
    xs, w, sc, z, b = int4_case(seed, t, n_in, n_out, group, x, scales, zeros, y if base else None)
    ref, slack = int4_ref(xs, w, sc, z, b, group)
    buf, out = out_like(t, n_out, TYPES[y], *y_at)
    if in_place:
        out.copy_(b)
    S.spmv_int4_run(to_dev(xs, *x_at), to_dev(w, *w_at), to_dev(sc), out, group, zeros=to_dev(z), base=out if in_place else to_dev(b))
    close(out, ref, ROUND[TYPES[y]] * ref.abs() + slack + TINY[TYPES[y]], f"{t} x {n_in} -> {n_out}, groups of {group}")
    assert untouched(buf, t, n_out, y_at[0] or n_out, y_at[1])


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 100000])
@pytest.mark.parametrize("t", [1, 2, 8, 9, 16, 17, 32, 33, 64, 65, 150])
def test_int4_tokens_and_groups(t, group, x):
    int4_check(t, 1312, 100, group, x=x, zeros=t % 2 == 0, base=t % 3 == 0, scales="f32" if t % 4 else x)


@pytest.mark.parametrize("x,y", [("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n_in,n_out", [(1, 1), (2, 3), (31, 5), (32, 32), (33, 16), (127, 17), (128, 33), (129, 64), (255, 31), (640, 257),
                                        (1000, 40), (2048, 48), (5003, 70), (12288, 33)])
def test_int4_sizes(n_in, n_out, x, y):
    for t, group in ((1, 32), (5, 128), (19, 64)):
        int4_check(t, n_in, n_out, group, x=x, y=y, scales=x, zeros=n_out % 2 == 1, base=t == 5, seed=n_in)


@pytest.mark.parametrize("t", [1, 7, 24, 64])
@pytest.mark.parametrize("w_at", [(700, 0), (656, 16), (657, 0), (660, 3), (656, 8), (672, 1)])
@pytest.mark.parametrize("x_at", [(1312, 0), (1313, 0), (1320, 8), (1400, 5)])
def test_int4_rows_anywhere(t, w_at, x_at):
    int4_check(t, 1312, 75, 64, x="bf16", x_at=x_at, w_at=w_at, y_at=(80, 3), base=True)
    int4_check(t, 1311, 75, 128, x="f16", x_at=x_at, w_at=w_at, y_at=(80, 3), base=True, in_place=True)


def test_int4_no_columns_and_no_tokens():
    x, w, sc, z, b = int4_case(1, 3, 0, 5, 32, base="f32")
    out = torch.empty(3, 5, device=DEV)
    S.spmv_int4_run(x.to(DEV), w.to(DEV), sc.to(DEV), out, 32, zeros=z.to(DEV), base=b.to(DEV))
    assert torch.equal(out.cpu(), b)
    S.spmv_int4_run(x.to(DEV), w.to(DEV), sc.to(DEV), out, 32)
    assert torch.equal(out.cpu(), torch.zeros(3, 5))
    x, w, sc, z, b = int4_case(1, 0, 64, 5, 32)
    S.spmv_int4_run(x.to(DEV), w.to(DEV), sc.to(DEV), torch.empty(0, 5, device=DEV), 32)


@pytest.mark.parametrize("t", [1, 5, 20, 64])
def test_int4_special_values(t):
    """Infinities, NaN, the largest numbers and subnormals of x stay in their own token."""
    xs, w, sc, z, _ = int4_case(5, t, 300, 40, 64)
    xs[0, 7] = INF
    if t > 4:
        xs[1, 130] = float("nan")
        xs[2] = 2.0 ** -24
        xs[3] = 65504.0
        xs[4] = 0.0
    ref, slack = int4_ref(xs, w, sc, z, None, 64)
    out = torch.empty(t, 40, device=DEV)
    S.spmv_int4_run(to_dev(xs), to_dev(w), to_dev(sc), out, 64, zeros=to_dev(z))
    close(out, ref, U * ref.abs() + slack)


@pytest.mark.parametrize("t", [1, 12, 24, 40])
@pytest.mark.parametrize("n_in,group", [(300, 32), (300, 64), (300, 128), (300, 300), (130, 64), (257, 32)])
def test_int4_infinite_scale(t, n_in, group):
    # the last group's scale is infinite: infinity of products of one sign, whatever is behind the last column
    w = torch.randint(9, 16, (40, n_in), dtype=torch.uint8)
    w = torch.cat([w, w.new_zeros(40, 1)], 1)[:, :(n_in + 1) // 2 * 2]
    w = (w[:, ::2] | w[:, 1::2] << 4).contiguous()
    x = torch.rand(t, n_in).add(0.5).half()
    scales = torch.ones(40, -(-n_in // group))
    scales[::2, -1] = math.inf
    y = torch.zeros(t, 40, device=DEV)
    S.spmv_int4_run(to_dev(x), to_dev(w), to_dev(scales), y, group)
    y = y.cpu()
    assert bool((y[:, ::2] == math.inf).all()) and bool(y[:, 1::2].isfinite().all())


@pytest.mark.parametrize("t", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("n_in,n_out,group", [(12288, 33, 32), (12288, 5000, 32), (4096, 12288, 64), (8192, 9000, 128), (5003, 4100, 32), (4097, 6000, 128)])
def test_int4_many_times(t, n_in, n_out, group):
    """The same bits in every one of many calls, one right after the other."""
    xs, w, sc, z, _ = int4_case(7, t, n_in, n_out, group, x="bf16", scales="bf16")
    args = [to_dev(v) for v in (xs, w, sc)]
    z, outs = to_dev(z), torch.empty(60, t, n_out, dtype=torch.bfloat16, device=DEV)
    for k in range(60):
        S.spmv_int4_run(*args, outs[k], group, zeros=z)
    assert bool((outs == outs[0]).all())
    at = torch.randperm(n_out, generator=gen(8))[:40]
    ref, slack = int4_ref(xs, w[at], sc[at], z.cpu()[at], None, group)
    close(outs[0][:, at.to(DEV)], ref, ROUND[torch.bfloat16] * ref.abs() + slack)


@pytest.mark.parametrize("t", [1, 6, 16, 64, 200])
def test_int4_repeats_and_tokens_apart(t):
    """The same bits again, and a token's bits whatever the others hold."""
    xs, w, sc, z, _ = int4_case(2, t, 2000, 300, 128)
    args = [to_dev(v) for v in (w, sc, z)]
    outs = []
    for k in range(3):
        x = to_dev(xs)
        if k == 2:
            x[: t - 1] = 1.0
        out = torch.empty(t, 300, device=DEV)
        S.spmv_int4_run(x, args[0], args[1], out, 128, zeros=args[2])
        outs.append(out.cpu())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0][-1], outs[2][-1])


# ----------------------------------------------------------------- verify

def verify_ref(target, draft, tokens, offsets, au, su, temperature):
    """The rules of the header, request by request, in 64 bits."""
    def cleaned(row):
        row = row.float().clone()
        row[row.isnan()] = -INF
        return row.clamp(max=torch.finfo(torch.float32).max).double()

    def softmax(row, t):
        m = row.max()
        if m == -INF:
            return torch.zeros_like(row)
        e = torch.exp((row - m) / t)
        e[e < 2.0 ** -126] = 0.0
        return e / e.sum()

    v = target.shape[1]
    n = len(offsets) - 1
    out, accepted = {}, []
    for i in range(n):
        lo, hi = offsets[i], offsets[i + 1]
        t = 1.0 if temperature is None else float(temperature[i])
        t = t if t <= 0 or t != t else min(max(t, 1e-30), 1e30)
        taken, got = hi - lo, []
        weights = None
        for j in range(hi - lo + 1):
            row = cleaned(target[lo + i + j])
            x = int(tokens[lo + j]) if j < hi - lo else -1
            inside = 0 <= x < v
            if not t > 0:
                top = int((row == row.max()).nonzero()[0]) if row.max() > -INF else -1
                if j < hi - lo and inside and x == top:
                    got.append(x)
                    continue
                taken = j
                got.append(top)
                break
            p = softmax(row, t)
            if j == hi - lo:
                weights = p
                break
            q = None if draft is None else softmax(cleaned(draft[lo + j]), t)
            if inside and float(au[lo + j]) * (1.0 if q is None else float(q[x])) < float(p[x]):
                got.append(x)
                continue
            taken = j
            weights = p.clone()
            if q is not None:
                weights = (p - q).clamp(min=0)
            elif inside:
                weights[x] = 0
            weights = weights if float(weights.sum()) > 0 else p
            break
        if weights is not None:
            run = weights.cumsum(0)
            at = ((weights > 0) & (run > float(su[i]) * run[-1])).nonzero()
            pos = (weights > 0).nonzero()
            got.append(int(at[0]) if len(at) else int(pos[-1]) if len(pos) else -1)
        accepted.append(taken)
        for k in range(hi - lo + 1):
            out[lo + i + k] = got[k] if k < len(got) else -1
    return out, accepted


def verify_check(target, draft, tokens, offsets, au, su, temperature, t_at=(None, 0), d_at=(None, 0), stream=None, offsets_dev=None):
    out, accepted = verify_ref(target, draft, tokens, offsets, au, su, temperature)
    n, d = len(offsets) - 1, len(tokens)
    got = torch.full((d + n,), -77, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -77, dtype=torch.int32, device=DEV)
    S.spmv_verify_drafts(to_dev(target, *t_at), to_dev(draft, *d_at), to_dev(tokens), torch.tensor(offsets).to(DEV), to_dev(au), to_dev(su),
                         got, acc, temperature=to_dev(temperature), stream=stream)
    got = got.cpu().tolist()
    assert acc.cpu().tolist() == accepted
    assert {k: got[k] for k in out} == out
    assert all(got[k] == -77 for k in range(d + n) if k not in out)
    return out, accepted


def verify_case(seed, counts, v, dtype="f32", std=3.0, error=0.5, temperature=None, point=False, masked=0.0, extra=0):
    g = gen(seed)
    n, d = len(counts), sum(counts) + extra
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    target = torch.randn(d + n, v, generator=g) * std
    rows = [o + i + j for i, (o, c) in enumerate(zip(offsets, counts)) for j in range(c)] + [0] * extra
    draft = target[rows] + torch.randn(d, v, generator=g) * error if d else torch.empty(0, v)
    if masked:
        out = torch.rand(1, v, generator=g) < masked
        out[0, v // 2] = False
        target = torch.where(out, -INF, target)
        draft = torch.where(out, -INF, draft)
    noise = -torch.log(-torch.log(torch.rand(d, v, generator=g).clamp(1e-7, 1 - 1e-7)))
    tokens = (draft + noise).argmax(1).int() if d else torch.empty(0, dtype=torch.int32)
    if temperature == "mixed":
        temperature = torch.rand(n, generator=g) + 0.5
        temperature[::3] = 0.0
    return (target.to(TYPES[dtype]), None if point else draft.to(TYPES[dtype]), tokens, offsets, torch.rand(d, generator=g),
            torch.rand(n, generator=g), temperature)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v", [1, 2, 7, 33, 1000, 4099, 32000])
@pytest.mark.parametrize("point", [False, True])
def test_verify_vocabularies(v, dtype, point):
    verify_check(*verify_case(v, [3, 0, 1, 5, 2, 0, 4], v, dtype=dtype, temperature="mixed", point=point))


@pytest.mark.parametrize("counts", [[0], [1], [40], [0, 0, 0], [17, 16, 15, 33], [1] * 300, [2, 0, 3] * 50])
def test_verify_counts(counts):
    verify_check(*verify_case(len(counts), counts, 513, error=0.1))
    verify_check(*verify_case(len(counts), counts, 513, error=0.1, temperature=torch.zeros(len(counts)), masked=0.5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("counts", [[5, 0, 3, 7, 1, 2, 4, 6] * 24, [200, 0, 1, 0, 70, 16, 15, 17] * 2 + [1] * 900, [0] * 700 + [400] + [0] * 300])
def test_verify_many_rows(counts, point, dtype):
    """Calls in which rows behind a rejected draft are left out: short lists, a
    few long ones among many short ones, nearly all empty."""
    case = list(verify_case(len(counts), counts, 601, dtype=dtype, error=0.2, point=point, temperature="mixed"))
    verify_check(*case)


def test_verify_many_rows_next_to_the_border():
    """As above with random numbers next to p(x) / q(x), and special rows."""
    target, draft, tokens, offsets, au, su, _ = verify_case(28, [3] * 300, 700, error=0.3)
    rows = torch.arange(900) + torch.arange(900) // 3
    p = torch.softmax(target[rows].double(), 1).gather(1, tokens.long()[:, None])[:, 0]
    q = torch.softmax(draft.double(), 1).gather(1, tokens.long()[:, None])[:, 0]
    for step in (-1, 0, 1):
        u = (p / q).float().clamp(max=1 - 2.0 ** -24)
        u = (u.view(torch.int32) + step).view(torch.float32).clamp(min=0, max=1 - 2.0 ** -24)
        verify_check(target, draft, tokens, offsets, u, su, None)
    target[5::40] = -INF
    draft[7::30] = -INF
    target[11::50, ::3] = float("nan")
    tokens[::17] = 700
    verify_check(target, draft, tokens, offsets, au, su, None)


@pytest.mark.parametrize("t_at,d_at", [((1003, 0), (1003, 0)), ((1001, 1), (1008, 3)), ((1200, 5), (1001, 7)), ((0, 2), (0, 4))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_rows_anywhere(t_at, d_at, dtype):
    case = list(verify_case(3, [2, 3, 1], 1001, dtype=dtype, temperature="mixed", masked=0.3))
    if t_at[0] == 0:  # one row used for all
        case[0], case[1] = case[0][:1].expand(9, -1), case[1][:1].expand(6, -1)
    verify_check(*case, t_at=t_at, d_at=d_at)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_verify_flat_rows(dtype):
    """Borders a few 10^-6 apart: fp32's running sums would miss some of these."""
    verify_check(*verify_case(11, [1] * 96, 100003, dtype=dtype, std=0.01, error=0.02))
    verify_check(*verify_case(12, [0] * 200, 50257, dtype=dtype, std=0.3))


def test_verify_next_to_the_border():
    """Random numbers on both sides of p(x) / q(x), as near as fp32 has them."""
    target, draft, tokens, offsets, au, su, _ = verify_case(21, [1] * 400, 700, error=1.0)
    p = torch.softmax(target[::2].double(), 1).gather(1, tokens.long()[:, None])[:, 0]
    q = torch.softmax(draft.double(), 1).gather(1, tokens.long()[:, None])[:, 0]
    for step in (-3, -1, 0, 1, 3):
        u = (p / q).float().clamp(max=1 - 2.0 ** -24)
        u = (u.view(torch.int32) + step).view(torch.float32).clamp(min=0, max=1 - 2.0 ** -24)
        verify_check(target, draft, tokens, offsets, u, su, None)


def test_verify_ends_of_the_random_numbers():
    case = list(verify_case(22, [2] * 40, 333, masked=0.6))
    for u, r in ((0.0, 0.0), (1 - 2.0 ** -24, 1 - 2.0 ** -24), (0.0, 1 - 2.0 ** -24)):
        case[4], case[5] = torch.full((80,), u), torch.full((40,), r)
        verify_check(*case)


def test_verify_equal_rows_are_accepted():
    """Where the drafter is the target, every draft stands, however large the random number."""
    target, _, tokens, offsets, _, su, _ = verify_case(23, [4] * 30, 5000, error=0.0)
    draft = torch.stack([target[5 * (k // 4) + k % 4] for k in range(120)])
    _, accepted = verify_check(target, draft, tokens, offsets, torch.full((120,), 1 - 2.0 ** -24), su, None)
    assert accepted == [4] * 30


@pytest.mark.parametrize("greedy", [False, True])
def test_verify_special_rows(greedy):
    """Rows with nothing above minus infinity, NaN, plus infinity, the type's
    lowest and largest value, equal logits, drafts outside the vocabulary."""
    target, draft, tokens, offsets, au, su, _ = verify_case(24, [2] * 14, 300)
    big = torch.finfo(torch.float32).max
    target[0] = -INF                      # no token at the first place
    target[4] = -INF                      # none at the second
    target[7, ::2] = float("nan")
    target[9] = -big
    target[12, 5], target[12, 77] = INF, INF
    target[15] = float("nan")
    target[18] = 1.0                      # all equal
    target[21] = big
    target[24], draft[16] = -INF, 0.0
    target[24, 17] = 0.5                  # one token left
    draft[18] = -INF                      # the drafter has nothing
    draft[20, 3] = INF
    tokens[22], tokens[24], tokens[26] = -1, 300, 2 ** 31 - 1
    t = torch.zeros(14) if greedy else torch.full((14,), 0.7)
    verify_check(target, draft, tokens, offsets, au, su, t)
    verify_check(target, None, tokens, offsets, au, su, t)


def test_verify_temperatures():
    case = list(verify_case(25, [2] * 12, 200))
    case[6] = torch.tensor([0.0, -1.0, float("nan"), 1e-38, 1e-20, 1e-3, 0.1, 1.0, 10.0, 1e10, INF, 3e38])
    verify_check(*case)


def test_verify_padded_batch():
    """Drafts behind the last request are left alone, and their rows."""
    case = verify_case(26, [2, 0, 3], 500, extra=4)
    verify_check(*case)


@pytest.mark.parametrize("offsets", [[3, 1, 7, -5], [-9, 2, 2, 99], [0, 99, 0, 6], [6, 6, 6, 6]])
def test_verify_offsets_out_of_range_stay_inside(offsets):
    """Offsets that are none: some result, nothing written outside the outputs."""
    target, draft, tokens, _, au, su, _ = verify_case(27, [2, 2, 2], 400)
    got = torch.full((9 + 64,), -77, dtype=torch.int32, device=DEV)
    acc = torch.full((3 + 64,), -77, dtype=torch.int32, device=DEV)
    S.spmv_verify_drafts(to_dev(target), to_dev(draft), to_dev(tokens), torch.tensor(offsets).to(DEV), to_dev(au), to_dev(su), got[:9], acc[:3])
    assert (got[9:] == -77).all() and (acc[3:] == -77).all()


def test_verify_captured_and_replayed():
    """One graph for both launches; new inputs in the same place at each replay."""
    cases = [verify_case(30 + k, [2, 0, 3], 3001, temperature=torch.tensor([1.0, 0.7, 0.0])) for k in range(3)]
    dev = [to_dev(x) if isinstance(x, torch.Tensor) else torch.tensor(x).to(DEV) for x in cases[0]]
    got = torch.empty(8, dtype=torch.int32, device=DEV)
    acc = torch.empty(3, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.spmv_verify_drafts(dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], got, acc, temperature=dev[6])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.spmv_verify_drafts(dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], got, acc, temperature=dev[6])
    for case in cases:
        for k in (0, 1, 2, 4, 5):
            dev[k].copy_(case[k])
        graph.replay()
        out, accepted = verify_ref(*case)
        assert acc.cpu().tolist() == accepted and got.cpu().tolist() == [out[k] for k in range(8)]


# ---------------------------------------------------------------- distill

def distill_case(seed, n, v, k, dtype="f32", top_type="f32", rest=False, temperature=1.0, pad=True, twice=False, std=2.0):
    g = gen(seed)
    z = randn(g, n, v, dtype=dtype, std=std)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] if v >= k else torch.randint(0, v, (k,), generator=g) for _ in range(n)]).int() if n else torch.empty(0, k).int()
    t = randn(g, n, k, dtype=top_type, std=2.0, mean=2.0)
    if pad and k > 1:
        ids[torch.rand(n, k, generator=g) < 0.2] = -1
        ids[:, -1] = v if n % 2 else 2 ** 31 - 1
        if n > 3:
            ids[n // 2] = -1
    if twice and k > 3:
        ids[:, 2] = ids[:, 0]
        ids[:, k // 2] = ids[:, 0]
    sums = None
    if rest:
        valid = (ids >= 0) & (ids < v)
        s = torch.where(valid, torch.exp(t.double() / temperature), 0.0).sum(1)
        sums = (s * (1.0 + 0.4 * torch.rand(n, generator=g)) + 1e-3).log().float()
    return z, ids, t, sums


def distill_ref(z, ids, t, sums, temperature):
    """Loss, stats, gradient for dloss = 1 and their tolerances, from the
    formulas in 64 bits, row by row."""
    n, v = z.shape
    loss, dl = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    stats, ds = torch.zeros(n, 3, dtype=torch.float64), torch.zeros(n, 3, dtype=torch.float64)
    grad, dg = torch.zeros(n, v, dtype=torch.float64), torch.zeros(n, v, dtype=torch.float64)
    for i in range(n):
        row = z[i].double()
        valid = (ids[i] >= 0) & (ids[i] < v)
        at, a = ids[i][valid].long(), t[i][valid].double() / temperature
        if len(at) == 0 or (sums is None and (a == -INF).all()):
            continue
        lp = a - (torch.logsumexp(a, 0) if sums is None else sums[i].double())
        p = lp.exp()
        m = row[~row.isnan()].max()
        d = (row - m) / temperature
        e = d.exp()
        off = torch.where(e > 0, e * ((4 + 3 * d.abs() / math.log(2)) * U + K * U), 0.0)
        listed = torch.zeros(v, dtype=torch.bool)
        listed[at] = True
        total, left = e.sum(), e[~listed].sum()
        d_total, d_left = off.sum() / total, off[~listed].sum() / left if left > 0 else 0.0
        lq = d[at] - total.log()
        d_lp = K * U * (torch.where(p > 0, lp.abs(), 0.0) + 1 + (0 if sums is None else 2 * sums[i].double().abs()))
        d_lq = K * U * (lq.abs() + 1) + d_total
        some = p > 0
        loss[i] = (p * (lp - lq))[some].sum()
        dl[i] = (p * (d_lp * (1 + (lp - lq).abs()) + d_lq + K * U * (lp - lq).abs()))[some].sum()
        factor, d_factor = 1.0, 0.0
        if sums is not None:
            r, d_r = max(0.0, float(1 - p.sum())), float((p * d_lp).sum() + K * U)
            if listed.all():
                r = d_r = 0.0
            if r > 0:
                loss[i] += r * (math.log(r) - (left / total).log())
            if d_r > 0 and left > 0:
                lr = abs(math.log(max(r, d_r))) + float((left / total).log().abs())
                dl[i] += d_r * (lr + 2) + r * (d_total + d_left + K * U * (lr + 1))
                factor = 1 - r * total / left
                d_factor = (d_r + r * (d_total + d_left + 4 * U)) * total / left
        stats[i] = torch.stack([m, total, left if sums is not None else torch.zeros_like(left)])
        ds[i] = torch.stack([torch.zeros_like(m), d_total * total, d_left * left if sums is not None else torch.zeros_like(left)])
        q, d_q = e / total, off / total + e / total * (d_total + 4 * U)
        grad[i] = q * torch.where(listed, 1.0, factor)
        dg[i] = torch.where(listed, d_q, d_q * abs(factor) + q * (d_factor + 4 * U))
        grad[i].index_add_(0, at, -p)
        dg[i].index_add_(0, at, p * d_lp + 8 * U * p)
        dg[i] += 4 * U * grad[i].abs()
    return loss, dl, stats, ds, grad, dg


def distill_check(z, ids, t, sums, temperature=1.0, z_at=(None, 0), o_at=(None, 0), in_place=False, dloss=None):
    n, v = z.shape
    loss_ref, dl, stats_ref, ds, grad_ref, dg = distill_ref(z, ids, t, sums, temperature)
    zd, idd, td, sd = to_dev(z, *z_at), to_dev(ids), to_dev(t), to_dev(sums)
    loss, stats = torch.full((n,), 7.0, device=DEV), torch.full((n, 3), 7.0, device=DEV)
    S.spmv_distill(zd, idd, td, loss, temperature=temperature, log_sums=sd, stats=stats)
    close(loss, loss_ref, dl + 1e-37, "loss")
    close(stats, stats_ref, ds + U * stats_ref.abs() + 1e-37, "stats")
    bare = torch.full((n,), 7.0, device=DEV)
    S.spmv_distill(zd, idd, td, bare, temperature=temperature, log_sums=sd)
    assert torch.equal(bare, loss) or bare.isnan().any()
    g = torch.ones(n) if dloss is None else dloss
    buf, out = out_like(n, v, z.dtype, *o_at)
    if in_place:
        buf, out = None, zd
    S.spmv_distill_backward(to_dev(g) if dloss is None else dloss.to(DEV), zd, idd, td, stats, out, temperature=temperature, log_sums=sd)
    scale = (g.double() / temperature)[:, None]
    ref = grad_ref * scale
    close(out, ref, ROUND[z.dtype] * ref.abs() + dg * scale.abs() * (1 + ROUND[z.dtype]) + TINY[z.dtype], "gradient")
    if buf is not None:
        assert untouched(buf, n, v, o_at[0] or v, o_at[1])
    return loss, stats


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,top_type", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("v", [1, 2, 5, 8, 17, 100, 2047, 4096, 32003])
def test_distill_vocabularies(v, dtype, top_type, rest):
    distill_check(*distill_case(v, 9, v, min(v, 20), dtype, top_type, rest, 1.0), 1.0)
    distill_check(*distill_case(v, 3, v, min(v, 7), dtype, top_type, rest, 2.5), 2.5)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("k", [0, 1, 2, 31, 64, 255, 257, 1000, 1024])
def test_distill_list_lengths(k, rest):
    distill_check(*distill_case(k, 5, 3001, k, "f32", "f32", rest))
    distill_check(*distill_case(k, 5, 3001, k, "bf16", "f32", rest, twice=True))


@pytest.mark.parametrize("n,v", [(1, 70001), (2, 300007), (40, 9001), (151, 5000), (700, 1025)])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_rows(n, v, rest):
    distill_check(*distill_case(n, n, v, 12, "bf16", "f32", rest, 1.5), 1.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z_at,o_at", [((1001, 0), (1001, 0)), ((1008, 1), (1008, 1)), ((1001, 3), (1002, 3)), ((1100, 7), (1003, 0))])
def test_distill_rows_anywhere(z_at, o_at, dtype):
    case = distill_case(5, 6, 1001, 30, dtype, "f32", True)
    distill_check(*case, z_at=z_at, o_at=o_at)
    distill_check(*case, z_at=z_at, in_place=True)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_every_token_listed(rest):
    z, _, _, _ = distill_case(6, 4, 50, 1)
    ids = torch.stack([torch.randperm(50, generator=gen(k)) for k in range(4)]).int()
    t = randn(gen(7), 4, 50)
    sums = torch.logsumexp(t.double(), 1).float() if rest else None
    distill_check(z, ids, t, sums)


def test_distill_few_left():
    """Where nearly all of the probability is listed, what is left of it keeps its digits."""
    z, ids, t, _ = distill_case(8, 6, 5000, 3, pad=False, std=0.5)
    for i in range(6):
        z[i, ids[i].long()] = 18.0 + torch.arange(3.0)
    sums = (torch.exp(t.double()).sum(1) * (1 + 1e-4)).log().float()
    distill_check(z, ids, t, sums)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_special_values(rest):
    """Rows of minus infinity, NaN and infinities as the formula has them, and
    teachers with nothing above minus infinity."""
    z, ids, t, sums = distill_case(9, 10, 200, 6, rest=rest, pad=False)
    big = torch.finfo(torch.float32).max
    z[0, 50:] = -INF                      # a masked vocabulary, listed tokens among it
    z[1, :150] = -big
    z[2, int(ids[2, 0])] = -INF
    z[3] = z[3].clamp(max=0) - 1e30
    t[4, 1:] = -INF
    t[5] = -INF
    z[6, 3], z[7, 3] = float("nan"), INF
    if rest:
        sums[5] = 0.0
    n = 8
    distill_check(z[:n], ids[:n], t[:n], None if sums is None else sums[:n])


def test_distill_gradient_of_one_loss_for_all():
    case = distill_case(10, 33, 777, 10, "f32", "f32", True)
    distill_check(*case, dloss=torch.full((1,), 0.25).expand(33))
    distill_check(*case, dloss=torch.randn(66, generator=gen(1))[::2])


def test_distill_gradient_against_differences():
    """Central differences of the loss in 64 bits, at some logits of each row:
    their own error is of the order of step^2."""
    z, ids, t, sums = distill_case(12, 4, 60, 6, rest=True, temperature=1.5, twice=True)
    _, stats = distill_check(z, ids, t, sums, 1.5)
    out = torch.empty_like(z, device=DEV)
    S.spmv_distill_backward(torch.ones(4, device=DEV), to_dev(z), to_dev(ids), to_dev(t), stats, out, temperature=1.5, log_sums=to_dev(sums))
    step = 2.0 ** -10
    for v in list(range(0, 60, 7)) + [int(x) for x in ids[0, :3]]:
        if v < 0 or v >= 60:
            continue
        up, down = z.double(), z.double()
        up[:, v] += step
        down[:, v] -= step
        slope = (distill_ref(up, ids, t, sums, 1.5)[0] - distill_ref(down, ids, t, sums, 1.5)[0]) / (2 * step)
        assert (out[:, v].cpu().double() - slope).abs().max() <= 1e-5


def test_distill_repeats():
    case = [to_dev(x) for x in distill_case(13, 20, 20011, 50, "bf16", "f32", True, twice=True)]
    got = []
    for _ in range(2):
        loss, stats, grad = torch.empty(20, device=DEV), torch.empty(20, 3, device=DEV), torch.empty_like(case[0])
        S.spmv_distill(case[0], case[1], case[2], loss, log_sums=case[3], stats=stats)
        S.spmv_distill_backward(loss, case[0], case[1], case[2], stats, grad, log_sums=case[3])
        got.append((loss.cpu(), stats.cpu(), grad.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_distill_no_rows():
    z = torch.empty(0, 10, device=DEV)
    ids, t = torch.empty(0, 3, dtype=torch.int32, device=DEV), torch.empty(0, 3, device=DEV)
    S.spmv_distill(z, ids, t, torch.empty(0, device=DEV))
    S.spmv_distill_backward(torch.empty(0, device=DEV), z, ids, t, torch.empty(0, 3, device=DEV), z)


# --------------------------------------------------- streams, graphs, far rows

def test_int4_captured_and_replayed():
    """Calls of every kernel in one graph, replayed on new inputs in the same place."""
    cases = [int4_case(40 + k, t, 1000, 260, g, x="bf16", scales="bf16", base="f32") + (g,)
             for k, (t, g) in enumerate([(1, 128), (12, 64), (30, 32), (64, 128), (70, 256)])]
    dev = [[v.to(DEV) for v in c[:5]] for c in cases]
    outs = [torch.empty(c[0].shape[0], 260, device=DEV) for c in cases]

    def run():
        for d, o, c in zip(dev, outs, cases):
            S.spmv_int4_run(d[0], d[1], d[2], o, c[5], zeros=d[3], base=d[4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (0, 100):
        for k, (d, c) in enumerate(zip(dev, cases)):
            x = randn(gen(seed + k), *c[0].shape, dtype="bf16")
            d[0].copy_(x)
            outs[k].fill_(float("nan"))
        graph.replay()
        for k, (o, c) in enumerate(zip(outs, cases)):
            x = randn(gen(seed + k), *c[0].shape, dtype="bf16")
            ref, slack = int4_ref(x, *c[1:])
            close(o, ref, U * ref.abs() + slack)


def test_int4_on_many_streams():
    """Calls of different kernels at work at the same time, each right."""
    cases = [int4_case(50 + k, t, 3000, 2000, 128, zeros=False) for k, t in enumerate([1, 16, 32, 64] * 3)]
    dev = [[None if v is None else v.to(DEV) for v in c] for c in cases]
    outs = [torch.empty(c[0].shape[0], 2000, device=DEV) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, o, st in zip(dev, outs, streams):
            S.spmv_int4_run(d[0], d[1], d[2], o, 128, stream=st)
    torch.cuda.synchronize()
    for o, c in zip(outs, cases):
        ref, slack = int4_ref(*c, 128)
        close(o, ref, U * ref.abs() + slack)


def test_verify_and_distill_on_a_given_stream():
    """A stream that is not the current one, while the current one is busy."""
    case = verify_case(61, [3, 1, 0, 4], 20000, temperature="mixed")
    st = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    verify_check(*case, stream=st)
    z, ids, t, sums = distill_case(62, 6, 5000, 9, rest=True)
    dev = [v.to(DEV) for v in (z, ids, t, sums)]
    loss, stats, out = torch.empty(6, device=DEV), torch.empty(6, 3, device=DEV), torch.empty_like(dev[0])
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    S.spmv_distill(dev[0], dev[1], dev[2], loss, log_sums=dev[3], stats=stats, stream=st)
    S.spmv_distill_backward(torch.ones(6, device=DEV), dev[0], dev[1], dev[2], stats, out, log_sums=dev[3], stream=st)
    st.synchronize()
    loss_ref, dl, _, _, grad, dg = distill_ref(z, ids, t, sums, 1.0)
    close(loss, loss_ref, dl + 1e-37)


def test_distill_captured_and_replayed():
    """Both directions in one graph; new logits in the same place at each replay."""
    z, ids, t, sums = distill_case(63, 5, 3001, 20, rest=True)
    dev = [v.to(DEV) for v in (z, ids, t, sums)]
    loss, stats, out = torch.empty(5, device=DEV), torch.empty(5, 3, device=DEV), torch.empty_like(dev[0])
    ones = torch.ones(1, device=DEV).expand(5)

    def run():
        S.spmv_distill(dev[0], dev[1], dev[2], loss, log_sums=dev[3], stats=stats)
        S.spmv_distill_backward(ones, dev[0], dev[1], dev[2], stats, out, log_sums=dev[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (64, 65):
        new = randn(gen(seed), 5, 3001, std=2.0)
        dev[0].copy_(new)
        graph.replay()
        loss_ref, dl, _, _, grad, dg = distill_ref(new, ids, t, sums, 1.0)
        close(loss, loss_ref, dl + 1e-37)
        close(out, grad, U * grad.abs() + dg + 1e-37)


def far_rows(t, fill):
    """The rows of t on the GPU, 2^31 + 16 elements apart."""
    stride = 2 ** 31 + 16
    buf = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=DEV)
    view = buf.as_strided(t.shape, (stride, 1))
    view.copy_(t) if fill else None
    return view


def test_rows_far_apart():
    """Offsets past 32 bits in every matrix."""
    z, ids, t, sums = distill_case(66, 3, 2000, 9, "bf16", rest=True)
    zd = far_rows(z, True)
    loss, stats = torch.empty(3, device=DEV), torch.empty(3, 3, device=DEV)
    dev = [v.to(DEV) for v in (ids, t, sums)]
    S.spmv_distill(zd, dev[0], dev[1], loss, log_sums=dev[2], stats=stats)
    S.spmv_distill_backward(torch.ones(3, device=DEV), zd, dev[0], dev[1], stats, zd, log_sums=dev[2])
    loss_ref, dl, _, _, grad, dg = distill_ref(z, ids, t, sums, 1.0)
    close(loss, loss_ref, dl + 1e-37)
    close(zd, grad, 2.0 ** -8 * grad.abs() + 1.01 * dg + TINY[torch.bfloat16])
    del zd
    case = verify_case(67, [1], 3000, dtype="bf16")
    got, acc = torch.empty(2, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    S.spmv_verify_drafts(far_rows(case[0], True), case[1].to(DEV), case[2].to(DEV), torch.tensor(case[3]).to(DEV), case[4].to(DEV), case[5].to(DEV),
                         got, acc)
    out, accepted = verify_ref(*case)
    assert acc.tolist() == accepted and got.tolist() == [out[0], out[1]]
    for n in (3, 20, 40):
        x, w, sc, zp, base = int4_case(68, n, 200, 3, 64, base="f32")
        y = torch.empty(n, 3, device=DEV)
        S.spmv_int4_run(to_dev(x), far_rows(w, True), sc.to(DEV), y, 64, zeros=zp.to(DEV), base=base.to(DEV))
        ref, slack = int4_ref(x, w, sc, zp, base, 64)
        close(y, ref, U * ref.abs() + slack)
    x, w, sc, zp, _ = int4_case(69, 2, 200, 130, 64)
    y = far_rows(torch.empty(2, 130), False)
    S.spmv_int4_run(far_rows(x, True), w.to(DEV), sc.to(DEV), y, 64, zeros=zp.to(DEV))
    ref, slack = int4_ref(x, w, sc, zp, None, 64)
    close(y, ref, U * ref.abs() + slack)


def test_int4_one_row_and_one_matrix_for_all():
    """Expanded inputs: one token for all, one row of base for all, one row of weights for all."""
    for t in (5, 40):
        x, w, sc, zp, base = int4_case(70, t, 700, 150, 128, base="f32")
        y = torch.empty(t, 150, device=DEV)
        S.spmv_int4_run(x[:1].to(DEV).expand(t, -1), w[:1].to(DEV).expand(150, -1), sc.to(DEV), y, 128, zeros=zp.to(DEV), base=base[:1].to(DEV).expand(t, -1))
        ref, slack = int4_ref(x[:1].expand(t, -1), w[:1].expand(150, -1), sc, zp, base[:1].expand(t, -1), 128)
        close(y, ref, U * ref.abs() + slack)


def test_the_readmes_calls_run():
    """The calls of these operators as README.md prints them."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code, = [c for c in re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S) if "spmv_distill" in c]
    w, sc, zp = int4_case(80, 3, 256, 40, 128)[1:4]
    x = randn(gen(81), 3, 256, dtype="f16")
    logits, teacher = randn(gen(82), 5, 90), randn(gen(83), 5, 8)
    names = dict(S=S, x=x.to(DEV), weights=w.to(DEV), scales=sc.to(DEV), zeros=zp.to(DEV), y=torch.empty(3, 40, device=DEV),
                 target_logits=randn(gen(84), 5, 90).to(DEV), draft_logits=randn(gen(85), 3, 90).to(DEV),
                 draft_tokens=torch.tensor([3, 5, 7], dtype=torch.int32, device=DEV), offsets=torch.tensor([0, 2, 3], device=DEV),
                 accept_uniforms=torch.rand(3, generator=gen(86)).to(DEV), sample_uniforms=torch.rand(2, generator=gen(87)).to(DEV),
                 tokens=torch.empty(5, dtype=torch.int32, device=DEV), accepted=torch.empty(2, dtype=torch.int32, device=DEV),
                 temperature=torch.tensor([1.0, 0.7], device=DEV), logits=logits.to(DEV), top_logits=teacher.to(DEV),
                 top_tokens=torch.arange(0, 80, 10, dtype=torch.int32).expand(5, -1).contiguous().to(DEV),
                 loss=torch.empty(5, device=DEV), stats=torch.empty(5, 3, device=DEV), dloss=torch.ones(5, device=DEV))
    exec(code, names)
    ref, slack = int4_ref(x, w, sc, zp, None, 128)
    close(names["y"], ref, U * ref.abs() + slack)
    assert bool((names["accepted"] >= 0).all()) and bool((names["loss"] > 0).all())
    # q - p of a row sums to nothing (dloss / temperature = 1/2, 90 terms of at most 1 rounded a few times)
    assert bool((names["logits"].double().sum(1).abs() <= 90 * 16 * U).all())
