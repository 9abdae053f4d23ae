"""Measured cases of the operators around a pruned layer: the layer norm that
feeds its product, in both directions; the low-rank adapters of many requests
beside the product; and the penalties, biases and grammar masks on the logits
that an output head's product gives.

``run`` computes a case with elementary torch operations in 32 bits
(``own = False``) or through the library's entry points (``own = True``);
``exact`` gives the same values in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # The residual stream of one decoded token (fp32, as the products leave
        # it) normalised into the fp16 vector that a 12288 x 12288 pruned
        # layer's product reads: latency is all that counts.
        {"name": "norm, one token", "op": "norm", "rows": 1, "cols": 12288, "x": "f32", "y": "f16", "params": "f16", "stats": False},
        # The same over the tokens of a batch of prompts.
        {"name": "norm, prompts", "op": "norm", "rows": 4096, "cols": 12288, "x": "f32", "y": "f16", "params": "f16", "stats": False},
        # A forward pass that keeps the statistics for its backward pass, with
        # an odd width (rows start at any alignment).
        {"name": "norm, odd width", "op": "norm", "rows": 1023, "cols": 5003, "x": "bf16", "y": "bf16", "params": "f32", "stats": True},
        # Recovery training of a pruned model's norms: a small ragged batch ...
        {"name": "norm gradient, small", "op": "norm_grad", "rows": 513, "cols": 4099, "x": "f32", "y": "f16", "params": "f32"},
        # ... and a full one at the width of the pruned layers.
        {"name": "norm gradient, full", "op": "norm_grad", "rows": 8192, "cols": 12288, "x": "bf16", "y": "bf16", "params": "f32"},
        # One request's token through its adapter.
        {"name": "adapters, one token", "op": "adapters", "tokens": 1, "n_in": 12288, "n_out": 12288, "rank": 16, "slots": 8,
         "x": "f16", "y": "f32", "prompts": False, "ragged": False},
        # A decode batch: a token of each of 48 requests, 32 adapters of mixed
        # ranks, some requests without one.
        {"name": "adapters, decode batch", "op": "adapters", "tokens": 48, "n_in": 12288, "n_out": 12288, "rank": 64, "slots": 32,
         "x": "f16", "y": "f32", "prompts": False, "ragged": True},
        # Prompts of a few requests, each with its adapter.
        {"name": "adapters, prompts", "op": "adapters", "tokens": 4096, "n_in": 12288, "n_out": 12288, "rank": 32, "slots": 8,
         "x": "f16", "y": "f32", "prompts": True, "ragged": False},
        # Short prompts, an odd width on both sides and an odd rank.
        {"name": "adapters, odd sizes", "op": "adapters", "tokens": 333, "n_in": 5003, "n_out": 4099, "rank": 20, "slots": 12,
         "x": "bf16", "y": "bf16", "prompts": True, "ragged": True},
        # One request's logits.
        {"name": "logits, one request", "op": "logits", "requests": 1, "vocab": 32000, "history": 1000, "biases": 50, "x": "f32", "y": "f32"},
        # A serving batch over a large vocabulary, with long histories.
        {"name": "logits, batch", "op": "logits", "requests": 256, "vocab": 128000, "history": 8192, "biases": 300, "x": "f32", "y": "f32"},
        # An odd vocabulary in 16 bits.
        {"name": "logits, odd vocabulary", "op": "logits", "requests": 37, "vocab": 50257, "history": 2000, "biases": 100, "x": "bf16", "y": "f32"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 128, the others of any parity."""
    n = _spread(rng, lo, hi)
    n = max(128, n // 128 * 128) if rng.random() < 0.5 else n
    return n + 128 if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "adapters", "logits"])
    if op in ("norm", "norm_grad"):
        x, y = rng.choice([("f32", "f16"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")])
        cols = _width(rng, 64, 12288)
        rows = _spread(rng, 1 if op == "norm" else 16, 8192)
        case = {"op": op, "rows": rows, "cols": cols, "x": x, "y": y, "params": rng.choice(["f32", x])}
        if op == "norm":
            case["stats"] = rng.random() < 0.5
        elif x == "f32":
            case["rows"] = min(case["rows"], 4096)
        return case
    if op == "adapters":
        prompts = rng.random() < 0.5
        x = rng.choice(["f16", "bf16"])
        return {"op": op, "tokens": _spread(rng, 32, 4096) if prompts else _spread(rng, 1, 256), "n_in": _width(rng, 256, 12288),
                "n_out": _width(rng, 256, 12288), "rank": rng.choice([4, 8, 16, 20, 32, 64, 128]), "slots": _spread(rng, 1, 8 if prompts else 64),
                "x": x, "y": rng.choice(["f32", x]), "prompts": prompts, "ragged": rng.random() < 0.5}
    x = rng.choice(["f32", "f16", "bf16"])
    return {"op": op, "requests": _spread(rng, 1, 256), "vocab": _width(rng, 1000, 128000), "history": _spread(rng, 1, 8192),
            "biases": _spread(rng, 1, 300), "x": x, "y": rng.choice(["f32", x])}


# ------------------------------------------------------------------ inputs

def _ragged(gen, rows, longest):
    """Lengths between 0 and `longest` (the first row has the longest), and
    their running offsets."""
    n = (torch.rand(rows, generator=gen) * (longest + 1)).long().clamp_(max=longest)
    n[0] = longest
    if rows > 2:
        n[rows // 2] = 0
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _frequent(gen, n, vocab):
    """Token ids as text has them: a few very frequent, most of them rare."""
    u = torch.rand(n, generator=gen, device=gen.device)
    rank = (torch.exp(u * math.log(vocab)) - 1).long().clamp_(max=vocab - 1)
    return ((rank * 7919 + 13) % vocab).int()


def prepare(case, seed):
    dev = torch.Generator(device=DEVICE).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    s = {"op": case["op"]}

    def normal(*size, dtype="f32", std=1.0, mean=0.0):
        return (torch.randn(*size, generator=dev, device=DEVICE) * std + mean).to(TYPES[dtype])

    if case["op"] in ("norm", "norm_grad"):
        n, d = case["rows"], case["cols"]
        # a residual stream: a mean of its own in every row, a few large columns
        x = torch.randn(n, d, generator=dev, device=DEVICE) * 1.5 + torch.randn(n, 1, generator=dev, device=DEVICE) * 0.5
        x[:, :: max(1, d // 7)] *= 8.0
        s["x"], s["eps"] = x.to(TYPES[case["x"]]), 1e-5
        s["weight"], s["bias"] = normal(d, dtype=case["params"], std=0.2, mean=1.0), normal(d, dtype=case["params"], std=0.1)
        s["y_type"] = TYPES[case["y"]]
        if case["op"] == "norm":
            s["stats"] = case["stats"]
            s["y"] = torch.empty(n, d, dtype=s["y_type"], device=DEVICE)
            s["mean"], s["rstd"] = (torch.empty(n, device=DEVICE) for _ in range(2)) if s["stats"] else (None, None)
        else:
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = (((xf - s["mean"][:, None]) ** 2).mean(1) + s["eps"]).rsqrt()
            s["dy"] = normal(n, d, dtype=case["y"], std=0.05)
            s["dx"], s["dweight"], s["dbias"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        return s
    if case["op"] == "adapters":
        t, n_in, n_out, r, n = (case[k] for k in ("tokens", "n_in", "n_out", "rank", "slots"))
        s["x"] = normal(t, n_in, dtype=case["x"])
        s["a"] = normal(n, r, n_in, dtype=case["x"], std=n_in ** -0.5)
        s["b"] = normal(n, n_out, r, dtype=case["x"], std=0.1)
        s["base"] = normal(t, n_out, dtype=case["y"], std=0.7)
        s["y"] = torch.empty_like(s["base"])
        if case["prompts"]:  # runs of tokens with one adapter, a run for each request
            requests = min(t, 2 * n)
            starts = torch.randperm(t, generator=cpu)[: requests - 1].sort().values
            run_of = torch.zeros(t, dtype=torch.int64)
            run_of[starts] = 1
            ids = torch.randint(0, n, (requests,), generator=cpu)[run_of.cumsum(0).clamp_(max=requests - 1)]
        else:  # a token of each request, one in eight without an adapter
            ids = torch.randint(0, n, (t,), generator=cpu)
            if t > 1:
                ids[torch.rand(t, generator=cpu) < 0.125] = -1
        s["ids"] = ids.int().to(DEVICE)
        ranks = torch.full((n,), r)
        if case["ragged"]:
            ranks = torch.tensor([max(1, r >> int(k)) for k in torch.randint(0, 3, (n,), generator=cpu)])
        s["ranks"] = ranks.int().to(DEVICE)
        s["scales"] = torch.rand(n, generator=dev, device=DEVICE) * 1.5 + 0.5
        return s
    t, v = case["requests"], case["vocab"]
    s["logits"] = normal(t, v, dtype=case["x"], std=3.0)
    s["y"] = torch.empty(t, v, dtype=TYPES[case["y"]], device=DEVICE)
    for kind, longest in (("prompt", case["history"]), ("output", max(1, case["history"] // 4))):
        offsets = _ragged(cpu, t, longest)
        s[kind + "_offsets"] = offsets.to(DEVICE)
        s[kind + "_tokens"] = _frequent(dev, int(offsets[-1]), v)
    plain = (torch.rand(t, generator=dev, device=DEVICE) < 0.25)  # requests without penalties
    for kind, lo, hi, off in (("repetition", 1.0, 1.3, 1.0), ("frequency", 0.0, 0.8, 0.0), ("presence", -0.2, 0.8, 0.0)):
        p = torch.rand(t, generator=dev, device=DEVICE) * (hi - lo) + lo
        s[kind] = torch.where(plain, torch.full_like(p, off), p)
    offsets = _ragged(cpu, t, min(case["biases"], v))
    s["bias_offsets"] = offsets.to(DEVICE)
    s["bias_tokens"] = torch.randint(0, v, (int(offsets[-1]),), generator=dev, device=DEVICE).int()
    s["bias_values"] = torch.randn(int(offsets[-1]), generator=dev, device=DEVICE) * 4.0
    # one request in three answers in a grammar; a grammar's state allows few tokens
    masks = max(1, t // 3)
    rows = torch.full((t,), -1)
    rows[torch.randperm(t, generator=cpu)[:masks]] = torch.arange(masks)
    s["mask_rows"] = rows.int().to(DEVICE)
    words = (v + 31) // 32
    bits = [torch.randint(-2 ** 31, 2 ** 31, (masks, words), generator=dev, device=DEVICE, dtype=torch.int64) for _ in range(4)]
    s["mask"] = (bits[0] & bits[1] & bits[2] & bits[3]).int()
    return s


# ------------------------------------------------------------ the operators

def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = ((c * c).mean(1) + s["eps"]).rsqrt()
    y = (c * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(s["y_type"])
    return {"y": y, "mean": mean, "rstd": rstd} if s["stats"] else {"y": y}


def _norm_grad_plain(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(s["weight"].dtype), "dbias": dy.sum(0).to(s["bias"].dtype)}


def _adapters_plain(s):
    n, r, n_in = s["a"].shape
    n_out = s["b"].shape[1]
    # every adapter's products for every token, those of other slots (and of
    # ranks that a slot does not have) set to zero
    h = (s["x"].float() @ s["a"].float().view(n * r, n_in).T).view(-1, n, r)
    slots = torch.arange(n, device=h.device)
    kept = (s["ids"][:, None] == slots)[:, :, None] & (torch.arange(r, device=h.device) < s["ranks"][:, None])
    h = torch.where(kept, h * s["scales"][:, None], 0.0)
    delta = h.view(-1, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, n_out)
    return (s["base"].float() + delta).to(s["base"].dtype)


def _counts(tokens, offsets, shape):
    row = torch.repeat_interleave(torch.arange(shape[0], device=tokens.device), offsets.diff(), output_size=tokens.numel())
    n = torch.zeros(shape[0] * shape[1], dtype=torch.int32, device=tokens.device)
    n.index_add_(0, row * shape[1] + tokens, torch.ones_like(tokens))
    return n.view(shape)


def _logits_plain(s):
    x = s["logits"].float()
    shape = x.shape
    out = _counts(s["output_tokens"], s["output_offsets"], shape)
    seen = (_counts(s["prompt_tokens"], s["prompt_offsets"], shape) > 0) | (out > 0)
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * out - s["presence"][:, None] * (out > 0)
    row = torch.repeat_interleave(torch.arange(shape[0], device=x.device), s["bias_offsets"].diff(), output_size=s["bias_values"].numel())
    bias = torch.zeros(shape[0] * shape[1], device=x.device).index_add_(0, row * shape[1] + s["bias_tokens"], s["bias_values"])
    x = x + bias.view(shape)
    token = torch.arange(shape[1], device=x.device)
    allowed = (s["mask"][s["mask_rows"].clamp(min=0).long()][:, token // 32] >> (token % 32)) & 1
    x = torch.where((allowed == 1) | (s["mask_rows"] < 0)[:, None], x, -math.inf)
    return x.to(s["y"].dtype)


def run(state):
    s = state
    if not own:
        return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "adapters": _adapters_plain, "logits": _logits_plain}[s["op"]](s)
    import sparse_matrix_vector_gb300 as S
    if s["op"] == "norm":
        S.spmv_layernorm(s["x"], s["weight"], s["bias"], s["y"], eps=s["eps"], mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]} if s["stats"] else {"y": s["y"]}
    if s["op"] == "norm_grad":
        S.spmv_layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if s["op"] == "adapters":
        S.spmv_adapters_run(s["x"], s["a"], s["b"], s["ids"], s["y"], base=s["base"], ranks=s["ranks"], scales=s["scales"])
        return s["y"]
    S.spmv_logits_process(s["logits"], s["y"], prompt=(s["prompt_tokens"], s["prompt_offsets"]), output=(s["output_tokens"], s["output_offsets"]),
                          repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                          bias=(s["bias_tokens"], s["bias_values"], s["bias_offsets"]), mask=s["mask"], mask_rows=s["mask_rows"])
    return s["y"]


# ------------------------------------------------------------- what it takes

def work(case):
    """The bytes of the inputs, read once, and of the outputs, written once,
    and the operations of the formulas."""
    if case["op"] == "norm":
        n, d = case["rows"], case["cols"]
        return {"bytes": n * d * (BYTES[case["x"]] + BYTES[case["y"]]) + 2 * d * BYTES[case["params"]] + (8 * n if case["stats"] else 0), "flops": 8 * n * d}
    if case["op"] == "norm_grad":
        n, d = case["rows"], case["cols"]
        return {"bytes": n * d * (2 * BYTES[case["x"]] + BYTES[case["y"]]) + 3 * d * BYTES[case["params"]] + 8 * n, "flops": 16 * n * d}
    if case["op"] == "adapters":
        t, n_in, n_out, r = (case[k] for k in ("tokens", "n_in", "n_out", "rank"))
        # of t tokens over n slots, so many slots are expected to be met
        met = case["slots"] * (1 - (1 - 1 / case["slots"]) ** (min(t, 2 * case["slots"]) if case["prompts"] else t))
        mean_rank = r * (7 / 12 if case["ragged"] else 1)
        tokens_met = t * (1 if case["prompts"] or t == 1 else 7 / 8)
        return {"bytes": int(tokens_met * n_in * BYTES[case["x"]] + 2 * t * n_out * BYTES[case["y"]] + met * mean_rank * (n_in + n_out) * BYTES[case["x"]]),
                "flops": int(2 * tokens_met * mean_rank * (n_in + n_out))}
    t, v = case["requests"], case["vocab"]
    mean = 1.0 if t == 1 else 0.5
    lists = mean * t * (4 * case["history"] + 4 * max(1, case["history"] // 4) + 8 * min(case["biases"], v))
    return {"bytes": int(t * v * (BYTES[case["x"]] + BYTES[case["y"]]) + lists + max(1, t // 3) * v / 8), "flops": 6 * t * v}


# ------------------------------------------------------- the same in 64 bits

def _exact_norm(s):
    x = s["x"].double()
    var, mean = torch.var_mean(x, dim=1, correction=0)
    rstd = 1.0 / torch.sqrt(var + s["eps"])
    y = torch.addcmul(s["bias"].double(), (x - mean[:, None]).mul_(rstd[:, None]), s["weight"].double())
    return {"y": y, "mean": mean, "rstd": rstd} if s["stats"] else {"y": y}


def _exact_norm_grad(s):
    n, d = s["x"].shape
    dx = torch.empty(n, d, dtype=torch.float64, device=s["x"].device)
    dw, db = (torch.zeros(d, dtype=torch.float64, device=s["x"].device) for _ in range(2))
    for lo in range(0, n, 1024):  # in blocks of rows, for memory's sake
        k = slice(lo, lo + 1024)
        r = s["rstd"][k].double().unsqueeze(1)
        xhat = (s["x"][k].double() - s["mean"][k].double().unsqueeze(1)) * r
        dy = s["dy"][k].double()
        dw += torch.einsum("nd,nd->d", dy, xhat)
        db += dy.sum(0)
        g = dy * s["weight"].double()
        along = torch.einsum("nd,nd->n", g, xhat).unsqueeze(1)
        dx[k] = r / d * (d * g - g.sum(1, keepdim=True) - xhat * along)
    return {"dx": dx, "dweight": dw, "dbias": db}


def _exact_adapters(s):
    y = s["base"].double()
    ids, ranks = s["ids"].tolist(), s["ranks"].tolist()
    for slot in sorted(set(ids) - {-1}):
        at = torch.tensor([i for i, k in enumerate(ids) if k == slot], device=y.device)
        a, b = s["a"][slot, : ranks[slot]].double(), s["b"][slot, :, : ranks[slot]].double()
        y[at] += (s["x"][at].double() @ a.T @ b.T) * s["scales"][slot].double()
    return y


def _exact_logits(s):
    x = s["logits"].double()
    v = x.shape[1]
    at = {k: s[k + "_offsets"].tolist() for k in ("prompt", "output", "bias")}
    bit = torch.arange(32, device=x.device)
    for i, row in enumerate(s["mask_rows"].tolist()):
        prompt, output, biased = (slice(at[k][i], at[k][i + 1]) for k in ("prompt", "output", "bias"))
        met = torch.unique(torch.cat([s["prompt_tokens"][prompt], s["output_tokens"][output]]).long())
        l, rep = x[i, met], s["repetition"][i].double()
        x[i, met] = torch.where(l > 0, l / rep, l * rep)
        told, n = torch.unique(s["output_tokens"][output].long(), return_counts=True)
        x[i, told] -= s["frequency"][i].double() * n + s["presence"][i].double()
        x[i].index_put_((s["bias_tokens"][biased].long(),), s["bias_values"][biased].double(), accumulate=True)
        if row >= 0:
            x[i, ((s["mask"][row].unsqueeze(1) >> bit) & 1).reshape(-1)[:v] == 0] = -math.inf
    return x


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "adapters": _exact_adapters, "logits": _exact_logits}[s["op"]](s)
