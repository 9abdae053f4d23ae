"""Measured cases of the operators that put a pruned model beside the dense
one that it came from: products with 4-bit weights and group scales (the other
way to make a layer small, for the layers that pruning would hurt); the
verification of tokens that the pruned model drafted against the dense model's
probabilities; and the distillation from the dense model's top logits that
recovers a pruned model, in both directions.

``run`` computes a case with elementary torch operations (``own = False``) or
through the library's entry points (``own = True``); ``exact`` gives the same
values in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
NONE = -math.inf


def listed():
    return [
        # One token through a layer of the width of the pruned ones, kept dense in 4 bits.
        {"name": "int4, one token", "op": "int4", "tokens": 1, "n_in": 12288, "n_out": 12288, "group": 128, "x": "f16", "y": "f32", "scales": "f16", "zeros": False, "base": False},
        # The drafted tokens of one request, verified together; zero points.
        {"name": "int4, drafted tokens", "op": "int4", "tokens": 6, "n_in": 4096, "n_out": 12288, "group": 64, "x": "bf16", "y": "bf16", "scales": "bf16", "zeros": True, "base": False},
        # A decode batch, added to the residual stream.
        {"name": "int4, decode batch", "op": "int4", "tokens": 64, "n_in": 12288, "n_out": 12288, "group": 128, "x": "f16", "y": "f32", "scales": "f16", "zeros": True, "base": True},
        # An odd width on both sides: rows of packed weights start at any byte.
        {"name": "int4, odd sizes", "op": "int4", "tokens": 11, "n_in": 5003, "n_out": 4099, "group": 32, "x": "bf16", "y": "f32", "scales": "f32", "zeros": False, "base": False},
        # One request's five drafted tokens: latency.
        {"name": "verify, one request", "op": "verify", "requests": 1, "drafts": 5, "vocab": 32000, "x": "f32", "point": False, "greedy": False, "masked": False},
        # A serving batch over a large vocabulary: ragged drafts, some requests greedy, some in a grammar.
        {"name": "verify, batch", "op": "verify", "requests": 64, "drafts": 7, "vocab": 128000, "x": "f32", "point": False, "greedy": True, "masked": True},
        # An odd vocabulary in 16 bits, with drafts that carry no probabilities (looked up in the text so far).
        {"name": "verify, odd vocabulary", "op": "verify", "requests": 37, "drafts": 4, "vocab": 50257, "x": "bf16", "point": True, "greedy": True, "masked": False},
        # The loss of a few tokens.
        {"name": "distill, few tokens", "op": "distill", "rows": 7, "vocab": 32000, "top": 50, "x": "f32", "top_type": "f32", "rest": False, "temperature": 2.0},
        # The loss of a batch of sequences.
        {"name": "distill, batch", "op": "distill", "rows": 4096, "vocab": 128000, "top": 64, "x": "bf16", "top_type": "f32", "rest": True, "temperature": 1.0},
        # An odd vocabulary, the teacher's logits in 16 bits.
        {"name": "distill, odd vocabulary", "op": "distill", "rows": 1001, "vocab": 50257, "top": 20, "x": "f16", "top_type": "f16", "rest": False, "temperature": 1.5},
        # The gradient of a small ragged batch ...
        {"name": "distill gradient, odd", "op": "distill_grad", "rows": 333, "vocab": 50257, "top": 20, "x": "f32", "top_type": "f32", "rest": False, "temperature": 1.5},
        # ... and of a full one.
        {"name": "distill gradient, batch", "op": "distill_grad", "rows": 2048, "vocab": 128000, "top": 64, "x": "bf16", "top_type": "f32", "rest": True, "temperature": 1.0},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 128, the others of any parity."""
    n = _spread(rng, lo, hi)
    return max(128, n // 128 * 128) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["int4", "verify", "distill", "distill_grad"])
    if op == "int4":
        x = rng.choice(["f16", "bf16"])
        return {"op": op, "tokens": _spread(rng, 1, 64), "n_in": _width(rng, 256, 12288), "n_out": _width(rng, 256, 12288), "group": rng.choice([32, 64, 128, 256]),
                "x": x, "y": rng.choice(["f32", x]), "scales": rng.choice(["f32", x]), "zeros": rng.random() < 0.5, "base": rng.random() < 0.5}
    if op == "verify":
        return {"op": op, "requests": _spread(rng, 1, 64), "drafts": _spread(rng, 1, 7), "vocab": _width(rng, 1000, 128000), "x": rng.choice(["f32", "f16", "bf16"]),
                "point": rng.random() < 0.3, "greedy": rng.random() < 0.5, "masked": rng.random() < 0.5}
    x = rng.choice(["f32", "f16", "bf16"])
    vocab = _width(rng, 1000, 128000)
    rows = _spread(rng, 1 if op == "distill" else 8, 4096 if op == "distill" else 2048)
    most = 10 ** 9 // (vocab * BYTES[x] * (1 if op == "distill" else 2))
    return {"op": op, "rows": min(rows, most), "vocab": vocab, "top": _spread(rng, 1, 128), "x": x, "top_type": rng.choice(["f32", x]),
            "rest": rng.random() < 0.5, "temperature": rng.choice([1.0, 1.0, 1.5, 2.0])}


# ------------------------------------------------------------------ inputs

def _draft_counts(n, most):
    """Drafted tokens of n requests: from `most` down to none, in turn."""
    return (most - torch.arange(n)) % (most + 1)


def prepare(case, seed):
    dev = torch.Generator(device=DEVICE).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    s = dict(case)

    def normal(*size, dtype="f32", std=1.0, mean=0.0):
        return (torch.randn(*size, generator=dev, device=DEVICE) * std + mean).to(TYPES[dtype])

    def uniform(*size):
        return torch.rand(*size, generator=dev, device=DEVICE)

    if case["op"] == "int4":
        t, n_in, n_out, group = (case[k] for k in ("tokens", "n_in", "n_out", "group"))
        groups = -(-n_in // group)
        s["x"] = normal(t, n_in, dtype=case["x"])
        # rounded weights lie around the zero point, few at the ends; the sum
        # of four numbers of two bits, 0 to 12, and a fifth of one bit, twice
        bits = [torch.randint(0, 256, (n_out, (n_in + 1) // 2), generator=dev, device=DEVICE, dtype=torch.uint8) for _ in range(4)]
        nibbles = [sum((b >> (h + 2 * k)) & 3 for b in bits[:2] for k in range(2)) + ((bits[2] >> h) & 1) + ((bits[3] >> h) & 1) * 2 for h in (0, 4)]
        s["weights"] = nibbles[0] | (nibbles[1] << 4)
        s["scales"] = (uniform(n_out, groups) * 0.5 + 0.75).mul_(0.3 * n_in ** -0.5).to(TYPES[case["scales"]])
        s["zeros"] = torch.randint(5, 11, (n_out, groups), generator=dev, device=DEVICE, dtype=torch.uint8) if case["zeros"] else None
        s["base"] = normal(t, n_out, dtype=case["y"]) if case["base"] else None
        s["y"] = torch.empty(t, n_out, dtype=TYPES[case["y"]], device=DEVICE)
        return s
    if case["op"] == "verify":
        n, most, v = case["requests"], case["drafts"], case["vocab"]
        counts = _draft_counts(n, most)[torch.randperm(n, generator=cpu)]
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        d = int(offsets[-1])
        s["offsets"] = offsets.to(DEVICE)
        row = torch.arange(d) + torch.repeat_interleave(torch.arange(n), counts)  # the target's row of each draft
        target = normal(d + n, v, std=4.0)
        # the drafter's logits are the target's with an error; the requests of
        # a grammar have their mask on both
        draft = target[row.to(DEVICE)] + normal(d, v, std=0.5)
        if case["masked"]:
            in_grammar = torch.rand(n, generator=cpu) < 0.3
            allowed = uniform(1, v) < 0.2
            out = torch.repeat_interleave(in_grammar, counts + 1).to(DEVICE)
            target = torch.where(out[:, None] & ~allowed, NONE, target)
            draft = torch.where(out[row.to(DEVICE)][:, None] & ~allowed, NONE, draft)
        t = uniform(n) * 0.6 + 0.6
        if case["greedy"]:
            t[torch.rand(n, generator=cpu).to(DEVICE) < 0.3] = 0.0
        s["temperature"] = t
        # each draft was picked from the drafter's distribution (by Gumbel's rule)
        per = torch.repeat_interleave(t, counts.to(DEVICE), output_size=d)[:, None]
        noise = -torch.log(-torch.log(uniform(d, v).clamp_(1e-7, 1 - 1e-7)))
        s["draft_tokens"] = (draft + noise * per).argmax(1).int()
        s["target"], s["draft"] = target.to(TYPES[case["x"]]), None if case["point"] else draft.to(TYPES[case["x"]])
        s["accept_uniforms"], s["sample_uniforms"] = uniform(d), uniform(n)
        s["tokens"] = torch.empty(d + n, dtype=torch.int32, device=DEVICE)
        s["accepted"] = torch.empty(n, dtype=torch.int32, device=DEVICE)
        return s
    n, v, k = case["rows"], case["vocab"], case["top"]
    logits = torch.randn(n, v, generator=dev, device=DEVICE).mul_(2.0)
    # the teacher's largest logits, where the student is not far off, and its
    # sum over the whole vocabulary; some positions have fewer of them
    top = uniform(n, k).mul_(6.0).add_(6.0).sort(1, descending=True).values
    at = torch.randint(0, v, (n, 1), generator=dev, device=DEVICE) + torch.arange(k, device=DEVICE) * max(1, v // (2 * k))
    tokens = (at % v).int()
    logits.scatter_(1, tokens.long(), top + normal(n, k))
    s["logits"] = logits.to(TYPES[case["x"]])
    del logits
    tokens[torch.arange(k, device=DEVICE)[None] >= torch.randint(max(1, k - 4), k + 1, (n, 1), generator=dev, device=DEVICE)] = -1
    tokens[n // 2 if n > 2 else n:] = torch.where(uniform(n - (n // 2 if n > 2 else n), 1) < 0.1, -1, tokens[n // 2 if n > 2 else n:])  # padded positions
    s["top_tokens"], s["top_logits"] = tokens, top.to(TYPES[case["top_type"]])
    listed_sum = torch.where(tokens >= 0, s["top_logits"].double().div(case["temperature"]).exp(), 0.0).sum(1)
    s["log_sums"] = (listed_sum * (1.02 + uniform(n) * 0.3)).clamp(min=1e-3).log().float() if case["rest"] else None
    if case["op"] == "distill":
        s["loss"], s["stats"] = torch.empty(n, device=DEVICE), torch.empty(n, 3, device=DEVICE)
    else:
        s["stats"] = _distill_stats(s)
        # of the mean over the rows, in fp16 with a loss scale
        s["dloss"] = torch.full((1,), (1024.0 if case["x"] == "f16" else 1.0) / n, device=DEVICE).expand(n)
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ------------------------------------------------------------ the operators

def _int4_plain(s):
    w = torch.stack([s["weights"] & 15, s["weights"] >> 4], 2).view(s["n_out"], -1)[:, : s["n_in"]].float()
    at = torch.arange(s["n_in"], device=w.device) // s["group"]
    w = (w - (8.0 if s["zeros"] is None else s["zeros"].float()[:, at])) * s["scales"].float()[:, at]
    y = s["x"].float() @ w.T
    return (y if s["base"] is None else s["base"].float() + y).to(s["y"].dtype)


def _softmax_parts(logits, t):
    """exp((l - max) / t) of each row, and the rows' sums in 64 bits."""
    l = logits.float()
    e = torch.exp((l - l.max(1, keepdim=True).values) / t[:, None])
    return e, e.sum(1, dtype=torch.float64)


def _verify_plain(s):
    n, v, dev = s["requests"], s["vocab"], s["target"].device
    d = s["draft_tokens"].numel()
    first, counts = s["offsets"][:-1], s["offsets"].diff()
    request = torch.repeat_interleave(torch.arange(n, device=dev), counts, output_size=d)
    draft, token = torch.arange(d, device=dev), s["draft_tokens"].long()
    greedy = s["temperature"] == 0
    t = torch.where(greedy, 1.0, s["temperature"])
    ids = torch.arange(v, device=dev, dtype=torch.int32)
    best = torch.where(s["target"] == s["target"].amax(1, keepdim=True), ids, v).amin(1)  # the lowest of equals
    e, total = _softmax_parts(s["target"][draft + request], t[request])
    p = e.gather(1, token[:, None])[:, 0] / total
    q = torch.ones_like(p)
    if s["draft"] is not None:
        e, total = _softmax_parts(s["draft"], t[request])
        q = e.gather(1, token[:, None])[:, 0] / total
    ok = torch.where(greedy[request], best[draft + request] == token, s["accept_uniforms"] * q < p)
    place = draft - first[request]
    accepted = counts.scatter_reduce(0, request, torch.where(ok, counts[request], place), "amin")
    # the row that the last token is drawn from, its weights and their running sum: in 64 bits, next to borders
    row = first + torch.arange(n, device=dev) + accepted
    e = torch.exp((s["target"][row].double() - s["target"][row].max(1, keepdim=True).values.double()) / t[:, None].double())
    w = e / e.sum(1, keepdim=True)
    if d > 0:
        at = (first + accepted).clamp(max=d - 1)
        if s["draft"] is None:
            q = torch.zeros_like(w).scatter_(1, token[at][:, None], 1.0)
        else:
            e = torch.exp((s["draft"][at].double() - s["draft"][at].max(1, keepdim=True).values.double()) / t[:, None].double())
            q = e / e.sum(1, keepdim=True)
        w = torch.where((accepted < counts)[:, None], (w - q).clamp(min=0.0), w)
    running = w.cumsum(1)
    drawn = (running <= s["sample_uniforms"].double()[:, None] * running[:, -1:]).sum(1).clamp(max=v - 1)
    drawn = torch.where(greedy, best[row], drawn)
    tokens = torch.full((d + n,), -1, dtype=torch.int32, device=dev)
    tokens[draft + request] = torch.where(place < accepted[request], s["draft_tokens"], -1)
    tokens[row] = drawn.int()
    return {"tokens": tokens, "accepted": accepted.int()}


def _teacher(s):
    """The teacher's probabilities, 0 where nothing is listed, and what is left of them."""
    valid = (s["top_tokens"] >= 0) & (s["top_tokens"] < s["vocab"])
    a = torch.where(valid, s["top_logits"].double() / s["temperature"], NONE)
    whole = torch.logsumexp(a, 1) if s["log_sums"] is None else s["log_sums"].double()
    p = torch.where(valid, torch.exp(a - whole[:, None]), 0.0)
    rest = torch.zeros_like(whole) if s["log_sums"] is None else (1.0 - p.sum(1)).clamp(min=0.0)
    return valid, p.float(), rest.float()


def _distill_stats(s):
    """Each row's largest logit, and the sums over the vocabulary and over the
    tokens that are not listed of exp((logit - largest) / temperature); zeros
    for a position at which nothing is listed."""
    z = s["logits"].float()
    m = z.max(1, keepdim=True).values
    e = z.sub_(m).div_(s["temperature"]).exp_() if z is not s["logits"] else torch.exp((z - m) / s["temperature"])
    total = e.sum(1)
    valid = s["top_tokens"] >= 0
    e[torch.arange(z.shape[0], device=z.device)[:, None].expand_as(valid)[valid], s["top_tokens"][valid].long()] = 0.0
    stats = torch.stack([m[:, 0], total, e.sum(1) if s["rest"] else torch.zeros_like(total)], 1)
    return torch.where(valid.any(1, keepdim=True), stats, 0.0)


def _distill_plain(s):
    stats = _distill_stats(s)
    valid, p, r = _teacher(s)
    m, total, rest = stats.unbind(1)
    at = s["top_tokens"].clamp(min=0).long()
    log_q = (s["logits"].gather(1, at).float() - m[:, None]) / s["temperature"] - total.log()[:, None]
    loss = torch.where(p > 0, p * (p.log() - log_q), 0.0).sum(1)
    loss = loss + torch.where(r > 0, r * (r.log() - (rest / total).log()), 0.0)
    return {"loss": torch.where(valid.any(1), loss, 0.0), "stats": stats}


def _distill_grad_plain(s):
    valid, p, r = _teacher(s)
    m, total, rest = s["stats"].unbind(1)
    q = torch.exp((s["logits"].float() - m[:, None]) / s["temperature"]) / total[:, None]
    rows = torch.arange(q.shape[0], device=q.device)[:, None].expand_as(s["top_tokens"])[valid]
    at = s["top_tokens"][valid].long()
    listed_q = q[rows, at]
    if s["rest"]:
        q = q * (1.0 - r * total / rest)[:, None]
    q[rows, at] = listed_q
    q.index_put_((rows, at), -p[valid], accumulate=True)
    g = s["dloss"] / s["temperature"]
    return torch.where(valid.any(1, keepdim=True), q * g[:, None], 0.0).to(s["logits"].dtype)


def run(state):
    s = state
    if not own:
        return {"int4": _int4_plain, "verify": _verify_plain, "distill": _distill_plain, "distill_grad": _distill_grad_plain}[s["op"]](s)
    import sparse_matrix_vector_gb300 as S
    if s["op"] == "int4":
        S.spmv_int4_run(s["x"], s["weights"], s["scales"], s["y"], s["group"], zeros=s["zeros"], base=s["base"])
        return s["y"]
    if s["op"] == "verify":
        S.spmv_verify_drafts(s["target"], s["draft"], s["draft_tokens"], s["offsets"], s["accept_uniforms"], s["sample_uniforms"], s["tokens"], s["accepted"],
                             temperature=s["temperature"])
        return {"tokens": s["tokens"], "accepted": s["accepted"]}
    if s["op"] == "distill":
        S.spmv_distill(s["logits"], s["top_tokens"], s["top_logits"], s["loss"], temperature=s["temperature"], log_sums=s["log_sums"], stats=s["stats"])
        return {"loss": s["loss"], "stats": s["stats"]}
    S.spmv_distill_backward(s["dloss"], s["logits"], s["top_tokens"], s["top_logits"], s["stats"], s["dlogits"], temperature=s["temperature"], log_sums=s["log_sums"])
    return s["dlogits"]


# ------------------------------------------------------------- what it takes

def work(case):
    """The bytes of the inputs, read once, and of the outputs, written once,
    and the operations of the formulas."""
    if case["op"] == "int4":
        t, n_in, n_out = (case[k] for k in ("tokens", "n_in", "n_out"))
        groups = -(-n_in // case["group"])
        return {"bytes": n_out * ((n_in + 1) // 2 + groups * (BYTES[case["scales"]] + case["zeros"])) + t * n_in * BYTES[case["x"]]
                + t * n_out * BYTES[case["y"]] * (1 + case["base"]), "flops": 2 * t * n_in * n_out}
    if case["op"] == "verify":
        n = case["requests"]
        d = int(_draft_counts(n, case["drafts"]).sum())
        rows = d + n + (0 if case["point"] else d)
        return {"bytes": rows * case["vocab"] * BYTES[case["x"]] + 16 * (d + n), "flops": 4 * rows * case["vocab"]}
    n, v, k = case["rows"], case["vocab"], case["top"]
    lists = n * (k * (4 + BYTES[case["top_type"]]) + 4 * case["rest"])
    if case["op"] == "distill":
        return {"bytes": n * v * BYTES[case["x"]] + lists + 16 * n, "flops": 4 * n * v}
    return {"bytes": 2 * n * v * BYTES[case["x"]] + lists + 12 * n, "flops": 4 * n * v}


# ------------------------------------------------------- the same in 64 bits

def _exact_int4(s):
    t, n_in, n_out, group = (s[k] for k in ("tokens", "n_in", "n_out", "group"))
    y = torch.zeros(t, n_out, dtype=torch.float64, device=s["x"].device)
    for lo in range(0, n_in, group):  # group by group
        hi = min(lo + group, n_in)
        cols = torch.arange(lo, hi, device=y.device)
        q = (s["weights"][:, cols // 2].int() >> (4 * (cols % 2))) & 15
        zero = 8 if s["zeros"] is None else s["zeros"][:, lo // group, None].int()
        y += (s["x"][:, lo:hi].double() @ (q - zero).double().T) * s["scales"][:, lo // group].double()
    return y if s["base"] is None else y + s["base"].double()


def _exact_rows(s):
    """Blocks of rows, for memory's sake: slice, listed entries of each row as
    a dense vector of the teacher's probabilities, whether listed, its rest."""
    n, v = s["logits"].shape
    step = max(1, 2 ** 25 // v)
    for lo in range(0, n, step):
        k = slice(lo, min(n, lo + step))
        tokens, t = s["top_tokens"][k].long(), s["top_logits"][k].double() / s["temperature"]
        valid = tokens >= 0
        weights = torch.exp(t - t.max()) * valid
        shift = t.max()
        p = weights / weights.sum(1, keepdim=True).clamp(min=1e-300) if s["log_sums"] is None else weights * torch.exp(shift - s["log_sums"][k].double())[:, None]
        dense = torch.zeros(tokens.shape[0], v + 1, dtype=torch.float64, device=t.device).scatter_add_(1, torch.where(valid, tokens, v), p)[:, :v]
        there = torch.zeros(tokens.shape[0], v + 1, dtype=torch.bool, device=t.device).scatter_(1, torch.where(valid, tokens, v), True)[:, :v]
        rest = torch.zeros_like(p[:, 0]) if s["log_sums"] is None else 1.0 - p.sum(1)
        yield k, dense, there, rest, valid.any(1)


def _exact_distill(s):
    n = s["logits"].shape[0]
    loss = torch.zeros(n, dtype=torch.float64, device=s["logits"].device)
    stats = torch.zeros(n, 3, dtype=torch.float64, device=s["logits"].device)
    for k, p, there, rest, any_listed in _exact_rows(s):
        z = s["logits"][k].double()
        m = z.amax(1, keepdim=True)
        log_q = torch.log_softmax(z / s["temperature"], 1)
        loss[k] = torch.where(any_listed, (torch.xlogy(p, p) - p * log_q).sum(1), 0.0)
        e = torch.exp((z - m) / s["temperature"])
        unlisted = torch.where(there, 0.0, e).sum(1)
        stats[k] = torch.stack([m[:, 0], e.sum(1), unlisted if s["rest"] else torch.zeros_like(unlisted)], 1) * any_listed[:, None]
        if s["rest"]:
            loss[k] += torch.where(any_listed, torch.xlogy(rest, rest) - rest * torch.log(unlisted / e.sum(1)), 0.0)
    return {"loss": loss, "stats": stats}


def _exact_distill_grad(s):
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device=s["logits"].device)
    for k, p, there, rest, any_listed in _exact_rows(s):
        m, total, unlisted = s["stats"][k].double().unbind(1)
        q = torch.exp((s["logits"][k].double() - m[:, None]) / s["temperature"]) / total[:, None]
        if s["rest"]:
            q = torch.where(there, q, q - q * (rest * total / unlisted)[:, None])
        out[k] = torch.where(any_listed[:, None], (q - p) * (s["dloss"][k].double() / s["temperature"])[:, None], 0.0)
    return out


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"int4": _exact_int4, "distill": _exact_distill, "distill_grad": _exact_distill_grad}[s["op"]](s)
