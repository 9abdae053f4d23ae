"""Python binding of the operators around a pruned layer and beside the dense
model it came from (include/spmv.h, last two sections), same names as the C
calls: layer norm and its gradient, low-rank adapters of many requests, the
logits' penalties, biases and grammar masks; products with 4-bit weights, the
verification of drafted tokens, distillation and its gradient.

Only argument marshalling lives here. Tensors are CUDA tensors of one device,
which is the current one; matrices have contiguous columns and any row
stride. Calls run on ``stream`` (default: the current torch stream) and do
not synchronize. A workspace that the caller does not give comes from torch's
caching allocator, from the pool of the stream that the call runs on; the
default stream's is kept for its next call, up to 64 MiB for each thread.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib
from ._lib import SPMV_BF16, SPMV_F16, SPMV_F32
from .api import SpmvError

_CODES = {torch.float32: SPMV_F32, torch.float16: SPMV_F16, torch.bfloat16: SPMV_BF16}
_F32, _I32, _I64 = torch.float32, torch.int32, torch.int64
_INT32_MAX = 2**31 - 1
_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (absent in CPU builds)
_library = None
# Workspaces of the default stream, one per thread and device, kept for the
# next call: its calls are in order, and it can be neither captured nor
# destroyed. (Taking one from the allocator between launches costs 4 us and
# makes the launches 2 us slower, of some 20 us a call.) Larger ones, whose
# calls take some 100 us and more, are not kept: a thread would hold its
# largest call's for good.
_kept = threading.local()
_KEPT_BYTES = 64 << 20


def _lib_handle():
    global _library
    if _library is None:
        _library = _lib.load()
    return _library


def _check(status: int, where: str) -> None:
    if status != 0:
        raise SpmvError(status, where)


def _too_large(where: str):
    """Sizes that the C call's 32-bit arguments would cut short."""
    raise SpmvError(8, where)  # SPMV_ERR_TOO_LARGE


def _dtype(t, what: str) -> int:
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be float32, float16 or bfloat16, got {t.dtype}") from None


def _rows(t, what: str):
    """(rows, columns, row stride) of a matrix, or of a vector as one row."""
    shape = t.shape
    if len(shape) == 2:
        n, d = shape
        stride, inner = t.stride()
        if inner != 1 and d > 1:
            raise ValueError(f"{what} must have contiguous columns")
        return n, d, stride
    if len(shape) == 1:
        d = shape[0]
        if d > 1 and t.stride(0) != 1:
            raise ValueError(f"{what} must be contiguous")
        return 1, d, d
    raise ValueError(f"{what} must be a matrix (or a vector: one row)")


def _vector(t, n: int, dtype, what: str) -> int:
    """Address of a contiguous vector of n elements; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} elements")
    return t.data_ptr()


def _same_device(first, *others) -> int:
    """The tensors' common CUDA device, which must be the current one."""
    dev = _current_device() if first.is_cuda else -1
    if dev < 0 or first.get_device() != dev:
        raise ValueError(f"tensors must be on the current CUDA device, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != dev:  # (-1: not a CUDA tensor)
            raise ValueError(f"tensors must be on the current CUDA device, got {t.device}")
    return dev


def _on(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev)
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    return 0 if handle == 1 else handle  # (two names of the default stream)


def _empty_on(handle: int, n_bytes: int, dev: int):
    """Memory of the pool of the stream that will use it. (A block of another
    stream's pool may still be in use by work queued there before it was
    freed, and be given away there while this stream is at work on it.)"""
    if handle == _raw_stream(dev):
        return torch.empty(n_bytes, dtype=torch.uint8, device=dev)
    stream = (torch.cuda.default_stream(dev) if handle == 0
              else torch.cuda.ExternalStream(handle, device=dev))
    with torch.cuda.stream(stream):
        return torch.empty(n_bytes, dtype=torch.uint8, device=dev)


def _workspace(given, n_bytes: int, handle: int, dev: int):
    """(address, bytes, owner) of a workspace; one that the caller does not
    give is safe to drop as soon as the call returns."""
    if given is not None:
        if given.data_ptr() % 16 or not given.is_contiguous():
            raise ValueError("workspace must be contiguous and 16-byte aligned")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if n_bytes == 0:
        return None, 0, None
    if handle == 0 and n_bytes <= _KEPT_BYTES:
        try:
            kept = _kept.by_device
        except AttributeError:
            kept = _kept.by_device = {}
        ws = kept.get(dev)
        if ws is None or ws.numel() < n_bytes:
            ws = kept[dev] = _empty_on(0, n_bytes, dev)
    else:
        ws = _empty_on(handle, n_bytes, dev)
    return ws.data_ptr(), n_bytes, ws


def _params(weight, bias, d: int, what: str):
    """Addresses of two vectors of one type (either may be None) and its code."""
    one = weight if weight is not None else bias
    if one is None:
        return 0, 0, SPMV_F32
    code = _dtype(one, what)
    return _vector(weight, d, one.dtype, what), _vector(bias, d, one.dtype, what), code


def spmv_layernorm(x, weight, bias, y, eps: float = 1e-5, mean=None, rstd=None,
                   stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias over each row of x (a vector is
    one row). y: of x's type, or of any type when x is float32; weight and
    bias (of one type) may be None; mean and rstd, if given, are float32
    vectors that receive the rows' statistics."""
    n, d, xs = _rows(x, "x")
    n_y, d_y, ys = _rows(y, "y")
    if n_y != n or d_y != d:
        raise ValueError("x and y must have the same shape")
    if d > _INT32_MAX:
        _too_large("spmv_layernorm")
    dev = _same_device(x, y, weight, bias, mean, rstd)
    w, b, p = _params(weight, bias, d, "weight and bias")
    _check(_lib_handle().spmv_layernorm(
        n, d, x.data_ptr(), _dtype(x, "x"), xs, w, b, p, eps, y.data_ptr(), _dtype(y, "y"), ys,
        _vector(mean, n, _F32, "mean"), _vector(rstd, n, _F32, "rstd"),
        _on(stream, dev)), "spmv_layernorm")


def spmv_layernorm_backward_workspace(n_rows: int, n_cols: int, want_params: bool = True) -> int:
    """Bytes of workspace that spmv_layernorm_backward needs (0 for sizes it refuses)."""
    if not 0 < n_cols <= _INT32_MAX:
        return 0
    return int(_lib_handle().spmv_layernorm_backward_workspace(n_rows, n_cols, int(want_params)))


def spmv_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace=None,
                            stream=None) -> None:
    """Gradient of spmv_layernorm: dx (of x's type) and, summed over the
    rows, dweight and dbias (of weight's type, or of one type if weight is
    None), each overwritten; any of the three may be None. dy may be an
    expanded row (row stride 0)."""
    n, d, xs = _rows(x, "x")
    n_dy, d_dy, dys = _rows(dy, "dy")
    if n_dy != n or d_dy != d:
        raise ValueError("dy and x must have the same shape")
    if d > _INT32_MAX:
        _too_large("spmv_layernorm_backward")
    code = _dtype(x, "x")
    dxs = 0
    if dx is not None:
        n_dx, d_dx, dxs = _rows(dx, "dx")
        if n_dx != n or d_dx != d:
            raise ValueError("dx and x must have the same shape")
        if dx.dtype != x.dtype:
            raise TypeError(f"dx must be {x.dtype}, got {dx.dtype}")
    dev = _same_device(x, dy, weight, mean, rstd, dx, dweight, dbias, workspace)
    w, dw, p = _params(weight, dweight, d, "weight and dweight")
    if w or dw:
        db = _vector(dbias, d, (weight if weight is not None else dweight).dtype, "dbias")
    else:
        _, db, p = _params(None, dbias, d, "dbias")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward call are needed")
    handle = _on(stream, dev)
    lib = _lib_handle()
    need = lib.spmv_layernorm_backward_workspace(n, d, 1 if dw or db else 0)
    wp, wn, _owner = _workspace(workspace, need, handle, dev)
    _check(lib.spmv_layernorm_backward(
        n, d, dy.data_ptr(), _dtype(dy, "dy"), dys, x.data_ptr(), code, xs, w, p,
        _vector(mean, n, _F32, "mean"), _vector(rstd, n, _F32, "rstd"),
        0 if dx is None else dx.data_ptr(), dxs, dw, db, wp, wn, handle),
        "spmv_layernorm_backward")


def spmv_adapters_workspace(n_tokens: int, n_slots: int, rank: int) -> int:
    """Bytes of workspace that spmv_adapters_run needs (0 for sizes it refuses)."""
    if min(n_tokens, n_slots, rank) < 0 or max(n_tokens, n_slots, rank) > _INT32_MAX:
        return 0
    return int(_lib_handle().spmv_adapters_workspace(n_tokens, n_slots, rank))


def spmv_adapters_run(x, a, b, slot_ids, y, base=None, ranks=None, scales=None, workspace=None,
                      stream=None) -> None:
    """y[t] = base[t] + scales[s] * b[s] @ (a[s] @ x[t]) with s = slot_ids[t];
    tokens whose slot id is outside [0, n_slots) get y[t] = base[t].
    x: (tokens, n_in) float16 or bfloat16 (a vector is one token); a: (slots,
    rank, n_in) and b: (slots, n_out, rank), contiguous, of x's type; y and
    base: (tokens, n_out), float32 or of x's type (base may be y, or None for
    zero); slot_ids, ranks (per slot, None: all of a's rank): int32; scales
    (per slot, None: 1): float32."""
    t, n_in, xs = _rows(x, "x")
    t_y, n_out, ys = _rows(y, "y")
    if t_y != t:
        raise ValueError("x and y must have the same number of tokens")
    slots, rank, a_in = a.shape
    if a_in != n_in or tuple(b.shape) != (slots, n_out, rank):
        raise ValueError(f"a must be (slots, rank, {n_in}) and b (slots, {n_out}, rank)")
    if (t > _INT32_MAX or n_in > _INT32_MAX or n_out > _INT32_MAX or slots > _INT32_MAX
            or rank > _INT32_MAX):
        _too_large("spmv_adapters_run")
    if a.dtype != x.dtype or b.dtype != x.dtype:
        raise TypeError("a and b must have x's type")
    if not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("a and b must be contiguous")
    bs = 0
    if base is not None:
        t_b, n_b, bs = _rows(base, "base")
        if t_b != t or n_b != n_out:
            raise ValueError("base and y must have the same shape")
        if base.dtype != y.dtype:
            raise TypeError(f"base must be {y.dtype}, got {base.dtype}")
    if slot_ids is None:
        raise ValueError("slot_ids is needed")
    dev = _same_device(x, y, a, b, slot_ids, base, ranks, scales, workspace)
    handle = _on(stream, dev)
    lib = _lib_handle()
    wp, wn, _owner = _workspace(workspace, lib.spmv_adapters_workspace(t, slots, rank), handle, dev)
    _check(lib.spmv_adapters_run(
        t, n_in, n_out, slots, rank, _dtype(x, "x"), x.data_ptr(), xs, a.data_ptr(),
        b.data_ptr(), _vector(slot_ids, t, _I32, "slot_ids"),
        _vector(ranks, slots, _I32, "ranks"),
        _vector(scales, slots, _F32, "scales"),
        None if base is None else base.data_ptr(), bs, y.data_ptr(), _dtype(y, "y"), ys, wp, wn,
        handle), "spmv_adapters_run")


def _list(pair, n: int, what: str):
    """Addresses of a ragged list's tokens and offsets (None: no list)."""
    if pair is None:
        return 0, 0
    tokens, offsets = pair
    return (_vector(tokens, tokens.numel(), _I32, what + " tokens"),
            _vector(offsets, n + 1, _I64, what + " offsets"))


def spmv_logits_process(logits, out, prompt=None, output=None, repetition=None, frequency=None,
                        presence=None, bias=None, mask=None, mask_rows=None,
                        stream=None) -> None:
    """Repetition, frequency and presence penalties, biases and grammar masks
    on logits (requests, vocab; a vector is one request), into out (float32 or
    of logits' type; may be logits itself).
    prompt, output: (tokens int32, offsets int64 of requests + 1): the tokens
    of each request's prompt, and those generated so far. repetition,
    frequency, presence: float32 per request. bias: (tokens int32, values
    float32, offsets int64). mask: int32 rows of ceil(vocab / 32) words, bit
    v % 32 of word v // 32 set where token v is allowed; mask_rows: int32 per
    request, the row of its mask or -1 (None: request i takes row i).
    include/spmv.h has the formula."""
    n, v, stride = _rows(logits, "logits")
    n_o, v_o, out_stride = _rows(out, "out")
    if n_o != n or v_o != v:
        raise ValueError("logits and out must have the same shape")
    if n > _INT32_MAX or v > _INT32_MAX:
        _too_large("spmv_logits_process")
    p_tok, p_off = _list(prompt, n, "prompt")
    o_tok, o_off = _list(output, n, "output")
    b_tok = b_val = b_off = 0
    if bias is not None:
        b_tok, b_off = _list((bias[0], bias[2]), n, "bias")
        b_val = _vector(bias[1], bias[0].numel(), _F32, "bias values")
    m_ptr = m_stride = n_masks = 0
    if mask is not None:
        if mask.dtype != torch.int32:
            raise TypeError(f"mask must be torch.int32, got {mask.dtype}")
        n_masks, words, m_stride = _rows(mask, "mask")
        if words != (v + 31) // 32:
            raise ValueError(f"mask must have {(v + 31) // 32} words in a row")
        if n_masks > _INT32_MAX:
            _too_large("spmv_logits_process")
        if mask_rows is None and n_masks < n:
            raise ValueError("mask must have a row for each request (or give mask_rows)")
        m_ptr = mask.data_ptr()
    lists = [t for group in (prompt, output, bias) if group is not None for t in group]
    dev = _same_device(logits, out, repetition, frequency, presence, mask, mask_rows, *lists)
    args = _lib.spmv_logits(
        n, v, logits.data_ptr(), stride, out.data_ptr(), out_stride, _dtype(logits, "logits"),
        _dtype(out, "out"), p_tok, p_off, o_tok, o_off, _vector(repetition, n, _F32, "repetition"),
        _vector(frequency, n, _F32, "frequency"), _vector(presence, n, _F32, "presence"), b_tok,
        b_val, b_off, m_ptr, m_stride, _vector(mask_rows, n, _I32, "mask_rows"), n_masks, 0)
    _check(_lib_handle().spmv_logits_process(ctypes.byref(args), _on(stream, dev)),
           "spmv_logits_process")


def spmv_int4_workspace(n_tokens: int, n_in: int) -> int:
    """Bytes of workspace that spmv_int4_run needs (0 for sizes it refuses)."""
    if min(n_tokens, n_in) < 0 or max(n_tokens, n_in) > _INT32_MAX:
        return 0
    return int(_lib_handle().spmv_int4_workspace(n_tokens, n_in))


def spmv_int4_run(x, weights, scales, y, group: int, zeros=None, base=None, workspace=None,
                  stream=None) -> None:
    """y[t] = base[t] + W @ x[t], W[o, i] = scales[o, i // group] * (q[o, i] - zeros[o, i // group]).
    x: (tokens, n_in) float16 or bfloat16 (a vector is one token); weights:
    (n_out, ceil(n_in / 2)) uint8, column i in the low (i even) or high half of
    byte i // 2; scales: (n_out, ceil(n_in / group)) contiguous, float32 or of
    x's type; zeros: the same of uint8 (None: 8); group: a power of two from 32 on,
    or at least n_in. y and base: (tokens, n_out), float32 or of x's type (base
    may be y, or None for zero)."""
    t, n_in, xs = _rows(x, "x")
    t_y, n_out, ys = _rows(y, "y")
    if t_y != t:
        raise ValueError("x and y must have the same number of tokens")
    if weights.dtype != torch.uint8:
        raise TypeError(f"weights must be torch.uint8, got {weights.dtype}")
    w_out, row_bytes, ws = _rows(weights, "weights")
    if w_out != n_out or row_bytes != (n_in + 1) // 2:
        raise ValueError(f"weights must be ({n_out}, {(n_in + 1) // 2})")
    if group < 1:
        raise ValueError("group must be at least 1")
    if t > _INT32_MAX or n_in > _INT32_MAX or n_out > _INT32_MAX:
        _too_large("spmv_int4_run")
    group = min(group, _INT32_MAX)
    groups = -(-n_in // group)
    if tuple(scales.shape) != (n_out, groups) or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous ({n_out}, {groups})")
    bs = 0
    if base is not None:
        t_b, n_b, bs = _rows(base, "base")
        if t_b != t or n_b != n_out:
            raise ValueError("base and y must have the same shape")
        if base.dtype != y.dtype:
            raise TypeError(f"base must be {y.dtype}, got {base.dtype}")
    dev = _same_device(x, y, weights, scales, zeros, base, workspace)
    handle = _on(stream, dev)
    lib = _lib_handle()
    wp, wn, _owner = _workspace(workspace, lib.spmv_int4_workspace(t, n_in), handle, dev)
    _check(lib.spmv_int4_run(
        t, n_in, n_out, group, _dtype(x, "x"), x.data_ptr(), xs, weights.data_ptr(), ws,
        scales.data_ptr(), _dtype(scales, "scales"),
        _vector(zeros, n_out * groups, torch.uint8, "zeros"),
        None if base is None else base.data_ptr(), bs, y.data_ptr(), _dtype(y, "y"), ys, wp, wn,
        handle), "spmv_int4_run")


def spmv_verify_workspace(n_requests: int, n_drafts: int, vocab: int) -> int:
    """Bytes of workspace that spmv_verify_drafts needs (0 for sizes it refuses)."""
    if min(n_requests, n_drafts, vocab) < 0 or max(n_requests, n_drafts, vocab) > _INT32_MAX:
        return 0
    return int(_lib_handle().spmv_verify_workspace(n_requests, n_drafts, vocab))


def spmv_verify_drafts(target, draft, draft_tokens, offsets, accept_uniforms, sample_uniforms,
                       tokens, accepted, temperature=None, workspace=None, stream=None) -> None:
    """Accept drafted tokens against the target's probabilities and draw one
    token more per request, by given random numbers in [0, 1).
    target: (drafts + requests, vocab) logits, a row more than drafts for each
    request; draft: (drafts, vocab) logits of the same type, or None where the
    drafts carry no probabilities; draft_tokens: int32 of all requests one
    after the other; offsets: int64 of requests + 1. accept_uniforms: float32
    per draft; sample_uniforms, temperature (None: 1; 0: greedy): float32 per
    request. tokens (drafts + requests, int32) receives each request's accepted
    drafts, the token drawn and -1 to its end, accepted (requests, int32) the
    number of drafts accepted. include/spmv.h has the rules."""
    rows, v, ts = _rows(target, "target")
    d = draft_tokens.numel()
    n = offsets.numel() - 1
    if n < 0 or rows != d + n:
        raise ValueError("target must have a row for each draft and one more for each request")
    if rows > _INT32_MAX or v > _INT32_MAX:
        _too_large("spmv_verify_drafts")
    ds = 0
    if draft is not None:
        rows_d, v_d, ds = _rows(draft, "draft")
        if rows_d != d or v_d != v:
            raise ValueError("draft must have a row for each draft and target's vocabulary")
        if draft.dtype != target.dtype:
            raise TypeError(f"draft must be {target.dtype}, got {draft.dtype}")
    if accept_uniforms is None or sample_uniforms is None or tokens is None or accepted is None:
        raise ValueError("the random numbers and both outputs are needed")
    dev = _same_device(target, draft, draft_tokens, offsets, accept_uniforms, sample_uniforms,
                       tokens, accepted, temperature, workspace)
    handle = _on(stream, dev)
    lib = _lib_handle()
    wp, wn, _owner = _workspace(workspace, lib.spmv_verify_workspace(n, d, v), handle, dev)
    _check(lib.spmv_verify_drafts(
        n, d, v, _dtype(target, "target"), target.data_ptr(), ts,
        None if draft is None else draft.data_ptr(), ds,
        _vector(draft_tokens, d, _I32, "draft_tokens"), _vector(offsets, n + 1, _I64, "offsets"),
        _vector(accept_uniforms, d, _F32, "accept_uniforms"),
        _vector(sample_uniforms, n, _F32, "sample_uniforms"),
        _vector(temperature, n, _F32, "temperature"), _vector(tokens, rows, _I32, "tokens"),
        _vector(accepted, n, _I32, "accepted"), wp, wn, handle), "spmv_verify_drafts")


def _top(logits, top_tokens, top_logits, where: str):
    """(rows, vocab, stride, top and its strides) of a distillation's inputs."""
    n, v, stride = _rows(logits, "logits")
    n_t, k, token_stride = _rows(top_tokens, "top_tokens")
    n_l, k_l, top_stride = _rows(top_logits, "top_logits")
    if n_t != n or n_l != n or k_l != k:
        raise ValueError("top_tokens and top_logits must have one shape, with logits' rows")
    if top_tokens.dtype != _I32:
        raise TypeError(f"top_tokens must be {_I32}, got {top_tokens.dtype}")
    if v > _INT32_MAX or k > _INT32_MAX:
        _too_large(where)
    return n, v, stride, k, token_stride, top_stride


def _stats(stats, n: int) -> int:
    if stats is not None and tuple(stats.shape) != (n, 3):
        raise ValueError(f"stats must be ({n}, 3)")
    return _vector(stats, 3 * n, _F32, "stats")


def spmv_distill(logits, top_tokens, top_logits, loss, temperature: float = 1.0, log_sums=None,
                 stats=None, stream=None) -> None:
    """loss[i]: the divergence of softmax(logits[i] / temperature) from the
    teacher's probabilities of its listed tokens. logits: (rows, vocab) (a
    vector is one row); top_tokens: (rows, top) int32, -1 where nothing is
    listed; top_logits: the same shape, any type. log_sums: float32 per row, the
    teacher's log sum over its vocabulary of exp(logit / temperature): the
    probabilities are then taken as they are and the rest counts as one more
    class (None: normalised over the listed tokens). loss: float32 per row;
    stats: (rows, 3) float32, what the gradient needs. include/spmv.h has the
    formula."""
    n, v, stride, k, token_stride, top_stride = _top(logits, top_tokens, top_logits, "spmv_distill")
    if loss is None:
        raise ValueError("loss is needed")
    dev = _same_device(logits, top_tokens, top_logits, loss, log_sums, stats)
    _check(_lib_handle().spmv_distill(
        n, v, logits.data_ptr(), _dtype(logits, "logits"), stride, k, top_tokens.data_ptr(),
        token_stride, top_logits.data_ptr(), _dtype(top_logits, "top_logits"), top_stride,
        _vector(log_sums, n, _F32, "log_sums"), temperature, _vector(loss, n, _F32, "loss"),
        _stats(stats, n), _on(stream, dev)), "spmv_distill")


def spmv_distill_backward(dloss, logits, top_tokens, top_logits, stats, dlogits,
                          temperature: float = 1.0, log_sums=None, stream=None) -> None:
    """Gradient of spmv_distill: dlogits (of logits' type and shape; may be
    logits itself) is overwritten. dloss: float32 per row, or one expanded over
    the rows; stats: the forward call's, with the same temperature and
    log_sums."""
    n, v, stride, k, token_stride, top_stride = _top(logits, top_tokens, top_logits,
                                                     "spmv_distill_backward")
    n_o, v_o, out_stride = _rows(dlogits, "dlogits")
    if n_o != n or v_o != v:
        raise ValueError("dlogits and logits must have the same shape")
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be {logits.dtype}, got {dlogits.dtype}")
    if dloss.dtype != _F32:
        raise TypeError(f"dloss must be {_F32}, got {dloss.dtype}")
    if dloss.dim() > 1 or dloss.numel() != n:
        raise ValueError(f"dloss must have {n} elements")
    if stats is None:
        raise ValueError("stats of the forward call are needed")
    dev = _same_device(logits, top_tokens, top_logits, dloss, log_sums, stats, dlogits)
    _check(_lib_handle().spmv_distill_backward(
        n, v, dloss.data_ptr(), dloss.stride(0) if dloss.dim() else 0, logits.data_ptr(),
        _dtype(logits, "logits"), stride, k, top_tokens.data_ptr(), token_stride,
        top_logits.data_ptr(), _dtype(top_logits, "top_logits"), top_stride,
        _vector(log_sums, n, _F32, "log_sums"), temperature, _stats(stats, n), dlogits.data_ptr(),
        out_stride, _on(stream, dev)), "spmv_distill_backward")
