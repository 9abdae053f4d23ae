"""CPU tests of the operators around a pruned layer: what the C entry points
and the Python wrappers refuse (validation comes before any device call), and
their workspace sizes. Nothing here launches a kernel."""
import ctypes

import pytest

import sparse_matrix_vector_gb300 as S
from sparse_matrix_vector_gb300 import _lib

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, TOO_LARGE = 0, 1, 5, 8
F32, F16, BF16 = 0, 1, 2
# made-up 16-byte aligned addresses far apart: refused calls never read them
X, Y, W, B, M, R, WS, DX, DW, DB = (0x10000000 * k for k in range(1, 11))


def layernorm(lib, **kw):
    a = dict(n=4, d=8, x=X, xt=F32, xs=8, w=W, b=B, pt=F32, eps=1e-5, y=Y, yt=F16, ys=8, m=M, r=R)
    a.update(kw)
    return lib.spmv_layernorm(a["n"], a["d"], a["x"], a["xt"], a["xs"], a["w"], a["b"], a["pt"],
                              a["eps"], a["y"], a["yt"], a["ys"], a["m"], a["r"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(d=-4), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(xt=7), INVALID), (dict(yt=-1), INVALID), (dict(pt=3), INVALID),
    (dict(x=X + 2), INVALID), (dict(y=Y + 1), INVALID), (dict(w=W + 2), INVALID),
    (dict(b=B + 1), INVALID), (dict(m=M + 2), INVALID), (dict(r=R + 2), INVALID),
    (dict(xs=-8), INVALID), (dict(ys=7), INVALID), (dict(ys=0), INVALID),
    (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y=X), INVALID),                      # fp16 output over fp32 input
    (dict(y=X + 64, yt=F32), INVALID),         # overlap that is not in place
    (dict(y=X, yt=F32, ys=16), INVALID),       # in place with another stride
    (dict(n=2**62, xs=2**10, ys=2**10), INVALID),
    (dict(xt=F16, yt=BF16), UNSUPPORTED), (dict(xt=BF16, yt=F32), UNSUPPORTED),
    (dict(d=2**31 - 1, xs=2**31, ys=2**31), TOO_LARGE),
    (dict(n=0), OK), (dict(n=0, x=None, y=None, m=None, r=None, w=None, b=None), OK),
])
def test_layernorm_refuses(spmv_lib, kw, status):
    assert layernorm(spmv_lib, **kw) == status


def backward(lib, **kw):
    a = dict(n=4, d=8, dy=Y, dyt=F16, dys=8, x=X, xt=F32, xs=8, w=W, pt=F32, m=M, r=R, dx=DX,
             dxs=8, dw=DW, db=DB, ws=WS, wn=1 << 40)
    a.update(kw)
    return lib.spmv_layernorm_backward(a["n"], a["d"], a["dy"], a["dyt"], a["dys"], a["x"],
                                       a["xt"], a["xs"], a["w"], a["pt"], a["m"], a["r"],
                                       a["dx"], a["dxs"], a["dw"], a["db"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(dy=None), INVALID), (dict(x=None), INVALID),
    (dict(m=None), INVALID), (dict(r=None), INVALID), (dict(dyt=9), INVALID),
    (dict(dxs=4), INVALID), (dict(dx=DX + 2), INVALID), (dict(dy=Y + 1), INVALID),
    (dict(w=W + 1), INVALID), (dict(dw=DW + 2), INVALID), (dict(db=DB + 2), INVALID),
    (dict(ws=WS + 8), INVALID), (dict(n=5000, ws=None), INVALID), (dict(n=5000, wn=0), INVALID),
    (dict(dx=X), INVALID), (dict(dx=Y), INVALID), (dict(dx=Y + 32, dyt=F32), INVALID),
    (dict(xt=F16, dyt=BF16), UNSUPPORTED), (dict(d=2**31 - 1, xs=2**31, dys=2**31, dxs=2**31),
                                            TOO_LARGE),
    (dict(n=0, dw=None, db=None), OK),
])
def test_layernorm_backward_refuses(spmv_lib, kw, status):
    assert backward(spmv_lib, **kw) == status


def test_layernorm_backward_workspace(spmv_lib):
    size = S.spmv_layernorm_backward_workspace
    assert size(100, 64, False) == 0 and size(0, 64) == 0
    assert size(-1, 64) == 0 and size(4, 0) == 0
    assert size(1, 64) >= 0 and size(100000, 12288) >= size(1, 12288)
    n = size(4096, 1000)
    assert n > 0 and backward(spmv_lib, n=4096, d=1000, xs=1000, dys=1000, dxs=1000,
                              wn=n - 1) == INVALID


def adapters(lib, **kw):
    a = dict(t=4, i=64, o=32, s=3, r=8, dt=F16, x=X, xs=64, a=W, b=B, ids=M, ranks=R, scales=DB,
             base=DX, bs=32, y=Y, yt=F32, ys=32, ws=WS, wn=1 << 40)
    a.update(kw)
    return lib.spmv_adapters_run(a["t"], a["i"], a["o"], a["s"], a["r"], a["dt"], a["x"], a["xs"],
                                 a["a"], a["b"], a["ids"], a["ranks"], a["scales"], a["base"],
                                 a["bs"], a["y"], a["yt"], a["ys"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), INVALID), (dict(i=-1), INVALID), (dict(o=-1), INVALID), (dict(s=-1), INVALID),
    (dict(r=-1), INVALID), (dict(dt=5), INVALID), (dict(yt=5), INVALID), (dict(x=None), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(ids=None), INVALID),
    (dict(y=None), INVALID), (dict(x=X + 1), INVALID), (dict(a=W + 1), INVALID),
    (dict(b=B + 1), INVALID), (dict(ids=M + 2), INVALID), (dict(ranks=R + 1), INVALID),
    (dict(scales=DB + 2), INVALID), (dict(base=DX + 2), INVALID), (dict(y=Y + 2), INVALID),
    (dict(ws=WS + 4), INVALID), (dict(xs=-1), INVALID), (dict(ys=31), INVALID),
    (dict(bs=-2), INVALID), (dict(base=Y + 128), INVALID), (dict(base=Y, bs=64), INVALID),
    (dict(x=Y), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(dt=F16, yt=BF16), UNSUPPORTED),
    (dict(dt=BF16, yt=F16), UNSUPPORTED), (dict(r=257), TOO_LARGE), (dict(s=16385), TOO_LARGE),
    (dict(t=0), OK), (dict(t=0, x=None, y=None, base=None, ids=None, ws=None, wn=0), OK),
    (dict(o=0), OK),
])
def test_adapters_refuses(spmv_lib, kw, status):
    assert adapters(spmv_lib, **kw) == status


def test_adapters_workspace(spmv_lib):
    size = S.spmv_adapters_workspace
    assert size(-1, 2, 8) == 0 and size(4, -1, 8) == 0 and size(4, 2, 257) == 0
    assert size(0, 2, 8) == 0
    n = size(5000, 8, 16)
    if n:
        assert adapters(spmv_lib, t=5000, s=8, r=16, wn=n - 1) == INVALID
        assert adapters(spmv_lib, t=5000, s=8, r=16, ws=None) == INVALID


def logits(lib, **kw):
    a = _lib.spmv_logits(n_requests=4, vocab=100, logits=X, stride=100, out=Y, out_stride=100,
                         dtype=F32, out_dtype=F32, prompt_tokens=W, prompt_offsets=W + 4096,
                         output_tokens=B, output_offsets=B + 4096, repetition=M, frequency=R,
                         presence=WS, bias_tokens=DW, bias_values=DW + 4096,
                         bias_offsets=DW + 8192, mask=DB, mask_stride=4, mask_rows=DX, n_masks=2)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.spmv_logits_process(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_requests=-1), INVALID), (dict(vocab=-1), INVALID), (dict(n_masks=-1), INVALID),
    (dict(dtype=4), INVALID), (dict(out_dtype=4), INVALID), (dict(logits=None), INVALID),
    (dict(out=None), INVALID), (dict(logits=X + 2), INVALID), (dict(out=Y + 2), INVALID),
    (dict(stride=-1), INVALID), (dict(out_stride=99), INVALID), (dict(out=X + 400), INVALID),
    (dict(out=X, out_stride=128), INVALID), (dict(prompt_offsets=None), INVALID),
    (dict(output_offsets=None), INVALID), (dict(bias_offsets=None), INVALID),
    (dict(bias_values=None), INVALID), (dict(prompt_offsets=W + 4), INVALID),
    (dict(bias_offsets=DW + 4), INVALID), (dict(prompt_tokens=W + 2), INVALID),
    (dict(repetition=M + 2), INVALID), (dict(mask=DB + 2), INVALID), (dict(mask_stride=-4), INVALID),
    (dict(mask_rows=DX + 1), INVALID),
    (dict(dtype=F16, out_dtype=BF16), UNSUPPORTED), (dict(dtype=F32, out_dtype=F16), UNSUPPORTED),
    (dict(n_requests=0), OK), (dict(vocab=0), OK),
])
def test_logits_refuses(spmv_lib, kw, status):
    assert logits(spmv_lib, **kw) == status


def test_logits_null_args(spmv_lib):
    assert spmv_lib.spmv_logits_process(None, None) == INVALID


def test_logits_struct_layout_matches_c(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    ct = _lib.spmv_logits
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "spmv.h"', 'int main(void) {',
             'printf("%zu\\n", sizeof(spmv_logits));']
    lines += [f'printf("%zu\\n", offsetof(spmv_logits, {f}));' for f, _ in ct._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(ct)] + [getattr(ct, f).offset for f, _ in ct._fields_]


def test_plans_refuse_bf16(spmv_lib):
    """The type that only these operators take is no matrix's."""
    import numpy as np
    h = S.api._host_csr(np.array([0, 1]), np.array([0]), np.ones(1, np.float16), 4)
    h.struct.value_dtype = BF16
    info = _lib.spmv_plan_info()
    assert spmv_lib.spmv_plan_inspect(ctypes.byref(h.struct), 0, None, ctypes.byref(info)) == INVALID


def _t(*size, dtype=torch.float32):
    return torch.zeros(*size, dtype=dtype)


@pytest.mark.parametrize("call,error", [
    (lambda: S.spmv_layernorm(_t(4, 8), None, None, _t(4, 8)), ValueError),       # not on a GPU
    (lambda: S.spmv_layernorm(_t(4, 8), None, None, _t(4, 7)), ValueError),       # shapes
    (lambda: S.spmv_layernorm(_t(8, 4).T, None, None, _t(4, 8)), ValueError),     # columns apart
    (lambda: S.spmv_layernorm(_t(2, 4, 8), None, None, _t(2, 4, 8)), ValueError),
    (lambda: S.spmv_layernorm_backward(_t(4, 8), _t(4, 8), None, None, None, _t(4, 8, dtype=torch.float16),
                                       None, None), TypeError),
    (lambda: S.spmv_layernorm_backward(_t(4, 8), _t(4, 7), None, None, None, None, None, None), ValueError),
    (lambda: S.spmv_adapters_run(_t(4, 8), _t(2, 3, 9), _t(2, 5, 3), _t(4), _t(4, 5)), ValueError),
    (lambda: S.spmv_adapters_run(_t(4, 8), _t(2, 3, 8), _t(2, 6, 3), _t(4), _t(4, 5)), ValueError),
    (lambda: S.spmv_adapters_run(_t(4, 8), _t(2, 3, 8, dtype=torch.float16), _t(2, 5, 3), _t(4), _t(4, 5)),
     TypeError),
    (lambda: S.spmv_adapters_run(_t(4, 8), _t(2, 3, 8), _t(2, 5, 3), None, _t(4, 5)), ValueError),
    (lambda: S.spmv_adapters_run(_t(4, 8), _t(2, 3, 8), _t(2, 5, 3), _t(4), _t(3, 5)), ValueError),
    (lambda: S.spmv_logits_process(_t(4, 8), _t(4, 9)), ValueError),
    (lambda: S.spmv_logits_process(_t(4, 8), _t(4, 8), mask=_t(4, 1)), TypeError),
    (lambda: S.spmv_logits_process(_t(4, 40), _t(4, 40), mask=_t(4, 1, dtype=torch.int32)), ValueError),
    (lambda: S.spmv_logits_process(_t(4, 8), _t(4, 8), mask=_t(3, 1, dtype=torch.int32)), ValueError),
    (lambda: S.spmv_logits_process(_t(4, 8), _t(4, 8), prompt=(_t(3), _t(5, dtype=torch.int64))), TypeError),
    (lambda: S.spmv_logits_process(_t(4, 8), _t(4, 8), prompt=(_t(3, dtype=torch.int32), _t(4, dtype=torch.int64))),
     ValueError),
])
def test_wrappers_refuse(spmv_lib, call, error):
    with pytest.raises(error):
        call()
