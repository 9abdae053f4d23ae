"""CPU tests of the operators that put a pruned model beside the dense one it
came from: what the C entry points and the Python wrappers refuse (validation
comes before any device call), and their workspace sizes. Nothing here
launches a kernel."""
import pytest

import sparse_matrix_vector_gb300 as S

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, TOO_LARGE = 0, 1, 5, 8
F32, F16, BF16 = 0, 1, 2
# made-up 16-byte aligned addresses far apart: refused calls never read them
X, W, SC, Z, B, Y, WS, A1, A2, A3, A4, A5 = (0x10000000 * k for k in range(1, 13))
HUGE = 2 ** 31 - 1


def int4(lib, **kw):
    a = dict(t=4, i=256, o=32, g=64, dt=F16, x=X, xs=256, w=W, ws=128, sc=SC, st=F32, z=Z, b=B, bs=32, y=Y, yt=F32, ys=32, wk=WS,
             wn=1 << 40)
    a.update(kw)
    return lib.spmv_int4_run(a["t"], a["i"], a["o"], a["g"], a["dt"], a["x"], a["xs"], a["w"], a["ws"], a["sc"], a["st"], a["z"], a["b"],
                             a["bs"], a["y"], a["yt"], a["ys"], a["wk"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(wk=None), INVALID), (dict(wn=64), INVALID), (dict(wk=WS + 8), INVALID), (dict(wk=Y), INVALID), (dict(wk=X), INVALID), (dict(wk=W), INVALID),
    (dict(t=-1), INVALID), (dict(i=-1), INVALID), (dict(o=-1), INVALID), (dict(g=0), INVALID), (dict(g=-32), INVALID),
    (dict(dt=4), INVALID), (dict(st=-1), INVALID), (dict(yt=9), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(sc=None), INVALID), (dict(y=None), INVALID), (dict(x=X + 1), INVALID), (dict(sc=SC + 2), INVALID), (dict(b=B + 2), INVALID),
    (dict(y=Y + 2), INVALID), (dict(xs=-1), INVALID), (dict(ws=-1), INVALID), (dict(ys=31), INVALID), (dict(ys=0), INVALID),
    (dict(bs=-1), INVALID), (dict(b=Y + 64), INVALID), (dict(b=Y, bs=64), INVALID), (dict(x=Y), INVALID), (dict(w=Y + 16), INVALID),
    (dict(sc=Y), INVALID), (dict(z=Y + 3), INVALID), (dict(wk=SC), INVALID), (dict(wk=Z), INVALID), (dict(wk=B), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(yt=BF16), UNSUPPORTED), (dict(st=BF16), UNSUPPORTED), (dict(dt=BF16, yt=F16), UNSUPPORTED),
    (dict(g=16), UNSUPPORTED), (dict(g=48), UNSUPPORTED), (dict(g=255), UNSUPPORTED), (dict(g=96), UNSUPPORTED),
    (dict(t=2 ** 18 + 1), TOO_LARGE), (dict(i=2 ** 30 + 1, g=HUGE), TOO_LARGE), (dict(o=2 ** 30 + 1), TOO_LARGE),
    (dict(t=0), OK), (dict(o=0), OK), (dict(t=0, x=None, w=W, y=None, b=None), OK),
])
def test_int4_refuses(spmv_lib, kw, status):
    assert int4(spmv_lib, **kw) == status


def test_int4_workspace(spmv_lib):
    size = S.spmv_int4_workspace
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 0) == 0 and size(4, -64) == 0
    assert size(2 ** 32 + 4, 64) == 0 and size(4, 2 ** 32 + 64) == 0 and size(2 ** 18 + 1, 64) == 0
    n = size(4, 256)
    assert n > 0 and int4(spmv_lib, wn=n - 1) == INVALID


def verify(lib, **kw):
    a = dict(n=3, d=5, v=100, dt=F32, t=X, ts=100, q=W, qs=100, tok=SC, off=Z, au=B, su=A1, temp=A2, out=Y, acc=A3, ws=WS, wn=1 << 40)
    a.update(kw)
    return lib.spmv_verify_drafts(a["n"], a["d"], a["v"], a["dt"], a["t"], a["ts"], a["q"], a["qs"], a["tok"], a["off"], a["au"], a["su"],
                                  a["temp"], a["out"], a["acc"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(d=-1), INVALID), (dict(v=0), INVALID), (dict(dt=3), INVALID), (dict(t=None), INVALID),
    (dict(tok=None), INVALID), (dict(off=None), INVALID), (dict(au=None), INVALID), (dict(su=None), INVALID), (dict(out=None), INVALID),
    (dict(acc=None), INVALID), (dict(ws=None), INVALID), (dict(wn=16), INVALID), (dict(ws=WS + 8), INVALID), (dict(t=X + 2), INVALID),
    (dict(q=W + 1), INVALID), (dict(tok=SC + 2), INVALID), (dict(off=Z + 4), INVALID), (dict(au=B + 1), INVALID), (dict(su=A1 + 2), INVALID),
    (dict(temp=A2 + 3), INVALID), (dict(out=Y + 1), INVALID), (dict(acc=A3 + 2), INVALID), (dict(ts=-1), INVALID), (dict(qs=-100), INVALID),
    (dict(out=X), INVALID), (dict(acc=W + 400), INVALID), (dict(out=SC + 4), INVALID), (dict(out=Z), INVALID), (dict(acc=A1), INVALID),
    (dict(acc=A2), INVALID), (dict(out=B), INVALID), (dict(acc=Y + 8), INVALID), (dict(out=WS + 16), INVALID), (dict(ws=X), INVALID),
    (dict(v=HUGE, ts=2 ** 32, qs=2 ** 32), TOO_LARGE), (dict(n=2 ** 24, d=2 ** 24), TOO_LARGE), (dict(n=2 ** 23, v=2 ** 30), TOO_LARGE),
    (dict(n=0), OK), (dict(n=0, d=0, t=None, q=None, tok=None, off=None, au=None, su=None, out=None, acc=None, ws=None, wn=0), OK),
])
def test_verify_refuses(spmv_lib, kw, status):
    assert verify(spmv_lib, **kw) == status


def test_verify_workspace(spmv_lib):
    size = S.spmv_verify_workspace
    assert size(0, 0, 100) == 0 and size(-1, 4, 100) == 0 and size(3, -1, 100) == 0 and size(3, 4, 0) == 0
    assert size(2 ** 32 + 3, 4, 100) == 0 and size(3, 2 ** 32 + 4, 100) == 0 and size(3, 4, 2 ** 32 + 100) == 0
    n = size(3, 5, 100)
    assert n > 0 and verify(spmv_lib, wn=n - 1) == INVALID
    assert size(64, 400, 128000) >= size(64, 400, 1000)


def distill(lib, **kw):
    a = dict(n=4, v=100, z=X, dt=BF16, zs=100, k=8, ids=W, is_=8, t=SC, tt=F32, ts=8, sums=Z, temp=1.0, loss=Y, stats=A1)
    a.update(kw)
    return lib.spmv_distill(a["n"], a["v"], a["z"], a["dt"], a["zs"], a["k"], a["ids"], a["is_"], a["t"], a["tt"], a["ts"], a["sums"],
                            a["temp"], a["loss"], a["stats"], None)


COMMON = [
    (dict(n=-1), INVALID), (dict(v=0), INVALID), (dict(v=-5), INVALID), (dict(k=-1), INVALID), (dict(dt=3), INVALID), (dict(tt=-2), INVALID),
    (dict(z=None), INVALID), (dict(ids=None), INVALID), (dict(t=None), INVALID), (dict(z=X + 1), INVALID), (dict(ids=W + 2), INVALID),
    (dict(t=SC + 2), INVALID), (dict(sums=Z + 1), INVALID), (dict(stats=A1 + 2), INVALID), (dict(zs=-1), INVALID), (dict(is_=-8), INVALID),
    (dict(ts=-1), INVALID), (dict(temp=0.0), INVALID), (dict(temp=-1.0), INVALID), (dict(temp=float("nan")), INVALID),
    (dict(temp=float("inf")), INVALID), (dict(temp=1e-45), INVALID), (dict(temp=1e-39), INVALID),
    (dict(k=1025, is_=1025, ts=1025), TOO_LARGE), (dict(n=2 ** 27 + 1), TOO_LARGE), (dict(v=HUGE), TOO_LARGE),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(loss=None), INVALID), (dict(loss=Y + 1), INVALID), (dict(loss=X + 8), INVALID), (dict(loss=W), INVALID), (dict(loss=SC + 4), INVALID),
    (dict(loss=Z), INVALID), (dict(stats=X), INVALID), (dict(stats=W + 4), INVALID), (dict(stats=Z), INVALID), (dict(stats=Y + 4), INVALID),
    (dict(n=0), OK), (dict(n=0, z=None, ids=None, t=None, sums=None, loss=None, stats=None), OK),
])
def test_distill_refuses(spmv_lib, kw, status):
    assert distill(spmv_lib, **kw) == status


def distill_backward(lib, **kw):
    a = dict(n=4, v=100, dl=B, dls=1, z=X, dt=BF16, zs=100, k=8, ids=W, is_=8, t=SC, tt=F32, ts=8, sums=Z, temp=1.0, stats=A1, out=Y, os=100)
    a.update(kw)
    return lib.spmv_distill_backward(a["n"], a["v"], a["dl"], a["dls"], a["z"], a["dt"], a["zs"], a["k"], a["ids"], a["is_"], a["t"], a["tt"],
                                     a["ts"], a["sums"], a["temp"], a["stats"], a["out"], a["os"], None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dl=None), INVALID), (dict(dl=B + 2), INVALID), (dict(dls=-1), INVALID), (dict(stats=None), INVALID), (dict(out=None), INVALID),
    (dict(out=Y + 1), INVALID), (dict(os=99), INVALID), (dict(os=0), INVALID), (dict(out=X + 16), INVALID), (dict(out=X, os=128), INVALID),
    (dict(out=W), INVALID), (dict(out=SC), INVALID), (dict(out=Z), INVALID), (dict(out=A1), INVALID), (dict(out=B), INVALID),
    (dict(n=0), OK),
])
def test_distill_backward_refuses(spmv_lib, kw, status):
    assert distill_backward(spmv_lib, **kw) == status


# ------------------------------------------------------- the Python wrappers

def _t(*size, dtype=torch.float32):
    return torch.empty(*size, dtype=dtype)


def _int4(**kw):
    a = dict(x=_t(2, 256, dtype=torch.float16), weights=_t(8, 128, dtype=torch.uint8), scales=_t(8, 4), y=_t(2, 8), group=64)
    a.update(kw)
    S.spmv_int4_run(**a)


def _verify(**kw):
    a = dict(target=_t(8, 50), draft=_t(5, 50), draft_tokens=_t(5, dtype=torch.int32), offsets=_t(4, dtype=torch.int64), accept_uniforms=_t(5),
             sample_uniforms=_t(3), tokens=_t(8, dtype=torch.int32), accepted=_t(3, dtype=torch.int32))
    a.update(kw)
    S.spmv_verify_drafts(**a)


def _distill(**kw):
    a = dict(logits=_t(4, 50), top_tokens=_t(4, 6, dtype=torch.int32), top_logits=_t(4, 6), loss=_t(4))
    a.update(kw)
    S.spmv_distill(**a)


def _distill_backward(**kw):
    a = dict(dloss=_t(4), logits=_t(4, 50), top_tokens=_t(4, 6, dtype=torch.int32), top_logits=_t(4, 6), stats=_t(4, 3), dlogits=_t(4, 50))
    a.update(kw)
    S.spmv_distill_backward(**a)


@pytest.mark.parametrize("call,error", [
    (lambda: _int4(y=_t(3, 8)), ValueError), (lambda: _int4(weights=_t(8, 128)), TypeError), (lambda: _int4(weights=_t(8, 127, dtype=torch.uint8)), ValueError),
    (lambda: _int4(weights=_t(7, 128, dtype=torch.uint8)), ValueError), (lambda: _int4(scales=_t(8, 3)), ValueError),
    (lambda: _int4(scales=_t(8, 8)[:, ::2]), ValueError), (lambda: _int4(group=0), ValueError), (lambda: _int4(base=_t(2, 7)), ValueError),
    (lambda: _int4(base=_t(2, 8, dtype=torch.float16)), TypeError), (lambda: _int4(x=_t(256, 2, dtype=torch.float16).T), ValueError),
    (lambda: _int4(), ValueError),  # not CUDA tensors
    (lambda: _verify(target=_t(7, 50)), ValueError), (lambda: _verify(draft=_t(4, 50)), ValueError), (lambda: _verify(draft=_t(5, 51)), ValueError),
    (lambda: _verify(draft=_t(5, 50, dtype=torch.float16)), TypeError), (lambda: _verify(offsets=_t(0, dtype=torch.int64)), ValueError),
    (lambda: _verify(sample_uniforms=None), ValueError), (lambda: _verify(tokens=None), ValueError), (lambda: _verify(), ValueError),
    (lambda: _distill(top_tokens=_t(4, 6)), TypeError), (lambda: _distill(top_logits=_t(4, 5)), ValueError), (lambda: _distill(loss=None), ValueError),
    (lambda: _distill(top_tokens=_t(3, 6, dtype=torch.int32)), ValueError), (lambda: _distill(), ValueError),
    (lambda: _distill_backward(dlogits=_t(4, 49)), ValueError), (lambda: _distill_backward(dlogits=_t(4, 50, dtype=torch.float16)), TypeError),
    (lambda: _distill_backward(dloss=_t(3)), ValueError), (lambda: _distill_backward(dloss=_t(4, dtype=torch.float16)), TypeError),
    (lambda: _distill_backward(stats=None), ValueError), (lambda: _distill_backward(), ValueError),
])
def test_wrappers_refuse(spmv_lib, call, error):
    with pytest.raises(error):
        call()


def _meta(*size, dtype=torch.float16):
    return torch.empty(*size, dtype=dtype, device="meta")


FAR = 2 ** 32 + 8  # (cut to 8 by a 32-bit argument)
U8, I32, I64 = torch.uint8, torch.int32, torch.int64


@pytest.mark.parametrize("call", [
    lambda: S.spmv_int4_run(_meta(2, FAR), _meta(5, FAR // 2, dtype=U8), _meta(5, 1), _meta(2, 5), FAR),
    lambda: S.spmv_int4_run(_meta(2, 64), _meta(FAR, 32, dtype=U8), _meta(FAR, 1), _meta(2, FAR), 64),
    lambda: S.spmv_int4_run(_meta(FAR, 64), _meta(5, 32, dtype=U8), _meta(5, 1), _meta(FAR, 5), 64),
    lambda: S.spmv_verify_drafts(_meta(3, FAR), None, _meta(2, dtype=I32), _meta(2, dtype=I64), None, None, None, None),
    lambda: S.spmv_verify_drafts(_meta(FAR + 1, 8), None, _meta(FAR, dtype=I32), _meta(2, dtype=I64), None, None, None, None),
    lambda: S.spmv_distill(_meta(2, FAR), _meta(2, 3, dtype=I32), _meta(2, 3), _meta(2)),
    lambda: S.spmv_distill(_meta(2, 8), _meta(2, FAR, dtype=I32), _meta(2, FAR), _meta(2)),
    lambda: S.spmv_distill_backward(_meta(2), _meta(2, FAR), _meta(2, 3, dtype=I32), _meta(2, 3), None, _meta(2, FAR)),
])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(S.SpmvError) as e:
        call()
    assert e.value.status == TOO_LARGE
