"""Host-side checks of the learner's calls (grouped bf16 products, residual
norms, expert combine, gradient clipping) in both builds: argument errors
return the documented status before any HIP call, and empty problems return
success without launching; and the binding's refusals that need no GPU."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
F32, BF16 = 0, 1
A = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced


def at(off):
    return ctypes.c_void_p(0x10000 + off)


@pytest.fixture(scope="module", params=["product", "checked"])
def L(request):
    import nvfp4_token_quantization_amd as nv
    return nv.load(nv.PRODUCT_LIB_PATH if request.param == "product" else nv.CHECKED_LIB_PATH)


def status(f, order, good, **kw):
    return f(*[dict(good, **kw)[k] for k in order.split()])


def test_grouped_forward(L):
    order = "x a_rows index m off groups w n k y type stream"
    good = dict(x=A, a_rows=8, index=None, m=8, off=A, groups=2, w=A, n=16, k=24, y=A, type=F32, stream=None)

    def f(**kw):
        return status(L.nvfp4_bf16_grouped_gemm, order, good, **kw)
    for kw in (dict(groups=0), dict(m=-1), dict(a_rows=-1), dict(n=-8), dict(k=-8), dict(type=2), dict(off=None),
               dict(x=None), dict(w=None), dict(y=None), dict(m=9)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(groups=1025), dict(n=12), dict(k=20), dict(n=(1 << 20) + 8), dict(k=(1 << 20) + 8), dict(m=1 << 31, a_rows=1 << 31),
               dict(index=A, a_rows=1 << 26, k=16), dict(m=(1 << 31) - 8, a_rows=(1 << 31) - 8, n=1 << 20)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=at(8)), dict(w=at(2)), dict(y=at(4)), dict(off=at(2)), dict(index=at(1))):
        assert f(**kw) == MISALIGNED, kw
    assert f(m=0, x=None, w=None, y=None) == OK
    assert f(n=0, w=None, y=None) == OK


def test_grouped_dgrad(L):
    order = "dy m off groups w n k dx type stream"
    good = dict(dy=A, m=8, off=A, groups=2, w=A, n=16, k=24, dx=A, type=BF16, stream=None)

    def f(**kw):
        return status(L.nvfp4_bf16_grouped_dgrad, order, good, **kw)
    for kw in (dict(groups=0), dict(m=-1), dict(type=-1), dict(off=None), dict(dy=None), dict(w=None), dict(dx=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(groups=1025), dict(n=12), dict(k=20), dict(m=1 << 31)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dy=at(8)), dict(w=at(2)), dict(dx=at(4)), dict(off=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(m=0, dy=None, dx=None) == OK
    assert f(k=0, dx=None) == OK


def test_grouped_wgrad(L):
    order = "dy m x a_rows index off groups n k add dw type stream"
    good = dict(dy=A, m=8, x=A, a_rows=8, index=None, off=A, groups=2, n=16, k=24, add=None, dw=A, type=F32, stream=None)

    def f(**kw):
        return status(L.nvfp4_bf16_grouped_wgrad, order, good, **kw)
    for kw in (dict(groups=0), dict(m=-1), dict(type=3), dict(off=None), dict(dy=None), dict(x=None), dict(dw=None),
               dict(a_rows=7)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(groups=1025), dict(n=12), dict(k=20), dict(index=A, a_rows=1 << 26, k=16),
               dict(groups=1024, n=1 << 20, k=1 << 20)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dy=at(8)), dict(x=at(8)), dict(add=at(4)), dict(dw=at(4)), dict(off=at(2)), dict(index=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(n=0, dw=None) == OK


NORM = "x xt r rt w1 g grows w2 pt rows d scale eps rout h amax q sb s stream"
NORM_GOOD = dict(x=A, xt=F32, r=A, rt=BF16, w1=A, g=A, grows=0, w2=A, pt=F32, rows=4, d=32, scale=1.0, eps=1e-6, rout=A,
                 h=A, amax=None, q=None, sb=None, s=None, stream=None)


def test_residual_norm(L):
    def f(**kw):
        return status(L.nvfp4_residual_norm, NORM, NORM_GOOD, **kw)
    q = dict(q=A, sb=A, s=A)
    for kw in (dict(rows=-1), dict(d=0), dict(xt=2), dict(rt=2), dict(pt=9), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(scale=float("nan")), dict(x=None), dict(q=A), dict(q=A, sb=A), dict(s=A),
               dict(rout=None, h=None), dict(w2=None), dict(w2=None, h=None, amax=A), dict(g=None, grows=1)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(d=16385), dict(d=24, **q), dict(rows=(1 << 31) + 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=at(2)), dict(r=at(1)), dict(rout=at(1)), dict(w1=at(2)), dict(g=at(2)), dict(w2=at(2)), dict(h=at(1)),
               dict(amax=at(2)), dict(q, q=at(8)), dict(q, x=at(4)), dict(q, h=at(2)), dict(q, s=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(rows=0, x=None) == OK


def test_residual_norm_backward(L):
    order = "x xt r rt w1 g grows w2 pt dh dr rows d scale eps dx dxt drin dw1 dg dw2 ws bytes stream"
    good = dict(x=A, xt=F32, r=A, rt=BF16, w1=A, g=A, grows=0, w2=A, pt=F32, dh=A, dr=A, rows=4, d=32, scale=1.0, eps=1e-6,
                dx=A, dxt=BF16, drin=A, dw1=A, dg=A, dw2=A, ws=A, bytes=1 << 30, stream=None)

    def f(**kw):
        return status(L.nvfp4_residual_norm_backward, order, good, **kw)
    for kw in (dict(rows=-1), dict(d=0), dict(xt=2), dict(rt=2), dict(pt=2), dict(dxt=2), dict(eps=-1.0), dict(w1=None),
               dict(w2=None), dict(g=None), dict(x=None), dict(dx=None), dict(dh=None, dr=None), dict(r=None),
               dict(g=None, dg=None, grows=1)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(d=16385), dict(rows=(1 << 31) + 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=at(2)), dict(r=at(1)), dict(dr=at(1)), dict(drin=at(1)), dict(w1=at(2)), dict(dh=at(1)), dict(dx=at(1)),
               dict(dw1=at(2)), dict(dw2=at(2)), dict(dg=at(2)), dict(ws=at(8))):
        assert f(**kw) == MISALIGNED, kw
    assert f(rows=0, dw1=None, dw2=None, dg=None) == OK
    w = L.nvfp4_residual_norm_backward_workspace
    assert w(0, 32) == 0 and w(4, 0) == 0 and w(4, 32) == 4 * 2 * 32 * 4
    assert w(1 << 20, 2560) < 1 << 27


def test_moe_combine(L):
    order = "y yt yrows slot p tokens topk d out ot stream"
    good = dict(y=A, yt=F32, yrows=8, slot=A, p=A, tokens=4, topk=2, d=32, out=A, ot=BF16, stream=None)

    def f(**kw):
        return status(L.nvfp4_moe_combine, order, good, **kw)
    for kw in (dict(yt=2), dict(ot=2), dict(yrows=-1), dict(tokens=-1), dict(topk=0), dict(d=-1), dict(y=None), dict(slot=None),
               dict(out=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(topk=65), dict(tokens=1 << 31), dict(d=(1 << 24) + 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(y=at(2)), dict(out=at(1)), dict(slot=at(2)), dict(p=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(tokens=0, slot=None, out=None) == OK
    assert f(d=0, y=None, out=None) == OK


def test_moe_combine_backward(L):
    order = "dout dt y yt yrows slot p tokens topk d dy dyt dp stream"
    good = dict(dout=A, dt=BF16, y=A, yt=F32, yrows=8, slot=A, p=A, tokens=4, topk=2, d=32, dy=A, dyt=BF16, dp=A, stream=None)

    def f(**kw):
        return status(L.nvfp4_moe_combine_backward, order, good, **kw)
    for kw in (dict(dt=2), dict(yt=2), dict(dyt=2), dict(tokens=-1), dict(topk=0), dict(dout=None), dict(y=None),
               dict(slot=None), dict(dy=None, dp=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(topk=65), dict(tokens=1 << 31)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dout=at(1)), dict(y=at(2)), dict(dy=at(1)), dict(slot=at(2)), dict(p=at(2)), dict(dp=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(tokens=0, dout=None) == OK


def test_clip_grad_norm(L):
    f = L.nvfp4_clip_grad_norm

    def arrays(ptr=0x10000, count=5, kind=F32, out=0x20000):
        return ((ctypes.c_void_p * 1)(ptr), None if out is None else (ctypes.c_void_p * 1)(out), (ctypes.c_int64 * 1)(count),
                (ctypes.c_int32 * 1)(kind))

    def call(tensors=1, max_norm=1.0, norm=A, ws=A, size=1 << 20, **kw):
        return f(*arrays(**kw), tensors, max_norm, norm, ws, size, None)
    for kw in (dict(tensors=-1), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(count=-1), dict(kind=2), dict(ptr=None),
               dict(out=0), dict(out=None, norm=None), dict(ws=None), dict(size=64)):
        assert call(**kw) == INVALID, kw
    assert f(None, None, None, None, 1, 1.0, A, A, 1 << 20, None) == INVALID
    assert call(count=(1 << 36) + 1) == SHAPE
    for kw in (dict(ptr=0x10002), dict(out=0x20002), dict(ptr=0x10001, kind=BF16), dict(norm=at(2)), dict(ws=at(4))):
        assert call(**kw) == MISALIGNED, kw
    w = L.nvfp4_clip_grad_norm_workspace
    assert w(0) == 0 and 0 < w(1) == w(2) <= w(1000)


def test_binding_refuses_cpu_tensors_and_overlaps():
    import nvfp4_token_quantization_amd as nv
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    i32 = torch.zeros(4, 1, dtype=torch.int32)
    for bad in (lambda: nv.nvfp4_bf16_grouped_gemm(x, i32, x), lambda: nv.nvfp4_residual_norm(x, x),
                lambda: nv.nvfp4_moe_combine(x, i32), lambda: nv.nvfp4_clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError):
            bad()
    nv._disjoint([0, 32], [64, 32], [32, 32])
    nv._disjoint([0, 16], [64, 64], [32, 0])
    for grads, outs in (([0, 16], None), ([0, 0], None), ([0, 32], [32, 0]), ([0, 32], [64, 80]), ([0, 32], [16, 128]),
                        ([0, 64], [64, 128])):
        with pytest.raises(ValueError):
            nv._disjoint(grads, grads if outs is None else outs, [32, 32])


def test_binding_finds_outputs_in_one_memory():
    import nvfp4_token_quantization_amd as nv
    buf = torch.zeros(64)
    nv._no_overlap(buf[:32], "out", buf[32:], None, buf[:0])
    nv._no_overlap(buf[:0], "out", buf)
    for other in (buf, buf[31:], buf[:1], buf.view(torch.uint8)[127:128]):
        with pytest.raises(ValueError):
            nv._no_overlap(buf[:32], "out", other)
