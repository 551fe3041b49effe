"""Host-side checks of the gate, embedding and vocabulary-loss calls in both
builds: argument errors return the documented status before any HIP call, and
empty problems return success without launching; and the binding's refusals
that need no GPU."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
F32, BF16 = 0, 1
A = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


def at(off):
    return ctypes.c_void_p(0x10000 + off)


@pytest.fixture(scope="module", params=["product", "checked"])
def L(request):
    import nvfp4_token_quantization_amd as nv
    return nv.load(nv.PRODUCT_LIB_PATH if request.param == "product" else nv.CHECKED_LIB_PATH)


def caller(f, order, good):
    return lambda **kw: f(*[dict(good, **kw)[k] for k in order.split()])


def test_gate(L):
    f = caller(L.nvfp4_moe_gate, "x e valid t n k norm w c s loss ws bytes stream",
               dict(x=A, e=A, valid=A, t=4, n=8, k=2, norm=1, w=A, c=A, s=A, loss=A, ws=A, bytes=1 << 30, stream=None))
    for kw in (dict(t=-1), dict(n=0), dict(k=0), dict(k=9), dict(x=None), dict(e=None), dict(w=None), dict(c=None), dict(s=None),
               dict(loss=None), dict(t=5000, ws=None), dict(t=5000, bytes=64), dict(bytes=-1)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=1025), dict(n=65, k=65), dict(t=1 << 30), dict(t=1 << 31, k=1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=at(2)), dict(e=at(1)), dict(w=at(2)), dict(c=at(2)), dict(s=at(1)), dict(loss=at(2)), dict(ws=at(8))):
        assert f(**kw) == MISALIGNED, kw
    assert f(t=0, x=None, e=None, w=None, c=None, s=None, loss=None) == OK
    w = L.nvfp4_moe_gate_workspace
    assert w(0, 8) == 0 and w(1, 8) == 0 and w(64, 128) == 0 and w(-1, 8) == 0 and w(5, 0) == 0
    assert w(65, 128) == 2 * (2 * 128 + 1) * 4 and w(1 << 24, 1021) == 256 * (2 * 1024 + 1) * 4


def test_gate_backward(L):
    f = caller(L.nvfp4_moe_gate_backward, "x e valid c t n k norm dw dl dx stream",
               dict(x=A, e=A, valid=None, c=A, t=4, n=8, k=2, norm=1, dw=A, dl=A, dx=A, stream=None))
    for kw in (dict(t=-1), dict(n=0), dict(k=0), dict(k=9), dict(x=None), dict(e=None), dict(dx=None), dict(dw=None, dl=None),
               dict(c=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=1025), dict(n=65, k=65), dict(t=1 << 30)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=at(2)), dict(e=at(1)), dict(c=at(2)), dict(dw=at(2)), dict(dl=at(2)), dict(dx=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(t=0, x=None, dx=None) == OK


def test_embedding(L):
    f = caller(L.nvfp4_embedding, "t tt vocab ids n d scale out ot stream",
               dict(t=A, tt=BF16, vocab=9, ids=A, n=4, d=16, scale=1.0, out=A, ot=F32, stream=None))
    for kw in (dict(tt=2), dict(ot=-1), dict(n=-1), dict(vocab=-1), dict(d=-1), dict(t=None), dict(ids=None), dict(out=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=(1 << 24) + 1), dict(d=(1 << 20) + 1), dict(vocab=(1 << 31) - 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(t=at(1)), dict(tt=F32, t=at(2)), dict(out=at(2)), dict(ids=at(2))):
        assert f(**kw) == MISALIGNED, kw
    assert f(n=0, ids=None, out=None) == OK
    assert f(d=0, t=None, out=None) == OK


def test_embedding_backward(L):
    f = caller(L.nvfp4_embedding_backward, "g gt ids n vocab d scale add out ot ws bytes stream",
               dict(g=A, gt=BF16, ids=A, n=4, vocab=9, d=16, scale=1.0, add=None, out=A, ot=F32, ws=A, bytes=1 << 30, stream=None))
    for kw in (dict(gt=2), dict(ot=2), dict(n=-1), dict(vocab=-1), dict(d=-1), dict(g=None), dict(ids=None), dict(out=None),
               dict(ws=None), dict(bytes=63), dict(bytes=-1)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=(1 << 24) + 1), dict(d=(1 << 20) + 1), dict(vocab=(1 << 31) - 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(g=at(1)), dict(out=at(2)), dict(add=at(2)), dict(ids=at(1)), dict(ws=at(8))):
        assert f(**kw) == MISALIGNED, kw
    assert f(vocab=0, out=None) == OK
    assert f(d=0, g=None, out=None) == OK
    assert f(n=0, add=A, ws=None, bytes=0, g=None, ids=None) == OK  # in place: nothing to do
    w = L.nvfp4_embedding_backward_workspace
    assert w(0, 16) == 0 and w(4, 0) == 0 and w(-1, 16) == 0 and w((1 << 24) + 1, 16) == 0
    assert w(4, 16) == 64 and w(20, 16) == 16 * 20 + 3 * 2 * 16 * 4


def test_vocab_loss(L):
    f = caller(L.nvfp4_vocab_loss, "h w t rows vocab k scale loss lse ws bytes stream",
               dict(h=A, w=A, t=A, rows=4, vocab=100, k=16, scale=1.0, loss=A, lse=A, ws=A, bytes=1 << 40, stream=None))
    for kw in (dict(rows=-1), dict(vocab=-1), dict(k=-8), dict(scale=NAN), dict(scale=INF), dict(h=None), dict(w=None), dict(t=None),
               dict(loss=None), dict(lse=None), dict(ws=None), dict(bytes=64)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(k=12), dict(k=(1 << 20) + 8), dict(vocab=(1 << 24) + 1), dict(rows=(1 << 24) + 1),
               dict(rows=1 << 24, vocab=1 << 24)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(h=at(8)), dict(w=at(8)), dict(t=at(2)), dict(loss=at(2)), dict(lse=at(1)), dict(ws=at(8))):
        assert f(**kw) == MISALIGNED, kw
    assert f(rows=0, h=None, t=None, loss=None, lse=None, ws=None, bytes=0) == OK
    w = L.nvfp4_vocab_loss_workspace
    assert w(0, 100, 16) == 0 and w(-1, 100, 16) == 0 and w(4, 100, 12) == 0 and 0 < w(4, 100, 16) < w(4, 1000, 16)


def test_vocab_loss_backward(L):
    f = caller(L.nvfp4_vocab_loss_backward, "h w t lse d rows vocab k scale add dh dw dwt ws bytes stream",
               dict(h=A, w=A, t=A, lse=A, d=A, rows=4, vocab=100, k=16, scale=1.0, add=None, dh=A, dw=A, dwt=F32, ws=A,
                    bytes=1 << 40, stream=None))
    for kw in (dict(rows=-1), dict(vocab=-1), dict(k=-8), dict(scale=NAN), dict(scale=-INF), dict(dwt=2), dict(h=None), dict(w=None),
               dict(t=None), dict(lse=None), dict(d=None), dict(dh=None, dw=None), dict(ws=None), dict(bytes=64)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(k=12), dict(vocab=(1 << 24) + 1), dict(rows=(1 << 24) + 1), dict(rows=1 << 24, vocab=1 << 24),
               dict(vocab=1 << 24, k=1 << 20)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(h=at(8)), dict(w=at(4)), dict(t=at(2)), dict(lse=at(2)), dict(d=at(1)), dict(add=at(8)), dict(dh=at(8)),
               dict(dw=at(4)), dict(ws=at(8))):
        assert f(**kw) == MISALIGNED, kw
    assert f(k=0, h=None, w=None) == OK
    assert f(rows=0, dw=None, ws=None, bytes=0) == OK
    w = L.nvfp4_vocab_loss_backward_workspace
    assert w(0, 100, 16) == 16 and w(-1, 100, 16) == 0 and w(4, 100, 12) == 0
    # dz of a piece, never of the whole of a large problem
    assert w(8192, 131072, 2048) < 2 * 8192 * 131072


def test_binding_refusals():
    import nvfp4_token_quantization_amd as nv
    x, i = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    b, t = x.to(torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: nv.nvfp4_moe_gate(x, i), lambda: nv.nvfp4_moe_gate_backward(x, i, d_weights=x[:, :2]),
                lambda: nv.nvfp4_embedding(x, t), lambda: nv.nvfp4_embedding_backward(x, t, 9),
                lambda: nv.nvfp4_vocab_loss(b, b, t), lambda: nv.nvfp4_vocab_loss_backward(b, b, t, x[0, :4], x[0, :4])):
        with pytest.raises(ValueError, match="GPU"):
            bad()
    for bad in (lambda: nv.nvfp4_moe_gate([1], i), lambda: nv.nvfp4_embedding(None, t), lambda: nv.nvfp4_vocab_loss(b, 3, t)):
        with pytest.raises((TypeError, ValueError)):
            bad()


def test_sizes_past_what_a_launch_holds(L):
    f = caller(L.nvfp4_embedding_backward, "g gt ids n vocab d scale add out ot ws bytes stream",
               dict(g=A, gt=BF16, ids=A, n=4, vocab=9, d=16, scale=1.0, add=None, out=A, ot=F32, ws=A, bytes=1 << 60, stream=None))
    assert f(vocab=(1 << 29) + 1) == SHAPE
    assert f(n=1 << 24, d=1 << 20) == SHAPE
    f = caller(L.nvfp4_vocab_loss, "h w t rows vocab k scale loss lse ws bytes stream",
               dict(h=A, w=A, t=A, rows=1 << 20, vocab=1 << 20, k=16, scale=1.0, loss=A, lse=A, ws=A, bytes=1 << 60, stream=None))
    assert f() == SHAPE  # 2^24 tiles of 256 x 256
    f = caller(L.nvfp4_vocab_loss_backward, "h w t lse d rows vocab k scale add dh dw dwt ws bytes stream",
               dict(h=A, w=A, t=A, lse=A, d=A, rows=4, vocab=100, k=16, scale=1.0, add=None, dh=A, dw=A, dwt=F32, ws=A,
                    bytes=1 << 60, stream=None))
    assert f(rows=1 << 20, vocab=1 << 20) == SHAPE
    assert f(rows=1 << 24, k=1 << 20) == SHAPE
