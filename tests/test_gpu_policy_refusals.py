"""What the binding refuses of the gate, embedding and vocabulary-loss calls
before anything is launched, on device tensors."""
import pytest
import torch

import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
DEV = "cuda:0"


def z(*s, dtype=F32):
    return torch.zeros(*s, dtype=dtype, device=DEV)


def refused(f, *kinds):
    with pytest.raises(kinds or (ValueError, TypeError)):
        f()


def test_gate():
    x, e = z(6, 8), z(6, 2, dtype=I32)
    c, dw, dl = z(9, dtype=I32), z(6, 2), z(1)[0]
    G, B = nv.nvfp4_moe_gate, nv.nvfp4_moe_gate_backward
    refused(lambda: G(x.double(), e), TypeError)
    refused(lambda: G(x.t(), e), ValueError)
    refused(lambda: G(x, e.long()), TypeError)
    refused(lambda: G(x, e[:5]), ValueError)
    refused(lambda: G(x, e, valid=z(6)), TypeError)
    refused(lambda: G(x, e, valid=z(5, dtype=torch.bool)), ValueError)
    refused(lambda: G(x, z(6, 9, dtype=I32)), nv.NVFP4Error)
    refused(lambda: G(x, e, out={"weight": dw}), ValueError)
    refused(lambda: G(x, e, out={"weights": x[:, :2]}), ValueError)
    refused(lambda: G(x, e, out={"prob_sums": x.view(-1)[:8]}), ValueError)
    buf = z(9)
    refused(lambda: G(x, e, out={"prob_sums": buf[:8], "loss": buf[7]}), ValueError)
    big, be = z(5000, 8), z(5000, 2, dtype=I32)
    refused(lambda: G(big, be, workspace=z(8, dtype=torch.uint8)), nv.NVFP4Error)
    refused(lambda: G(big, be, workspace=z(1 << 20)), TypeError)
    refused(lambda: B(x, e, c), ValueError)
    refused(lambda: B(x, e, d_loss=dl), ValueError)
    refused(lambda: B(x, e, c[:8], d_loss=dl), ValueError)
    refused(lambda: B(x, e, c, d_loss=z(2)), ValueError)
    refused(lambda: B(x, e, c, d_weights=dw[:5]), ValueError)
    refused(lambda: B(x, e, c, d_weights=dw, out=x), ValueError)
    refused(lambda: B(x, e, c, d_weights=dw, out=z(6, 7)), ValueError)


def test_embedding():
    t, ids, g = z(9, 16), z(5, dtype=I32), z(5, 16)
    F, B = nv.nvfp4_embedding, nv.nvfp4_embedding_backward
    refused(lambda: F(t.half(), ids), TypeError)
    refused(lambda: F(t, ids.long()), TypeError)
    refused(lambda: F(t.t(), ids), ValueError)
    refused(lambda: F(t, ids, out_dtype=torch.float16), TypeError)
    refused(lambda: F(t, ids, out=t[:5]), ValueError)
    refused(lambda: F(t, ids, out=z(5, 15)), ValueError)
    refused(lambda: B(g[:4], ids, 9), ValueError)
    refused(lambda: B(g, ids, -1), ValueError)
    refused(lambda: B(g, ids, 9, add=z(8, 16)), ValueError)
    refused(lambda: B(g, ids, 9, add=t.to(BF16), out=t), TypeError)
    refused(lambda: B(g, ids, 5, out=g), ValueError)
    buf = z(12, 16)
    refused(lambda: B(g, ids, 9, add=buf[:9], out=buf[1:10]), ValueError)
    refused(lambda: B(g, ids, 9, workspace=z(8, dtype=torch.uint8)), nv.NVFP4Error)
    ws = z(1 << 16, dtype=torch.uint8)
    refused(lambda: B(g, ids, 9, out=ws[:576].view(F32).view(9, 16), workspace=ws), ValueError)


def test_vocab_loss():
    h, w, t, v = z(6, 16, dtype=BF16), z(40, 16, dtype=BF16), z(6, dtype=I32), z(6)
    F, B = nv.nvfp4_vocab_loss, nv.nvfp4_vocab_loss_backward
    refused(lambda: F(h.float(), w, t), TypeError)
    refused(lambda: F(h, w[:, :8].contiguous(), t), ValueError)
    refused(lambda: F(h, w, t[:5]), ValueError)
    refused(lambda: F(h, w, t.long()), TypeError)
    refused(lambda: F(h, w, t, scale=float("nan")), nv.NVFP4Error)
    refused(lambda: F(z(6, 12, dtype=BF16), z(4, 12, dtype=BF16), t), nv.NVFP4Error)
    refused(lambda: F(h, w, t, out={"nll": v}), ValueError)
    refused(lambda: F(h, w, t, out={"loss": v, "lse": v}), ValueError)
    refused(lambda: F(h, w, t, workspace=z(16, dtype=torch.uint8)), nv.NVFP4Error)
    refused(lambda: B(h, w, t, v[:5], v), ValueError)
    refused(lambda: B(h, w, t, v, v.double()), TypeError)
    refused(lambda: B(h, w, t, v, v, want_dh=False, want_dw=False), ValueError)
    refused(lambda: B(h, w, t, v, v, want_dw=False, add=z(40, 16)), ValueError)
    refused(lambda: B(h, w, t, v, v, add=z(39, 16)), ValueError)
    refused(lambda: B(h, w, t, v, v, dw_dtype=torch.float16), TypeError)
    refused(lambda: B(h, w, t, v, v, add=z(40, 16), out={"dw": z(40, 16, dtype=BF16)}), TypeError)
    refused(lambda: B(h, w, t, v, v, out={"dh": h}), ValueError)
    refused(lambda: B(h, w, t, v, v, out={"dw": w}), ValueError)
    buf = z(41, 16)
    refused(lambda: B(h, w, t, v, v, add=buf[:40], out={"dw": buf[1:]}), ValueError)
    refused(lambda: B(h, w, t, v, v, workspace=z(16, dtype=torch.uint8)), nv.NVFP4Error)
    # and a call that none of these spoiled
    assert (F(h, w, t)["loss"] > 3).all()
