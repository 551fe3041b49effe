"""The learner's operators as they are used together: one mixture-of-experts
block, forward and backward, with the router, the quantizers and the NVFP4
products around them.

  x = residual + gate * norm(attention output);  h = norm(x)     (quantized too)
  route h, up-projection, SwiGLU, down-projection, sum over experts
  x' = x + gate * norm(that sum)

and back to every gradient (dequantized backward: the gradients go through the
bf16 values of the quantized weights), then clipping.  The reference is the
same chain in 64 bits with autograd, on the chain's own rounded activations.
"""
import pytest
import torch

import learner_refs as ref
import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
T, D, F, E, K, EPS = 300, 256, 128, 16, 4, 1e-6


def inputs(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0, mean=0.0):
        return torch.randn(*s, generator=g) * std + mean
    w = {"attn": n(T, D), "residual": n(T, D), "w_post": n(D, std=0.1, mean=1.0), "w_pre": n(D, std=0.1, mean=1.0),
         "gate": n(D, std=0.2, mean=0.5), "w_post2": n(D, std=0.1, mean=1.0), "gate2": n(D, std=0.2, mean=0.5),
         "logits": n(T, E)}
    w = {k: v.to(DEV) for k, v in w.items()}
    w["residual"] = w["residual"].to(BF16)
    w["up"] = n(E, 2 * F, D, std=0.06).to(BF16).to(DEV)
    w["down"] = n(E, D, F, std=0.09).to(BF16).to(DEV)
    w["d_out"] = n(T, D, std=0.1).to(BF16).to(DEV)
    return w


def dequantized(weight):
    """The bf16 values of a quantized weight: what the backward pass multiplies by."""
    q, sb, s, _ = nv.nvfp4_quantize_weight(weight)
    return (q, sb, s), nv.nvfp4_dequantize_rows(q, sb, s, rows_per_scale=weight.shape[1])


def swiglu_grad(gate_up, dh):
    g, u = gate_up.float().chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1).to(BF16)


def block(w):
    """Forward and backward of the block on the library's calls."""
    a = {}
    a["up_q"], a["up"] = dequantized(w["up"])
    a["down_q"], a["down"] = dequantized(w["down"])
    first = nv.nvfp4_residual_norm(w["attn"], w["residual"], w["w_pre"], post_weight=w["w_post"], gate=w["gate"], eps=EPS,
                                   quantize=True)
    a["x"], a["h"] = first["residual"], first["h"]
    rt = nv.nvfp4_moe_route(w["logits"], K)
    a["rt"] = rt
    chosen = torch.gather(w["logits"], 1, rt["experts"].long())
    a["p"] = torch.softmax(chosen, dim=1)
    # the NVFP4 forward product on the fused norm's quantized rows, and its bf16 counterpart
    a["gu_fp4"] = nv.nvfp4_grouped_gemm((first["q"], first["sb"], first["s"]), rt["offsets"], a["up_q"],
                                        row_index=rt["row_index"])
    a["h_deq"] = nv.nvfp4_dequantize_rows(first["q"], first["sb"], first["s"])
    a["gu"] = nv.nvfp4_bf16_grouped_gemm(a["h_deq"], rt["offsets"], a["up"], row_index=rt["row_index"])
    a["act"] = nv.nvfp4_swiglu_quantize_rows(a["gu"], want_h=True, quantize=False)["h"]
    a["y"] = nv.nvfp4_bf16_grouped_gemm(a["act"], rt["offsets"], a["down"])
    a["moe"] = nv.nvfp4_moe_combine(a["y"], rt["slot_of"], a["p"], out_dtype=F32)
    a["out"] = nv.nvfp4_residual_norm(a["moe"], a["x"], None, post_weight=w["w_post2"], gate=w["gate2"], eps=EPS)["residual"]
    # backward
    g = nv.nvfp4_residual_norm_backward(a["moe"], a["out"], None, d_residual=w["d_out"], post_weight=w["w_post2"],
                                        gate=w["gate2"], eps=EPS)
    a["d_post2"], a["d_gate2"], a["d_moe"] = g["d_post_weight"], g["d_gate"], g["dx"]
    c = nv.nvfp4_moe_combine_backward(a["d_moe"], a["y"], rt["slot_of"], a["p"])
    a["d_p"], a["d_y"] = c["d_weights"], c["dy"]
    a["d_act"] = nv.nvfp4_bf16_grouped_dgrad(a["d_y"], rt["offsets"], a["down"])
    a["d_down"] = nv.nvfp4_bf16_grouped_wgrad(a["d_y"], a["act"], rt["offsets"])
    a["d_gu"] = swiglu_grad(a["gu"], a["d_act"])
    a["d_rows"] = nv.nvfp4_bf16_grouped_dgrad(a["d_gu"], rt["offsets"], a["up"])
    a["d_up"] = nv.nvfp4_bf16_grouped_wgrad(a["d_gu"], a["h_deq"], rt["offsets"], row_index=rt["row_index"])
    a["d_h"] = nv.nvfp4_moe_combine(a["d_rows"], rt["slot_of"])
    g = nv.nvfp4_residual_norm_backward(w["attn"], a["x"], w["w_pre"], dh=a["d_h"], d_residual=g["d_residual"],
                                        post_weight=w["w_post"], gate=w["gate"], eps=EPS)
    a["d_attn"], a["d_residual"] = g["dx"], g["d_residual"]
    a["d_post"], a["d_pre"], a["d_gate"] = g["d_post_weight"], g["d_norm_weight"], g["d_gate"]
    return a


GRADS = ("d_up", "d_down", "d_post", "d_pre", "d_gate", "d_post2", "d_gate2")


def reference(w, a):
    """Every gradient by autograd in 64 bits over the plain chain, its
    activations replaced by the block's own where those are rounded."""
    leaf = {k: w[k].double().requires_grad_() for k in ("attn", "residual", "w_post", "w_pre", "gate", "w_post2", "gate2")}
    leaf["up"], leaf["down"] = a["up"].double().requires_grad_(), a["down"].double().requires_grad_()
    p = a["p"].double().requires_grad_()

    def norm(v, weight):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * weight

    def at(value, stored):  # the stored activation, with the exact one's gradient
        return value + (stored.double() - value).detach()
    x = at(leaf["residual"] + leaf["gate"] * norm(leaf["attn"], leaf["w_post"]), a["x"])
    h = at(norm(x, leaf["w_pre"]), a["h_deq"])
    rt, rows = a["rt"], a["rt"]["row_index"].long()
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), (rt["offsets"][1:] - rt["offsets"][:-1]).long())
    gu = at((h[rows][:, None, :] * leaf["up"][expert]).sum(2), a["gu"])
    gate, up = gu.chunk(2, dim=1)
    act = at(torch.nn.functional.silu(gate) * up, a["act"])
    y = at((act[:, None, :] * leaf["down"][expert]).sum(2), a["y"])
    moe = at((y[rt["slot_of"].long()] * p[:, :, None]).sum(1), a["moe"])
    out = x + leaf["gate2"] * norm(moe, leaf["w_post2"])
    out.backward(w["d_out"].double())
    return out.detach(), {"d_attn": leaf["attn"].grad, "d_residual": leaf["residual"].grad, "d_p": p.grad,
                          "d_up": leaf["up"].grad, "d_down": leaf["down"].grad, "d_post": leaf["w_post"].grad,
                          "d_pre": leaf["w_pre"].grad, "d_gate": leaf["gate"].grad, "d_post2": leaf["w_post2"].grad,
                          "d_gate2": leaf["gate2"].grad}


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


# Backward, a gradient's bf16 roundings on its way: d_out's residual gradient, d_moe, d_y, d_gu, d_h, then its own.
# Each is at most 2^-8 of an element, so of the 2-norm; at most six in a row.
CHAIN = 6 * 2.0 ** -8


def test_block_forward_and_backward():
    w = inputs(1)
    a = block(w)
    out, want = reference(w, a)
    assert off(a["out"], out) <= 2 * 2.0 ** -8  # x and out are rounded once each
    # the NVFP4 product and the bf16 one of the dequantized operands: dequantizing rounds S s_b q to bf16, at most 2^-8
    # of an element, on both sides, so a product is off by at most 2 x 2^-8 + 2^-16 of itself (and fp32 sums of 256)
    size = nv.nvfp4_bf16_grouped_gemm(a["h_deq"].abs(), a["rt"]["offsets"], a["up"].abs(), row_index=a["rt"]["row_index"])
    assert ((a["gu_fp4"] - a["gu"]).abs() <= (2 * 2.0 ** -8 + 2.0 ** -15) * size).all()
    for name, value in want.items():
        assert off(a[name], value) <= CHAIN, name


def test_clipping_the_blocks_gradients_and_repeats():
    w = inputs(2)
    a = block(w)
    b = block(w)
    for name in a:
        if isinstance(a[name], torch.Tensor):
            assert torch.equal(a[name], b[name]), name  # the same bits on every run
    grads = [a[k] for k in GRADS]
    total = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    kept = [g.clone() for g in grads]
    norm = nv.nvfp4_clip_grad_norm(grads, 0.25)
    assert abs(float(norm) - float(total)) <= 2.0 ** -23 * float(total)
    after = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    assert abs(float(after) - 0.25) <= 0.25 * 2.0 ** -20  # 1e-6 / norm and one rounding an element
    for g, k in zip(grads, kept):
        assert torch.equal(g * 0 + k * (0.25 / (float(total) + 1e-6)) > 0, k > 0)


def test_block_in_a_graph():
    """The whole block captured once and replayed on new inputs, with eager
    work between the replays, gives the eager bits."""
    w = inputs(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(w)
    for seed in (4, 5, 6, 7):
        new = inputs(seed)
        for k in w:
            w[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        eager = block(new)
        for name in GRADS + ("out", "d_attn", "d_residual", "d_p"):
            assert torch.equal(held[name], eager[name]), (seed, name)


def test_gradients_of_microbatches_add_up_in_place():
    w = inputs(8)
    a = block(w)
    acc = torch.zeros_like(a["d_up"])
    for _ in range(2):
        nv.nvfp4_bf16_grouped_wgrad(a["d_gu"], a["h_deq"], a["rt"]["offsets"], row_index=a["rt"]["row_index"], add=acc, out=acc)
    # x + x is exact; the sums inside each call have the same bits
    assert torch.equal(acc, a["d_up"] * 2)


def test_clipped_gradients_of_the_block_element_by_element():
    a = block(inputs(2))
    grads = [a[k] for k in GRADS]
    total = float(torch.stack([g.double().square().sum() for g in grads]).sum().sqrt())
    kept = [g.clone() for g in grads]
    nv.nvfp4_clip_grad_norm(grads, 0.25)
    for name, g, k in zip(GRADS, grads, kept):
        want = k.double() * (0.25 / (total + 1e-6))
        ref.close(g, want, 4 * ref.U * want.abs(), name)
