"""A policy's learner step from the library's calls as they are used together:
tokens in through the embedding, a mixture-of-experts layer with the router's
gate, log-probabilities of the targets out, and back to every gradient, the
table's from both of its ends.

  x = embedding(table, ids);  h = norm(x);  route and gate h's router logits
  x' = x + sum over experts;  g = norm(x');  loss = vocabulary loss of g over table
  total = sum d_loss loss + COEF balance loss

The last tokens are padding: no id, not counted by the gate, no target.  The
reference is the same chain in 64 bits with autograd, on the chain's own rounded
activations.
"""
import pytest
import torch

import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
DEV = "cuda:0"
T, PAD, D, E, K, VOCAB, EPS, COEF, SCALE, TEMP = 300, 40, 128, 16, 3, 1003, 1e-6, 0.05, 4.0, 0.8


def inputs(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g) * std + mean).to(DEV)
    w = {"table": n(VOCAB, D, std=0.2).to(BF16), "router": n(E, D, std=0.2), "experts": n(E, D, D, std=0.1).to(BF16),
         "w1": n(D, std=0.1, mean=1.0), "w2": n(D, std=0.1, mean=1.0), "d_loss": n(T, std=1.0 / T),
         "coef": torch.tensor(COEF, device=DEV)}
    ids = (torch.rand(T, generator=g) ** 3 * VOCAB).to(I32)
    targets = torch.roll(ids, -1)
    targets[torch.rand(T, generator=g) < 0.2] = -1  # the prompt
    ids[T - PAD:] = targets[T - PAD - 1:] = -1
    w["ids"], w["targets"] = ids.to(DEV), targets.to(DEV)
    w["valid"] = w["ids"] >= 0
    return w


def step(w):
    a = {}
    a["x"] = nv.nvfp4_embedding(w["table"], w["ids"], scale=SCALE, out_dtype=F32)
    a["h"] = nv.nvfp4_residual_norm(a["x"], None, w["w1"], residual_dtype=F32, eps=EPS)["h"]
    a["logits"] = a["h"].float() @ w["router"].t()
    rt = a["rt"] = nv.nvfp4_moe_route(a["logits"], K)
    gate = nv.nvfp4_moe_gate(a["logits"], rt["experts"], valid=w["valid"])
    a["weights"], a["counts"], a["balance"] = gate["weights"], gate["counts"], gate["loss"]
    a["y"] = nv.nvfp4_bf16_grouped_gemm(a["h"], rt["offsets"], w["experts"], row_index=rt["row_index"])
    a["moe"] = nv.nvfp4_moe_combine(a["y"], rt["slot_of"], a["weights"], out_dtype=F32)
    second = nv.nvfp4_residual_norm(a["moe"], a["x"], w["w2"], eps=EPS)
    a["x2"], a["g"] = second["residual"], second["h"]
    out = nv.nvfp4_vocab_loss(a["g"], w["table"], w["targets"], scale=TEMP)
    a["loss"], a["lse"] = out["loss"], out["lse"]
    # backward
    b = nv.nvfp4_vocab_loss_backward(a["g"], w["table"], w["targets"], a["lse"], w["d_loss"], scale=TEMP)
    a["d_table"] = b["dw"]
    n2 = nv.nvfp4_residual_norm_backward(a["moe"], a["x2"], w["w2"], dh=b["dh"], eps=EPS, dx_dtype=F32)
    a["d_w2"] = n2["d_norm_weight"]
    c = nv.nvfp4_moe_combine_backward(n2["dx"], a["y"], rt["slot_of"], a["weights"])
    a["d_experts"] = nv.nvfp4_bf16_grouped_wgrad(c["dy"], a["h"], rt["offsets"], row_index=rt["row_index"])
    rows = nv.nvfp4_bf16_grouped_dgrad(c["dy"], rt["offsets"], w["experts"])
    d_logits = nv.nvfp4_moe_gate_backward(a["logits"], rt["experts"], a["counts"], d_weights=c["d_weights"], d_loss=w["coef"],
                                          valid=w["valid"])
    a["d_router"] = d_logits.t() @ a["h"].float()
    d_h = nv.nvfp4_moe_combine(rows, rt["slot_of"], out_dtype=F32) + d_logits @ w["router"]
    n1 = nv.nvfp4_residual_norm_backward(a["x"], a["x"], w["w1"], dh=d_h.to(BF16), d_residual=n2["d_residual"], eps=EPS,
                                         dx_dtype=F32)
    a["d_w1"] = n1["d_norm_weight"]
    # the table's other end, onto the gradient that the loss gave it
    nv.nvfp4_embedding_backward(n1["d_residual"], w["ids"], VOCAB, scale=SCALE, add=a["d_table"], out=a["d_table"])
    return a


GRADS = ("d_table", "d_experts", "d_router", "d_w1", "d_w2")


def reference(w, a):
    leaf = {k: w[k].double().requires_grad_() for k in ("table", "router", "experts", "w1", "w2")}

    def at(value, stored):  # the stored activation, with the exact one's gradient
        return value + (stored.double() - value).detach()

    def norm(v, weight):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * weight
    ok = w["valid"]
    x = at(torch.where(ok[:, None], leaf["table"][w["ids"].long().clamp(min=0)] * SCALE, 0.0), a["x"])
    h = at(norm(x, leaf["w1"]), a["h"])
    logits = at(h @ leaf["router"].t(), a["logits"])
    chosen = a["rt"]["experts"].long()
    p = torch.softmax(logits, 1)
    mine = p.gather(1, chosen)
    weights = torch.where(ok[:, None], mine / mine.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(chosen[ok].reshape(-1), minlength=E).double()
    balance = E * (counts / counts.sum() * p[ok].mean(0)).sum()
    y = at((leaf["experts"][chosen] * h[:, None, None, :]).sum(3), a["y"][a["rt"]["slot_of"].long()])
    x2 = at(x + (y * weights[:, :, None]).sum(1), a["x2"])
    g = at(norm(x2, leaf["w2"]), a["g"])
    z = TEMP * (g @ leaf["table"].t())
    has = w["targets"] >= 0
    loss = torch.logsumexp(z, 1) - z.gather(1, w["targets"].long().clamp(min=0)[:, None])[:, 0]
    (((loss * w["d_loss"].double())[has]).sum() + COEF * balance).backward()
    return (weights.detach(), balance.detach(), torch.where(has, loss, 0.0).detach(), torch.cat([counts, ok.sum()[None]]),
            {"d_" + k: v.grad for k, v in leaf.items()})


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


# bf16 roundings of a gradient in a row: dz, dh, dy, d_h; each at most 2^-8 of an element, so of the 2-norm
CHAIN = 4 * 2.0 ** -8


def test_step_forward_and_backward():
    w = inputs(1)
    a = step(w)
    weights, balance, loss, counts, want = reference(w, a)
    # fp32 arithmetic on stored activations throughout
    assert off(a["weights"], weights) <= 2.0 ** -18 and abs(float(a["balance"] - balance)) <= 2.0 ** -18 * float(balance)
    assert torch.equal(a["counts"].double(), counts)
    assert off(a["loss"], loss) <= 2.0 ** -18 and (a["loss"][w["targets"] < 0] == 0).all()
    for name in GRADS:
        assert off(a[name], want[name]) <= CHAIN, (name, off(a[name], want[name]))


def test_step_repeats_and_in_a_graph():
    w = inputs(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = step(w), step(w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for name in GRADS + ("loss", "balance", "weights"):
        assert torch.equal(a[name], b[name]), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(w)
    for seed in (3, 4, 5, 6):
        new = inputs(seed)
        for k in w:
            w[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        eager = step(new)
        for name in GRADS + ("loss", "balance", "weights"):
            assert torch.equal(held[name], eager[name]), (seed, name)


def test_step_in_the_checked_build():
    w = inputs(7)
    saved = nv._lib
    try:
        nv._lib = nv.load(nv.PRODUCT_LIB_PATH)
        a = step(w)
        nv._lib = nv.load(nv.CHECKED_LIB_PATH)
        b = step(w)
    finally:
        nv._lib = saved
    for name in GRADS + ("loss", "balance", "weights"):
        assert torch.equal(a[name], b[name]), name
