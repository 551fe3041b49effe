"""GPU tests of the router's gate and its gradient against the definition in 64
bits.

Bounds: U is the fp32 unit, D the largest distance of a row's logits from its
maximum, of which rounding in the argument of an exponential keeps D U; an
exponential is within 2 U of its argument's, a sum of E terms within E U, a
quotient within U.  So p and the weights are within R = (2 D + 2 E + 16) U of
themselves (and an underflow step), a sum over T tokens within R + T U.
"""
import pytest
import torch

import nvfp4_token_quantization_amd as nv
from learner_refs import U

pytestmark = pytest.mark.gpu

F32, I32, F64 = torch.float32, torch.int32, torch.float64
DEV = "cuda:0"
TINY = 2.0 ** -126


def inputs(T, E, K, seed=0, spread=2.0, valid=0.0):
    g = torch.Generator().manual_seed(seed + T + 31 * E + K)
    logits = (torch.randn(T, E, generator=g) * spread).to(DEV)
    experts = nv.nvfp4_moe_route(logits, K)["experts"] if T else torch.empty(0, K, dtype=I32, device=DEV)
    mask = (torch.rand(T, generator=g) >= valid).to(DEV) if valid else None
    return logits, experts, mask, torch.randn(T, K, generator=g).to(DEV), torch.tensor(0.37, device=DEV)


def exact(logits, experts, valid, normalize):
    T, E = logits.shape
    K = experts.shape[1]
    ok = torch.ones(T, dtype=torch.bool, device=DEV) if valid is None else valid.bool()
    x = torch.where(ok[:, None], logits.double(), 0.0)
    p = torch.softmax(x, 1)
    has = (experts >= 0) & (experts < E) & ok[:, None]
    at = experts.long().clamp(0, E - 1)
    mine = torch.where(has, p.gather(1, at), 0.0)
    w = torch.where(has, mine / mine.sum(1, keepdim=True).clamp(min=1e-300), 0.0) if normalize else mine
    counts = torch.bincount(at[has], minlength=E)
    n = int(ok.sum())
    sums = torch.where(ok[:, None], p, 0.0).sum(0)
    total = int(counts.sum())
    loss = float(E * (counts.double() * sums).sum() / (total * n)) if total else 0.0
    span = (x.amax(1) - x.amin(1))[:, None] if T else x.new_zeros(0, 1)
    rel = (2 * span + 2 * E + 16) * U
    return dict(ok=ok, p=p, has=has, at=at, w=w, counts=torch.cat([counts, torch.tensor([n], device=DEV)]), sums=sums,
                loss=loss, rel=rel)


def exact_back(logits, experts, valid, normalize, counts, dw, dloss):
    e = exact(logits, experts, valid, normalize)
    T, E = logits.shape
    c = counts.double()
    total, n = float(c[:E].sum()), float(c[E])
    up = (float(dloss) * E * c[:E] / (total * n) if dloss is not None and total and n else torch.zeros(E, dtype=F64, device=DEV))[None]
    p, rel = e["p"], e["rel"]
    got = p * (up - (p * up).sum(1, keepdim=True))
    size = p * (up.abs() + (p * up.abs()).sum(1, keepdim=True))
    if dw is not None:
        d = torch.where(e["has"], dw.double(), 0.0)
        w = e["w"]
        dot, adot = (w * d).sum(1, keepdim=True), (w * d.abs()).sum(1, keepdim=True)
        if normalize:
            got = got.scatter_add(1, e["at"], w * (d - dot))
            size = size.scatter_add(1, e["at"], w * (d.abs() + adot))
        else:
            got = got.scatter_add(1, e["at"], w * d) - p * dot
            size = size.scatter_add(1, e["at"], w * d.abs()) + p * adot
    zero = torch.zeros_like(got)
    return torch.where(e["ok"][:, None], got, zero), torch.where(e["ok"][:, None], (3 * rel + 64 * U) * size + TINY, zero)


def check(got, e):
    assert torch.equal(got["counts"].long(), e["counts"].long())
    err = (got["weights"].double() - e["w"]).abs()
    assert (err <= 2 * e["rel"] * e["w"] + TINY * e["has"]).all(), float((err - 2 * e["rel"] * e["w"]).max())
    T = len(e["w"])
    lim = ((e["rel"] + T * U) * torch.where(e["ok"][:, None], e["p"], 0.0)).sum(0)
    assert ((got["prob_sums"].double() - e["sums"]).abs() <= lim + TINY * T).all()
    r = float(e["rel"].max()) + (T + 8) * U if T else U
    assert abs(float(got["loss"]) - e["loss"]) <= r * abs(e["loss"])


SHAPES = [(1, 1, 1), (1, 5, 3), (3, 16, 16), (64, 17, 4), (65, 32, 20), (300, 33, 8), (63, 64, 33), (1000, 128, 8),
          (129, 128, 64), (500, 129, 8), (65, 256, 40), (40, 300, 8), (33, 512, 64), (100, 513, 8), (17, 1024, 64),
          (5000, 8, 2), (17000, 60, 4)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_forward(T, E, K, normalize, masked):
    logits, experts, valid, _, _ = inputs(T, E, K, valid=masked)
    got = nv.nvfp4_moe_gate(logits, experts, valid=valid, normalize=normalize)
    check(got, exact(logits, experts, valid, normalize))
    alone = nv.nvfp4_moe_gate(logits, experts, valid=valid, normalize=normalize, balance=False)
    assert list(alone) == ["weights"] and torch.equal(alone["weights"], got["weights"])


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
def test_backward(T, E, K, normalize, parts):
    logits, experts, valid, dw, dl = inputs(T, E, K, valid=0.2)
    counts = nv.nvfp4_moe_gate(logits, experts, valid=valid, normalize=normalize)["counts"]
    dw, dl = dw if parts != "loss" else None, dl if parts != "weights" else None
    got = nv.nvfp4_moe_gate_backward(logits, experts, counts, d_weights=dw, d_loss=dl, valid=valid, normalize=normalize)
    want, bound = exact_back(logits, experts, valid, normalize, counts, dw, dl)
    err = (got.double() - want).abs()
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-300)).max())


def test_choices_that_are_no_expert_or_come_twice():
    T, E, K = 200, 40, 6
    logits, experts, _, dw, dl = inputs(T, E, K)
    experts[::3, 1] = -1
    experts[1::3, 2] = E
    experts[2::3, 0] = -2 ** 31
    experts[5] = -7           # a token without any choice
    experts[:, 4] = experts[:, 3]  # an expert named twice
    for normalize in (True, False):
        e = exact(logits, experts, None, normalize)
        got = nv.nvfp4_moe_gate(logits, experts, normalize=normalize)
        check(got, e)
        assert (got["weights"][5] == 0).all()
        dw[5] = float("nan")  # of no choice: read into nothing
        back = nv.nvfp4_moe_gate_backward(logits, experts, got["counts"], d_weights=dw, d_loss=dl, normalize=normalize)
        want, bound = exact_back(logits, experts, None, normalize, got["counts"], dw, dl)
        assert ((back.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T", [50, 3000])
def test_padding_tokens_reach_nothing(T):
    logits, experts, valid, dw, dl = inputs(T, 24, 3, valid=0.5)
    a = nv.nvfp4_moe_gate(logits, experts, valid=valid)
    ga = nv.nvfp4_moe_gate_backward(logits, experts, a["counts"], d_weights=dw, d_loss=dl, valid=valid)
    logits[~valid] = float("nan")
    experts[~valid] = 2 ** 31 - 1
    dw[~valid] = float("inf")
    b = nv.nvfp4_moe_gate(logits, experts, valid=valid.to(torch.uint8))
    gb = nv.nvfp4_moe_gate_backward(logits, experts, b["counts"], d_weights=dw, d_loss=dl, valid=valid)
    for key in a:
        assert torch.equal(a[key], b[key]), key
    assert torch.equal(ga, gb) and (gb[~valid] == 0).all()
    none = torch.zeros(T, dtype=torch.bool, device=DEV)
    c = nv.nvfp4_moe_gate(logits, experts, valid=none)
    assert all((v == 0).all() for v in c.values())
    assert (nv.nvfp4_moe_gate_backward(logits, experts, c["counts"], d_weights=dw, d_loss=dl, valid=none) == 0).all()


def test_extreme_logits():
    T, E, K = 70, 20, 4
    logits, experts, _, dw, dl = inputs(T, E, K)
    logits[0] = 1e30
    logits[1] = -3e38
    logits[2, :10] = -float("inf")
    logits[3] = torch.linspace(-80, 80, E, device=DEV)
    experts[2] = torch.tensor([0, 12, 15, 3], device=DEV)
    for normalize in (True, False):
        got = nv.nvfp4_moe_gate(logits, experts, normalize=normalize)
        x = logits.double()
        x[2, :10] = -1e5  # exp underflows to the same zero
        e = exact(x, experts, None, normalize)
        e["rel"][:] = (2 * 160 + 2 * E + 16) * U
        check(got, e)
        assert got["weights"][2, 0] == 0 and got["weights"][2, 3] == 0
    logits[4, 0] = float("nan")
    logits[5, 0] = float("inf")
    got = nv.nvfp4_moe_gate(logits, experts, normalize=False)["weights"]
    assert torch.isnan(got[4]).all() and torch.isnan(got[5]).any() and torch.isfinite(got[6:]).all()
    assert torch.isfinite(got[:4]).all()


def test_no_tokens():
    logits, experts, _, dw, dl = inputs(0, 12, 3)
    got = nv.nvfp4_moe_gate(logits, experts)
    assert (got["counts"] == 0).all() and (got["prob_sums"] == 0).all() and got["loss"] == 0
    assert nv.nvfp4_moe_gate_backward(logits, experts, got["counts"], d_weights=dw, d_loss=dl).shape == (0, 12)


def test_an_even_load_has_loss_one():
    T, E = 480, 24
    logits = torch.zeros(T, E, device=DEV)
    experts = (torch.arange(T * 2, device=DEV) % E).to(I32).view(T, 2)
    got = nv.nvfp4_moe_gate(logits, experts)
    assert abs(float(got["loss"]) - 1) < (T + 64) * U and (got["counts"][:E] == 40).all()
    assert torch.equal(got["weights"], torch.full((T, 2), 0.5, device=DEV))


def test_counts_of_several_ranks():
    """Two halves of a batch as two ranks: losses and gradients by the summed counts are the whole batch's."""
    logits, experts, valid, dw, dl = inputs(400, 16, 2, valid=0.2)
    whole = nv.nvfp4_moe_gate(logits, experts, valid=valid)
    halves = [nv.nvfp4_moe_gate(logits[i:i + 200], experts[i:i + 200], valid=valid[i:i + 200]) for i in (0, 200)]
    counts = halves[0]["counts"] + halves[1]["counts"]
    assert torch.equal(counts, whole["counts"])
    c = counts.double()
    loss = sum(16 * float((c[:16] * h["prob_sums"].double()).sum() / (c[:16].sum() * c[16])) for h in halves)
    assert abs(loss - float(whole["loss"])) <= 500 * U * loss
    g = [nv.nvfp4_moe_gate_backward(logits[i:i + 200], experts[i:i + 200], counts, d_weights=dw[i:i + 200], d_loss=dl,
                                    valid=valid[i:i + 200]) for i in (0, 200)]
    assert torch.equal(torch.cat(g), nv.nvfp4_moe_gate_backward(logits, experts, counts, d_weights=dw, d_loss=dl, valid=valid))


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    logits, experts, valid, dw, dl = inputs(30, 12, 3, valid=0.2)
    counts = nv.nvfp4_moe_gate(logits, experts, valid=valid, normalize=normalize)["counts"]
    g = nv.nvfp4_moe_gate_backward(logits, experts, counts, d_weights=dw, d_loss=dl, valid=valid, normalize=normalize)
    c = counts.double()

    def total(x):
        p = torch.softmax(x, 1)
        m = p.gather(1, experts.long())
        m = m / m.sum(1, keepdim=True) if normalize else m
        s = p[valid].sum(0)
        return float((m * dw.double())[valid].sum() + float(dl) * 12 * (c[:12] * s).sum() / (c[:12].sum() * c[12]))
    a = torch.randn(30, 12, generator=torch.Generator().manual_seed(2)).to(DEV).double()
    x, eps = logits.double(), 1e-5
    num = (total(x + eps * a) - total(x - eps * a)) / (2 * eps)
    # the difference is off by the third derivative times eps^2 and 64-bit noise over eps
    bound = exact_back(logits, experts, valid, normalize, counts, dw, dl)[1]
    assert abs(float((g.double() * a).sum()) - num) <= float((bound * a.abs()).sum()) + 1e-8


def test_given_tensors_streams_and_graphs():
    logits, experts, valid, dw, dl = inputs(3000, 64, 6, valid=0.1)
    ref = nv.nvfp4_moe_gate(logits, experts, valid=valid)
    need = nv.lib().nvfp4_moe_gate_workspace(3000, 64)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    out = {k: torch.full_like(v, 7) for k, v in ref.items()}
    got = nv.nvfp4_moe_gate(logits, experts, valid=valid, out=out, workspace=ws[:need])
    assert all(got[k] is out[k] and torch.equal(out[k], ref[k]) for k in ref) and (ws[need:] == 255).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = nv.nvfp4_moe_gate(logits, experts, valid=valid)
    s.synchronize()
    assert all(torch.equal(b[k], ref[k]) for k in ref)
    dx = torch.empty_like(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_moe_gate(logits, experts, valid=valid, out=out, workspace=ws[:need])
        nv.nvfp4_moe_gate_backward(logits, experts, out["counts"], d_weights=dw, d_loss=dl, valid=valid, out=dx)
    for step in range(4):
        l2, e2, v2, _, _ = inputs(3000, 64, 6, seed=step, valid=0.1 + 0.2 * step)
        logits.copy_(l2)
        experts.copy_(e2)
        valid.copy_(v2)
        graph.replay()
        torch.cuda.synchronize()
        ref = nv.nvfp4_moe_gate(logits, experts, valid=valid)
        assert all(torch.equal(out[k], ref[k]) for k in ref)
        assert torch.equal(dx, nv.nvfp4_moe_gate_backward(logits, experts, ref["counts"], d_weights=dw, d_loss=dl, valid=valid))
