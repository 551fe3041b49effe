"""GPU tests of the expert combine, forward and backward, against its 64-bit
form, through the layouts nvfp4_moe_route writes and others."""
import itertools

import pytest
import torch

import learner_refs as ref
import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def make(tokens, topk, d, y=F32, out=BF16, extra=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows = tokens * topk + extra
    return dict(y=torch.randn(rows, d, generator=g).to(y).to(DEV),
                slot=torch.randperm(rows, generator=g)[:tokens * topk].to(torch.int32).view(tokens, topk).to(DEV),
                p=torch.rand(tokens, topk, generator=g).to(DEV), dout=torch.randn(tokens, d, generator=g).to(out).to(DEV))


def check(c, out=BF16, dy=BF16, weights=True):
    p = c["p"] if weights else None
    ok = (c["slot"] >= 0) & (c["slot"] < c["y"].shape[0])
    at = torch.where(ok, c["slot"], torch.zeros_like(c["slot"])).long()
    pd = torch.where(ok, (p if weights else torch.ones_like(c["p"])).double(), torch.zeros((), dtype=torch.float64, device=DEV))
    y = c["y"].double()[at] * ok[..., None]
    got = nv.nvfp4_moe_combine(c["y"], c["slot"], p, out_dtype=out)
    term = pd[..., None] * y
    ref.close(got, term.sum(1), (c["slot"].shape[1] + 1) * ref.U * term.abs().sum(1), "out")
    back = nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], p, out={
        "dy": torch.full(c["y"].shape, 5.0, dtype=dy, device=DEV)})
    g = c["dout"].double()
    want = torch.full(c["y"].shape, 5.0, dtype=torch.float64, device=DEV)
    want[at[ok]] = (pd[..., None] * g[:, None, :])[ok]
    ref.close(back["dy"], want, ref.U * want.abs(), "dy")
    if weights:
        dot = y * g[:, None, :]
        ref.close(back["d_weights"], dot.sum(2), (dot.shape[2] + 8) * ref.U * dot.abs().sum(2), "d_weights")
    else:
        assert set(back) == {"dy"}


@pytest.mark.parametrize("d", [1, 7, 8, 65, 512, 520, 2048, 2049, 9000])
@pytest.mark.parametrize("topk", [1, 2, 8, 11, 64])
def test_sizes(d, topk):
    check(make(5, topk, d, seed=d + topk))


@pytest.mark.parametrize("y,out,dy", list(itertools.product([F32, BF16], repeat=3)))
def test_types(y, out, dy):
    for d in (264, 77):
        c = make(40, 3, d, y, out, seed=d)
        check(c, out, dy)
        check(c, out, dy, weights=False)


@pytest.mark.parametrize("tokens,topk,d", [(1, 2, 72), (2, 2, 72), (63, 2, 72), (1000, 2, 72), (20000, 2, 72), (2_200_000, 1, 1030)],
                         ids=lambda v: str(v))
def test_token_counts(tokens, topk, d):
    if tokens > 10 ** 6:  # more pieces than a launch has blocks, and offsets past 4 GiB
        y = (torch.arange(tokens, device=DEV) % 251).to(BF16)[:, None].expand(tokens, d).contiguous()
        slot = torch.arange(tokens, device=DEV, dtype=torch.int32).flip(0)[:, None].contiguous()
        got = nv.nvfp4_moe_combine(y, slot)
        assert torch.equal(got, y.flip(0))
        back = nv.nvfp4_moe_combine_backward(got, y, slot)
        assert torch.equal(back["dy"], y)
        return
    check(make(tokens, topk, d, extra=3, seed=tokens))


def test_slots_outside_and_rows_unnamed():
    c = make(50, 4, 520, extra=9)
    c["slot"][::3, 1] = -1
    c["slot"][::4, 2] = c["y"].shape[0]
    c["slot"][7, 0] = 2 ** 31 - 1
    c["slot"][9] = -2 ** 31
    check(c)
    # a dropped choice adds nothing even if its weight is not a number, nor does an unnamed row
    named = torch.zeros(c["y"].shape[0], dtype=torch.bool, device=DEV)
    ok = (c["slot"] >= 0) & (c["slot"] < c["y"].shape[0])
    named[c["slot"][ok].long()] = True
    want = nv.nvfp4_moe_combine(c["y"], c["slot"], c["p"])
    c["p"][~ok] = float("nan")
    c["y"][~named] = float("inf")
    assert torch.equal(nv.nvfp4_moe_combine(c["y"], c["slot"], c["p"]), want)


def test_a_row_named_twice_forward():
    y = torch.randn(3, 40, device=DEV)
    slot = torch.tensor([[1, 1, 2], [0, 1, 0]], dtype=torch.int32, device=DEV)
    got = nv.nvfp4_moe_combine(y, slot, out_dtype=F32)
    ref.close(got, y.double()[slot.long()].sum(1), 4 * ref.U * y.double().abs()[slot.long()].sum(1))


def test_the_routers_layout():
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(300, 16, generator=g).to(DEV)
    rt = nv.nvfp4_moe_route(logits, 4)
    x = torch.randn(300, 264, generator=g).to(BF16).to(DEV)
    routed = x[rt["row_index"].long()]
    assert torch.equal(nv.nvfp4_moe_combine(routed, rt["slot_of"], out_dtype=F32), x.float() * 4)


def test_graph_replays_and_repeats():
    c = make(200, 8, 520)
    out = nv.nvfp4_moe_combine(c["y"], c["slot"], c["p"])
    back = nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], c["p"])
    o, b = torch.empty_like(out), {k: torch.empty_like(v) for k, v in back.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_moe_combine(c["y"], c["slot"], c["p"], out=o)
        nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], c["p"], out=b)
    for _ in range(4):
        o.zero_()
        for t in b.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and all(torch.equal(b[k], back[k]) for k in back)
        nv.nvfp4_moe_combine(c["y"], c["slot"], c["p"])


def test_gradients_against_differences():
    c = make(4, 3, 20, F32, F32, seed=6)

    def loss(y, p):
        return float(((y[c["slot"].long()] * p[..., None]).sum(1) * c["dout"].double()).sum())
    y, p = c["y"].double(), c["p"].double()
    back = nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], c["p"], dy_dtype=F32)
    for name, t in (("dy", y), ("d_weights", p)):
        for at in range(0, t.numel(), 3):
            two = []
            for sign in (1, -1):
                w = t.clone()
                w.view(-1)[at] += sign * 1e-3
                two.append(loss(w, p) if name == "dy" else loss(y, w))
            # the loss is linear in each: differences are exact but for 64-bit rounding
            assert abs((two[0] - two[1]) / 2e-3 - float(back[name].reshape(-1)[at])) <= 1e-5 * 20


def test_empty():
    y = torch.randn(0, 16, device=DEV)
    slot = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    assert (nv.nvfp4_moe_combine(y, slot) == 0).all()
    assert nv.nvfp4_moe_combine(y, slot[:0]).shape == (0, 16)
    back = nv.nvfp4_moe_combine_backward(torch.ones(3, 16, device=DEV), y, slot, torch.ones(3, 2, device=DEV))
    assert (back["d_weights"] == 0).all()


def test_refusals():
    c = make(6, 2, 16)
    f, b = nv.nvfp4_moe_combine, nv.nvfp4_moe_combine_backward
    for bad in (lambda: f(c["y"], c["slot"], c["p"][:3]), lambda: f(c["y"], c["slot"].view(-1)), lambda: f(c["y"].t(), c["slot"]),
                lambda: f(c["y"], c["slot"], out=c["y"][:6]), lambda: b(c["dout"][:2], c["y"], c["slot"]),
                lambda: f(c["y"].cpu(), c["slot"]), lambda: b(c["dout"], c["y"], c["slot"], out={"dy": c["y"]})):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(c["y"], c["slot"].long()), lambda: f(c["y"].half(), c["slot"]),
                lambda: f(c["y"], c["slot"], c["p"].double()), lambda: f(c["y"], c["slot"], out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(nv.NVFP4Error):
        f(c["y"], torch.zeros(1, 65, dtype=torch.int32, device=DEV))


def test_refuses_outputs_in_one_memory():
    c = make(6, 2, 16)
    dy = torch.empty(c["y"].shape, dtype=torch.float32, device=DEV)
    dw = dy.view(-1)[:12].view(6, 2)
    with pytest.raises(ValueError):
        nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], c["p"], out={"dy": dy, "d_weights": dw})


def test_outputs_of_other_names():
    c = make(6, 2, 16)
    dw = torch.full((6, 2), 7.0, device=DEV)
    for name in ("dw", "dx", "d_weight"):
        with pytest.raises(ValueError):
            nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], c["p"], out={name: dw})
    back = nv.nvfp4_moe_combine_backward(c["dout"], c["y"], c["slot"], out={"d_weights": dw})
    assert set(back) == {"dy"} and (dw == 7).all()
