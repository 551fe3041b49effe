"""GPU tests of the vocabulary loss (nvfp4_vocab_loss and its backward pass)
against the definition in 64 bits.

Bounds: U is the fp32 unit.  A logit is a sum of k exact products in fp32 and
one scaling, so within (k + 4) U scale sum|h w| of the exact one (E, the
largest of a row).  The exponentials see that error, that of their argument
(D U for arguments up to D) and a few U of their own; sums of V terms add V U,
the logarithm and the last sums a few U of lse.  dz is rounded once to bf16
(half a step, 2^-8), so dh and dw are within 2^-8 plus the probability's own
error of the sum of the magnitudes of their terms, plus fp32 sums, plus one
rounding to their type.  A probability below fp32's smallest normal number,
2^-126, may come out as zero, and so may a dz that a product reads: each is then
off by less than 2^-126.
"""
import pytest
import torch

import nvfp4_token_quantization_amd as nv
from learner_refs import HALF, U, close

pytestmark = pytest.mark.gpu

F32, BF16, I32, F64 = torch.float32, torch.bfloat16, torch.int32, torch.float64
DEV = "cuda:0"
TINY = 2.0 ** -126


def inputs(rows, vocab, k, seed=0, ignored=0.25, std=1.0):
    g = torch.Generator().manual_seed(seed + 7 * rows + vocab + k)
    h = torch.randn(rows, k, generator=g).to(BF16).to(DEV)
    w = (torch.randn(vocab, k, generator=g) * std / max(k, 1) ** 0.5).to(BF16).to(DEV)
    t = torch.randint(0, max(vocab, 1), (rows,), generator=g, dtype=I32)
    if ignored:
        t[torch.rand(rows, generator=g) < ignored] = -1
    d = torch.randn(rows, generator=g) / max(rows, 1)
    return h, w, t.to(DEV), d.to(DEV)


def exact_loss(h, w, t, scale):
    """(loss, lse, bound) of the rows with a target; zeros elsewhere."""
    rows, k = h.shape
    V = w.shape[0]
    has = (t >= 0) & (t < V)
    z = scale * torch.mm(h.double(), w.double().t().contiguous())
    mag = abs(scale) * torch.mm(h.double().abs(), w.double().abs().t().contiguous())
    zt = z.gather(1, t.long().clamp(0, max(V - 1, 0))[:, None])[:, 0] if V else z.new_zeros(rows)
    lse = torch.logsumexp(z, 1) if V else z.new_zeros(rows)
    err = (k + 4) * U * mag.amax(1) if V else z.new_zeros(rows)
    span = (z - zt[:, None]).abs().amax(1) if V else z.new_zeros(rows)
    bound = 2 * err + (2 * span + V + 32) * U + 8 * U * (lse.abs() + zt.abs())
    zero = torch.zeros_like(lse)
    return torch.where(has, lse - zt, zero), torch.where(has, lse, zero), torch.where(has, bound, zero)


def exact_grads(h, w, t, lse, d, scale, add=None):
    """{name: (exact, fp32 bound)} with dz's rounding in the bound; lse as given."""
    rows, k = h.shape
    V = w.shape[0]
    has = (t >= 0) & (t < V)
    at = torch.nonzero(has)[:, 0]
    hd, wd, tt = h[at].double(), w.double(), t[at].long()
    z = scale * torch.mm(hd, wd.t().contiguous())
    err = (k + 4) * U * abs(scale) * torch.mm(hd.abs(), wd.abs().t().contiguous())
    l = lse[at].double()[:, None]
    p = torch.exp(z - l)
    perr = p * (err + (2 * (z - l).abs() + 4 * l.abs() + 8) * U) * 1.01 + TINY
    one = torch.zeros_like(p)
    one[torch.arange(len(at), device=h.device), tt] = 1
    c = scale * d[at].double()[:, None]
    dz = c * (p - one)
    dzerr = c.abs() * perr + (HALF[BF16] + 4 * U) * (dz.abs() + c.abs() * perr) + TINY
    dh = torch.zeros(rows, k, dtype=F64, device=h.device)
    bh = torch.zeros_like(dh)
    dh[at] = torch.mm(dz, wd)
    bh[at] = torch.mm(dzerr + (V + 8) * U * dz.abs(), wd.abs())
    dw = torch.mm(dz.t().contiguous(), hd)
    bw = torch.mm((dzerr + (rows + 8) * U * dz.abs()).t().contiguous(), hd.abs())
    if add is not None:
        dw = dw + add.double()
        bw = bw + 2 * U * (dw.abs() + add.double().abs())
    return {"dh": (dh, bh), "dw": (dw, bw)}


def check_loss(got, want):
    for name, v in zip(("loss", "lse"), want):
        err = (got[name].double() - v).abs()
        assert (err <= want[2] + U * v.abs()).all(), (name, float((err - want[2]).max()))


SIZES = [(1, 1, 8), (1, 7, 64), (3, 255, 8), (5, 257, 72), (63, 1000, 64), (64, 129, 200), (65, 1000, 136),
         (128, 513, 64), (129, 300, 520), (200, 2049, 72), (256, 256, 64), (300, 5003, 264), (700, 1537, 128)]


@pytest.mark.parametrize("rows,vocab,k", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_forward(rows, vocab, k, scale):
    h, w, t, _ = inputs(rows, vocab, k, std=3.0)
    check_loss(nv.nvfp4_vocab_loss(h, w, t, scale=scale), exact_loss(h, w, t, scale))


@pytest.mark.parametrize("rows,vocab,k", SIZES)
@pytest.mark.parametrize("dtype,added", [(F32, False), (F32, True), (BF16, False), (BF16, True)])
def test_backward(rows, vocab, k, dtype, added):
    h, w, t, d = inputs(rows, vocab, k, std=3.0)
    lse = nv.nvfp4_vocab_loss(h, w, t, scale=0.8)["lse"]
    add = torch.randn(vocab, k, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV) if added else None
    got = nv.nvfp4_vocab_loss_backward(h, w, t, lse, d, scale=0.8, add=add, dw_dtype=dtype)
    assert got["dw"].dtype == dtype and got["dh"].dtype == BF16
    for name, (want, bound) in exact_grads(h, w, t, lse, d, 0.8, add).items():
        close(got[name], want, bound, name)


@pytest.mark.parametrize("rows,vocab,k", [(9000, 9000, 64), (40, 70001, 64), (2500, 40000, 136), (100, 30000, 2056)])
def test_several_pieces_and_splits(rows, vocab, k):
    h, w, t, d = inputs(rows, vocab, k, std=2.0)
    got = nv.nvfp4_vocab_loss(h, w, t)
    check_loss(got, exact_loss(h, w, t, 1.0))
    g = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, dw_dtype=BF16)
    for name, (want, bound) in exact_grads(h, w, t, got["lse"], d, 1.0).items():
        close(g[name], want, bound, name)


@pytest.mark.parametrize("rows", [1, 60, 100, 300, 1100])
def test_rows_without_a_target(rows):
    h, w, t, d = inputs(rows, 777, 72, ignored=0.0)
    t[:] = -1
    out = nv.nvfp4_vocab_loss(h, w, t)
    assert (out["loss"] == 0).all() and (out["lse"] == 0).all()
    g = nv.nvfp4_vocab_loss_backward(h, w, t, out["lse"], d)
    assert (g["dh"] == 0).all() and (g["dw"] == 0).all()
    # one row among them, the last; what the others hold reaches nothing
    t[-1] = 776
    t[:-1] = torch.tensor([777, -5, 2 ** 31 - 1, -2 ** 31], dtype=I32).repeat(rows)[:rows - 1].to(DEV)
    h[:-1] = float("nan")
    d[:-1] = float("inf")
    out = nv.nvfp4_vocab_loss(h, w, t)
    one = nv.nvfp4_vocab_loss(h[-1:], w, t[-1:])
    check_loss({k: v[-1:] for k, v in out.items()}, exact_loss(h[-1:], w, t[-1:], 1.0))
    assert (out["loss"][:-1] == 0).all() and (out["lse"][:-1] == 0).all()
    g = nv.nvfp4_vocab_loss_backward(h, w, t, out["lse"], d)
    assert (g["dh"][:-1] == 0).all()
    want = exact_grads(h[-1:], w, t[-1:], out["lse"][-1:], d[-1:], 1.0)
    close(g["dh"][-1:], *want["dh"], "dh")
    close(g["dw"], *want["dw"], "dw")
    check_loss(one, exact_loss(h[-1:], w, t[-1:], 1.0))


def test_empty_problems():
    h, w, t, d = inputs(5, 40, 16)
    none = torch.empty(0, 16, dtype=BF16, device=DEV)
    out = nv.nvfp4_vocab_loss(none, w, t[:0])
    assert out["loss"].shape == (0,)
    add = torch.randn(40, 16, device=DEV)
    g = nv.nvfp4_vocab_loss_backward(none, w, t[:0], out["lse"], d[:0], add=add)
    assert torch.equal(g["dw"], add) and g["dh"].shape == (0, 16)
    assert (nv.nvfp4_vocab_loss_backward(none, w, t[:0], out["lse"], d[:0])["dw"] == 0).all()
    out = nv.nvfp4_vocab_loss(h, none, t)  # no vocabulary: no row has a target
    assert (out["loss"] == 0).all()
    g = nv.nvfp4_vocab_loss_backward(h, none, t, out["lse"], d)
    assert (g["dh"] == 0).all() and g["dw"].shape == (0, 16)
    # k == 0: every logit is zero
    z = torch.empty(5, 0, dtype=BF16, device=DEV)
    out = nv.nvfp4_vocab_loss(z, torch.empty(40, 0, dtype=BF16, device=DEV), t.clamp(min=0))
    assert (out["loss"].double() - torch.log(torch.tensor(40.0, dtype=F64))).abs().max() < 16 * U * 4


@pytest.mark.parametrize("rows", [3, 100, 200])
def test_targets_far_below_the_others(rows):
    """Sums past fp32 relative to the target's logit: losses up to 2 x 10^4."""
    vocab, k = 1500, 64
    h, w, t, d = inputs(rows, vocab, k, ignored=0.0)
    w *= 0.05
    h[:, 0] = torch.linspace(1, 100, rows, device=DEV).to(BF16)
    w[:, 0] = torch.linspace(-100, 100, vocab, device=DEV).to(BF16)
    t[:] = torch.arange(rows, device=DEV, dtype=I32)
    out = nv.nvfp4_vocab_loss(h, w, t)
    want = exact_loss(h, w, t, 1.0)
    assert float(want[0].max()) > 1e4
    check_loss(out, want)
    # and the other way: the target far above, the loss a tiny number or zero
    t[:] = vocab - 1
    check_loss(nv.nvfp4_vocab_loss(h, w, t), exact_loss(h, w, t, 1.0))
    g = nv.nvfp4_vocab_loss_backward(h, w, t, out["lse"], d)
    for name, (v, bound) in exact_grads(h, w, t, out["lse"], d, 1.0).items():
        close(g[name], v, bound, name)


def test_infinite_logits():
    vocab, k = 600, 16
    h = torch.ones(70, k, dtype=BF16, device=DEV)
    w = torch.zeros(vocab, k, dtype=BF16, device=DEV)
    w[::2, 0] = -float("inf")  # half of the vocabulary has probability 0
    t = torch.arange(1, 71, dtype=I32, device=DEV) * 2 + 1
    out = nv.nvfp4_vocab_loss(h, w, t)
    ln = torch.log(torch.tensor(300.0, dtype=F64))
    assert ((out["loss"].double() - ln).abs() < 64 * U).all() and ((out["lse"].double() - ln).abs() < 64 * U).all()
    t[3] = 4  # a target of probability 0
    out = nv.nvfp4_vocab_loss(h, w, t)
    assert out["loss"][3] == float("inf") and abs(float(out["lse"][3]) - float(ln)) < 1e-5
    w[5, 0] = float("inf")
    assert torch.isnan(nv.nvfp4_vocab_loss(h, w, t)["loss"]).all()
    w[5, 0] = float("nan")
    assert torch.isnan(nv.nvfp4_vocab_loss(h, w, t)["loss"]).all()


@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_other_rows_reach_no_row(bad):
    h, w, t, d = inputs(300, 1000, 72, ignored=0.0)
    a = nv.nvfp4_vocab_loss(h, w, t)
    ga = nv.nvfp4_vocab_loss_backward(h, w, t, a["lse"], d)
    h2, d2 = h.clone(), d.clone()
    h2[7] = float(bad)
    d2[7] = float(bad)
    b = nv.nvfp4_vocab_loss(h2, w, t)
    keep = torch.arange(300, device=DEV) != 7
    assert torch.equal(a["loss"][keep], b["loss"][keep]) and not torch.isfinite(b["loss"][7])
    gb = nv.nvfp4_vocab_loss_backward(h2, w, t, b["lse"], d2)
    assert torch.equal(ga["dh"][keep], gb["dh"][keep])


def test_the_given_tensors_are_used():
    h, w, t, d = inputs(130, 700, 72)
    big = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)  # NaN patterns in the workspace
    out = {"loss": torch.full((130,), 9.0, device=DEV), "lse": torch.full((130,), 9.0, device=DEV)}
    got = nv.nvfp4_vocab_loss(h, w, t, out=out, workspace=big)
    assert got["loss"] is out["loss"] and torch.equal(got["loss"], nv.nvfp4_vocab_loss(h, w, t)["loss"])
    ref = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d)
    big.fill_(255)
    o = {"dh": torch.full((130, 72), 9.0, dtype=BF16, device=DEV), "dw": torch.full((700, 72), 9.0, device=DEV)}
    g = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, out=o, workspace=big)
    assert g["dw"] is o["dw"] and torch.equal(g["dw"], ref["dw"]) and torch.equal(g["dh"], ref["dh"])
    # in place onto earlier gradients, and one gradient alone
    before = torch.randn(700, 72, device=DEV)
    want = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, add=before)["dw"]
    buf = before.clone()
    g = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, add=buf, want_dh=False, out={"dw": buf})
    assert list(g) == ["dw"] and torch.equal(buf, want)
    g = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, want_dw=False)
    assert list(g) == ["dh"] and torch.equal(g["dh"], ref["dh"])


@pytest.mark.parametrize("rows", [40, 300])
def test_outputs_end_where_they_end(rows):
    """Bytes around the outputs and the workspace stay as they were."""
    vocab, k = 1003, 72
    h, w, t, d = inputs(rows, vocab, k)
    need = nv.lib().nvfp4_vocab_loss_backward_workspace(rows, vocab, k)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    dw = torch.full((vocab + 2, k), 5.0, device=DEV)
    dh = torch.full((rows + 2, k), 5.0, dtype=BF16, device=DEV)
    lse = nv.nvfp4_vocab_loss(h, w, t)["lse"]
    nv.nvfp4_vocab_loss_backward(h, w, t, lse, d, out={"dw": dw[1:-1], "dh": dh[1:-1]}, workspace=ws[:need])
    assert (dw[0] == 5).all() and (dw[-1] == 5).all() and (dh[0] == 5).all() and (dh[-1] == 5).all()
    assert (ws[need:] == 77).all()
    need = nv.lib().nvfp4_vocab_loss_workspace(rows, vocab, k)
    ws.fill_(77)
    loss = torch.full((rows + 2,), 5.0, device=DEV)
    l = torch.full((rows + 2,), 5.0, device=DEV)
    nv.nvfp4_vocab_loss(h, w, t, out={"loss": loss[1:-1], "lse": l[1:-1]}, workspace=ws[:need])
    assert (ws[need:] == 77).all()
    for v in (loss, l):
        assert v[0] == 5 and v[-1] == 5
    assert torch.equal(l[1:-1], lse)


def test_gradients_against_differences():
    """d(sum d_loss loss) along random directions of h and w, from bf16 points
    one step apart on both sides, in 64 bits for the difference itself."""
    h, w, t, d = inputs(20, 300, 64, ignored=0.2, std=2.0)
    lse = nv.nvfp4_vocab_loss(h, w, t)["lse"]
    g = nv.nvfp4_vocab_loss_backward(h, w, t, lse, d)

    def total(hh, ww):
        z = hh @ ww.t()
        l = torch.logsumexp(z, 1) - z.gather(1, t.long().clamp(min=0)[:, None])[:, 0]
        return float((l * d.double())[t >= 0].sum())
    gen = torch.Generator().manual_seed(3)
    hd, wd, eps = h.double(), w.double(), 1e-4
    ah = torch.randn(20, 64, generator=gen).to(DEV).double()
    aw = torch.randn(300, 64, generator=gen).to(DEV).double()
    # a difference's own error is of the order of eps^2; the gradients' that of dz's rounding
    num = (total(hd + eps * ah, wd) - total(hd - eps * ah, wd)) / (2 * eps)
    bound = exact_grads(h, w, t, lse, d, 1.0)
    slack = float((bound["dh"][1] * ah.abs()).sum()) + HALF[BF16] * float((g["dh"].double() * ah).abs().sum())
    assert abs(float((g["dh"].double() * ah).sum()) - num) <= slack + 1e-6 * abs(num)
    num = (total(hd, wd + eps * aw) - total(hd, wd - eps * aw)) / (2 * eps)
    assert abs(float((g["dw"].double() * aw).sum()) - num) <= float((bound["dw"][1] * aw.abs()).sum()) + 1e-6 * abs(num)


def test_equal_calls_equal_bits_and_streams():
    h, w, t, d = inputs(500, 3000, 264)
    a = nv.nvfp4_vocab_loss(h, w, t)
    ga = nv.nvfp4_vocab_loss_backward(h, w, t, a["lse"], d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = nv.nvfp4_vocab_loss(h, w, t)
        gb = nv.nvfp4_vocab_loss_backward(h, w, t, b["lse"], d)
    s.synchronize()
    for x, y in ((a, b), (ga, gb)):
        for key in x:
            assert torch.equal(x[key], y[key]), key


def test_in_graphs_that_share_a_workspace():
    h, w, t, d = inputs(200, 2000, 136)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    out = {k: torch.empty(200, device=DEV) for k in ("loss", "lse")}
    grads = {"dh": torch.empty_like(h), "dw": torch.empty(2000, 136, device=DEV)}

    def fwd():
        nv.nvfp4_vocab_loss(h, w, t, out=out, workspace=ws)

    def bwd():
        nv.nvfp4_vocab_loss_backward(h, w, t, out["lse"], d, out=grads, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd()
        bwd()
    torch.cuda.current_stream().wait_stream(side)
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gf):
        fwd()
    with torch.cuda.graph(gb):
        bwd()
    for step in range(4):
        h2, _, t2, d2 = inputs(200, 2000, 136, seed=step + 1, ignored=0.1 * step)
        h.copy_(h2)
        t.copy_(t2)
        d.copy_(d2)
        gf.replay()
        gb.replay()
        torch.cuda.synchronize()
        e = nv.nvfp4_vocab_loss(h, w, t)
        eg = nv.nvfp4_vocab_loss_backward(h, w, t, e["lse"], d)
        for key in e:
            assert torch.equal(out[key], e[key])
        for key in eg:
            assert torch.equal(grads[key], eg[key])


def test_a_table_past_four_gigabytes():
    vocab, k = 1 << 20, 1032  # dw 4.3 GB, w 2.2 GB
    g = torch.Generator(device=DEV).manual_seed(0)
    w = torch.empty(vocab, k, dtype=BF16, device=DEV)
    for lo in range(0, vocab, 1 << 17):
        w[lo:lo + (1 << 17)] = torch.randn(1 << 17, k, generator=g, device=DEV).mul_(0.1)
    h = torch.randn(3, k, generator=g, device=DEV).to(BF16)
    t = torch.tensor([vocab - 1, 5, vocab // 2 + 77], dtype=I32, device=DEV)
    d = torch.tensor([0.5, -1.0, 2.0], device=DEV)
    out = nv.nvfp4_vocab_loss(h, w, t)
    z = torch.cat([h.double() @ w[lo:lo + (1 << 17)].double().t().contiguous() for lo in range(0, vocab, 1 << 17)], 1)
    lse = torch.logsumexp(z, 1)
    mag = k * U * float(h.abs().double().amax() * w.abs().double().amax()) * k ** 0.5 * 4
    assert ((out["lse"].double() - lse).abs() < mag + 64 * U * lse.abs()).all()
    got = nv.nvfp4_vocab_loss_backward(h, w, t, out["lse"], d)
    p = torch.exp(z - lse[:, None])
    p[torch.arange(3), t.long()] -= 1
    dz = p * d.double()[:, None]
    for rows in (slice(0, 300), slice(vocab // 2, vocab // 2 + 300), slice(vocab - 300, vocab)):
        want = torch.mm(dz[:, rows].t().contiguous(), h.double())
        size = torch.mm(dz[:, rows].abs().t().contiguous(), h.double().abs())
        assert ((got["dw"][rows].double() - want).abs() <= (HALF[BF16] + 1e-3) * size).all()


# pieces of the vocabulary: of 2^29 elements of dz, of 2048 columns at least and of 2^21 at most
@pytest.mark.parametrize("rows,vocab,k", [(40001, 14003, 16), (270001, 2500, 8), (300, 2 ** 21 + 77, 8), (3, 4500001, 8)])
def test_pieces_of_the_vocabulary(rows, vocab, k):
    h, w, t, d = inputs(rows, vocab, k, std=2.0)
    t[0] = vocab - 1
    got = nv.nvfp4_vocab_loss(h, w, t)
    check_loss(got, exact_loss(h, w, t, 1.0))
    g = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d)
    for name, (want, bound) in exact_grads(h, w, t, got["lse"], d, 1.0).items():
        close(g[name], want, bound, name)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [5, 70, 333])
def test_an_infinite_row_of_the_table(rows):
    """A table row that every logit of is -infinity has probability 0 and a zero
    gradient, whatever lies past the last row with a target."""
    h, w, t, d = inputs(rows, 1000, 64, ignored=0.0)
    h[:, 0] = h[:, 0].abs() + 1
    w[5, 0] = -float("inf")
    t[t == 5] = 6
    t[-2:] = -1
    got = nv.nvfp4_vocab_loss(h, w, t)
    assert torch.isfinite(got["loss"]).all()
    dw = nv.nvfp4_vocab_loss_backward(h, w, t, got["lse"], d, want_dh=False)["dw"]
    assert (dw[5] == 0).all() and torch.isfinite(dw).all()
