"""GPU tests of the residual norms, forward and backward, against their 64-bit
form: every combination of parts and types, widths from 1 to 16384, the fused
quantization, gradients against differences, graphs and refusals."""
import itertools

import pytest
import torch

import learner_refs as ref
import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
EPS = 1e-6
WIDTHS = [1, 7, 8, 64, 71, 504, 512, 513, 520, 1024, 2048, 2560, 4100, 8192, 8200, 9001, 16384]


def make(rows, d, x=F32, r=BF16, p=F32, post=True, gate="channel", residual=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, dtype=F32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)
    c = dict(x=t(rows, d, dtype=x, std=3.0), residual=t(rows, d, dtype=r, std=2.0) if residual else None,
             norm_weight=t(d, dtype=p, std=0.3, mean=1.0), post_weight=t(d, dtype=p, std=0.3, mean=1.0) if post else None,
             gate={"none": lambda: None, "channel": lambda: t(d, dtype=p),
                   "element": lambda: t(rows, d, dtype=p)}[gate]())
    c["dh"], c["dr"] = t(rows, d, dtype=BF16), t(rows, d, dtype=r)
    return c


def forward(c, scale=0.7, **kw):
    return nv.nvfp4_residual_norm(c["x"], c["residual"], c["norm_weight"], post_weight=c["post_weight"], gate=c["gate"],
                                  scale=scale, eps=EPS, **kw)


def check_forward(c, got, scale=0.7):
    r, bound = ref.norm_forward(c["x"], c["residual"], c["norm_weight"], c["post_weight"], c["gate"], scale, EPS)
    ref.close(got["residual"], r, bound, "residual")
    if "h" in got:  # of the stored residual
        h = ref.norm_of(got["residual"], c["norm_weight"], EPS)
        ref.close(got["h"], h, 64 * ref.U * h.abs(), "h")


def backward(c, r, scale=0.7, **kw):
    return nv.nvfp4_residual_norm_backward(c["x"], r, c["norm_weight"], c["dh"], c["dr"], post_weight=c["post_weight"],
                                           gate=c["gate"], scale=scale, eps=EPS, **kw)


def check_backward(c, r, got, scale=0.7):
    want = ref.norm_backward(c["x"], r, c["norm_weight"], c["dh"], c["dr"], c["post_weight"], c["gate"], scale, EPS)
    assert set(got) == set(want)
    for key, (w, bound) in want.items():
        ref.close(got[key], w, bound, key)


@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d):
    c = make(9, d, seed=d)
    got = forward(c)
    check_forward(c, got)
    check_backward(c, got["residual"], backward(c, got["residual"]))


@pytest.mark.parametrize("x,r,p", list(itertools.product([F32, BF16], repeat=3)))
@pytest.mark.parametrize("d", [264, 77])
def test_types(x, r, p, d):
    for post, gate in itertools.product([True, False], ["none", "channel", "element"]):
        c = make(6, d, x, r, p, post, gate, seed=d)
        got = forward(c)
        assert got["residual"].dtype == r and got["h"].dtype == BF16
        check_forward(c, got)
        for dx in (F32, BF16):
            back = backward(c, got["residual"], dx_dtype=dx)
            assert back["dx"].dtype == dx and back["d_residual"].dtype == r
            check_backward(c, got["residual"], back)


@pytest.mark.parametrize("rows", [1, 2, 255, 1025, 5000])
def test_row_counts(rows):
    c = make(rows, 136, seed=rows)
    got = forward(c)
    check_forward(c, got)
    check_backward(c, got["residual"], backward(c, got["residual"]))


def test_parts_left_out():
    c = make(33, 264, residual=False)
    got = forward(c)
    assert got["residual"].dtype == BF16
    check_forward(c, got)
    got = forward(c, residual_dtype=F32)
    assert got["residual"].dtype == F32
    check_forward(c, got)
    # without the norm that follows (the last block), and its backward pass
    c = make(33, 264)
    c["norm_weight"] = None
    got = forward(c)
    assert set(got) == {"residual"}
    check_forward(c, got)
    c["dh"] = None
    check_backward(c, got["residual"], backward(c, got["residual"]))
    # only one of the two gradients
    c = make(33, 264)
    r = forward(c)["residual"]
    for gone in ("dh", "dr"):
        k = dict(c)
        k[gone] = None
        check_backward(k, r, backward(k, r))


@pytest.mark.parametrize("d", [16, 48, 512, 528, 2560, 8192, 16384])
@pytest.mark.parametrize("r", [F32, BF16])
def test_quantized_rows_have_the_quantizers_bits(d, r):
    c = make(21, d, r=r, seed=d)
    c["x"][3] = 0
    c["residual"][3] = 0
    c["x"][4] *= 1e6
    got = forward(c, want_amax=True, quantize=True)
    plain = forward(c)
    assert torch.equal(got["h"], plain["h"]) and torch.equal(got["residual"], plain["residual"])
    assert torch.equal(got["amax"], got["h"].float().abs().amax(1))
    q, sb, s = nv.nvfp4_quantize_rows(got["h"])
    assert torch.equal(got["q"], q) and torch.equal(got["sb"], sb) and torch.equal(got["s"], s)
    only = forward(c, want_h=False, quantize=True)
    assert set(only) == {"residual", "q", "sb", "s"} and torch.equal(only["q"], q)


def test_extremes():
    c = make(8, 264)
    c["x"][0] = 0            # a row of zeros
    c["x"][1] = 1e-30        # squares below fp32
    c["residual"][1] = 0
    c["x"][2] *= 1e15
    got = forward(c)
    check_forward(c, got)
    c["x"][3, 5] = float("nan")
    c["x"][4, 6] = float("inf")
    bad = forward(c)
    assert bad["h"][3].isnan().all() and bad["h"][4].isnan().any()
    keep = [0, 1, 2, 5, 6, 7]
    assert torch.equal(bad["h"][keep], got["h"][keep])  # each row by itself


def test_rows_do_not_depend_on_the_batch():
    c = make(3000, 528)
    whole = forward(c, quantize=True)
    part = dict(c, x=c["x"][1234:1241].contiguous(), residual=c["residual"][1234:1241].contiguous())
    few = forward(part, quantize=True)
    for key in ("residual", "h", "q", "sb", "s"):
        assert torch.equal(few[key], whole[key][1234:1241])


def test_offsets_past_32_bits():
    """Rows beyond 4 GiB of each operand have the bits they have on their own."""
    rows, d = 1_060_000, 1024
    c = make(8, d, seed=3)
    x = torch.empty(rows, d, dtype=F32, device=DEV)
    r = torch.empty(rows, d, dtype=F32, device=DEV)
    x[-8:], r[-8:] = c["x"], c["residual"].float()
    x[:-8] = 1.0
    r[:-8] = 0.5
    few = dict(c, x=x[-8:].clone(), residual=r[-8:].clone())
    want = forward(few)
    got = forward(dict(c, x=x, residual=r), out={"residual": r})
    for key in want:
        assert torch.equal(got[key][-8:], want[key])
    dh = torch.zeros(rows, d, dtype=BF16, device=DEV)
    dr = torch.zeros(rows, d, dtype=F32, device=DEV)
    dh[-8:], dr[-8:] = c["dh"], c["dr"].float()
    few.update(dh=dh[-8:].clone(), dr=dr[-8:].clone())
    want = backward(few, want["residual"])
    got = backward(dict(c, x=x, dh=dh, dr=dr), r, out={"d_residual": dr})
    for key in ("dx", "d_residual"):
        assert torch.equal(got[key][-8:], want[key])
    # the other rows' gradients are zero, so the column sums are the few rows', added in another order
    for key, (w, bound) in ref.norm_backward(few["x"], r[-8:], c["norm_weight"], few["dh"], few["dr"], c["post_weight"],
                                             c["gate"], 0.7, EPS).items():
        if key in ("d_post_weight", "d_norm_weight", "d_gate"):
            ref.close(got[key], w, bound, key)


def test_in_place_and_unaligned_rows():
    c = make(50, 520)
    want = forward(c)
    kept = c["residual"].clone()
    got = forward(dict(c, residual=kept), out={"residual": kept})
    assert got["residual"].data_ptr() == kept.data_ptr()
    assert torch.equal(kept, want["residual"]) and torch.equal(got["h"], want["h"])
    back = backward(c, want["residual"])
    dr = c["dr"].clone()
    again = backward(dict(c, dr=dr), want["residual"], out={"d_residual": dr})
    assert torch.equal(dr, back["d_residual"]) and torch.equal(again["dx"], back["dx"])
    # rows that start off 16 bytes take the narrow loads
    odd = torch.empty(50 * 520 + 1, dtype=F32, device=DEV)[1:].view(50, 520)
    odd.copy_(c["x"])
    got = forward(dict(c, x=odd))
    check_forward(c, got)
    with pytest.raises(nv.NVFP4Error):
        forward(dict(c, x=odd[:, :512].contiguous().view(-1)[:0].new_empty(50 * 512 + 1)[1:].view(50, 512),
                     residual=None, norm_weight=c["norm_weight"][:512].contiguous(),
                     post_weight=None, gate=None), quantize=True)


@pytest.mark.parametrize("gate", ["none", "channel", "element"])
def test_gradients_against_differences(gate):
    """Each gradient against central differences of the 64-bit forward form."""
    rows, d, scale = 3, 24, 0.7
    c = make(rows, d, F32, F32, F32, True, gate, seed=5)
    loss_h, loss_r = c["dh"].double(), c["dr"].double()
    names = ["x", "residual", "norm_weight", "post_weight"] + ([] if gate == "none" else ["gate"])
    v = {k: (None if c[k] is None else c[k].double()) for k in ("x", "residual", "norm_weight", "post_weight", "gate")}

    def loss(v):
        r, _ = ref.norm_forward(v["x"], v["residual"], v["norm_weight"], v["post_weight"], v["gate"], scale, EPS)
        return float((ref.norm_of(r, v["norm_weight"], EPS) * loss_h).sum() + (r * loss_r).sum())

    r = forward(c, scale)["residual"]
    got = backward(c, r, scale, dx_dtype=F32)
    key = {"x": "dx", "residual": "d_residual", "norm_weight": "d_norm_weight", "post_weight": "d_post_weight",
           "gate": "d_gate"}
    for name in names:
        size = float(got[key[name]].abs().max())
        for at in range(0, v[name].numel(), 5):
            step, two = 1e-4, []
            for sign in (1, -1):
                w = dict(v, **{name: v[name].clone()})
                w[name].view(-1)[at] += sign * step
                two.append(loss(w))
            diff = (two[0] - two[1]) / (2 * step)
            # third-order term of the differences and the fp32 rounding of r' and the sums
            assert abs(diff - float(got[key[name]].reshape(-1)[at])) <= 1e-4 * max(size, 1.0), (name, at)


def test_backward_repeats_bit_for_bit():
    c = make(3000, 520)
    r = forward(c)["residual"]
    first = backward(c, r)
    ws = torch.empty(nv.lib().nvfp4_residual_norm_backward_workspace(3000, 520), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        again = backward(c, r, workspace=ws)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_graph_replays():
    c = make(300, 528)
    r = forward(c)["residual"]
    want_f, want_b = forward(c, want_amax=True, quantize=True), backward(c, r)
    out_f = {k: torch.empty_like(v) for k, v in want_f.items()}
    out_b = {k: torch.empty_like(v) for k, v in want_b.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(c, want_amax=True, quantize=True, out=out_f)
        backward(c, r, out=out_b)
    for i in range(4):
        for t in list(out_f.values()) + list(out_b.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out_f[k], want_f[k]) for k in want_f)
        assert all(torch.equal(out_b[k], want_b[k]) for k in want_b)
        backward(c, r)


def test_no_rows():
    c = make(0, 264)
    got = forward(c, quantize=True)
    assert got["h"].shape == (0, 264)
    back = backward(c, got["residual"])
    for key in ("d_norm_weight", "d_post_weight", "d_gate"):
        assert (back[key] == 0).all()


def test_refusals():
    c = make(4, 264)
    for kw in (dict(residual=c["residual"][:3]), dict(norm_weight=c["norm_weight"][:8]), dict(gate=c["gate"][:8]),
               dict(x=c["x"].t()), dict(x=c["x"].cpu())):
        with pytest.raises(ValueError):
            forward(dict(c, **kw))
    for kw in (dict(x=c["x"].half()), dict(norm_weight=c["norm_weight"].bfloat16())):
        with pytest.raises(TypeError):
            forward(dict(c, **kw))
    with pytest.raises(ValueError):
        forward(dict(c, norm_weight=None), quantize=True)
    with pytest.raises(ValueError):
        forward(c, out={"residual": c["x"].view(BF16).view(-1)[:4 * 264].view(4, 264)})  # overlaps x
    with pytest.raises(ValueError):
        backward(dict(c, dh=None, dr=None), c["residual"])
    with pytest.raises(nv.NVFP4Error):
        forward(make(2, 24), quantize=True)          # d % 16
    with pytest.raises(nv.NVFP4Error):
        forward(make(2, 16385))                      # too wide
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_residual_norm(c["x"], c["residual"], c["norm_weight"], eps=-1.0)
    with pytest.raises(nv.NVFP4Error):
        backward(c, c["residual"], workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_refuses_outputs_and_workspaces_in_one_memory():
    c = make(4, 264)
    buf = torch.empty(4, 264, dtype=BF16, device=DEV)
    one = dict(c, residual=c["residual"].to(BF16))
    with pytest.raises(ValueError):
        forward(one, out={"residual": buf, "h": buf})
    stored = forward(one)["residual"]
    one["dr"] = one["dr"].to(BF16)
    with pytest.raises(ValueError):
        backward(one, stored, out={"dx": buf, "d_residual": buf})
    with pytest.raises(ValueError):
        backward(one, stored, out={"d_residual": one["dh"]})
    space = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    dx = space[:4 * 264 * 2].view(BF16).view(4, 264)
    with pytest.raises(ValueError):
        backward(one, stored, out={"dx": dx}, workspace=space)
    # in place where the calls allow it
    kept = one["dr"].clone()
    want = backward(dict(one, dr=kept), stored)
    got = backward(one, stored, out={"d_residual": one["dr"]})
    assert torch.equal(got["d_residual"], want["d_residual"]) and torch.equal(got["dx"], want["dx"])


def sized(rows, d, size, gate, r):
    """Rows of x and of the stored residual of about `size`, a dh with a part
    along the residual's rows, so that the projection term is as large as the
    others, and a dr of the gradient's own size."""
    c = make(rows, d, F32, r, F32, True, gate, seed=d)
    c["x"] = c["x"] / 3 * size
    stored = (c["residual"].float() / 2 * size).to(r)
    c["dh"] = (stored.float() / size + c["dh"].float()).to(BF16)
    c["dr"] = (c["dr"].float() / size).to(r)
    return c, stored


@pytest.mark.parametrize("size,eps", [(1e12, EPS), (1e14, EPS), (1e15, EPS), (1e17, EPS), (1e-13, 0.0), (1e-16, 0.0),
                                      (1e-15, 1e-33)])
@pytest.mark.parametrize("d,gate,r", [(264, "channel", BF16), (264, "element", F32), (77, "channel", F32), (8200, "none", BF16)])
def test_backward_of_very_large_and_very_small_rows(size, eps, d, gate, r):
    """rho^3 leaves fp32 long before the row of squares does."""
    c, stored = sized(7, d, size, gate, r)
    for dr in (c["dr"], None):
        got = nv.nvfp4_residual_norm_backward(c["x"], stored, c["norm_weight"], c["dh"], dr, post_weight=c["post_weight"],
                                              gate=c["gate"], scale=0.7, eps=eps, dx_dtype=F32)
        want = ref.norm_backward(c["x"], stored, c["norm_weight"], c["dh"], dr, c["post_weight"], c["gate"], 0.7, eps)
        assert set(got) == set(want)
        for key, (w, bound) in want.items():
            ref.close(got[key], w, bound, key)


@pytest.mark.parametrize("d", [264, 77, 8200])
def test_backward_of_zero_and_not_finite_rows(d):
    c = make(9, d, seed=d)
    stored = forward(c)["residual"]
    c["x"][1] = 0
    stored[2] = 0
    c["x"][3] = 0
    stored[3] = 0
    c["dh"][4] = 0
    c["dr"][4] = 0
    got = backward(c, stored)
    check_backward(c, stored, got)
    bad, bad_stored = dict(c, x=c["x"].clone(), dh=c["dh"].clone()), stored.clone()
    bad["x"][0, 5] = float("nan")
    bad["dh"][5, 7] = float("inf")
    bad_stored[8, 9] = float("nan")
    again = backward(bad, bad_stored)
    keep = [1, 2, 3, 4, 6, 7]
    for key in ("dx", "d_residual"):  # each row by itself
        assert torch.equal(again[key][keep], got[key][keep]), key
    assert again["dx"][0].isnan().all() and torch.equal(again["d_residual"][0], got["d_residual"][0])
    assert again["d_residual"][8].isnan().all() and again["dx"][8].isnan().all()
    assert again["dx"][5].isnan().any()


def test_outputs_of_other_names():
    """A name that the call does not know is refused before anything is
    written; an output it knows but was not asked for stays as it is."""
    c = make(5, 264)
    kept = {"residual": torch.full((5, 264), 3.0, dtype=BF16, device=DEV)}
    for name in ("residual_out", "d_residual", "H"):
        with pytest.raises(ValueError):
            forward(c, out=dict(kept, **{name: torch.empty(5, 264, dtype=BF16, device=DEV)}))
    assert (kept["residual"] == 3).all()
    amax = torch.full((5,), 7.0, device=DEV)
    got = forward(c, out={"amax": amax})
    assert "amax" not in got and (amax == 7).all()
    stored = got["residual"]
    with pytest.raises(ValueError):
        backward(c, stored, out={"d_x": torch.empty(5, 264, dtype=BF16, device=DEV)})
    gate = torch.full((264,), 7.0, device=DEV)
    back = backward(dict(c, gate=None), stored, out={"d_gate": gate})
    assert "d_gate" not in back and (gate == 7).all()
