"""GPU tests of the learner's calls in the checked build: the same bits as the
product library on valid inputs, decreasing offsets and non-finite rows to be
quantized refused with NVFP4_ERROR_PRECONDITION before anything is written."""
import pytest
import torch

import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


@pytest.fixture
def use():
    saved = nv._lib

    def pick(which):
        nv._lib = nv.load(nv.CHECKED_LIB_PATH if which == "checked" else nv.PRODUCT_LIB_PATH)
    yield pick
    nv._lib = saved


def calls():
    g = torch.Generator().manual_seed(1)

    def n(*s, dtype=BF16):
        return torch.randn(*s, generator=g).to(dtype).to(DEV)
    off = torch.tensor([0, 30, 30, 75], dtype=torch.int32, device=DEV)
    x, w, dy = n(75, 136), n(3, 72, 136), n(75, 72)
    r, nw = n(20, 256), n(256, dtype=F32)
    b = n(20, 256, dtype=F32)
    y, slot, p = n(40, 136, dtype=F32), torch.arange(40, dtype=torch.int32, device=DEV).view(20, 2), n(20, 2, dtype=F32)
    dout = n(20, 136)
    return off, b, {
        "forward": lambda **k: nv.nvfp4_bf16_grouped_gemm(x, off, w, **k),
        "dgrad": lambda **k: nv.nvfp4_bf16_grouped_dgrad(dy, off, w, **k),
        "wgrad": lambda **k: nv.nvfp4_bf16_grouped_wgrad(dy, x, off, **k),
        "norm": lambda **k: nv.nvfp4_residual_norm(b, r, nw, quantize=True, **k),
        "norm backward": lambda **k: nv.nvfp4_residual_norm_backward(b, r, nw, dh=r, d_residual=r, **k),
        "combine": lambda **k: nv.nvfp4_moe_combine(y, slot, p, **k),
        "combine backward": lambda **k: nv.nvfp4_moe_combine_backward(dout, y, slot, p, **k),
        "clip": lambda **k: nv.nvfp4_clip_grad_norm([b], 1.0, norm_only=True),
    }


def flat(v):
    return [v] if isinstance(v, torch.Tensor) else [v[k] for k in sorted(v)]


def test_same_bits_as_the_product_library(use):
    _, _, c = calls()
    for name, f in c.items():
        use("product")
        a = flat(f())
        use("checked")
        assert all(torch.equal(u, v) for u, v in zip(a, flat(f()))), name


def test_decreasing_offsets_are_refused(use):
    off, _, c = calls()
    use("checked")
    off[2] = 20
    for name, shape in (("forward", (75, 72)), ("dgrad", (75, 136)), ("wgrad", (3, 72, 136))):
        out = torch.full(shape, 9.0, device=DEV)
        with pytest.raises(nv.NVFP4Error) as e:
            c[name](out=out)
        assert e.value.status == nv.ERROR_PRECONDITION
        assert (out == 9).all(), name
    off[2] = 30
    c["forward"]()  # a valid call after refused ones


def test_rows_to_quantize_must_be_finite(use):
    _, b, c = calls()
    use("checked")
    b[19, 255] = float("nan")
    out = {"residual": torch.full((20, 256), 9.0, dtype=BF16, device=DEV)}
    with pytest.raises(nv.NVFP4Error) as e:
        c["norm"](out=out)
    assert e.value.status == nv.ERROR_PRECONDITION and (out["residual"] == 9).all()


@pytest.mark.parametrize("name", ["norm_weight", "post_weight", "gate", "gate by row"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_parameters_of_rows_to_quantize_must_be_finite(use, name, dtype):
    g = torch.Generator().manual_seed(2)

    def n(*s, t=dtype):
        return torch.randn(*s, generator=g).to(t).to(DEV)
    x, r = n(20, 256, t=F32), n(20, 256, t=BF16)
    p = {"norm_weight": n(256), "post_weight": n(256), "gate": n(20, 256) if name == "gate by row" else n(256)}
    use("checked")
    for kw in (dict(quantize=True), dict(want_amax=True)):
        nv.nvfp4_residual_norm(x, r, **p, **kw)
        for value in ("nan", "inf"):
            bad = dict(p)
            key = name.split()[0]
            bad[key] = p[key].clone()
            bad[key].view(-1)[-1] = float(value)
            out = {"residual": torch.full((20, 256), 9.0, dtype=BF16, device=DEV)}
            with pytest.raises(nv.NVFP4Error) as e:
                nv.nvfp4_residual_norm(x, r, **bad, out=out, **kw)
            assert e.value.status == nv.ERROR_PRECONDITION and (out["residual"] == 9).all()
            # without anything quantized such a parameter is IEEE arithmetic's business
            nv.nvfp4_residual_norm(x, r, **bad)
