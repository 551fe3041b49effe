"""GPU tests of the bf16 products grouped by expert (forward, dgrad, wgrad)
against their 64-bit form: ragged and empty experts, one row and none, odd
widths, rows through an index, outputs in both types, what a call leaves
untouched, graphs, streams and repeatability."""
import pytest
import torch

import learner_refs as ref
import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def bf16(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(BF16).to(DEV)


def case(counts, n, k, tokens=0, seed=0):
    """Operands of a layout with counts[e] rows per expert; tokens > 0: X is
    read through an index into that many rows."""
    g = torch.Generator().manual_seed(seed)
    M = sum(counts)
    offsets, index = ref.route_layout(counts, max(tokens, 1), g, DEV)
    return dict(offsets=offsets, index=index if tokens else None, x=bf16(g, tokens or M, k),
                w=bf16(g, len(counts), n, k, std=0.1), dy=bf16(g, M, n))


def run(way, c, **kw):
    if way == "forward":
        return nv.nvfp4_bf16_grouped_gemm(c["x"], c["offsets"], c["w"], row_index=c["index"], **kw)
    if way == "dgrad":
        return nv.nvfp4_bf16_grouped_dgrad(c["dy"], c["offsets"], c["w"], **kw)
    return nv.nvfp4_bf16_grouped_wgrad(c["dy"], c["x"], c["offsets"], row_index=c["index"], **kw)


def want(way, c, add=None):
    if way == "forward":
        return ref.product(way, c["x"], c["offsets"], c["w"], c["index"])
    if way == "dgrad":
        return ref.product(way, c["dy"], c["offsets"], c["w"])
    return ref.product(way, c["dy"], c["offsets"], c["x"], c["index"], add=add)


WAYS = ("forward", "dgrad", "wgrad")
LAYOUTS = {
    "one row": [1],
    "one row of many": [0, 1, 0],
    "few": [3, 0, 1, 2, 0, 7],
    "tile edges": [31, 32, 33, 63, 64, 65, 127, 128, 129],
    "large tiles": [255, 256, 257, 0, 300],
    "one expert": [700],
    "ends empty": [0, 0, 40, 0, 513, 0, 0],
}
WIDTHS = [(8, 8), (64, 64), (72, 200), (136, 520), (256, 256), (264, 1032), (512, 96)]


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("gather", [False, True], ids=["in place", "gathered"])
def test_layouts(way, layout, gather):
    c = case(LAYOUTS[layout], 136, 264, tokens=50 if gather else 0, seed=len(layout))
    ref.close(run(way, c), *want(way, c), way)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("out", [F32, BF16])
def test_widths(way, n, k, out):
    c = case([5, 0, 130, 64, 19], n, k, tokens=77, seed=n + k)
    got = run(way, c, out_dtype=out)
    assert got.dtype == out
    ref.close(got, *want(way, c), way)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("groups", [64, 65, 256, 300, 1024])
def test_many_experts(way, groups):
    g = torch.Generator().manual_seed(groups)
    counts = torch.randint(0, 4, (groups,), generator=g).tolist()
    counts[groups // 2] = 150
    c = case(counts, 64, 72, tokens=33, seed=groups)
    ref.close(run(way, c), *want(way, c), way)


@pytest.mark.parametrize("way", WAYS)
def test_long_sums_of_one_sign(way):
    """Same-sign products, where roundings add up instead of cancelling."""
    c = case([1900], 264, 2056, tokens=500, seed=9)
    for key in ("x", "w", "dy"):
        c[key] = c[key].abs()
    ref.close(run(way, c), *want(way, c), way)


@pytest.mark.parametrize("way", ("forward", "wgrad"))
def test_indices_outside_x_are_zero_rows(way):
    c = case([70, 0, 45], 72, 136, tokens=20, seed=3)
    c["index"][::5] = -1
    c["index"][3::7] = 20
    c["index"][60] = 2 ** 31 - 1
    c["index"][61] = -2 ** 31
    ref.close(run(way, c), *want(way, c), way)


@pytest.mark.parametrize("way", WAYS)
def test_rows_behind_the_last_expert(way):
    """NaN rows that no expert owns reach no result; their output rows stay as they were."""
    c = case([60, 30], 72, 136, seed=4)
    c["offsets"] = torch.tensor([10, 60, 83], dtype=torch.int32, device=DEV)
    for key in ("x", "dy"):
        c[key][:10] = float("nan")
        c[key][83:] = float("inf")
    y, bound = want(way, c)
    if way == "wgrad":
        ref.close(run(way, c), y, bound, way)
        return
    out = torch.full((100, y.shape[1]), 7.0, device=DEV)
    got = run(way, c, out=out)
    assert got.data_ptr() == out.data_ptr()
    ref.close(got[10:83], y[10:83], bound[10:83], way)
    assert (got[:10] == 7).all() and (got[83:] == 7).all()


@pytest.mark.parametrize("way", WAYS)
def test_nan_of_one_expert_stays_there(way):
    c = case([40, 33, 50], 72, 136, seed=5)
    c["x"][40:73] = float("nan")
    c["dy"][40:73] = float("nan")
    got, (y, bound) = run(way, c), want(way, c)
    keep = [0, 2] if way == "wgrad" else [i for i in range(123) if not 40 <= i < 73]
    ref.close(got[keep], y[keep], bound[keep], way)
    assert got[1 if way == "wgrad" else slice(40, 73)].isnan().all()


@pytest.mark.parametrize("way", WAYS)
def test_offsets_are_clamped(way):
    c = case([50, 50, 50], 64, 72, seed=6)
    c["offsets"] = torch.tensor([-5, 60, 60, 900], dtype=torch.int32, device=DEV)  # expert 1 owns nothing
    ref.close(run(way, c), *want(way, c), way)


@pytest.mark.parametrize("out", [F32, BF16])
def test_wgrad_adds_up(out):
    c = case([5, 0, 200, 64], 72, 136, tokens=77, seed=7)
    g = torch.Generator().manual_seed(1)
    add = torch.randn(4, 72, 136, generator=g).to(out).to(DEV)
    y, bound = want("wgrad", c, add=add)
    before = add.clone()
    ref.close(run("wgrad", c, add=add, out_dtype=out), y, bound, "apart")
    assert torch.equal(add, before)
    got = run("wgrad", c, add=add, out=add)
    assert got.data_ptr() == add.data_ptr()
    ref.close(got, y, bound, "in place")


def test_empty_sums_give_zeros():
    off = torch.tensor([0, 3, 3, 10], dtype=torch.int32, device=DEV)
    x, w = torch.empty(12, 0, dtype=BF16, device=DEV), torch.empty(3, 16, 0, dtype=BF16, device=DEV)
    out = torch.full((12, 16), 5.0, device=DEV)
    nv.nvfp4_bf16_grouped_gemm(x, off, w, out=out)
    assert (out[:10] == 0).all() and (out[10:] == 5).all()
    dy, w = torch.empty(12, 0, dtype=BF16, device=DEV), torch.empty(3, 0, 16, dtype=BF16, device=DEV)
    out = torch.full((12, 16), 5.0, device=DEV)
    nv.nvfp4_bf16_grouped_dgrad(dy, off, w, out=out)
    assert (out[:10] == 0).all() and (out[10:] == 5).all()
    # nothing to write at all
    none = torch.empty(0, 16, dtype=BF16, device=DEV)
    assert nv.nvfp4_bf16_grouped_gemm(none, off, torch.zeros(3, 8, 16, dtype=BF16, device=DEV)).shape == (0, 8)
    # every index outside an x without rows
    idx = torch.zeros(12, dtype=torch.int32, device=DEV)
    got = nv.nvfp4_bf16_grouped_gemm(none, off, torch.ones(3, 8, 16, dtype=BF16, device=DEV), row_index=idx)
    assert (got[:10] == 0).all()
    dy = torch.ones(12, 8, dtype=BF16, device=DEV)
    assert (nv.nvfp4_bf16_grouped_wgrad(dy, none, off, row_index=idx) == 0).all()


def test_wgrad_of_no_rows():
    c = case([0, 0], 72, 136, seed=8)
    assert (run("wgrad", c) == 0).all()
    add = torch.ones(2, 72, 136, device=DEV)
    assert (run("wgrad", c, add=add) == 1).all()


@pytest.mark.parametrize("way", WAYS)
def test_unaligned_row_counts_and_taller_outputs(way):
    c = case([17, 3], 72, 136, seed=10)
    if way == "wgrad":
        return
    cols = 72 if way == "forward" else 136
    out = torch.full((64, cols), 3.0, dtype=BF16, device=DEV)
    got = run(way, c, out=out)
    y, bound = want(way, c)
    ref.close(got[:20], y, bound, way)
    assert (got[20:] == 3).all()


@pytest.mark.parametrize("way", WAYS)
def test_repeatable_and_row_independent(way):
    c = case([300, 40, 0, 513], 136, 264, tokens=90, seed=11)
    first = run(way, c)
    for _ in range(3):
        assert torch.equal(run(way, c), first)


@pytest.mark.parametrize("way", WAYS)
def test_graph_replays(way):
    c = case([130, 0, 45], 136, 264, tokens=60, seed=12)
    eager = run(way, c)
    out = torch.empty_like(eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(way, c, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(way, c, out=out)
    for i in range(4):
        out.fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        # the host never reads the layout: a replay follows new offsets
        run(way, c)
    moved = c["offsets"].clone()
    c["offsets"].copy_(torch.tensor([0, 100, 150, 175], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref.close(out, *want(way, c), way)
    c["offsets"].copy_(moved)


def test_on_another_stream():
    c = case([130, 0, 45], 136, 264, tokens=60, seed=13)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = {way: run(way, c) for way in WAYS}
    s.synchronize()
    for way in WAYS:
        ref.close(got[way], *want(way, c), way)


def test_offsets_past_32_bits():
    """A weight and an output whose byte offsets pass 4 GiB: the last expert's rows."""
    n, k, E = 2048, 2048, 520  # 4.36 GB of weights
    g = torch.Generator(device=DEV).manual_seed(14)
    w = torch.empty(E, n, k, dtype=BF16, device=DEV)
    w[0] = torch.randn(n, k, generator=g, device=DEV).to(BF16)
    w[-1] = torch.randn(n, k, generator=g, device=DEV).to(BF16)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = 3
    offsets[-1] = 40
    x = torch.randn(40, k, generator=g, device=DEV).to(BF16)
    dy = torch.randn(40, n, generator=g, device=DEV).to(BF16)
    few = torch.tensor([0, 3, 40], dtype=torch.int32, device=DEV)
    ends = torch.stack([w[0], w[-1]])
    ref.close(nv.nvfp4_bf16_grouped_gemm(x, offsets, w), *ref.product("forward", x, few, ends), "forward")
    ref.close(nv.nvfp4_bf16_grouped_dgrad(dy, offsets, w), *ref.product("dgrad", dy, few, ends), "dgrad")
    dw = nv.nvfp4_bf16_grouped_wgrad(dy, x, offsets, out_dtype=BF16, out=w)  # the weights are no longer needed
    y, bound = ref.product("wgrad", dy, few, x)
    ref.close(dw[0], y[0], bound[0], "wgrad first")
    ref.close(dw[-1], y[1], bound[1], "wgrad last")
    assert (dw[1:-1] == 0).all()


def test_refusals():
    c = case([5, 6], 64, 72, seed=15)
    x, w, dy, off = c["x"], c["w"], c["dy"], c["offsets"]
    f, dg, wg = nv.nvfp4_bf16_grouped_gemm, nv.nvfp4_bf16_grouped_dgrad, nv.nvfp4_bf16_grouped_wgrad
    for bad in (lambda: f(x.float(), off, w), lambda: f(x, off.long(), w), lambda: f(x, off, w, out_dtype=torch.float16),
                lambda: wg(dy, x, off, add=torch.zeros(2, 64, 72, device=DEV),
                           out=torch.zeros(2, 64, 72, dtype=BF16, device=DEV))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(x[:, :64], off, w), lambda: f(x[:, ::2], off, w[:, :, :36].contiguous()),
                lambda: f(x, off[:2], w), lambda: f(x, off, w, m_total=12), lambda: f(x.cpu(), off, w),
                lambda: f(x, off, w, out=torch.empty(10, 64, device=DEV)), lambda: dg(dy, off, w[:, :56].contiguous()),
                lambda: wg(dy, x[:10], off), lambda: wg(dy, x, off, add=torch.zeros(2, 64, 64, device=DEV)),
                lambda: f(x, off, w, out=w.view(-1)[:704].view(11, 64)),
                lambda: wg(dy, x, off, row_index=off)):
        with pytest.raises(ValueError):
            bad()
    for n, k in ((60, 72), (64, 68)):
        with pytest.raises(nv.NVFP4Error):
            f(torch.zeros(11, k, dtype=BF16, device=DEV), off, torch.zeros(2, n, k, dtype=BF16, device=DEV))


# (way, counts, n, k): layouts that reach every tile shape the calls choose
# from on 256 CUs, ragged in rows, columns and the summed dimension
SHAPES = {
    "forward 256x256": ("forward", [1000, 0, 1700, 396, 1000], 12296, 72),
    "forward 192x128": ("forward", [700, 64, 193, 1091], 2440, 200),
    "forward 128x128": ("forward", [7, 30, 0, 1] * 16, 1032, 136),
    "forward 64x128": ("forward", [130, 64, 1, 40], 2440, 264),
    "forward 64x64": ("forward", [3, 0, 5, 1], 1032, 264),
    "forward 64x64 split": ("forward", [3, 0, 70], 264, 2312),
    "dgrad 128x256": ("dgrad", [300, 129, 0, 128, 1], 136, 8200),
    "dgrad 64x128": ("dgrad", [130, 64, 1, 40], 264, 2440),
    "dgrad 64x64": ("dgrad", [3, 0, 5, 1], 264, 1032),
    "dgrad 64x64 split": ("dgrad", [3, 0, 70], 2312, 264),
    "wgrad 256x128": ("wgrad", [140, 0, 1, 33, 257, 64, 128, 129], 1000, 1032),
    "wgrad 128x128": ("wgrad", [140, 0, 1, 33, 257, 64, 128, 129], 520, 1032),
    "wgrad 64x128": ("wgrad", [140, 0, 1, 33], 520, 1032),
    "wgrad 64x64": ("wgrad", [140, 0, 1, 33], 136, 1032),
    "wgrad 64x64 split": ("wgrad", [3000, 0, 130, 1500], 136, 264),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("out", [F32, BF16])
def test_every_tile_shape(shape, out):
    way, counts, n, k = SHAPES[shape]
    c = case(counts, n, k, tokens=0 if way == "dgrad" else 333, seed=n)
    if c["index"] is not None:
        c["index"][::7] = -1
    got = run(way, c, out_dtype=out)
    ref.close(got, *want(way, c), shape)
    assert torch.equal(run(way, c, out_dtype=out), got)


@pytest.mark.parametrize("shape", [s for s in SHAPES if not s.startswith("dgrad")])
def test_every_tile_shape_in_place_rows(shape):
    way, counts, n, k = SHAPES[shape]
    c = case(counts, n, k, seed=k)
    ref.close(run(way, c), *want(way, c), shape)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", [(136, 264), (1032, 2312)])
def test_rows_depend_on_their_own_rows_alone(way, n, k):
    """Other values (and no numbers at all) in the other rows, at the same
    sizes and offsets, leave a row's bits (an expert's, for wgrad) alone."""
    c = case([300, 40, 0, 513], n, k, seed=16)
    first = run(way, c)
    for value in (2.5, float("nan"), float("inf")):
        o = dict(c, x=c["x"].clone(), dy=c["dy"].clone())
        if way == "wgrad":
            for t in (o["x"], o["dy"]):
                t[:300], t[340:] = value, value
            assert torch.equal(run(way, o)[1], first[1])
            continue
        other = torch.arange(853, device=DEV) % 3 != 0
        o["x"][other], o["dy"][other] = value, value
        got = run(way, o)
        assert torch.equal(got[~other], first[~other])
        assert not torch.equal(got[other], first[other])


def test_wgrad_output_has_the_groups_exactly():
    c = case([17, 3], 72, 136, seed=10)
    for groups in (1, 3):
        with pytest.raises(ValueError):
            run("wgrad", c, out=torch.empty(groups, 72, 136, device=DEV))
