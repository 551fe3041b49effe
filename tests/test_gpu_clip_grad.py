"""GPU tests of the global gradient norm and clipping against 64 bits."""
import math

import pytest
import torch

import learner_refs as ref
import nvfp4_token_quantization_amd as nv

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def tensors(sizes, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to((F32, BF16)[i % 2]).to(DEV) for i, n in enumerate(sizes)]


def exact(grads, max_norm):
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check(grads, max_norm, got, norm):
    want, c = exact(grads, max_norm)
    assert norm.dtype == F32 and norm.dim() == 0
    assert abs(float(norm) - want) <= 2 * ref.U * want  # one rounding, and the fp64 sums'
    for i, (g, o) in enumerate(zip(grads, got)):
        assert o.dtype == g.dtype
        w = g.double() * c
        ref.close(o, w, 4 * ref.U * w.abs(), "tensor %d" % i)


SIZES = {"one value": [1], "few": [3, 5, 0, 1, 9], "chunk edges": [8191, 8192, 8193, 16384, 16385, 2048],
         "over a list": [17 + i for i in range(97)], "over two lists": [i % 5 for i in range(250)],
         "large": [3_000_001, 77, 2_500_000], "empty": [0, 0]}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes(sizes, max_norm):
    grads = tensors(SIZES[sizes], seed=3)
    kept = [t.clone() for t in grads]
    out = [torch.full_like(t, 3.0) for t in grads]
    check(kept, max_norm, out, nv.nvfp4_clip_grad_norm(grads, max_norm, out=out))
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    norm = nv.nvfp4_clip_grad_norm(grads, max_norm)  # in place
    check(kept, max_norm, grads, norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    only = nv.nvfp4_clip_grad_norm(kept, max_norm, norm_only=True)
    assert torch.equal(only, norm)


@pytest.mark.parametrize("std", [1e-35, 1e-22, 1e25, 1e37])
def test_squares_outside_fp32(std):
    grads = tensors([1000, 77], std=std)
    out = [torch.empty_like(t) for t in grads]
    check(grads, std, out, nv.nvfp4_clip_grad_norm(grads, std, out=out))


def test_unaligned_views():
    base = torch.randn(50_001, device=DEV)
    half = torch.randn(50_001, device=DEV).to(BF16)
    grads = [base[1:], half[3:], base[:0]]
    out = [torch.empty(50_000, device=DEV), torch.empty(49_999, dtype=BF16, device=DEV)[1:], torch.empty(0, device=DEV)]
    check(grads, 0.1, out, nv.nvfp4_clip_grad_norm(grads, 0.1, out=out))
    kept = [t.clone() for t in grads]
    check(kept, 0.1, grads, nv.nvfp4_clip_grad_norm(grads, 0.1))


def test_not_finite():
    grads = tensors([100, 50])
    grads[0][3] = float("inf")
    out = [torch.empty_like(t) for t in grads]
    assert float(nv.nvfp4_clip_grad_norm(grads, 1.0, out=out)) == math.inf
    assert out[0][3].isnan() and (out[1] == 0).all()
    grads[1][4] = float("nan")
    assert math.isnan(float(nv.nvfp4_clip_grad_norm(grads, 1.0, out=out)))
    assert out[0].isnan().all() and out[1].isnan().all()


def test_zero_gradients_and_zero_limit():
    grads = [torch.zeros(100, device=DEV)]
    assert float(nv.nvfp4_clip_grad_norm(grads, 1.0)) == 0 and (grads[0] == 0).all()
    grads = tensors([100])
    nv.nvfp4_clip_grad_norm(grads, 0.0)
    assert (grads[0] == 0).all()


def test_graph_replays_and_two_graphs_at_once():
    """Two captured calls with workspaces of their own, replayed on two streams."""
    sets = [tensors([70_000, 513, 9], seed=s) for s in (1, 2)]
    outs = [[torch.empty_like(t) for t in g] for g in sets]
    want = []
    for g in sets:
        o = [torch.empty_like(t) for t in g]
        want.append((nv.nvfp4_clip_grad_norm(g, 1.0, out=o), o))
    spaces = [torch.empty(nv.lib().nvfp4_clip_grad_norm_workspace(3), dtype=torch.uint8, device=DEV) for _ in sets]
    torch.cuda.synchronize()
    graphs, norms = [], []
    for g, o, ws in zip(sets, outs, spaces):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norms.append(nv.nvfp4_clip_grad_norm(g, 1.0, out=o, workspace=ws))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (n, o), norm, got in zip(want, norms, outs):
            assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(o, got))


def test_refusals():
    g = tensors([16, 16])
    for bad in (lambda: nv.nvfp4_clip_grad_norm([], 1.0), lambda: nv.nvfp4_clip_grad_norm([g[0], g[0]], 1.0),
                lambda: nv.nvfp4_clip_grad_norm([g[0], g[0][4:]], 1.0), lambda: nv.nvfp4_clip_grad_norm(g, 1.0, out=g[:1]),
                lambda: nv.nvfp4_clip_grad_norm([g[0].cpu()], 1.0), lambda: nv.nvfp4_clip_grad_norm([g[0][::2]], 1.0),
                lambda: nv.nvfp4_clip_grad_norm([g[0][:8], g[0][8:]], 1.0, out=[g[0][8:], g[0][:8]]),
                lambda: nv.nvfp4_clip_grad_norm(g, 1.0, out=g, norm_only=True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nv.nvfp4_clip_grad_norm([g[0].double()], 1.0)
    for bad in (-1.0, float("nan")):
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_clip_grad_norm(g, bad)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_clip_grad_norm(g, 1.0, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    # the same tensors out as in, given by the caller, are in place
    kept = [t.clone() for t in g]
    check(kept, 1.0, g, nv.nvfp4_clip_grad_norm(g, 1.0, out=list(g)))


def test_refuses_a_workspace_in_a_gradient():
    g = [torch.ones(1 << 16, device=DEV), torch.ones(8, device=DEV)]
    out = [torch.empty_like(t) for t in g]
    for space in (g[0], out[0]):
        with pytest.raises(ValueError):
            nv.nvfp4_clip_grad_norm(g, 1.0, out=out, workspace=space.view(torch.uint8))


@pytest.mark.parametrize("std,max_norm", [(1e37, 1e-3), (1e37, 0.5), (1e20, 1e-30), (1e38, 1e-33), (1e3, 1e-34)])
def test_factors_below_fp32(std, max_norm):
    """max_norm / norm under fp32's normal range (down to 1e-73 here), results
    inside it: max_norm, the factor and the product are rounded once each."""
    for sizes in ([1000, 77], [9000, 16384]):
        grads = tensors(sizes, std=std)
        for t in grads:
            t.clamp_(-3e38, 3e38)  # a draw past the type's range would be infinite
        out = [torch.empty_like(t) for t in grads]
        norm, (want, c) = nv.nvfp4_clip_grad_norm(grads, max_norm, out=out), exact(grads, max_norm)
        assert float(norm) == math.inf if want > 3.5e38 else abs(float(norm) - want) <= 2 * ref.U * want
        for i, (g, o) in enumerate(zip(grads, out)):
            w = g.double() * c
            ref.close(o, w, 4 * ref.U * w.abs(), "tensor %d" % i)
