"""GPU tests of the embedding lookup and its gradient by sorted tokens against
the definition in 64 bits.  A row of n tokens is summed in fp32 in some order:
within n U of the sum of the magnitudes, then scaled, added and rounded once
each."""
import pytest
import torch

import nvfp4_token_quantization_amd as nv
from learner_refs import U, close

pytestmark = pytest.mark.gpu

F32, BF16, I32, F64 = torch.float32, torch.bfloat16, torch.int32, torch.float64
DEV = "cuda:0"


def ids_of(n, vocab, how, seed=0):
    g = torch.Generator().manual_seed(seed + n + vocab)
    if how == "even":
        t = torch.randint(0, vocab, (n,), generator=g)
    elif how == "one":
        t = torch.full((n,), vocab - 1)
    elif how == "sorted":
        t = torch.arange(n) * vocab // max(n, 1)
    elif how == "skewed":
        t = (torch.rand(n, generator=g) ** 8 * vocab).long()
    else:  # with ids that are not in the table
        t = torch.randint(-vocab, 2 * vocab, (n,), generator=g)
        t[::7] = -2 ** 31
        t[3::7] = 2 ** 31 - 1
    return t.to(I32).to(DEV)


def randn(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def exact_grad(dout, ids, vocab, scale, add=None):
    i = ids.reshape(-1).long()
    ok = (i >= 0) & (i < vocab)
    d = dout.reshape(-1, dout.shape[-1])[ok].double()
    zero = torch.zeros(vocab, dout.shape[-1], dtype=F64, device=DEV)
    sums = zero.index_add(0, i[ok], d)
    size = zero.index_add(0, i[ok], d.abs())
    n = torch.bincount(i[ok], minlength=vocab)[:, None].double()
    want, bound = scale * sums, abs(scale) * size * (n + 2) * U
    if add is not None:
        want = want + add.double()
        bound = bound + 2 * U * (want.abs() + add.double().abs())
    return want, bound


@pytest.mark.parametrize("n,vocab,d", [(1, 1, 1), (1, 50, 512), (5, 3, 7), (64, 1000, 520), (333, 77, 513), (1000, 5000, 2048)])
@pytest.mark.parametrize("table,out", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_lookup(n, vocab, d, table, out):
    t, ids = randn(vocab, d, dtype=table), ids_of(n, vocab, "strange")
    got = nv.nvfp4_embedding(t, ids, scale=1.7, out_dtype=out)
    i = ids.long()
    ok = (i >= 0) & (i < vocab)
    # one product in fp32, one rounding: the bits of torch's own
    s = torch.tensor(1.7, dtype=F32, device=DEV)
    want = torch.where(ok[:, None], t[i.clamp(0, vocab - 1)].float() * s, 0.0).to(out)
    assert torch.equal(got, want)


SHAPES = [(1, 1, 1), (1, 9, 512), (7, 5, 8), (63, 100, 64), (64, 100, 513), (65, 4, 1024), (500, 2000, 72), (2047, 300, 40),
          (2048, 31, 40), (2049, 31, 40), (4100, 1003, 513), (9000, 70000, 64), (20000, 500, 520)]


@pytest.mark.parametrize("n,vocab,d", SHAPES)
@pytest.mark.parametrize("how", ["even", "one", "sorted", "skewed", "strange"])
def test_gradient(n, vocab, d, how):
    ids, dout = ids_of(n, vocab, how), randn(n, d)
    close(nv.nvfp4_embedding_backward(dout, ids, vocab, scale=0.5), *exact_grad(dout, ids, vocab, 0.5), how)


@pytest.mark.parametrize("n,vocab,d", [(65, 4, 1024), (500, 2000, 72), (3000, 300, 513)])
@pytest.mark.parametrize("dout_type", [F32, BF16])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("added", ["none", "add", "in place"])
def test_gradient_types_and_sums(n, vocab, d, dout_type, out_type, added):
    ids, dout = ids_of(n, vocab, "skewed"), randn(n, d, dtype=dout_type)
    add = None if added == "none" else randn(vocab, d, dtype=out_type, seed=5)
    want = exact_grad(dout, ids, vocab, 2.5, add)
    untouched = torch.bincount(ids.long(), minlength=vocab) == 0
    before = None if add is None else add.clone()
    got = nv.nvfp4_embedding_backward(dout, ids, vocab, scale=2.5, add=add, out=add if added == "in place" else None,
                                      out_dtype=out_type)
    assert got.dtype == out_type
    close(got, *want, added)
    if add is not None:
        assert torch.equal(got[untouched], before[untouched])


def test_order_of_the_tokens_is_kept():
    """A row's tokens are added as they come: 1 + 2^-24 + 2^-24 ... in fp32."""
    n = 40
    dout = torch.full((n, 8), 2.0 ** -24, device=DEV)
    dout[0] = 1.0
    ids = torch.zeros(n, dtype=I32, device=DEV)
    a = nv.nvfp4_embedding_backward(dout, ids, 1)
    b = nv.nvfp4_embedding_backward(dout.flip(0).contiguous(), ids, 1)
    assert (b > a).all()


@pytest.mark.parametrize("n", [100, 5000])
def test_values_that_are_not_finite_stay_in_their_row(n):
    ids, dout = ids_of(n, 50, "even"), randn(n, 64)
    bad = int(ids[17])
    dout[17, 3] = float("nan")
    dout[17, 4] = float("inf")
    got = nv.nvfp4_embedding_backward(dout, ids, 50)
    assert torch.isnan(got[bad, 3]) and got[bad, 4] == float("inf")
    mask = torch.ones_like(got, dtype=torch.bool)
    mask[bad, 3] = mask[bad, 4] = False
    assert torch.isfinite(got[mask]).all()
    dout[3] = float("nan")  # a token outside the table
    ids[3] = -1
    ids[17] = 50
    assert torch.isfinite(nv.nvfp4_embedding_backward(dout, ids, 50)).all()


def test_empty_problems_and_shapes():
    table = randn(9, 16)
    none = torch.empty(0, dtype=I32, device=DEV)
    assert nv.nvfp4_embedding(table, none).shape == (0, 16)
    assert (nv.nvfp4_embedding_backward(table[:0], none, 9) == 0).all()
    assert torch.equal(nv.nvfp4_embedding_backward(table[:0], none, 9, add=table), table)
    buf = table.clone()
    assert torch.equal(nv.nvfp4_embedding_backward(table[:0], none, 9, add=buf, out=buf), table)
    two = torch.arange(6, dtype=I32, device=DEV).view(2, 3)
    out = nv.nvfp4_embedding(table, two, out_dtype=F32)
    assert torch.equal(out, table[:6].view(2, 3, 16))
    g = nv.nvfp4_embedding_backward(out, two, 9)
    assert torch.equal(g[:6], table[:6]) and (g[6:] == 0).all()
    assert (nv.nvfp4_embedding(table[:0], two) == 0).all()  # no vocabulary
    assert nv.nvfp4_embedding_backward(out, two, 0).shape == (0, 16)


@pytest.mark.parametrize("d", [513, 1024])
def test_outputs_end_where_they_end(d):
    n, vocab = 3000, 200
    ids, dout = ids_of(n, vocab, "skewed"), randn(n, d)
    need = nv.lib().nvfp4_embedding_backward_workspace(n, d)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    buf = torch.full((vocab + 2, d), 5.0, device=DEV)
    nv.nvfp4_embedding_backward(dout, ids, vocab, out=buf[1:-1], workspace=ws[:need])
    assert (buf[0] == 5).all() and (buf[-1] == 5).all() and (ws[need:] == 77).all()
    assert torch.equal(buf[1:-1], nv.nvfp4_embedding_backward(dout, ids, vocab))
    out = torch.full((n + 2, d), 5.0, dtype=BF16, device=DEV)
    nv.nvfp4_embedding(buf[1:-1], ids, out=out[1:-1])
    assert (out[0] == 5).all() and (out[-1] == 5).all()


def test_rows_whose_memory_is_not_aligned():
    flat = torch.randn(50 * 64 + 1, generator=torch.Generator().manual_seed(0)).to(DEV)
    table = flat[1:].view(50, 64)  # 4-byte aligned
    ids = ids_of(700, 50, "even")
    out = nv.nvfp4_embedding(table, ids, out_dtype=F32)
    assert torch.equal(out, table[ids.long()])
    buf = torch.empty(50 * 64 + 1, device=DEV)[1:].view(50, 64)
    close(nv.nvfp4_embedding_backward(out, ids, 50, out=buf), *exact_grad(out, ids, 50, 1.0))


def test_equal_calls_equal_bits_streams_and_graphs():
    n, vocab, d = 6000, 4000, 264
    ids, dout = ids_of(n, vocab, "skewed"), randn(n, d, dtype=BF16)
    a = nv.nvfp4_embedding_backward(dout, ids, vocab)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = nv.nvfp4_embedding_backward(dout, ids, vocab)
    s.synchronize()
    assert torch.equal(a, b)
    table, ws = randn(vocab, d), torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    grad, out = torch.zeros(vocab, d, device=DEV), torch.empty(n, d, dtype=BF16, device=DEV)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        nv.nvfp4_embedding(table, ids, out=out)
    with torch.cuda.graph(graphs[1]):
        nv.nvfp4_embedding_backward(dout, ids, vocab, add=grad, out=grad, workspace=ws)
    want = torch.zeros(vocab, d, device=DEV)
    for step in range(4):
        ids.copy_(ids_of(n, vocab, ["even", "one", "skewed", "strange"][step], seed=step))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nv.nvfp4_embedding(table, ids))
        want = nv.nvfp4_embedding_backward(dout, ids, vocab, add=want)
        assert torch.equal(grad, want)


def test_a_table_past_four_gigabytes():
    vocab, d = (1 << 20) + 77, 1032
    ids = torch.tensor([vocab - 1, 0, vocab - 1, vocab // 2, 3], dtype=I32, device=DEV)
    table = torch.zeros(vocab, d, device=DEV)
    table[ids.long()] = randn(5, d)
    out = nv.nvfp4_embedding(table, ids, out_dtype=F32)
    assert torch.equal(out, table[ids.long()])
    g = nv.nvfp4_embedding_backward(out, ids, vocab, out=table)
    assert torch.equal(g[vocab - 1], out[0] + out[2]) and torch.equal(g[vocab // 2], out[3])
    assert int((g != 0).any(1).sum()) == 4


# sorted runs of 2048 are merged by eights: one, two and three times, with runs that are short or missing
@pytest.mark.parametrize("n", [16384, 16385, 32768 + 2049, 131072, 131073, 300001])
def test_long_batches_by_permutation(n):
    """Every id once: each row of the table is its token's, to the bit."""
    g = torch.Generator().manual_seed(n)
    ids, dout = torch.randperm(n, generator=g).to(I32).to(DEV), randn(n, 8)
    got = nv.nvfp4_embedding_backward(dout, ids, n)
    assert torch.equal(got[ids.long()], dout)


@pytest.mark.parametrize("n,vocab", [(40000, 1), (140001, 7000), (140001, 300)])
@pytest.mark.parametrize("how", ["even", "skewed", "strange"])
def test_long_batches(n, vocab, how):
    ids, dout = ids_of(n, vocab, how), randn(n, 8)
    got = nv.nvfp4_embedding_backward(dout, ids, vocab)
    close(got, *exact_grad(dout, ids, vocab, 1.0), how)
    assert torch.equal(got, nv.nvfp4_embedding_backward(dout, ids, vocab))
