"""Plain 64-bit forms of the learner's operators (grouped bf16 products,
residual norms, expert combine, gradient clipping) and the error bounds the
GPU tests hold the kernels to.

U is the fp32 rounding unit; HALF the largest relative error of one rounding
to a type (half a step).  A sum of n terms in fp32, in any order, is within
n U sum|terms| of the exact one.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def spans(offsets, m_total):
    """Row ranges of the experts: offsets clamped to [0, m_total]."""
    out = []
    o = offsets.tolist()
    for a, b in zip(o[:-1], o[1:]):
        lo = min(max(a, 0), m_total)
        out.append((lo, min(max(b, lo), m_total)))
    return out


def gathered(x, row_index, m_total):
    x = x.double()
    if row_index is None:
        return x[:m_total]
    r = row_index[:m_total].long()
    ok = (r >= 0) & (r < x.shape[0])
    safe = torch.where(ok, r, torch.zeros_like(r))
    rows = x[safe] if x.shape[0] else torch.zeros(len(r), x.shape[1], dtype=torch.float64, device=x.device)
    return torch.where(ok[:, None], rows, torch.zeros_like(rows))


def product(way, a, offsets, b, row_index=None, m_total=None, add=None):
    """(exact, bound of an fp32 result) of the grouped product.  forward:
    a = x, b = w; dgrad: a = dy, b = w; wgrad: a = dy, b = x.  Rows that no
    expert owns are NaN in the exact result."""
    m_total = m_total if m_total is not None else (row_index.numel() if row_index is not None and way == "forward"
                                                   else a.shape[0])
    if way == "wgrad":
        x = gathered(b, row_index, m_total)
        n, k = a.shape[1], b.shape[1]
        y = torch.zeros(offsets.numel() - 1, n, k, dtype=torch.float64, device=a.device)
        bound = torch.zeros_like(y)
        for e, (lo, hi) in enumerate(spans(offsets, m_total)):
            if hi > lo:
                dy = a[lo:hi].double().t().contiguous()
                y[e] = dy @ x[lo:hi]
                bound[e] = (hi - lo + 1) * U * (dy.abs() @ x[lo:hi].abs())
        if add is not None:
            y += add.double()
            bound += U * (y.abs() + add.double().abs())
        return y, bound
    x = gathered(a, row_index, m_total)
    cols = b.shape[1] if way == "forward" else b.shape[2]
    y = torch.full((m_total, cols), float("nan"), dtype=torch.float64, device=a.device)
    bound = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(spans(offsets, m_total)):
        if hi > lo:
            w = b[e].double()
            w = w.t().contiguous() if way == "forward" else w
            y[lo:hi] = x[lo:hi] @ w
            bound[lo:hi] = (w.shape[0] + 1) * U * (x[lo:hi].abs() @ w.abs())
    return y, bound


def close(got, want, bound, what=""):
    """got is `want` up to the fp32 bound and one rounding to its type."""
    err = (got.double() - want).abs()
    lim = bound + HALF[got.dtype] * (want.abs() + bound) + 2.0 ** -133  # the last: one bf16 subnormal step
    bad = ~(err <= lim)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d entries out of bounds; first at %s: got %r, want %r, bound %g" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(lim[i])))


def norm_forward(x, residual, norm_weight, post_weight, gate, scale, eps):
    """(r', its fp32 bound) before rounding, in 64 bits; rows are normed by norm_of."""
    b = x.double()
    n = b if post_weight is None else norm_of(b, post_weight, eps)
    step = scale * n * (1.0 if gate is None else gate.double())
    r = step if residual is None else residual.double() + step
    return r, 64 * U * (step.abs() + (0 if residual is None else residual.double().abs()))


def norm_of(v, weight, eps):
    v = v.double()
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * weight.double()


def norm_backward(x, r, norm_weight, dh, dr, post_weight, gate, scale, eps):
    """{name: (exact, fp32 bound)} by the formulas, in 64 bits."""
    b, rr = x.double(), r.double()
    rows, d = b.shape
    one = torch.ones(d, dtype=torch.float64, device=x.device)
    g = one if gate is None else gate.double()
    t = torch.zeros_like(b) if dr is None else dr.double()
    at = t.abs()
    got = {}
    zero = torch.zeros(d, dtype=torch.float64, device=x.device)
    if dh is not None:
        q2 = 1 / torch.sqrt(rr.square().mean(1, keepdim=True) + eps)
        up = dh.double() * norm_weight.double()
        t = t + q2 * up - rr * q2 ** 3 * (up * rr).mean(1, keepdim=True)
        at = at + q2 * up.abs() + rr.abs() * q2 ** 3 * (up * rr).abs().mean(1, keepdim=True)
        dw2 = dh.double() * rr * q2
        got["d_norm_weight"] = (dw2.sum(0), (rows + 64) * U * dw2.abs().sum(0))
    elif norm_weight is not None:
        got["d_norm_weight"] = (zero, zero)
    got["d_residual"] = (t, 128 * U * at)
    dn, adn = scale * g * t, abs(scale) * g.abs() * at
    if post_weight is None:
        n = b
        got["dx"] = (dn, 160 * U * adn)
    else:
        w1 = post_weight.double()
        q1 = 1 / torch.sqrt(b.square().mean(1, keepdim=True) + eps)
        n = b * q1 * w1
        up, aup = dn * w1, adn * w1.abs()
        got["dx"] = (q1 * up - b * q1 ** 3 * (up * b).mean(1, keepdim=True),
                     256 * U * (q1 * aup + b.abs() * q1 ** 3 * (aup * b.abs()).mean(1, keepdim=True)))
        got["d_post_weight"] = ((dn * b * q1).sum(0), (rows + 256) * U * (adn * b.abs() * q1).sum(0))
    if gate is not None:
        dg, adg = scale * n * t, abs(scale) * n.abs() * at
        got["d_gate"] = (dg, 256 * U * adg) if gate.dim() == 2 else (dg.sum(0), (rows + 256) * U * adg.sum(0))
    return got


def route_layout(counts, topk_tokens, gen, device):
    """offsets of the given rows per expert and a row_index of random tokens."""
    offsets = torch.zeros(len(counts) + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(counts).cumsum(0)
    rows = torch.randint(0, topk_tokens, (int(offsets[-1]),), generator=gen, dtype=torch.int32)
    return offsets.to(device), rows.to(device)
