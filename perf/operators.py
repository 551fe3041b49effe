"""The learner's operators around the low-precision experts, as they are timed and compared.

Four families: bf16 products grouped by expert (forward, data gradient, weight
gradient), the norms after and before a block fused with its gate and residual
(forward, backward), the sum over a token's experts (forward, backward), and
the global gradient norm with clipping.  Each has a plain form in elementary
torch operations (`own` false), the library's calls (`own` true) and the exact
values in 64 bits.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # the up-projection of a mixture-of-experts layer in bf16: 4096 tokens, 8 of 128 experts each, Zipf popularity
        dict(name="experts up", op="product", way="forward", tokens=4096, experts=128, topk=8, n=1536, k=2048,
             gather=True, out="f32", accumulate=False, zipf=1.1),
        # data gradient of that layer's down-projection, against its dequantized weights
        dict(name="experts down dgrad", op="product", way="dgrad", tokens=4096, experts=128, topk=8, n=2048, k=768,
             gather=False, out="bf16", accumulate=False, zipf=1.1),
        # weight gradient of the up-projection, every expert's fp32 gradient written
        dict(name="experts up wgrad", op="product", way="wgrad", tokens=4096, experts=128, topk=8, n=1536, k=2048,
             gather=True, out="f32", accumulate=False, zipf=1.1),
        # rollout decode: 64 tokens, the weights of the experts they hit are the work
        dict(name="experts decode", op="product", way="forward", tokens=64, experts=128, topk=8, n=1536, k=2048,
             gather=True, out="f32", accumulate=False, zipf=1.1),
        # a small layer with odd widths, added onto the gradients of an earlier microbatch; some experts stay empty
        dict(name="small wgrad", op="product", way="wgrad", tokens=301, experts=8, topk=2, n=520, k=1032,
             gather=True, out="f32", accumulate=True, zipf=2.0),
        # between two blocks of a training batch: norm of the block's fp32 output, channel gate, bf16 residual, next norm
        dict(name="norms", op="norm", way="forward", rows=16384, d=2560, x="f32", residual="bf16", post=True,
             gate="channel"),
        # the same point when a few tokens are generated
        dict(name="norms decode", op="norm", way="forward", rows=7, d=2048, x="f32", residual="bf16", post=True,
             gate="channel"),
        # its backward pass
        dict(name="norms backward", op="norm", way="backward", rows=16384, d=2560, x="f32", residual="bf16", post=True,
             gate="channel"),
        # a token's sum over its experts, forward and backward
        dict(name="combine", op="combine", way="forward", tokens=4096, topk=8, d=2048, y="f32", out="bf16"),
        dict(name="combine backward", op="combine", way="backward", tokens=4096, topk=8, d=2048, y="f32", out="bf16"),
        # clipping before the optimizer: fp32 expert gradients and bf16 dense ones of one layer
        dict(name="clip layer", op="clip", big=24, rows=4096, cols=2560, small=36, width=2560, scale=0.01),
        # few small tensors (adapters, norms), where latency counts
        dict(name="clip few", op="clip", big=3, rows=129, cols=513, small=5, width=77, scale=0.01),
    ]


def _size(rng, lo, hi, step=1):
    return max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["product", "product", "product", "norm", "norm", "combine", "clip"])
    if op == "product":
        while True:
            E = _size(rng, 1, 256)
            c = dict(op=op, way=rng.choice(["forward", "dgrad", "wgrad"]), tokens=_size(rng, 1, 8192), experts=E,
                     topk=rng.randint(1, min(8, E)), n=_size(rng, 64, 4096, 8), k=_size(rng, 64, 4096, 8),
                     gather=rng.random() < 0.5, out=rng.choice(["f32", "bf16"]), accumulate=False,
                     zipf=rng.choice([0.0, 1.1, 2.0]))
            c["accumulate"] = c["way"] == "wgrad" and c["out"] == "f32" and rng.random() < 0.5
            c["gather"] = c["gather"] and c["way"] != "dgrad"
            if c["tokens"] * c["topk"] * c["n"] * c["k"] <= 32768 * 1536 * 2048 and \
                    c["experts"] * c["n"] * c["k"] * (2 if c["accumulate"] else 1) <= 128 * 1536 * 2048:
                return c
    if op == "norm":
        while True:
            c = dict(op=op, way=rng.choice(["forward", "backward"]), rows=_size(rng, 1, 16384),
                     d=_size(rng, 64, 8192, rng.choice([1, 8, 16])), x=rng.choice(["f32", "bf16"]),
                     residual=rng.choice(["f32", "bf16"]), post=rng.random() < 0.7,
                     gate=rng.choice(["none", "channel", "element"]))
            if c["rows"] * c["d"] * (2 if c["gate"] == "element" else 1) <= 16384 * 2560:
                return c
    if op == "combine":
        while True:
            c = dict(op=op, way=rng.choice(["forward", "backward"]), tokens=_size(rng, 1, 16384), topk=rng.randint(1, 8),
                     d=_size(rng, 64, 8192, rng.choice([1, 8])), y=rng.choice(["f32", "bf16"]),
                     out=rng.choice(["f32", "bf16"]))
            if c["tokens"] * c["topk"] * c["d"] <= 4096 * 8 * 2048:
                return c
    return dict(op=op, big=rng.randint(1, 24), rows=_size(rng, 16, 4096), cols=_size(rng, 64, 2560),
                small=rng.randint(0, 36), width=_size(rng, 1, 8192), scale=rng.choice([0.0001, 0.01]))


# ---------------------------------------------------------------------------
# inputs


def _route(c, seed, device):
    """A router's choices: Gaussian logits with a Zipf popularity over the experts, top-k of them, in the contiguous
    per-expert layout (offsets, token of each routed row, routed row of each choice)."""
    g = torch.Generator(device=device).manual_seed(seed)
    T, E, K = c["tokens"], c["experts"], c["topk"]
    rank = torch.randperm(E, generator=g, device=device).to(F32) + 1
    logits = torch.randn(T, E, generator=g, device=device) - c["zipf"] * torch.log(rank)
    chosen = logits.topk(K, dim=1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=device)
    offsets[1:] = torch.bincount(chosen, minlength=E).cumsum(0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * K, device=device)
    i32 = torch.int32
    return offsets.to(i32), (order // K).to(i32), slot.reshape(T, K).to(i32)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(1 + seed)

    def normal(*shape, std=1.0, dtype=F32, mean=0.0):
        t = torch.randn(*shape, generator=g, device=dev, dtype=F32)
        return t.mul_(std).add_(mean).to(dtype)

    s = {"c": c}
    if c["op"] == "product":
        s["offsets"], s["row_index"], _ = _route(c, seed, dev)
        # the host's copy of the rows per expert, as a program has it that multiplies expert by expert
        s["bounds"] = s["offsets"].tolist()
        M = c["tokens"] * c["topk"]
        if not c["gather"]:
            s["row_index"] = None
        if c["way"] != "wgrad":
            s["w"] = normal(c["experts"], c["n"], c["k"], std=0.02, dtype=BF16)
        if c["way"] != "dgrad":
            s["x"] = normal(c["tokens"] if c["gather"] else M, c["k"], dtype=BF16)
        if c["way"] != "forward":
            s["dy"] = normal(M, c["n"], std=0.1, dtype=BF16)
        s["before"] = normal(c["experts"], c["n"], c["k"]) if c["accumulate"] else None
    elif c["op"] == "norm":
        R, D = c["rows"], c["d"]
        s["x"] = normal(R, D, std=0.7, dtype=DTYPES[c["x"]])
        s["residual"] = normal(R, D, std=2.0, dtype=DTYPES[c["residual"]])
        s["norm_weight"] = normal(D, std=0.2, mean=1.0)
        s["post_weight"] = normal(D, std=0.2, mean=1.0) if c["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: normal(D, std=0.3, mean=0.5),
                     "element": lambda: normal(R, D, std=0.3, mean=0.5)}[c["gate"]]()
        if c["way"] == "backward":  # the residual input then stands for the saved new residual
            s["d_residual"] = normal(R, D, std=0.1, dtype=DTYPES[c["residual"]])
            s["dh"] = normal(R, D, std=0.1, dtype=BF16)
    elif c["op"] == "combine":
        M = c["tokens"] * c["topk"]
        s["slot_of"] = torch.randperm(M, generator=g, device=dev).to(torch.int32).reshape(c["tokens"], c["topk"])
        s["weights"] = torch.softmax(normal(c["tokens"], c["topk"]), dim=1)
        s["y"] = normal(M, c["d"], dtype=DTYPES[c["y"]])
        if c["way"] == "backward":
            s["dout"] = normal(c["tokens"], c["d"], std=0.1, dtype=DTYPES[c["out"]])
    else:
        sizes = [(c["rows"], c["cols"])] * c["big"] + [(c["width"] + i,) for i in range(c["small"])]
        s["grads"] = [normal(*z, std=c["scale"], dtype=(F32, BF16)[i % 2]) for i, z in enumerate(sizes)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import nvfp4_token_quantization_amd as nv
    c = s["c"]
    if c["op"] == "product":
        if c["way"] == "forward":
            return nv.nvfp4_bf16_grouped_gemm(s["x"], s["offsets"], s["w"], row_index=s["row_index"],
                                              out_dtype=DTYPES[c["out"]])
        if c["way"] == "dgrad":
            return nv.nvfp4_bf16_grouped_dgrad(s["dy"], s["offsets"], s["w"], out_dtype=DTYPES[c["out"]])
        return nv.nvfp4_bf16_grouped_wgrad(s["dy"], s["x"], s["offsets"], row_index=s["row_index"], add=s["before"],
                                           out_dtype=DTYPES[c["out"]])
    if c["op"] == "norm":
        if c["way"] == "forward":
            return nv.nvfp4_residual_norm(s["x"], s["residual"], s["norm_weight"], post_weight=s["post_weight"],
                                          gate=s["gate"], scale=0.5, eps=EPS)
        return nv.nvfp4_residual_norm_backward(s["x"], s["residual"], s["norm_weight"], s["dh"], s["d_residual"],
                                               post_weight=s["post_weight"], gate=s["gate"], scale=0.5, eps=EPS)
    if c["op"] == "combine":
        if c["way"] == "forward":
            return nv.nvfp4_moe_combine(s["y"], s["slot_of"], s["weights"], out_dtype=DTYPES[c["out"]])
        return nv.nvfp4_moe_combine_backward(s["dout"], s["y"], s["slot_of"], s["weights"], dy_dtype=BF16)
    norm = nv.nvfp4_clip_grad_norm(s["grads"], 1.0, out=s["out"])
    return {"norm": norm, "out": s["out"]}


def _plain(s):
    c = s["c"]
    if c["op"] == "product":
        out = DTYPES[c["out"]]
        spans = list(zip(s["bounds"][:-1], s["bounds"][1:]))
        if c["way"] != "dgrad":
            x = s["x"] if s["row_index"] is None else s["x"][s["row_index"].long()]
        if c["way"] == "forward":
            return torch.cat([(x[a:b].float() @ s["w"][e].float().T).to(out) for e, (a, b) in enumerate(spans)])
        if c["way"] == "dgrad":
            return torch.cat([(s["dy"][a:b].float() @ s["w"][e].float()).to(out) for e, (a, b) in enumerate(spans)])
        dw = torch.stack([s["dy"][a:b].float().T @ x[a:b].float() for a, b in spans])
        return (dw + s["before"] if c["accumulate"] else dw).to(out)
    if c["op"] == "norm":
        x, r, w2 = s["x"].float(), s["residual"].float(), s["norm_weight"]
        rho1 = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        n = x * rho1 * s["post_weight"] if c["post"] else x
        gate = 1.0 if s["gate"] is None else s["gate"]
        if c["way"] == "forward":
            r = (r + 0.5 * gate * n).to(DTYPES[c["residual"]])
            h = r.float() * torch.rsqrt(r.float().square().mean(1, keepdim=True) + EPS) * w2
            return {"residual": r, "h": h.to(BF16)}
        dh = s["dh"].float()
        rho2 = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
        t = s["d_residual"].float() + rho2 * w2 * dh - r * rho2 ** 3 * (dh * w2 * r).mean(1, keepdim=True)
        dn = 0.5 * gate * t
        got = {"d_residual": t.to(DTYPES[c["residual"]]), "d_norm_weight": (dh * r * rho2).sum(0)}
        if c["post"]:
            got["d_post_weight"] = (dn * x * rho1).sum(0)
            m = dn * s["post_weight"]
            dx = rho1 * m - x * rho1 ** 3 * (m * x).mean(1, keepdim=True)
        else:
            dx = dn
        got["dx"] = dx.to(BF16)
        if c["gate"] != "none":
            dg = 0.5 * n * t
            got["d_gate"] = dg.sum(0) if c["gate"] == "channel" else dg
        return got
    if c["op"] == "combine":
        y = s["y"][s["slot_of"].long()].float()
        if c["way"] == "forward":
            return (y * s["weights"][:, :, None]).sum(1).to(DTYPES[c["out"]])
        dout = s["dout"].float()
        dy = torch.empty(s["y"].shape, dtype=BF16, device=y.device)
        dy[s["slot_of"].long()] = (dout[:, None, :] * s["weights"][:, :, None]).to(BF16)
        return {"dy": dy, "d_weights": (y * dout[:, None, :]).sum(2)}
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
    factor = torch.clamp(1.0 / (norm + 1e-6), max=1.0).float()
    return {"norm": norm.float(), "out": [(t.float() * factor).to(t.dtype) for t in s["grads"]]}


# ---------------------------------------------------------------------------
# what a pass has to read, write and compute


def _hit(c):
    """Experts that get at least one row, for one draw of the router's choices."""
    offsets, _, _ = _route(c, 0, "cpu")
    return int((offsets[1:] > offsets[:-1]).sum())


def work(case):
    c = case
    if c["op"] == "product":
        M, n, k = c["tokens"] * c["topk"], c["n"], c["k"]
        rows_x = c["tokens"] if c["gather"] else M
        weights = _hit(c) * n * k * 2
        if c["way"] == "forward":
            moved = rows_x * k * 2 + weights + M * n * BYTES[c["out"]]
        elif c["way"] == "dgrad":
            moved = M * n * 2 + weights + M * k * BYTES[c["out"]]
        else:
            moved = M * n * 2 + rows_x * k * 2 + c["experts"] * n * k * (8 if c["accumulate"] else BYTES[c["out"]])
        return {"bytes": moved, "flops": 2 * M * n * k}
    if c["op"] == "norm":
        e, x, r = c["rows"] * c["d"], BYTES[c["x"]], BYTES[c["residual"]]
        gate = 4 if c["gate"] == "element" else 0
        if c["way"] == "forward":
            return {"bytes": e * (x + 2 * r + 2 + gate), "flops": 9 * e}
        return {"bytes": e * (x + 3 * r + 2 + 2 + 2 * gate), "flops": 24 * e}
    if c["op"] == "combine":
        M = c["tokens"] * c["topk"] * c["d"]
        if c["way"] == "forward":
            return {"bytes": M * BYTES[c["y"]] + c["tokens"] * c["d"] * BYTES[c["out"]], "flops": 2 * M}
        return {"bytes": M * (BYTES[c["y"]] + 2) + c["tokens"] * c["d"] * BYTES[c["out"]], "flops": 3 * M}
    # the factor needs every gradient before the first can be scaled: counted as one read and one write all the same
    sizes = [c["rows"] * c["cols"]] * c["big"] + [c["width"] + i for i in range(c["small"])]
    return {"bytes": sum(n * (4, 2)[i % 2] * 2 for i, n in enumerate(sizes)), "flops": 3 * sum(sizes)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "product":
        M = c["tokens"] * c["topk"]
        expert = torch.bucketize(torch.arange(M, device="cuda"), s["offsets"][1:].long(), right=True)
        token = torch.arange(M, device="cuda") if s["row_index"] is None else s["row_index"].long()
        rows, cols = {"forward": (M, c["n"]), "dgrad": (M, c["k"]), "wgrad": (c["n"], c["k"])}[c["way"]]
        if c["way"] == "wgrad":
            got = s["before"].double() if c["accumulate"] else torch.zeros(c["experts"], rows, cols, dtype=torch.float64,
                                                                           device="cuda")
        else:
            got = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            of = torch.nonzero(expert == e)[:, 0]
            if not len(of):
                continue
            if c["way"] == "forward":
                got[of] = torch.mm(s["x"][token[of]].double(), s["w"][e].double().t().contiguous())
            elif c["way"] == "dgrad":
                got[of] = torch.mm(s["dy"][of].double(), s["w"][e].double())
            else:
                got[e] += torch.mm(s["dy"][of].double().t().contiguous(), s["x"][token[of]].double())
        return got
    if c["op"] == "norm":
        D, a = c["d"], 0.5
        b, r, w2 = (s[key].double() for key in ("x", "residual", "norm_weight"))
        w1 = s["post_weight"].double() if c["post"] else None
        g = torch.ones(D, dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double()
        q1 = 1 / torch.sqrt((b * b).sum(1) / D + EPS)[:, None]
        n = b if w1 is None else b * q1 * w1
        if c["way"] == "forward":
            new = r + a * g * n
            kept = new.to(DTYPES[c["residual"]]).double()
            return {"residual": new, "h": kept / torch.sqrt((kept * kept).sum(1) / D + EPS)[:, None] * w2}
        # the gradients by the rule of products and quotients, norm by norm
        def through(v, q, up):  # of v -> v q(v), for the gradient `up` of its result
            return q * (up - v * q * ((up * v * q).sum(1) / D)[:, None])
        q2 = 1 / torch.sqrt((r * r).sum(1) / D + EPS)[:, None]
        dh = s["dh"].double()
        t = s["d_residual"].double() + through(r, q2, dh * w2)
        got = {"d_residual": t, "d_norm_weight": (dh * (r * q2)).sum(0)}
        got["dx"] = a * g * t if w1 is None else through(b, q1, a * g * t * w1)
        if w1 is not None:
            got["d_post_weight"] = (a * g * t * (b * q1)).sum(0)
        if c["gate"] == "channel":
            got["d_gate"] = (a * t * n).sum(0)
        elif c["gate"] == "element":
            got["d_gate"] = a * t * n
        return got
    if c["op"] == "combine":
        at, p = s["slot_of"].long(), s["weights"].double()
        if c["way"] == "forward":
            got = torch.zeros(c["tokens"], c["d"], dtype=torch.float64, device="cuda")
            for j in range(c["topk"]):
                got += p[:, j, None] * s["y"][at[:, j]].double()
            return got
        dout = s["dout"].double()
        dy, dp = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda"), torch.empty_like(p)
        for j in range(c["topk"]):
            dy[at[:, j]] = p[:, j, None] * dout
            dp[:, j] = (s["y"][at[:, j]].double() * dout).sum(1)
        return {"dy": dy, "d_weights": dp}
    total = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in s["grads"]))
    return {"norm": torch.tensor(total, dtype=torch.float64), "out": [t.double() * min(1.0, 1.0 / (total + 1e-6))
                                                                    for t in s["grads"]]}
