"""The two ends of a policy's learner step and the router's gate, as they are timed and compared.

Three families: the log-probability loss over a large vocabulary (forward,
backward), the embedding lookup (forward, backward) and the router's gate with
its balance loss (forward, backward).  Each has a plain form in elementary
torch operations (`own` false), the library's calls (`own` true) and the exact
values in 64 bits.
"""
import math

import torch

own = False

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
DTYPES = {"f32": F32, "bf16": BF16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # log-probabilities of a learner's batch: a quarter of the positions are prompt and padding, which have no target
        dict(name="loss", op="loss", way="forward", rows=8192, vocab=131072, k=2048, ignored=0.25, scale=1.0),
        # scoring 64 sampled tokens at the rollout's temperature: the table is the work
        dict(name="loss rollout", op="loss", way="forward", rows=64, vocab=131072, k=2560, ignored=0.0, scale=1.25),
        # gradients of that learner's batch for the last hidden rows and the table
        dict(name="loss backward", op="loss", way="backward", rows=8192, vocab=131072, k=2048, ignored=0.25, scale=1.0),
        # a short microbatch with a small table of odd length
        dict(name="loss backward small", op="loss", way="backward", rows=301, vocab=32003, k=1032, ignored=0.1,
             scale=0.7),
        # the batch's tokens looked up
        dict(name="embedding", op="embedding", way="forward", tokens=16384, vocab=131072, d=2560, table="bf16",
             out="bf16", zipf=1.0),
        # the same when a few tokens are generated
        dict(name="embedding decode", op="embedding", way="forward", tokens=64, vocab=131072, d=2048, table="bf16",
             out="bf16", zipf=1.0),
        # gradient of the whole table in fp32; tokens repeat as words do
        dict(name="embedding backward", op="embedding", way="backward", tokens=16384, vocab=131072, d=2048, dout="bf16",
             out="f32", zipf=1.0),
        # a short batch, mostly padding with one id, and a small table of odd width
        dict(name="embedding backward small", op="embedding", way="backward", tokens=4099, vocab=1003, d=513, dout="f32",
             out="f32", zipf=2.0),
        # the router's gate for a batch: weights over the 8 chosen of 128 experts, counts and the balance loss
        dict(name="gate", op="gate", way="forward", tokens=16384, experts=128, topk=8, normalize=True, ignored=0.1,
             zipf=1.1),
        # the same when a few tokens are generated
        dict(name="gate decode", op="gate", way="forward", tokens=64, experts=128, topk=8, normalize=True, ignored=0.0,
             zipf=1.1),
        # its backward pass
        dict(name="gate backward", op="gate", way="backward", tokens=16384, experts=128, topk=8, normalize=True,
             ignored=0.1, zipf=1.1),
        # a small layer of few experts, weights not renormalised
        dict(name="gate backward small", op="gate", way="backward", tokens=301, experts=8, topk=2, normalize=False,
             ignored=0.0, zipf=2.0),
    ]


def _size(rng, lo, hi, step=1):
    return max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["loss", "loss", "embedding", "embedding", "gate"])
    way = rng.choice(["forward", "backward"])
    if op == "loss":
        while True:
            c = dict(op=op, way=way, rows=_size(rng, 1, 8192), vocab=_size(rng, 500, 131072, rng.choice([1, 8, 128])),
                     k=_size(rng, 64, 4096, 8), ignored=rng.choice([0.0, 0.1, 0.5]), scale=rng.choice([1.0, 0.7, 1.25]))
            if _counted(c) * c["vocab"] * c["k"] <= 6144 * 131072 * 2048 and c["vocab"] * c["k"] <= 131072 * 2048:
                return c
    if op == "embedding":
        while True:
            c = dict(op=op, way=way, tokens=_size(rng, 1, 32768), vocab=_size(rng, 100, 131072),
                     d=_size(rng, 64, 8192, rng.choice([1, 8])), out=rng.choice(["f32", "bf16"]),
                     zipf=rng.choice([0.0, 1.0, 2.0]))
            c["table" if way == "forward" else "dout"] = rng.choice(["f32", "bf16"])
            if c["tokens"] * c["d"] <= 16384 * 2560 and c["vocab"] * c["d"] <= 131072 * 2048:
                return c
    while True:
        E = _size(rng, 1, 512)
        c = dict(op=op, way=way, tokens=_size(rng, 1, 16384), experts=E, topk=rng.randint(1, min(8, E)),
                 normalize=rng.random() < 0.5, ignored=rng.choice([0.0, 0.1, 0.5]), zipf=rng.choice([0.0, 1.1, 2.0]))
        if c["tokens"] * E <= 16384 * 128:
            return c


# ---------------------------------------------------------------------------
# inputs


def _counted(c):
    """Rows or tokens that are not left out."""
    n = c["rows"] if c["op"] == "loss" else c["tokens"]
    return n - int(n * c["ignored"])


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(1 + seed)

    def normal(*shape, std=1.0, dtype=F32):
        return torch.randn(*shape, generator=g, device=dev, dtype=F32).mul_(std).to(dtype)

    def tokens(n, vocab, zipf):  # ids as frequent as their rank says, ranks dealt at random
        rank = torch.randperm(vocab, generator=g, device=dev).to(F32) + 1
        return torch.multinomial(rank ** -zipf, n, replacement=True, generator=g).to(I32)

    def left_out(n, share):
        mask = torch.zeros(n, dtype=torch.bool, device=dev)
        mask[torch.randperm(n, generator=g, device=dev)[:int(n * share)]] = True
        return mask

    s = {"c": c}
    if c["op"] == "loss":
        s["h"] = normal(c["rows"], c["k"], dtype=BF16)
        s["w"] = normal(c["vocab"], c["k"], std=2.0 / math.sqrt(c["k"]), dtype=BF16)  # logits of a few units
        s["targets"] = tokens(c["rows"], c["vocab"], 1.0).masked_fill_(left_out(c["rows"], c["ignored"]), -1)
        if c["way"] == "backward":
            s["lse"] = _plain_loss(s)["lse"]  # saved by the forward pass
            s["d_loss"] = normal(c["rows"], std=1.0 / c["rows"])  # advantages over the batch
    elif c["op"] == "embedding":
        s["ids"] = tokens(c["tokens"], c["vocab"], c["zipf"])
        if c["way"] == "forward":
            s["table"] = normal(c["vocab"], c["d"], std=0.02, dtype=DTYPES[c["table"]])
        else:
            s["dout"] = normal(c["tokens"], c["d"], std=0.1, dtype=DTYPES[c["dout"]])
    else:
        T, E = c["tokens"], c["experts"]
        rank = torch.randperm(E, generator=g, device=dev).to(F32) + 1
        s["logits"] = normal(T, E) - c["zipf"] * torch.log(rank)
        s["experts"] = s["logits"].topk(c["topk"], dim=1).indices.to(I32)
        s["valid"] = ~left_out(T, c["ignored"]) if c["ignored"] else None
        if c["way"] == "backward":
            # the forward pass's counts: choices of each expert by the tokens that count, and those tokens
            keep = s["experts"] if s["valid"] is None else s["experts"][s["valid"]]
            s["counts"] = torch.cat([torch.bincount(keep.reshape(-1).long(), minlength=E),
                                     torch.tensor([len(keep)], device=dev)]).to(I32)
            s["d_weights"] = normal(T, c["topk"], std=0.1)
            s["d_loss"] = torch.tensor(0.01, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import nvfp4_token_quantization_amd as nv
    c = s["c"]
    if c["op"] == "loss":
        if c["way"] == "forward":
            return nv.nvfp4_vocab_loss(s["h"], s["w"], s["targets"], scale=c["scale"])
        return nv.nvfp4_vocab_loss_backward(s["h"], s["w"], s["targets"], s["lse"], s["d_loss"], scale=c["scale"],
                                            dw_dtype=BF16)
    if c["op"] == "embedding":
        if c["way"] == "forward":
            return nv.nvfp4_embedding(s["table"], s["ids"], scale=math.sqrt(c["d"]), out_dtype=DTYPES[c["out"]])
        return nv.nvfp4_embedding_backward(s["dout"], s["ids"], c["vocab"], scale=math.sqrt(c["d"]),
                                           out_dtype=DTYPES[c["out"]])
    if c["way"] == "forward":
        return nv.nvfp4_moe_gate(s["logits"], s["experts"], valid=s["valid"], normalize=c["normalize"])
    return nv.nvfp4_moe_gate_backward(s["logits"], s["experts"], s["counts"], d_weights=s["d_weights"],
                                      d_loss=s["d_loss"], valid=s["valid"], normalize=c["normalize"])


def _plain_loss(s):
    z = (s["h"].float() @ s["w"].float().T).mul_(s["c"]["scale"])
    top = z.amax(1)
    target = s["targets"].long()
    has = target >= 0
    zt = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    lse = top + z.sub_(top[:, None]).exp_().sum(1).log()
    return {"loss": torch.where(has, lse - zt, 0.0), "lse": torch.where(has, lse, 0.0)}


def _plain(s):
    c = s["c"]
    if c["op"] == "loss":
        if c["way"] == "forward":
            return _plain_loss(s)
        h, w, target = s["h"].float(), s["w"].float(), s["targets"].long()
        dz = (h @ w.T).mul_(c["scale"]).sub_(s["lse"][:, None]).exp_()
        one = torch.ones(c["rows"], 1, device=dz.device)
        dz.scatter_add_(1, target.clamp(min=0)[:, None], -one)
        dz.mul_(torch.where(target >= 0, s["d_loss"] * c["scale"], 0.0)[:, None])
        return {"dh": (dz @ w).to(BF16), "dw": (dz.T @ h).to(BF16)}
    if c["op"] == "embedding":
        if c["way"] == "forward":
            return (s["table"][s["ids"].long()].float() * math.sqrt(c["d"])).to(DTYPES[c["out"]])
        got = torch.zeros(c["vocab"], c["d"], device=s["dout"].device)
        got.index_add_(0, s["ids"].long(), s["dout"].float())
        return got.mul_(math.sqrt(c["d"])).to(DTYPES[c["out"]])
    E, at = c["experts"], s["experts"].long()
    p = (s["logits"] - s["logits"].amax(1, keepdim=True)).exp()
    p = p / p.sum(1, keepdim=True)
    mine = p.gather(1, at)
    total = mine.sum(1, keepdim=True)
    keep = torch.ones(c["tokens"], 1, device=p.device) if s["valid"] is None else s["valid"].float()[:, None]
    if c["way"] == "forward":
        chosen = torch.zeros_like(p).scatter_add_(1, at, keep.expand(-1, c["topk"]))
        counts = torch.cat([chosen.sum(0), keep.sum()[None]])
        sums = (p * keep).sum(0)
        share = counts[:E] / counts[:E].sum().clamp(min=1)
        return {"weights": (mine / total if c["normalize"] else mine) * keep, "counts": counts.to(I32),
                "prob_sums": sums, "loss": E * (share * sums).sum() / counts[E].clamp(min=1)}
    counts = s["counts"].float()
    up = (s["d_loss"] * E * counts[:E] / counts[:E].sum().clamp(min=1) / counts[E].clamp(min=1)).expand(c["tokens"], E)
    dw = s["d_weights"]
    got = p * (up - (p * up).sum(1, keepdim=True))
    if c["normalize"]:
        n = mine / total
        got = got.scatter_add(1, at, n * (dw - (n * dw).sum(1, keepdim=True)))
    else:
        got = got.scatter_add(1, at, mine * dw) - p * (mine * dw).sum(1, keepdim=True)
    return torch.where(keep > 0, got, 0.0)


# ---------------------------------------------------------------------------
# what a pass has to read, write and compute


def work(case):
    c = case
    if c["op"] == "loss":
        rows, V, k = c["rows"], c["vocab"], c["k"]
        n = _counted(c)
        if c["way"] == "forward":
            return {"bytes": n * k * 2 + V * k * 2 + rows * 12, "flops": 2 * n * V * k}
        # the logits again, then a product for each gradient
        return {"bytes": n * k * 2 + rows * k * 2 + V * k * 4 + rows * 12, "flops": 6 * n * V * k}
    if c["op"] == "embedding":
        n, V, d = c["tokens"], c["vocab"], c["d"]
        if c["way"] == "forward":
            # a row that several tokens name is read once
            return {"bytes": _distinct(n, V, c["zipf"]) * d * BYTES[c["table"]] + n * (d * BYTES[c["out"]] + 4),
                    "flops": n * d}
        return {"bytes": n * (d * BYTES[c["dout"]] + 4) + V * d * BYTES[c["out"]], "flops": 2 * n * d}
    T, E, K = c["tokens"], c["experts"], c["topk"]
    if c["way"] == "forward":
        return {"bytes": T * E * 4 + T * K * 8 + E * 8, "flops": 6 * T * E}
    return {"bytes": T * E * 8 + T * K * 8 + E * 4, "flops": 8 * T * E}


def _distinct(n, vocab, zipf):
    """Expected number of different ids among n tokens."""
    p = torch.arange(1, vocab + 1, dtype=torch.float64) ** -zipf
    return int(round(float((1 - (1 - p / p.sum()) ** n).sum())))


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "loss":
        rows, V, a = c["rows"], c["vocab"], c["scale"]
        h, w, t = s["h"].double(), s["w"].double(), s["targets"].long()
        kept = torch.nonzero((t >= 0) & (t < V))[:, 0]
        wt = w.t().contiguous()
        loss, lse = torch.zeros(rows, dtype=f64, device="cuda"), torch.zeros(rows, dtype=f64, device="cuda")
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
        for at in kept.split(1024):
            z = a * torch.mm(h[at], wt)
            if c["way"] == "forward":
                lse[at] = torch.logsumexp(z, 1)
                loss[at] = lse[at] - z[torch.arange(len(at), device="cuda"), t[at]]
                continue
            dz = torch.exp(z - s["lse"][at].double()[:, None])
            dz[torch.arange(len(at), device="cuda"), t[at]] -= 1
            dz *= a * s["d_loss"][at].double()[:, None]
            dh[at] = torch.mm(dz, w)
            dw += torch.mm(dz.t().contiguous(), h[at])
        return {"loss": loss, "lse": lse} if c["way"] == "forward" else {"dh": dh, "dw": dw}
    if c["op"] == "embedding":
        ids, a = s["ids"].long(), math.sqrt(c["d"])
        if c["way"] == "forward":
            return a * torch.index_select(s["table"], 0, ids).double()
        # tokens in the order of their ids: a row's sum is the difference of running sums, piece by piece of the columns
        order = torch.argsort(ids, stable=True)
        ends = torch.searchsorted(ids[order], torch.arange(c["vocab"] + 1, device="cuda"))
        got = torch.empty(c["vocab"], c["d"], dtype=f64, device="cuda")
        for lo in range(0, c["d"], 512):
            run = torch.zeros(c["tokens"] + 1, min(512, c["d"] - lo), dtype=f64, device="cuda")
            run[1:] = s["dout"][order, lo:lo + 512].double().cumsum(0)
            got[:, lo:lo + 512] = a * (run[ends[1:]] - run[ends[:-1]])
        return got
    E, K = c["experts"], c["topk"]
    T = c["tokens"]
    ok = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    x, at = s["logits"].double(), s["experts"].long()
    p = torch.softmax(x, 1)
    hit = torch.nn.functional.one_hot(at, E).to(f64)  # [T, K, E]
    chosen = hit.sum(1)
    pc = p * chosen
    norm = pc.sum(1) if c["normalize"] else torch.ones(T, dtype=f64, device="cuda")
    if c["way"] == "forward":
        weights = torch.stack([(p * hit[:, j]).sum(1) / norm for j in range(K)], 1)
        counts = torch.cat([chosen[ok].sum(0), ok.sum()[None].to(f64)])
        sums = p[ok].sum(0)
        loss = E * torch.dot(counts[:E], sums) / (counts[:E].sum() * counts[E]) if bool(ok.any()) else torch.zeros((), dtype=f64)
        return {"weights": torch.where(ok[:, None], weights, 0.0), "counts": counts.to(I32), "prob_sums": sums, "loss": loss}
    # d loss / d x by the chain through p: the weights are p at the chosen over `norm`
    cn = s["counts"].double()
    gp = s["d_loss"].double() * E * cn[:E] / (cn[:E].sum() * cn[E]) * torch.ones(T, 1, dtype=f64, device="cuda")
    dw = s["d_weights"].double()
    for j in range(K):
        gp = gp + hit[:, j] * (dw[:, j] / norm)[:, None]
    if c["normalize"]:
        picked = (p[:, None, :] * hit).sum(2)
        gp = gp - chosen * ((dw * picked).sum(1) / norm ** 2)[:, None]
    dx = p * gp - p * (p * gp).sum(1, keepdim=True)
    return torch.where(ok[:, None], dx, 0.0)
