"""What the operators between a history's encoder and its loss are measured on.

An encoder's blocks add their outputs to a stream of rows, one row per event,
and normalise it (layer norm, with the residual sum taken on the way); the
last normalised rows are scored against the table of all items, and the loss
is the softmax cross entropy of the item that came next.  Both operators are
measured alone (encoding, evaluation) and with their gradients (training).

``own`` says which side ``run`` computes: the plain form in elementary torch
operations (32 bits whatever the inputs' type, rounded once at the end), or
the framework's calls.  Both take what ``prepare`` makes.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one user's newest event on its way through a block
        dict(name="norm 1 row bf16", op="norm", dtype="bf16", rows=1, dim=256, residual=True, affine=True, pad=0),
        # the rows of a ranking batch's histories (60,515 events of 4 heads x 64)
        dict(name="norm stream bf16", op="norm", dtype="bf16", rows=60515, dim=256, residual=True, affine=True, pad=0),
        # fp32 pooled rows, a part of a wider buffer, normalised without weights
        dict(name="norm pooled fp32", op="norm", dtype="f32", rows=12029, dim=200, residual=False, affine=False, pad=56),
        # a block's norm in a training step
        dict(name="norm train bf16", op="norm train", dtype="bf16", rows=50523, dim=512, residual=True, affine=True, pad=0),
        # wide rows, fp16: the concatenated pooled rows of 32 tables
        dict(name="norm train wide f16", op="norm train", dtype="f16", rows=8192, dim=4096, residual=False, affine=True,
             pad=0),
        # a small model in fp32 with an odd width
        dict(name="norm train odd fp32", op="norm train", dtype="f32", rows=3727, dim=77, residual=True, affine=True, pad=0),
        # one user's held-out event scored against a catalogue
        dict(name="loss of 1 row bf16", op="loss", dtype="bf16", rows=1, items=50000, dim=64, scale=1.0, left_out=0.0, pad=0),
        # evaluation of a batch's last events against a catalogue beyond the cache
        dict(name="loss of 512 f16", op="loss", dtype="f16", rows=512, items=1000000, dim=128, scale=1.0, left_out=0.0,
             pad=0),
        # a small model's training step, some events without a label
        dict(name="loss train small bf16", op="loss train", dtype="bf16", rows=300, items=5000, dim=64, scale=1.0,
             left_out=0.1, pad=0),
        # a training step, a third of the padded batch's rows left out, rows of a wider buffer
        dict(name="loss train f16", op="loss train", dtype="f16", rows=4000, items=50021, dim=128, scale=1.0, left_out=0.3,
             pad=128),
        # the same in fp32, rows and items odd, with a temperature
        dict(name="loss train fp32", op="loss train", dtype="f32", rows=2050, items=20011, dim=96, scale=2.0, left_out=0.05,
             pad=0),
        # a large step over a large catalogue
        dict(name="loss train large bf16", op="loss train", dtype="bf16", rows=8192, items=131072, dim=256, scale=1.0,
             left_out=0.0, pad=0),
    ]


def draw(rng):
    """One more case of the listed ones' ranges."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["norm", "norm train", "loss", "loss train"])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), pad=rng.choice([0, 0, 8, 24, 129]))
        if op.startswith("norm"):
            c |= dict(rows=spread(1, 65536), dim=rng.choice([spread(1, 4096), 64 * rng.randint(1, 16)]),
                      residual=rng.random() < 0.5, affine=rng.random() < 0.8)
            if c["rows"] * c["dim"] > 3.3e7:
                continue
        else:
            c |= dict(rows=spread(1, 16384), items=spread(1, 1000000),
                      dim=rng.choice([16, 32, 48, 64, 96, 128, 192, 256, 384, 512, spread(1, 640)]),
                      scale=rng.choice([1.0, 1.0, 0.5, 2.5]), left_out=rng.choice([0.0, 0.0, 0.1, 0.5]))
            if c["rows"] * c["items"] > 1.08e9 or work(c)["flops"] > 1.65e12 or c["items"] * c["dim"] > 1.28e8:
                continue
        return c


def work(case):
    n, d, e = case["rows"], case["dim"], 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        streams = 4 if case["residual"] else 2  # x, residual in; sum, result out
        params, flops = 2 * d * e if case["affine"] else 0, 8 * n * d
        if case["op"] == "norm train":
            streams += 4 if case["residual"] else 3  # sum, upstream gradients (of both) in; gradient out
            params, flops = 2 * params, flops + 14 * n * d
        stats = 8 * n * (2 if case["op"] == "norm train" else 1)
        return {"bytes": streams * n * d * e + params + stats, "flops": flops}
    v = case["items"]
    if case["op"] == "loss":
        return {"bytes": (n + v) * d * e + 16 * n, "flops": 2 * n * v * d}
    # two products for the gradients; the logits' recomputation is not counted
    return {"bytes": 2 * (n + v) * d * e + 28 * n, "flops": 6 * n * v * d}


def prepare(case, seed):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    n, d = case["rows"], case["dim"]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std + mean).to(dt)

    st = {"case": case}
    wide = normal(n, d + case["pad"])
    if case["op"].startswith("norm"):
        # rows whose spread and mean differ, as a stream's rows do
        wide.mul_(torch.rand((n, 1), generator=g, device=dev).mul_(2).add_(0.25).to(dt))
        wide.add_(torch.randn((n, 1), generator=g, device=dev).mul_(0.5).to(dt))
        st["x"], st["eps"] = wide[:, :d], 1e-5
        st["residual"] = normal(n, d, std=2.0) if case["residual"] else None
        st["weight"] = normal(d, std=0.1, mean=1.0) if case["affine"] else None
        st["bias"] = normal(d, std=0.1) if case["affine"] else None
        if case["op"] == "norm train":
            st["grad"] = normal(n, d)
            st["grad_total"] = normal(n, d) if case["residual"] else None
    else:
        v = case["items"]
        st["x"] = wide[:, :d]
        st["table"] = normal(v, d, std=1.5 / math.sqrt(d))
        # items by popularity: the chance of item i falls as 1 / (i + 1)
        u = torch.rand((n,), generator=g, device=dev, dtype=torch.float64)
        st["targets"] = (torch.exp(u * math.log(v + 1.0)).long() - 1).clamp_(0, v - 1)
        left_out = torch.rand((n,), generator=g, device=dev) < case["left_out"]
        st["targets"][left_out] = -1
        if case["op"] == "loss train":
            # the mean over the labelled rows; fp16 gradients come with a loss scale
            labelled = (st["targets"] >= 0).sum().clamp_(min=1)
            st["grad"] = ((65536.0 if case["dtype"] == "f16" else 1.0) / labelled.float()).expand(n).contiguous()
    if own:
        import recommender_sparse_embeddings_gb300 as tbe

        # what a program keeps beside its weights: the handle, and a workspace of the batch's size
        train = case["op"].endswith("train")
        if case["op"].startswith("norm"):
            st["handle"] = tbe.tbe_layer_norm_create(d, dt, eps=st["eps"], weight=case["affine"], bias=case["affine"])
            if train:
                st["workspace"] = tbe.make_layer_norm_workspace(st["handle"], n, device=dev)
        else:
            st["handle"] = tbe.tbe_softmax_loss_create(d, dt, scale=case["scale"])
            st["workspace"] = tbe.make_softmax_loss_workspace(st["handle"], n, v, backward=train, device=dev)
    return st


# --------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if not own:
        return plain_norm(state) if op.startswith("norm") else plain_loss(state)
    import recommender_sparse_embeddings_gb300 as tbe

    h, x = state["handle"], state["x"]
    if op.startswith("norm"):
        w, b, r = state["weight"], state["bias"], state["residual"]
        out, total, stats = tbe.tbe_layer_norm_forward(h, x, weight=w, bias=b, residual=r)
        res = {"out": out, "total": total if r is not None else None}
        if op == "norm train":
            res["grad_x"], res["grad_weight"], res["grad_bias"] = tbe.tbe_layer_norm_backward(
                h, total, stats, state["grad"], weight=w, grad_total=state["grad_total"], workspace=state["workspace"])
        return res
    table, targets, ws = state["table"], state["targets"], state["workspace"]
    loss, lse = tbe.tbe_softmax_loss_forward(h, x, table, targets, workspace=ws)
    res = {"loss": loss, "lse": lse}
    if op == "loss train":
        res["grad_x"], res["grad_table"] = tbe.tbe_softmax_loss_backward(h, x, table, targets, lse, state["grad"],
                                                                         workspace=ws)
    return res


def plain_norm(state):
    x, r, w, b = state["x"], state["residual"], state["weight"], state["bias"]
    dt, res = x.dtype, {"total": None}
    t = x.float()
    if r is not None:
        res["total"] = (t + r.float()).to(dt)  # the stream as it is kept, and normalised
        t = res["total"].float()
    centred = t - t.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(-1, keepdim=True) + state["eps"])
    hat = centred * rstd
    y = hat if w is None else hat * w.float() + b.float()
    res["out"] = y.to(dt)
    if state["case"]["op"] == "norm train":
        g = state["grad"].float()
        a = g if w is None else g * w.float()
        gx = (a - a.mean(-1, keepdim=True) - hat * (a * hat).mean(-1, keepdim=True)) * rstd
        if r is not None:
            gx = gx + state["grad_total"].float()
        res["grad_x"] = gx.to(dt)
        res["grad_weight"] = (g * hat).sum(0).to(dt) if w is not None else None
        res["grad_bias"] = g.sum(0).to(dt) if w is not None else None
    return res


def plain_loss(state):
    case, targets = state["case"], state["targets"]
    x, w, dt = state["x"].float(), state["table"].float(), state["x"].dtype
    s = torch.matmul(x, w.t()).mul_(case["scale"])
    keep = targets >= 0
    at = targets.clamp(min=0)[:, None]
    picked = s.gather(1, at)[:, 0]
    most = s.amax(-1, keepdim=True)
    s.sub_(most).exp_()
    total = s.sum(-1, keepdim=True)
    lse = (most + total.log())[:, 0]
    res = {"loss": torch.where(keep, lse - picked, torch.zeros_like(lse)), "lse": lse}
    if case["op"] == "loss train":
        s.div_(total)
        s.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
        s.mul_((state["grad"] * keep * case["scale"])[:, None])
        res["grad_x"] = torch.matmul(s, w).to(dt)
        res["grad_table"] = torch.matmul(s.t(), x).to(dt)
    return res


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs in 64 bits from the definitions, the loss some rows at a time:
    y = (t - mean) / sqrt(var + eps) w + b with t the kept stream, loss_i = log sum_v exp(scale x_i.w_v) - scale x_i.w_target,
    and their derivatives."""
    st, f64 = prepare(case, seed), torch.float64
    x = st["x"].to(f64)
    if case["op"].startswith("norm"):
        kept = (x + st["residual"].to(f64)).to(st["x"].dtype) if case["residual"] else None
        t = x if kept is None else kept.to(f64)
        var, mean = torch.var_mean(t, dim=1, correction=0, keepdim=True)
        sd = torch.sqrt(var + st["eps"])
        hat = (t - mean) / sd
        w = st["weight"].to(f64) if case["affine"] else torch.ones(case["dim"], dtype=f64, device=x.device)
        res = {"total": t if case["residual"] else None, "out": hat * w + (st["bias"].to(f64) if case["affine"] else 0.0)}
        if case["op"] == "norm train":
            g = st["grad"].to(f64)
            slope = g * w
            # the derivative's projection: the parts along the ones and along hat fall out
            along = torch.einsum("nd,nd->n", slope, hat)[:, None] / case["dim"]
            res["grad_x"] = (slope - slope.sum(1, keepdim=True) / case["dim"] - along * hat) / sd
            if case["residual"]:
                res["grad_x"] = res["grad_x"] + st["grad_total"].to(f64)
            res["grad_weight"] = torch.einsum("nd,nd->d", g, hat) if case["affine"] else None
            res["grad_bias"] = g.sum(0) if case["affine"] else None
        return res
    w, n, v, scale = st["table"].to(f64), case["rows"], case["items"], case["scale"]
    loss, lse = torch.zeros(n, dtype=f64, device=x.device), torch.zeros(n, dtype=f64, device=x.device)
    train = case["op"] == "loss train"
    gx, gw = (torch.zeros_like(x), torch.zeros_like(w)) if train else (None, None)
    step = max(1, min(n, int(1e8) // v))
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        logits = scale * (x[lo:hi] @ w.t())
        lse[lo:hi] = torch.logsumexp(logits, 1)
        target = st["targets"][lo:hi]
        row = torch.nonzero(target >= 0)[:, 0]
        loss[lo + row] = lse[lo + row] - logits[row, target[row]]
        if train:
            d = torch.softmax(logits, 1)
            d[row, target[row]] -= 1.0
            d *= torch.where(target >= 0, st["grad"][lo:hi].to(f64), 0.0)[:, None]
            gx[lo:hi] = scale * (d @ w)
            gw += scale * (d.t() @ x[lo:hi])
            del d
        del logits
    res = {"loss": loss, "lse": lse}
    if train:
        res |= {"grad_x": gx, "grad_table": gw}
    return res
