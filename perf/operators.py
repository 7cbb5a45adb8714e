"""What the sequence operators beside the embedding tables are measured on.

A user's history is a run of events, one looked-up embedding row each.  The
operators work on such runs: attention over the ragged histories of a batch
(each event sees the `window` newest events up to itself and the history's
first `sinks` events; a learned bias is added by the bucket of the distance),
its gradients, and the attention of one new event per user over a paged cache
of keys and values, to which the event is appended first.

``own`` says which side ``run`` computes: the plain form in elementary torch
operations (32 bits whatever the inputs' type, rounded once at the end), or
the framework's calls.  Both take what ``prepare`` makes.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one request's few short histories, encoded while the user waits
        dict(name="encode 3 short bf16", op="forward", dtype="bf16", batch=3, mean=20, sigma=0.6, longest=40,
             heads=2, kv_heads=2, dim=32, window=0, sinks=0, buckets=16, max_distance=64, law=1),
        # a ranking batch's histories: many, ragged, mostly far under the longest
        dict(name="encode 512 ragged bf16", op="forward", dtype="bf16", batch=512, mean=120, sigma=0.7, longest=510,
             heads=4, kv_heads=4, dim=64, window=128, sinks=4, buckets=32, max_distance=128, law=2),
        # life-long histories in a few shared key-value heads, windowed
        dict(name="encode long window f16", op="forward", dtype="f16", batch=5, mean=4500, sigma=0.5, longest=8191,
             heads=16, kv_heads=4, dim=128, window=1024, sinks=16, buckets=32, max_distance=1024, law=3),
        # histories straight from fp32 pooled rows, all earlier events visible
        dict(name="encode 64 fp32", op="forward", dtype="f32", batch=64, mean=190, sigma=0.5, longest=400,
             heads=4, kv_heads=2, dim=64, window=0, sinks=0, buckets=32, max_distance=128, law=4),
        # a training step on a batch of ragged histories
        dict(name="train 256 ragged bf16", op="train", dtype="bf16", batch=256, mean=200, sigma=0.8, longest=1000,
             heads=8, kv_heads=8, dim=64, window=256, sinks=4, buckets=32, max_distance=256, law=5),
        # all earlier events visible, equal lengths cut at a power of two
        dict(name="train full bf16", op="train", dtype="bf16", batch=8, mean=2048, sigma=0.0, longest=2048,
             heads=8, kv_heads=8, dim=64, window=0, sinks=0, buckets=32, max_distance=128, law=6),
        # long histories, four query heads to a key-value head, fp16
        dict(name="train long window f16", op="train", dtype="f16", batch=4, mean=6000, sigma=0.4, longest=8191,
             heads=8, kv_heads=2, dim=128, window=2000, sinks=8, buckets=64, max_distance=2000, law=7),
        # a small model in fp32 with an odd head width
        dict(name="train 40 fp32", op="train", dtype="f32", batch=40, mean=90, sigma=0.6, longest=260,
             heads=2, kv_heads=1, dim=40, window=50, sinks=2, buckets=8, max_distance=50, law=8),
        # one user's next event
        dict(name="next event of 1 bf16", op="decode", dtype="bf16", batch=1, mean=300, sigma=0.0, longest=300,
             heads=4, kv_heads=4, dim=64, window=0, sinks=0, buckets=32, max_distance=128, page=16, law=9),
        # a serving batch over whole histories
        dict(name="next event of 128 bf16", op="decode", dtype="bf16", batch=128, mean=4000, sigma=0.5, longest=8190,
             heads=16, kv_heads=4, dim=128, window=0, sinks=0, buckets=32, max_distance=1024, page=64, law=10),
        # few users with very long histories, of which a window and the first events are read
        dict(name="next event windowed f16", op="decode", dtype="f16", batch=12, mean=30000, sigma=0.5, longest=65000,
             heads=8, kv_heads=2, dim=64, window=4096, sinks=16, buckets=64, max_distance=4096, page=32, law=11),
        # fp32 caches of middling length
        dict(name="next event of 200 fp32", op="decode", dtype="f32", batch=200, mean=700, sigma=0.7, longest=2000,
             heads=6, kv_heads=6, dim=48, window=0, sinks=0, buckets=0, max_distance=0, page=20, law=12),
    ]


def draw(rng):
    """One more case of the listed ones' ranges."""
    def spread(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n + 1 if n == 3072 else n  # no size has this value

    while True:
        op = rng.choice(["forward", "train", "decode"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        kv = rng.choice([1, 2, 4, 6, 8])
        heads = kv * rng.choice([1, 1, 2, 3, 4])
        if heads > 16:
            continue
        dim = rng.choice([16, 32, 40, 48, 64, 64, 80, 96, 128, 128])
        longest = spread(1, 60000 if op == "decode" else 8192)
        batch = spread(1, 512)
        c = dict(op=op, dtype=dtype, batch=batch, mean=max(1, int(longest * rng.uniform(0.3, 1.0))),
                 sigma=rng.choice([0.0, 0.4, 0.8]), longest=longest, heads=heads, kv_heads=kv, dim=dim,
                 window=rng.choice([0, spread(1, 4096)]), sinks=rng.choice([0, rng.randint(1, 64)]),
                 buckets=rng.choice([0, 8, 31, 32, 64]), max_distance=0, law=rng.randint(100, 999))
        if c["buckets"]:
            c["max_distance"] = max(c["buckets"] + 1, spread(20, 2048))
        if not c["window"]:
            c["sinks"] = 0
        if 3072 in (c["mean"], int(lengths_of(c).sum())):
            continue
        if op == "decode":
            c["page"] = rng.choice([1, 8, 16, 20, 32, 64, 128])
            if batch * longest * kv * dim > 2.5e8:  # under the largest listed cache
                continue
        elif batch * heads * longest * longest > 2.0e9 or work(c)["flops"] > (4e12 if dtype != "f32" else 2.5e11):
            continue
        return c


def lengths_of(case):
    """The lengths of the batch's histories, fixed by the case: log-normal about the mean, cut at the longest."""
    z = np.random.RandomState(case["law"]).standard_normal(case["batch"])
    n = np.rint(case["mean"] * np.exp(case["sigma"] * z - 0.5 * case["sigma"] ** 2))
    return np.clip(n, 1, case["longest"]).astype(np.int64)


def bucket_starts(case):
    """First distance of every bucket: one distance each in the first half, then growing by a constant factor up to max_distance."""
    n, most = case["buckets"], case["max_distance"]
    single = max(1, n // 2)
    starts = list(range(min(single, n)))
    for i in range(n - single):
        at = math.ceil(single * (most / single) ** (i / max(1, n - single)) - 1e-9)
        starts.append(max(starts[-1] + 1, at))
    return starts


def pairs_of(case):
    """Visible (query, key) pairs of the batch, of one head."""
    n, w, s = lengths_of(case), case["window"], case["sinks"]
    total = 0
    for length in n.tolist():
        i = np.arange(length, dtype=np.int64) if case["op"] != "decode" else np.array([length - 1])
        seen = i + 1 if w == 0 else np.minimum(i + 1, w) + np.minimum(s, np.maximum(0, i + 1 - w))
        total += int(seen.sum())
    return total


def work(case):
    n, e = int(lengths_of(case).sum()), 4 if case["dtype"] == "f32" else 2
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    pairs, bias = pairs_of(case), case["buckets"] * h * e
    if case["op"] == "decode":
        b = case["batch"]
        # the visible rows of the cache, the new rows in and into the cache, queries and outputs, the page table
        pages = math.ceil(pairs / case["page"]) * 4
        return {"bytes": 2 * pairs * hk * d * e + 4 * b * hk * d * e + 2 * b * h * d * e + bias + pages + 8 * b,
                "flops": 4 * pairs * h * d}
    rows = n * d * e
    if case["op"] == "forward":
        return {"bytes": rows * (2 * h + 2 * hk) + bias + 8 * (case["batch"] + 1), "flops": 4 * pairs * h * d}
    # forward: two products; backward: four more, the probabilities' recomputation not counted
    return {"bytes": rows * (4 * h + 4 * hk) + 2 * bias + 8 * (case["batch"] + 1), "flops": 12 * pairs * h * d}


def prepare(case, seed):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.RandomState((seed * 7919 + 13) % (1 << 31))
    n = host.permutation(lengths_of(case))
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    st = {"case": case, "scale": 1.0 / math.sqrt(d), "starts": bucket_starts(case) if case["buckets"] else None}
    st["bias"] = normal(case["buckets"], h, std=0.5) if case["buckets"] else None
    if case["op"] == "decode":
        page, b = case["page"], case["batch"]
        per = (n + page - 1) // page
        used, wide = int(per.sum()), int(per.max())
        order = host.permutation(used + 1)[:used]  # pages as an allocator hands them out over time
        table = np.zeros((b, wide), np.int32)
        at = 0
        for i, p in enumerate(per.tolist()):
            table[i, :p] = order[at:at + p]
            at += p
        st["k_pages"], st["v_pages"] = normal(used + 1, page, hk, d), normal(used + 1, page, hk, d)
        st["table"] = torch.from_numpy(table).to(dev)
        st["lengths"] = torch.from_numpy(n.astype(np.int32)).to(dev)  # with the new event
        st["before"] = st["lengths"] - 1
        st["one_each"] = torch.arange(b + 1, device=dev, dtype=torch.int64)
        st["q"], st["k"], st["v"] = normal(b, h, d), normal(b, hk, d), normal(b, hk, d)
    else:
        total = int(n.sum())
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(dev)
        st["longest"] = int(n.max())
        st["q"], st["k"], st["v"] = normal(total, h, d), normal(total, hk, d), normal(total, hk, d)
        if case["op"] == "train":
            st["grad"] = normal(total, h, d)
    if own:
        import recommender_sparse_embeddings_gb300 as tbe

        # what a program keeps beside its weights: the handle, and a workspace of the batch's size
        handle = tbe.tbe_attention_create(h, hk, d, dt, window=case["window"], sinks=case["sinks"],
                                          bucket_starts=st["starts"], scale=st["scale"])
        st["handle"] = handle
        if case["op"] == "decode":
            st["workspace"] = tbe.make_attention_decode_workspace(handle, b, wide * page, device=dev)
        else:
            st["workspace"] = tbe.make_attention_workspace(handle, total, case["batch"],
                                                           backward=case["op"] == "train", device=dev)
    return st


# --------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"forward": plain_forward, "train": plain_train, "decode": plain_decode}[op](state)
    import recommender_sparse_embeddings_gb300 as tbe

    h, ws, bias = state["handle"], state["workspace"], state["bias"]
    q, k, v = state["q"], state["k"], state["v"]
    if op == "decode":
        kp, vp, table = state["k_pages"], state["v_pages"], state["table"]
        tbe.tbe_attention_append(h, k, v, state["one_each"], state["before"], kp, vp, table)
        out = tbe.tbe_attention_decode(h, q, kp, vp, table, state["lengths"], bias=bias, workspace=ws)
        return {"out": out, "k_pages": kp, "v_pages": vp}
    out, lse = tbe.tbe_attention_forward(h, q, k, v, state["offsets"], bias=bias, workspace=ws)
    if op == "forward":
        return {"out": out}
    gq, gk, gv, gb = tbe.tbe_attention_backward(h, q, k, v, state["offsets"], out, lse, state["grad"], bias=bias,
                                                workspace=ws)
    return {"out": out, "grad_q": gq, "grad_k": gk, "grad_v": gv, "grad_bias": gb}


def padded(x, seq, pos, batch, longest, heads):
    """Ragged rows [N, heads, D] as fp32 [batch, kv_heads, group, longest, D] filled up with zeros."""
    out = torch.zeros((batch, longest) + x.shape[1:], dtype=torch.float32, device=x.device)
    out[seq, pos] = x.float()
    return out.permute(0, 2, 1, 3).unflatten(1, heads)


def plain_places(state):
    off = state["offsets"]
    at = torch.arange(state["q"].shape[0], device=off.device)
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)
    return seq, at - off[seq]


def plain_visible(dist, key, window, sinks):
    seen = dist >= 0
    if window:
        seen = seen & ((dist < window) | (key < sinks))
    return seen


def plain_probabilities(state, qp, kp):
    """Softmax over the visible keys, [B, Hk, G, L, L] in fp32, and the distances' buckets."""
    case, dev, longest = state["case"], qp.device, state["longest"]
    at = torch.arange(longest, device=dev)
    dist = at[:, None] - at[None, :]
    s = torch.matmul(qp, kp.transpose(-1, -2)).mul_(state["scale"])
    if state["bias"] is not None:
        starts = torch.tensor(state["starts"], device=dev)
        bucket = (torch.searchsorted(starts, at, right=True) - 1).contiguous()  # of each distance
        by_distance = state["bias"].float()[bucket].t().contiguous()  # [H, L]
        s.add_(by_distance[:, dist.clamp(min=0)].unflatten(0, (case["kv_heads"], -1)))
    else:
        bucket = None
    s.masked_fill_(~plain_visible(dist, at[None, :], case["window"], case["sinks"]), -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    return s.div_(s.sum(-1, keepdim=True)), bucket


def plain_attend(state):
    case = state["case"]
    b, longest, hk = case["batch"], state["longest"], case["kv_heads"]
    seq, pos = plain_places(state)
    qp = padded(state["q"], seq, pos, b, longest, (hk, -1))
    kp = padded(state["k"], seq, pos, b, longest, (hk, 1))
    vp = padded(state["v"], seq, pos, b, longest, (hk, 1))
    p, bucket = plain_probabilities(state, qp, kp)
    return seq, pos, qp, kp, vp, p, bucket


def ragged(x, seq, pos, dtype):
    """[B, Hk, G, L, D] back to the ragged rows [N, heads, D], rounded once."""
    return x.flatten(1, 2).permute(0, 2, 1, 3)[seq, pos].to(dtype)


def plain_forward(state):
    seq, pos, qp, kp, vp, p, _ = plain_attend(state)
    return {"out": ragged(torch.matmul(p, vp), seq, pos, state["q"].dtype)}


def plain_train(state):
    case, dt = state["case"], state["q"].dtype
    b, longest, hk = case["batch"], state["longest"], case["kv_heads"]
    seq, pos, qp, kp, vp, p, bucket = plain_attend(state)
    out = ragged(torch.matmul(p, vp), seq, pos, dt)
    gp = padded(state["grad"], seq, pos, b, longest, (hk, -1))
    gv = torch.matmul(p.transpose(-1, -2), gp).sum(2, keepdim=True)
    ds = torch.matmul(gp, vp.transpose(-1, -2))
    mean = torch.zeros(p.shape[:-1] + (1,), dtype=torch.float32, device=p.device)
    torch.sum(p * ds, -1, keepdim=True, out=mean)
    ds.sub_(mean).mul_(p)
    del p
    gq = torch.matmul(ds, kp).mul_(state["scale"])
    gk = torch.matmul(ds.transpose(-1, -2), qp).sum(2, keepdim=True).mul_(state["scale"])
    gb = None
    if bucket is not None:
        # sums along each diagonal (one distance), then over each bucket's distances
        both = ds.sum(0).flatten(0, 1)  # [H, L, L]
        at = torch.arange(longest, device=both.device)
        key = at[:, None] - at[None, :]  # [query, distance]
        by = both.gather(-1, key.clamp(min=0).expand_as(both)).mul_(key >= 0).sum(1)  # [H, distance]
        hot = (bucket[:, None] == torch.arange(case["buckets"], device=by.device)).float()
        gb = torch.matmul(by, hot).t().contiguous().to(dt)
    return {"out": out, "grad_q": ragged(gq, seq, pos, dt), "grad_k": ragged(gk, seq, pos, dt),
            "grad_v": ragged(gv, seq, pos, dt), "grad_bias": gb}


def plain_decode(state):
    case, q = state["case"], state["q"]
    kp, vp, table, n = state["k_pages"], state["v_pages"], state["table"].long(), state["lengths"].long()
    page, b, hk = case["page"], case["batch"], case["kv_heads"]
    last = n - 1
    where = table.gather(1, (last // page)[:, None])[:, 0]
    kp[where, last % page] = state["k"]
    vp[where, last % page] = state["v"]
    keys = kp[table].flatten(1, 2).permute(0, 2, 1, 3).float()  # [B, Hk, L, D]
    values = vp[table].flatten(1, 2).permute(0, 2, 1, 3).float()
    s = torch.matmul(q.float().unflatten(1, (hk, -1)), keys.transpose(-1, -2)).mul_(state["scale"])  # [B, Hk, G, L]
    at = torch.arange(s.shape[-1], device=q.device)
    dist = last[:, None] - at
    if state["bias"] is not None:
        bucket = torch.searchsorted(torch.tensor(state["starts"], device=q.device), dist.clamp(min=0), right=True) - 1
        s.add_(state["bias"].float()[bucket].permute(0, 2, 1).unflatten(1, (hk, -1)))
    s.masked_fill_(~plain_visible(dist, at, case["window"], case["sinks"])[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(s, values).div_(s.sum(-1, keepdim=True))
    return {"out": out.flatten(1, 2).to(q.dtype), "k_pages": kp, "v_pages": vp}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs in 64 bits, one history at a time, from the definitions:
    p_ij = exp(scale q_i.k_j + bias[bucket(i-j)]) / sum over visible j, out_i = sum_j p_ij v_j, and their derivatives."""
    if pairs_of(case) * case["heads"] * case["dim"] * (14 if case["op"] == "train" else 4) > 8e12:
        return None
    st = prepare(case, seed)
    group, w, sinks, scale = case["heads"] // case["kv_heads"], case["window"], case["sinks"], st["scale"]
    dev, f64 = st["q"].device, torch.float64
    bias = st["bias"].to(f64) if st["bias"] is not None else None

    def bucket_of(d):
        found = torch.full_like(d, -1)
        for first in st["starts"]:
            found += d >= first
        return found.clamp_(min=0)

    def logits(q, k, i, j):
        """[H, rows, keys] with -inf where the key is not seen."""
        s = scale * torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(group, 1))
        d = i[:, None] - j[None, :]
        if bias is not None:
            s = s + bias.t()[:, bucket_of(d)]
        hidden = (d < 0) if w == 0 else (d < 0) | ((d >= w) & (j[None, :] >= sinks))
        return s.masked_fill(hidden, float("-inf")), d

    if case["op"] == "decode":
        kp, vp, page = st["k_pages"].to(f64), st["v_pages"].to(f64), case["page"]
        table, n, out = st["table"].cpu().numpy(), st["lengths"].cpu().numpy(), []
        for b in range(case["batch"]):
            last = int(n[b]) - 1
            kp[table[b, last // page], last % page] = st["k"][b].to(f64)
            vp[table[b, last // page], last % page] = st["v"][b].to(f64)
            mine = torch.from_numpy(table[b, :last // page + 1].astype(np.int64)).to(dev)
            k, v = kp[mine].flatten(0, 1)[:last + 1], vp[mine].flatten(0, 1)[:last + 1]
            s, _ = logits(st["q"][b:b + 1].to(f64), k, torch.tensor([last], device=dev),
                          torch.arange(last + 1, device=dev))
            out.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.repeat_interleave(group, 1)))
        return {"out": torch.cat(out), "k_pages": kp, "v_pages": vp}

    off = st["offsets"].cpu().numpy()
    res = {"out": torch.zeros_like(st["q"], dtype=f64)}
    if case["op"] == "train":
        res |= {"grad_q": torch.zeros_like(st["q"], dtype=f64), "grad_k": torch.zeros_like(st["k"], dtype=f64),
                "grad_v": torch.zeros_like(st["v"], dtype=f64),
                "grad_bias": torch.zeros_like(bias) if bias is not None else None}
    for b in range(case["batch"]):
        lo, hi = int(off[b]), int(off[b + 1])
        at = torch.arange(hi - lo, device=dev)
        q, k, v = (st[x][lo:hi].to(f64) for x in ("q", "k", "v"))
        s, d = logits(q, k, at, at)
        p = torch.softmax(s, -1)
        del s
        wide_v = v.repeat_interleave(group, 1)
        res["out"][lo:hi] = torch.einsum("hij,jhd->ihd", p, wide_v)
        if case["op"] != "train":
            continue
        g = st["grad"][lo:hi].to(f64)
        fold = lambda x: x.unflatten(1, (-1, group)).sum(2)  # noqa: E731
        res["grad_v"][lo:hi] = fold(torch.einsum("hij,ihd->jhd", p, g))
        gs = torch.einsum("ihd,jhd->hij", g, wide_v)
        gs = p * (gs - (res["out"][lo:hi] * g).sum(-1).t()[:, :, None])
        del p
        res["grad_q"][lo:hi] = scale * torch.einsum("hij,jhd->ihd", gs, k.repeat_interleave(group, 1))
        res["grad_k"][lo:hi] = scale * fold(torch.einsum("hij,ihd->jhd", gs, q))
        if bias is not None:
            which = bucket_of(d)
            for c in range(case["buckets"]):
                if case["buckets"] and st["starts"][c] < hi - lo:
                    res["grad_bias"][c] += (gs * ((which == c) & (d >= 0))).sum((1, 2))
    return res
