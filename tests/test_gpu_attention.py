"""Attention over ragged histories on the GPU against 64-bit references."""

import numpy as np
import pytest
import torch

import attention_reference as ref
import recommender_sparse_embeddings_gb300 as tbe

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
LENGTHS = [1, 0, 63, 64, 65, 2, 127, 128, 129, 0, 300, 31]


class Batch:
    def __init__(self, dtype, heads, kv_heads, dim, lengths, window=0, sinks=0, starts=None, seed=0, scale=None,
                 index=torch.int64):
        g = torch.Generator().manual_seed(seed)
        n = sum(lengths)
        self.dtype, self.window, self.sinks, self.starts = dtype, window, sinks, starts
        self.scale = scale if scale is not None else dim ** -0.5
        self.off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)

        def normal(*shape):
            return torch.randn(shape, generator=g).to(dtype).cuda()

        self.q, self.k, self.v = normal(n, heads, dim), normal(n, kv_heads, dim), normal(n, kv_heads, dim)
        self.grad = normal(n, heads, dim)
        self.bias = normal(len(starts), heads) if starts else None
        self.offsets = torch.from_numpy(self.off).to(index).cuda()
        self.handle = tbe.tbe_attention_create(heads, kv_heads, dim, dtype, window, sinks, starts, self.scale)

    def run(self, stream=None):
        out, lse = tbe.tbe_attention_forward(self.handle, self.q, self.k, self.v, self.offsets, self.bias,
                                             stream=stream)
        gq, gk, gv, gb = tbe.tbe_attention_backward(self.handle, self.q, self.k, self.v, self.offsets, out, lse,
                                                    self.grad, self.bias, stream=stream)
        return {"out": out, "lse": lse, "grad_q": gq, "grad_k": gk, "grad_v": gv, "grad_bias": gb}

    def check(self, got=None):
        got = got or self.run()
        assert tbe.tbe_attention_get_error(self.handle) == tbe.TBE_OK
        b = None if self.bias is None else ref.f64(self.bias)
        want, bound = ref.attention(ref.f64(self.q), ref.f64(self.k), ref.f64(self.v), self.off, self.window,
                                    self.sinks, self.scale, self.starts, b, ref.f64(self.grad), self.dtype)
        for x in want:
            ref.close(got[x], want[x], bound[x], x)
        if b is None:
            assert got["grad_bias"] is None
        return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks,starts", [
    (0, 0, None),
    (0, 0, [0, 1, 2, 3, 5, 9, 17, 100]),
    (1, 0, [0]),
    (50, 3, [0, 1, 7, 49]),
    (64, 70, tuple(range(0, 200, 3))),
    (128, 128, [0, 64, 128]),
    (200, 1, None),
    (0, 0, [0, 1, 2, 5, 40, 150, 5000]),
    (90, 7, [0, 64, 2048]),
])
def test_masks_and_bias(dtype, window, sinks, starts):
    Batch(dtype, 2, 1, 64, LENGTHS, window, sinks, list(starts) if starts else None).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 1), (3, 3, 8), (2, 2, 16), (4, 1, 32), (6, 2, 40), (2, 1, 48),
                                                (3, 1, 63), (2, 2, 72), (4, 2, 96), (1, 1, 100), (4, 1, 128),
                                                (2, 1, 136), (1, 1, 256)])
def test_heads_and_widths(dtype, heads, kv_heads, dim):
    Batch(dtype, heads, kv_heads, dim, [130, 1, 0, 77, 259], 90, 5, [0, 1, 2, 4, 8, 80], seed=dim).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_history_with_window_and_sinks(dtype):
    """Many tiles behind the window, and the first tokens seen by all of them."""
    Batch(dtype, 2, 1, 64, [1900, 40], 150, 9, tbe.tbe_relative_buckets(32, 150), seed=3).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,sinks", [(64, 5), (64, 128), (128, 40)])
def test_sinks_seen_by_many_queries(dtype, dim, sinks):
    """Histories long enough that the first tile's far queries are work items
    of their own, joined; others in the batch are not split."""
    Batch(dtype, 2, 1, dim, [2500, 50, 0, 5000, 300], 70, sinks, [0, 1, 9, 60, 2000], seed=31).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_long_full_history(dtype, dim):
    Batch(dtype, 1, 1, dim, [1025], starts=[0, 1, 300, 1000], seed=4).check()


def test_many_short_histories():
    g = np.random.default_rng(5)
    Batch(torch.bfloat16, 2, 2, 32, g.integers(0, 9, 1500).tolist(), 4, 1, [0, 1, 2], seed=5).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks,starts", [(0, 0, [0, 1, 30]), (100, 3, [0, 2, 50, 4000]), (60, 0, None)])
def test_many_histories_taken_in_turn(dtype, dim, window, sinks, starts):
    """Two hundred histories of one to five key blocks, some empty, whose
    heads do not divide the number of CTAs: a CTA takes tiles of other heads,
    lengths and histories one after another."""
    g = np.random.default_rng(dim + window)
    lengths = np.where(g.random(200) < 0.1, 0, g.integers(1, 330, 200))
    Batch(dtype, 6, 3, dim, lengths.tolist(), window, sinks, starts, seed=32).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_token(dtype):
    b = Batch(dtype, 2, 2, 64, [1], 0, 0, [0])
    got = b.check()
    assert torch.equal(got["out"], b.v)  # one weight, 1
    assert not got["grad_q"].any() and not got["grad_k"].any() and not got["grad_bias"].any()


def test_no_tokens():
    for lengths in ([], [0, 0, 0]):
        b = Batch(torch.bfloat16, 2, 2, 64, lengths, starts=[0, 2])
        got = b.run()
        assert got["out"].shape == (0, 2, 64) and not got["grad_bias"].any()
        assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows_and_int32_offsets(dtype):
    """q, k, v as slices of one projection's rows, some at odd element
    offsets; gradients come back contiguous."""
    for pad in (0, 8, 3):
        b = Batch(dtype, 4, 2, 64, LENGTHS, 100, 2, [0, 3, 9], seed=6, index=torch.int32)
        n = b.q.shape[0]
        wide = torch.full((n, 8, 64 + pad), float("nan"), dtype=dtype, device="cuda")
        for name, lo, hi in (("q", 0, 4), ("k", 4, 6), ("v", 6, 8)):
            wide[:, lo:hi, :64] = getattr(b, name)
            setattr(b, name, wide[:, lo:hi, :64])
        turned = torch.empty((4, n, 64), dtype=dtype, device="cuda")
        turned.copy_(b.grad.transpose(0, 1))
        b.grad = turned.transpose(0, 1)
        b.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_broadcast_rows(dtype):
    b = Batch(dtype, 2, 2, 64, [70, 140], seed=7)
    b.k = b.k[:, :1].expand(-1, 2, -1)
    b.grad = b.grad[:1].expand(b.q.shape[0], -1, -1)
    b.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_neighbours_do_not_leak(dtype, bad):
    """Histories beside a history of non-finite rows, and rows behind the
    batch's end, do not change its results."""
    b = Batch(dtype, 2, 1, 64, [70, 33, 150], 60, 4, [0, 2], seed=8)
    clean = b.check()
    n = b.q.shape[0]
    for name in ("q", "k", "v", "grad"):
        t = getattr(b, name)
        wide = torch.full((n + 200,) + t.shape[1:], bad, dtype=dtype, device="cuda")
        wide[:n] = t
        wide[70:103] = bad
        setattr(b, name, wide[:n])
    got = b.run()
    for x in ("out", "grad_q", "grad_k", "grad_v"):
        for lo, hi in ((0, 70), (103, n)):
            assert torch.equal(got[x][lo:hi], clean[x][lo:hi]), (x, lo)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_see_nothing(dtype):
    """A bias of -inf hides its bucket's keys: rows left with no key give
    zeros and zero gradients; the others ignore the hidden keys."""
    b = Batch(dtype, 2, 2, 64, [40, 200], 0, 0, [0, 5], seed=9)
    b.bias[0] = -float("inf")  # distances 0..4: rows 0..4 see nothing
    got = b.run()
    bias = ref.f64(b.bias)
    want, bound = ref.attention(ref.f64(b.q), ref.f64(b.k), ref.f64(b.v), b.off, 0, 0, b.scale, b.starts, bias,
                                ref.f64(b.grad), dtype)
    for x in ("out", "lse", "grad_q", "grad_k", "grad_v"):
        ref.close(got[x], want[x], bound[x], x)
    assert not got["out"][:5].any() and not got["grad_q"][:5].any() and not got["grad_bias"][0].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_lowest_bias(dtype):
    """A bias of the type's lowest value leaves rows that have nothing else
    with equal weights, and vanishes beside any other key."""
    b = Batch(dtype, 1, 1, 64, [12], 0, 0, [0, 5], seed=10)
    b.bias[0] = torch.finfo(dtype).min
    out, _ = tbe.tbe_attention_forward(b.handle, b.q, b.k, b.v, b.offsets, b.bias)
    v = ref.f64(b.v)
    for i in range(5):
        mean = v[:i + 1].mean(0)
        if dtype != torch.float16:  # fp16's lowest does not swallow the logits
            ref.close(out[i], mean, 4 * ref.UNIT[dtype] * np.abs(v[:i + 1]).mean(0), f"row {i}")
    keep = ref.f64(b.bias)
    keep[0] = -np.inf
    want, bound = ref.attention(ref.f64(b.q), ref.f64(b.k), v, b.off, 0, 0, b.scale, b.starts, keep, dtype=dtype)
    ref.close(out[5:], want["out"][5:], bound["out"][5:], "out")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 63])
def test_lowest_bias_has_finite_gradients(dtype, dim):
    """Rows that see nothing but keys of the lowest bias pass no gradient; the
    others' gradients are those of a bias of -inf there."""
    b = Batch(dtype, 1, 1, dim, [12, 300], 0, 0, [0, 5], seed=33, scale=4.0)
    b.bias[0] = torch.finfo(dtype).min
    got = b.run()
    b.bias[0] = -float("inf")
    want = b.run()
    for x in ("grad_q", "grad_k", "grad_v"):
        assert torch.equal(got[x], want[x]), x
    assert torch.equal(got["grad_bias"][1], want["grad_bias"][1]) and not got["grad_bias"][0].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_logits(dtype):
    """Logits of several hundred, rising along the history: the running
    maximum moves in every tile."""
    b = Batch(dtype, 1, 1, 64, [500], seed=11, scale=1.0)
    ramp = torch.linspace(0, 6, 500, device="cuda")[:, None, None]
    b.q = (b.q.float().abs() + 0.5).to(dtype)
    b.k = (b.k.float() * 0.1 + ramp).to(dtype)
    b.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_deterministic_and_reused_workspace(dtype):
    b = Batch(dtype, 4, 2, 64, LENGTHS * 3, 100, 3, [0, 1, 2, 50], seed=12)
    first = b.run()
    ws = tbe.make_attention_workspace(b.handle, b.q.shape[0], len(b.off) - 1, True)
    ws.fill_(255)
    for _ in range(2):
        out, lse = tbe.tbe_attention_forward(b.handle, b.q, b.k, b.v, b.offsets, b.bias, workspace=ws)
        gs = tbe.tbe_attention_backward(b.handle, b.q, b.k, b.v, b.offsets, out, lse, b.grad, b.bias, workspace=ws)
        for x, y in zip((out, lse) + gs, first.values()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 200])
def test_a_workspace_serves_smaller_batches(dtype, dim):
    big = tbe.tbe_attention_create(1, 1, dim, dtype, 70, 3, [0, 2])
    for backward in (False, True):
        room = tbe.tbe_attention_workspace_bytes(big, 40000, 300, backward)
        for n, b in ((40000, 1), (39999, 300), (20000, 300), (19000, 10), (9000, 100), (1, 1), (0, 0)):
            assert 0 < tbe.tbe_attention_workspace_bytes(big, n, b, backward) <= room, (n, b)


def test_another_stream():
    b = Batch(torch.bfloat16, 2, 2, 64, [300, 100], 50, 2, [0, 4], seed=13)
    want = b.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = b.run(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for x in want:
        assert torch.equal(got[x], want[x])


def test_captured_in_a_graph():
    b = Batch(torch.bfloat16, 2, 2, 64, [300, 100], 50, 2, [0, 4], seed=14)
    want = b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.run()
    for t in got.values():
        t.zero_()
    g.replay()
    for x in want:
        assert torch.equal(got[x], want[x])


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_malformed_offsets_are_reported(index):
    b = Batch(torch.bfloat16, 1, 1, 64, [10, 20, 30], seed=15, index=index)
    for off in ([0, 10, 5, 60], [0, 10, 30, 59], [1, 10, 30, 60], [0, 70, 70, 60], [0, -5, 30, 60]):
        b.offsets = torch.tensor(off, dtype=index, device="cuda")
        b.run()
        assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_ERR_BAD_OFFSETS, off
        assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,histories,window,sinks", [(300, 101, 0, 0), (300, 301, 0, 0), (6000, 9, 64, 4)])
def test_overlapping_offsets_stay_in_bounds(dtype, tokens, histories, window, sinks):
    """Offsets that run back and forth name many times the tiles that N tokens
    have (and many times the sinks' far queries): reported, and nothing beyond
    the workspace is touched."""
    b = Batch(dtype, 2, 1, 64, [tokens], window, sinks, [0, 3], seed=34)
    b.offsets = torch.tensor([0, tokens] * (histories // 2 + 1), device="cuda")[:histories + 1]
    n = tbe.tbe_attention_workspace_bytes(b.handle, tokens, histories, True)
    room = torch.full((n + 65536,), 77, dtype=torch.uint8, device="cuda")
    out, lse = tbe.tbe_attention_forward(b.handle, b.q, b.k, b.v, b.offsets, b.bias, workspace=room[:n])
    tbe.tbe_attention_backward(b.handle, b.q, b.k, b.v, b.offsets, out, lse, b.grad, b.bias, workspace=room[:n])
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_ERR_BAD_OFFSETS
    assert (room[n:] == 77).all()


def test_gradients_match_differences():
    """Directional derivatives of the fp32 forward by central differences.
    With step h the truncation is about h^2 / 6 of a third derivative (of the
    order of the loss's own scale S = sqrt(#outputs)), and each loss carries
    about 2^-22 S sqrt(D) of rounding: h = 2^-6 balances to about 3e-4 S."""
    b = Batch(torch.float32, 2, 1, 64, [70, 5, 130], 40, 2, [0, 1, 3, 20], seed=16)
    got = b.run()
    up = ref.f64(b.grad)

    def loss():
        out, _ = tbe.tbe_attention_forward(b.handle, b.q, b.k, b.v, b.offsets, b.bias)
        return float((ref.f64(out) * up).sum())

    g = torch.Generator().manual_seed(17)
    size = np.sqrt(up.size)
    for name in ("q", "k", "v", "bias"):
        x = getattr(b, name)
        step = torch.randn(x.shape, generator=g).cuda()
        step /= step.norm()  # a step of length h in all
        h = 2.0 ** -6
        setattr(b, name, x + h * step)
        up_loss = loss()
        setattr(b, name, x - h * step)
        down = loss()
        setattr(b, name, x)
        want = (up_loss - down) / (2 * h)
        have = float((ref.f64(got["grad_" + name]) * ref.f64(step)).sum())
        assert abs(want - have) < 3e-4 * size, (name, want, have)


def test_refusals():
    b = Batch(torch.bfloat16, 4, 2, 64, [10, 20], 0, 0, [0, 3], seed=18)
    h, q, k, v, off, bias = b.handle, b.q, b.k, b.v, b.offsets, b.bias
    f = tbe.tbe_attention_forward
    for args in ((q[:, :3], k, v, off, bias), (q, k[:29], v, off, bias), (q, k, v.float(), off, bias),
                 (q, k, v, off.float(), bias), (q, k, v, off, None), (q, k, v, off, bias[:1]),
                 (q, k, v, off, bias.float()), (q.cpu(), k, v, off, bias),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), k, v, off, bias)):
        with pytest.raises(ValueError):
            f(h, *args)
    with pytest.raises(ValueError):
        f(h, q, k, v, off, bias, out=torch.empty(30, 4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(tbe.TBEError) as e:
        f(h, q, k, v, off, bias, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tbe.TBE_ERR_WORKSPACE_TOO_SMALL
    out, lse = f(h, q, k, v, off, bias)
    with pytest.raises(ValueError):
        tbe.tbe_attention_backward(h, q, k, v, off, out, lse[:1], b.grad, bias)
    with pytest.raises(ValueError):
        tbe.tbe_attention_backward(h, q, k, v, off, out, lse, b.grad[:, :1], bias)
    with pytest.raises(tbe.TBEError) as e:
        tbe.tbe_attention_backward(h, q, k, v, off, out, lse, b.grad, bias,
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tbe.TBE_ERR_WORKSPACE_TOO_SMALL
    h.close()
    with pytest.raises(RuntimeError):
        f(h, q, k, v, off, bias)


# ------------------------------------------------------------------ the cache


class Cache:
    """Pages filled with `fill` but for the histories' rows, in shuffled order."""

    def __init__(self, dtype, heads, kv_heads, dim, lengths, page, window=0, sinks=0, starts=None, seed=0,
                 fill=float("nan"), extra=2):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.window, self.sinks, self.starts, self.page = dtype, window, sinks, starts, page
        self.lengths, b = lengths, len(lengths)
        per = [(n + page - 1) // page for n in lengths]
        width = max(per + [1]) + 1
        order = torch.randperm(sum(per) + extra, generator=g).tolist()
        table = np.full((b, width), -1, np.int32)  # what no token needs is never looked up
        at = 0
        for i, p in enumerate(per):
            table[i, :p] = order[at:at + p]
            at += p

        def normal(*shape):
            return torch.randn(shape, generator=g).to(dtype)

        self.q = normal(b, heads, dim).cuda()
        self.bias = normal(len(starts), heads).cuda() if starts else None
        self.keys = [normal(n, kv_heads, dim) for n in lengths]
        self.values = [normal(n, kv_heads, dim) for n in lengths]
        self.k_pages = torch.full((sum(per) + extra, page, kv_heads, dim), fill, dtype=dtype).cuda()
        self.v_pages = self.k_pages.clone()
        self.table = torch.from_numpy(table).cuda()
        self.n = torch.tensor(lengths, dtype=torch.int32).cuda()
        self.handle = tbe.tbe_attention_create(heads, kv_heads, dim, dtype, window, sinks, starts)
        self.scale = dim ** -0.5

    def append(self, lo, hi, index=torch.int64):
        """Tokens [min(lo, n), min(hi, n)) of every history of n tokens."""
        part = [(min(lo, n), min(hi, n)) for n in self.lengths]
        off = torch.tensor(np.concatenate([[0], np.cumsum([y - x for x, y in part])]), dtype=index).cuda()
        k = torch.cat([t[x:y] for t, (x, y) in zip(self.keys, part)]).cuda()
        v = torch.cat([t[x:y] for t, (x, y) in zip(self.values, part)]).cuda()
        before = torch.tensor([x for x, _ in part], dtype=torch.int32).cuda()
        tbe.tbe_attention_append(self.handle, k, v, off, before, self.k_pages, self.v_pages, self.table)

    def check(self, **kw):
        out = tbe.tbe_attention_decode(self.handle, self.q, self.k_pages, self.v_pages, self.table, self.n,
                                       self.bias, **kw)
        assert tbe.tbe_attention_get_error(self.handle) == tbe.TBE_OK
        want, bound = ref.decode(ref.f64(self.q), [ref.f64(x) for x in self.keys], [ref.f64(x) for x in self.values],
                                 self.window, self.sinks, self.scale, self.starts,
                                 None if self.bias is None else ref.f64(self.bias), self.dtype)
        ref.close(out, want, bound, "out")
        return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 1), (2, 2, 16), (3, 1, 40), (4, 2, 63), (4, 1, 64), (2, 2, 96),
                                                (6, 1, 128), (16, 1, 128), (9, 1, 72), (2, 1, 200), (1, 1, 256)])
def test_decode_heads_and_widths(dtype, heads, kv_heads, dim):
    c = Cache(dtype, heads, kv_heads, dim, [0, 1, 16, 17, 129, 300], 16, 100, 3, [0, 1, 4, 64], seed=dim)
    c.append(0, 10 ** 6)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 7, 16, 20, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (33, 5), (64, 128), (1000, 9)])
def test_decode_pages_and_masks(dtype, page, window, sinks):
    c = Cache(dtype, 4, 2, 64, [1, 0, 5, 64, 65, 511, 129], page, window, sinks, [0, 1, 2, 8, 60], seed=page)
    c.append(0, 4, torch.int32)
    c.append(4, 10 ** 6)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [0, 1500])
def test_decode_split_and_joined(dtype, window):
    """Few long histories: chunks over many CTAs, joined; one short beside."""
    c = Cache(dtype, 4, 2, 64, [5000, 255, 256, 257, 1], 32, window, 8, tbe.tbe_relative_buckets(32, 900), seed=20)
    c.append(0, 10 ** 6)
    a = c.check()
    ws = tbe.make_attention_decode_workspace(c.handle, 5, c.table.shape[1] * 32)
    ws.fill_(255)
    assert torch.equal(a, c.check(workspace=ws))
    c.check(max_length=5000)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_equals_the_forward_call_s_last_row(dtype):
    """Token by token over the cache, the forward call's rows."""
    n = 40
    c = Cache(dtype, 2, 1, 64, [n], 8, 12, 3, [0, 1, 5], seed=21)
    g = torch.Generator().manual_seed(22)
    q = torch.randn((n, 2, 64), generator=g).to(dtype).cuda()
    off = torch.tensor([0, n]).cuda()
    want, _ = tbe.tbe_attention_forward(c.handle, q, c.keys[0].cuda(), c.values[0].cuda(), off, c.bias)
    for t in range(n):
        c.append(t, t + 1)
        length = torch.tensor([t + 1], dtype=torch.int32).cuda()
        got = tbe.tbe_attention_decode(c.handle, q[t:t + 1], c.k_pages, c.v_pages, c.table, length, c.bias)
        err = (got[0].float() - want[t].float()).abs().max()
        assert err <= 8 * ref.UNIT[dtype] * 4, (t, err)  # weights and result each rounded, values up to about 4


def test_append_keeps_what_it_does_not_write():
    c = Cache(torch.float16, 2, 2, 40, [9, 0, 20], 7, seed=23, fill=5.0)
    c.append(0, 3)
    c.append(3, 20)
    table = c.table.cpu().numpy()
    k = torch.full_like(c.k_pages.cpu(), 5.0)
    v = k.clone()
    for b, n in enumerate(c.lengths):
        for j in range(n):
            k[table[b, j // 7], j % 7] = c.keys[b][j]
            v[table[b, j // 7], j % 7] = c.values[b][j]
    assert torch.equal(c.k_pages.cpu(), k) and torch.equal(c.v_pages.cpu(), v)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_pages(dtype):
    """Keys and values interleaved in one buffer, heads before tokens."""
    c = Cache(dtype, 4, 2, 64, [70, 33], 16, 0, 0, [0, 9], seed=24)
    pages = c.k_pages.shape[0]
    both = torch.full((pages, 2, 2, 16, 64), float("nan"), dtype=dtype, device="cuda")
    c.k_pages, c.v_pages = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    c.append(0, 100)
    c.check()


def test_cache_positions_out_of_range_are_reported():
    c = Cache(torch.bfloat16, 2, 2, 64, [20, 30], 8, seed=25, fill=0.0)
    c.append(0, 100)
    h, width = c.handle, c.table.shape[1]
    one = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.arange(3).cuda()
    for before in ([-1, 0], [width * 8, 0], [2 ** 31 - 1, 0], [24, 0]):  # the last: a page the table does not name
        tbe.tbe_attention_append(h, one, one, off, torch.tensor(before, dtype=torch.int32).cuda(), c.k_pages.clone(),
                                 c.v_pages.clone(), c.table)
        assert tbe.tbe_attention_get_error(h) == tbe.TBE_ERR_INDEX_OOB, before
    for bad in (-1, width * 8 + 1, 2 ** 31 - 1):
        n = torch.tensor([bad, 30], dtype=torch.int32).cuda()
        out = tbe.tbe_attention_decode(h, c.q, c.k_pages, c.v_pages, c.table, n, c.bias)
        assert tbe.tbe_attention_get_error(h) == tbe.TBE_ERR_INDEX_OOB
        assert not out[0].any() and out[1].any()
    table = c.table.clone()
    table[0, 1] = c.k_pages.shape[0]
    tbe.tbe_attention_decode(h, c.q, c.k_pages, c.v_pages, table, c.n, c.bias)
    assert tbe.tbe_attention_get_error(h) == tbe.TBE_ERR_INDEX_OOB


def test_cache_refusals():
    c = Cache(torch.bfloat16, 4, 2, 64, [20, 30], 8, 0, 0, [0, 2], seed=26)
    d = tbe.tbe_attention_decode
    for args in ((c.q[:1], c.k_pages, c.v_pages, c.table, c.n, c.bias),
                 (c.q, c.k_pages, c.v_pages[1:], c.table, c.n, c.bias),
                 (c.q, c.k_pages, c.v_pages, c.table.long(), c.n, c.bias),
                 (c.q, c.k_pages, c.v_pages, c.table, c.n.long(), c.bias),
                 (c.q, c.k_pages, c.v_pages, c.table, c.n, None),
                 (c.q.half(), c.k_pages, c.v_pages, c.table, c.n, c.bias),
                 (c.q, c.k_pages[..., :32], c.v_pages[..., :32], c.table, c.n, c.bias)):
        with pytest.raises(ValueError):
            d(c.handle, *args)
    long = Cache(torch.bfloat16, 4, 2, 64, [2000], 8, 0, 0, [0, 2], seed=27)
    with pytest.raises(tbe.TBEError) as e:
        d(long.handle, long.q, long.k_pages, long.v_pages, long.table, long.n, long.bias,
          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tbe.TBE_ERR_WORKSPACE_TOO_SMALL


def test_long_cache_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31: the last pages of a buffer of
    more than 2^31 elements."""
    dim, page, hk = 128, 64, 4
    pages = 2 ** 31 // (page * hk * dim) + 40
    c = Cache(torch.bfloat16, 4, hk, dim, [900], page, seed=28, extra=1)
    big = [torch.empty((pages, page, hk, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.k_pages, c.v_pages = big
    c.table = torch.arange(pages - c.table.shape[1], pages, dtype=torch.int32, device="cuda")[None].contiguous()
    c.append(0, 900)
    c.check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 6)])
def test_many_tiles_on_every_sm(dim, window, sinks):
    """Thousands of tiles of several key blocks each, launched again and
    again: no wait may run out.  Against the fp32 path on the same values:
    the result's and the weights' rounding, the latter by the sum of
    magnitudes (the fp32 path on |v|)."""
    g = np.random.default_rng(dim + window)
    lengths = g.integers(1, 900, 120).tolist()
    b = Batch(torch.bfloat16, 8, 4, dim, lengths, window, sinks, [0, 1, 2, 9, 100], seed=30)
    first = b.run()
    for _ in range(10):
        again = b.run()
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK
    for x in first:
        assert torch.equal(first[x], again[x]), x
    h = tbe.tbe_attention_create(8, 4, dim, torch.float32, window, sinks, b.starts)
    q, k, v, bias = (t.float() for t in (b.q, b.k, b.v, b.bias))
    want, lse = tbe.tbe_attention_forward(h, q, k, v, b.offsets, bias)
    size, _ = tbe.tbe_attention_forward(h, q, k, v.abs(), b.offsets, bias)
    u = 2.0 ** -8
    assert ((first["out"].float() - want).abs() <= u * want.abs() + (u + 2.0 ** -14) * size).all()
    # gradients: by their size over the batch (the element-wise bounds are
    # checked on small batches): roundings of relative size u add up at random
    grads = tbe.tbe_attention_backward(h, q, k, v, b.offsets, want, lse, b.grad.float(), bias)
    for x, y in zip(("grad_q", "grad_k", "grad_v", "grad_bias"), grads):
        assert (first[x].float() - y).norm() <= 1.5 * u * y.norm(), x
