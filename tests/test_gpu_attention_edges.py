"""Attention at the edges of its contract: biases that hide keys or are of
large magnitude, streams and workspaces of the caller's choice, single caches
without pages.  References in 64 bits; helpers of the operators' main tests."""

import numpy as np
import pytest
import torch

import attention_reference as ref
import recommender_sparse_embeddings_gb300 as tbe
from test_gpu_attention import DTYPES, Batch, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("starts", [[0, 1, 30], [0, 5, 4000]])
@pytest.mark.parametrize("heads,kv_heads,histories", [(6, 3, 200), (8, 2, 5)])
def test_lowest_bias_in_some_heads(dim, starts, heads, kv_heads, histories):
    """The type's lowest value in the last bucket of every other head hides its
    keys there (every row has others), whatever the heads beside it hold: in
    batches whose tiles are taken in turn, and under query heads that share a
    key-value head."""
    g = np.random.default_rng(dim + histories)
    lengths = g.integers(1, 400, histories)
    lengths[0] = 4500 if starts[-1] > 400 else 700
    b = Batch(torch.bfloat16, heads, kv_heads, dim, lengths.tolist(), 0, 0, starts, seed=40)
    b.bias[-1, ::2] = -float("inf")
    want = b.run()
    b.bias[-1, ::2] = torch.finfo(torch.bfloat16).min
    for _ in range(3):
        got = b.run()
        for x in want:
            assert torch.equal(got[x], want[x]), x
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_stream_that_is_not_the_current_one(as_handle):
    """The calls' own memory belongs to the stream they launch on: what is
    allocated and filled on the current stream meanwhile is other memory."""
    b = Batch(torch.bfloat16, 2, 1, 64, [300, 100, 700], 50, 2, [0, 4], seed=41)
    want = b.run()
    c = Cache(torch.bfloat16, 4, 2, 64, [3000, 20], 16, seed=42)
    c.append(0, 10 ** 6)
    one = c.check()
    n, count = b.q.shape[0], len(b.off) - 1
    sizes = [tbe.tbe_attention_workspace_bytes(b.handle, n, count, x) for x in (False, True)]
    sizes.append(tbe.tbe_attention_decode_workspace_bytes(c.handle, 2, c.table.shape[1] * 16))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if as_handle else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the launches wait behind some 10 ms
    got = b.run(stream=stream)
    last = tbe.tbe_attention_decode(c.handle, c.q, c.k_pages, c.v_pages, c.table, c.n, c.bias, stream=stream)
    fill = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for size in sizes for _ in range(8)]
    torch.cuda.current_stream().wait_stream(s)
    for x in want:
        assert torch.equal(got[x], want[x]), x
    assert torch.equal(last, one)
    assert all((f == 255).all() for f in fill)
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK


@pytest.mark.parametrize("as_handle", [False, True])
def test_table_calls_on_a_stream_that_is_not_the_current_one(as_handle):
    g = torch.Generator().manual_seed(43)
    table = torch.randn((1000, 64), generator=g).cuda()
    h = tbe.tbe_create([table], "sum")
    ids = torch.randint(0, 1000, (5000,), generator=g).cuda()
    off = torch.arange(0, 5001, 5).cuda()
    up = torch.randn((1000, 64), generator=g).cuda()
    want = tbe.tbe_forward(h, ids, off, 1000)
    grad = tbe.tbe_per_sample_weight_grad(h, ids, off, 1000, up)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if as_handle else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = tbe.tbe_forward(h, ids, off, 1000, stream=stream)
    weights = tbe.tbe_per_sample_weight_grad(h, ids, off, 1000, up, stream=stream)
    space = tbe.make_workspace(h, 5000, 1000, stream=stream)
    both = tbe.tbe_forward_prepare(h, ids, off, 1000, space, stream=stream)
    size = space.numel()
    del space
    fill = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(both, want) and torch.equal(weights, grad)
    assert all((f == 255).all() for f in fill) and tbe.tbe_get_error(h) == tbe.TBE_OK


@pytest.mark.parametrize("dtype", DTYPES)
def test_workspaces_start_on_16_byte_boundaries(dtype):
    """Others are refused, by the binding and by the library; slices on a
    boundary are as good as the whole."""
    b = Batch(dtype, 2, 1, 64, [300, 20], 50, 2, [0, 4], seed=44)
    want = b.run()
    c = Cache(dtype, 4, 2, 64, [3000, 20], 16, seed=45)
    c.append(0, 10 ** 6)
    one = c.check()
    space = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def calls(ws):
        out, lse = tbe.tbe_attention_forward(b.handle, b.q, b.k, b.v, b.offsets, b.bias, workspace=ws)
        yield torch.equal(out, want["out"])
        gq = tbe.tbe_attention_backward(b.handle, b.q, b.k, b.v, b.offsets, want["out"], want["lse"], b.grad, b.bias,
                                        workspace=ws)[0]
        yield torch.equal(gq, want["grad_q"])
        yield torch.equal(c.check(workspace=ws), one)

    assert all(calls(space[16:])) and all(calls(space[4096 + 48:]))
    for at in (1, 4, 8, 20):
        with pytest.raises(ValueError):
            next(calls(space[at:]))
        with pytest.raises(ValueError):
            tbe.tbe_attention_backward(b.handle, b.q, b.k, b.v, b.offsets, want["out"], want["lse"], b.grad, b.bias,
                                       workspace=space[at:])
        with pytest.raises(ValueError):
            c.check(workspace=space[at:])


def test_the_library_refuses_misaligned_workspaces():
    b = Batch(torch.bfloat16, 2, 2, 64, [10], seed=46)
    lib, h = tbe.load_library(), b.handle.ptr
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    rows = [tbe._rows(b.handle, t, 10, 2, "x") for t in (b.q, b.k, b.v, b.grad)]
    out = [torch.empty_like(b.q) for _ in range(4)]
    lse = torch.empty((2, 10), device="cuda")
    off = b.offsets.data_ptr()
    for at in (1, 4, 8):
        ws = space.data_ptr() + at
        assert lib.tbe_attention_forward(h, *rows[:3], None, off, 1, 10, 1, out[0].data_ptr(), lse.data_ptr(), ws,
                                         1 << 19, None) == tbe.TBE_ERR_INVALID_ARG
        assert lib.tbe_attention_backward(h, *rows[:3], None, off, 1, 10, 1, out[0].data_ptr(), lse.data_ptr(),
                                          rows[3], *[t.data_ptr() for t in out[1:]], None, ws, 1 << 19,
                                          None) == tbe.TBE_ERR_INVALID_ARG
        pages = [tbe._pages(b.handle, t[None], (1, 10, 2, 64), "x") for t in (b.k, b.v)]
        table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        one = torch.ones(1, dtype=torch.int32, device="cuda")
        assert lib.tbe_attention_decode(h, rows[0], *pages, 1, 10, table.data_ptr(), 1, one.data_ptr(), 1, 10, None,
                                        out[0].data_ptr(), ws, 1 << 19, None) == tbe.TBE_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_head_whose_every_bucket_is_hidden(dtype, dim):
    """Over several tiles, beside a head that sees its keys: zeros, a statistic
    of -inf and no gradients."""
    b = Batch(dtype, 2, 2, dim, [300, 20], 0, 0, [0, 7], seed=50)
    b.bias[:, 0] = -float("inf")
    got = b.check()
    assert not got["out"][:, 0].any() and not got["grad_q"][:, 0].any() and not got["grad_v"][:, 0].any()
    assert (got["lse"][0] == -float("inf")).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_hidden_distant_keys_of_large_logits(dtype):
    """Keys far back are hidden by a bias of -inf; their logits (up to about
    1200) would not fit fp32's exponentials."""
    b = Batch(dtype, 1, 1, 64, [400], 0, 0, [0, 70], seed=51, scale=1.0)
    b.q = (b.q.float().abs() + 2).to(dtype)
    b.k = (b.k.float() * 0.1).to(dtype)
    b.k[:150] = 6
    b.bias[1] = -float("inf")
    b.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("last", [False, True])
def test_bias_of_distances_nobody_sees(dtype, bad, last):
    """Buckets that begin behind the window reach no result, whatever they
    hold; their gradient is zero."""
    b = Batch(dtype, 2, 1, 64, [300, 65], 50, 0, [0, 20, 60, 200], seed=52)
    b.bias[2:] = 0
    clean = b.run()
    b.bias[2] = bad
    if last:
        b.bias[3] = bad
    got = b.run()
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK
    for x in clean:
        assert torch.equal(got[x], clean[x]), x
    assert not got["grad_bias"][2:].any()


def _offsets_of(dtype):
    return [-6.0e4, 6.0e4] if dtype == torch.float16 else [-1.0e6, -1.0e9, -1.0e30, 1.0e9]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40, 63])
@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("shape", ["all", "near", "window"])
def test_bias_of_large_magnitude(dtype, dim, which, shape):
    """A softmax does not change when all the logits of a row move by the same
    amount: a large bias on every key that a row sees leaves the results of no
    bias, and the bounds are those of logits without it.

    all: every bucket.  near: the first bucket alone, so that the rows of short
    distances see nothing else; to the others its keys are hidden (a large
    negative value) or the only ones (a positive one).  window: the buckets
    that a window and its sinks reach, the rest at zero."""
    values = _offsets_of(dtype)
    if which >= len(values):
        pytest.skip("fp16 holds two of the values")
    value = values[which]
    window, sinks = (40, 3) if shape == "window" else (0, 0)
    b = Batch(dtype, 2, 1, dim, [200, 1, 70, 29, 150], window, sinks, [0, 30, 60, 190], seed=53 + which)
    zero = np.zeros((4, 2))
    if shape == "all":
        b.bias[:] = value
    elif shape == "near":
        b.bias[0] = value
        hide = np.where(np.arange(4)[:, None] == 0, 0.0, -np.inf) + zero
    else:
        # distances up to 39 are seen within the window, any by the sinks
        b.bias[:3] = value
        b.bias[3] = 0
    q, k, v, grad = (ref.f64(x) for x in (b.q, b.k, b.v, b.grad))
    got = b.run()
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK

    def want(bias, rows=None):
        g = grad if rows is None else grad * rows[:, None, None]
        return ref.attention(q, k, v, b.off, window, sinks, b.scale, b.starts, bias, g, dtype)

    if shape == "all":
        res, bound = want(zero)
    else:
        first = np.concatenate([np.arange(n) for n in np.diff(b.off)])
        if shape == "near":
            rows = first < 30  # rows that see the first bucket alone
            one = want(hide if value > 0 else zero, rows)
            rest = ref.f64(b.bias)
            rest[0] = -np.inf
            two = want(hide if value > 0 else rest, ~rows)
        else:
            rows = first < 190  # rows that see buckets of the value alone
            one = want(zero, rows)
            far = np.where(np.arange(4)[:, None] == 3, -np.inf if value > 0 else 0.0, 0.0 if value > 0 else -np.inf)
            two = want(far + zero, ~rows)
        res, bound = ({}, {})
        for x in one[0]:
            if x == "lse":
                continue
            if x == "out":
                pick = rows[:, None, None]
                res[x], bound[x] = np.where(pick, one[0][x], two[0][x]), np.where(pick, one[1][x], two[1][x])
            else:
                res[x], bound[x] = one[0][x] + two[0][x], one[1][x] + two[1][x]
    for x in res:
        if x != "lse":
            ref.close(got[x], res[x], bound[x], x)
    # the statistic holds the offset, in fp32's steps
    if shape == "all":
        lse = res["lse"] + float(b.bias[0, 0]) * np.log2(np.e)
        assert (np.abs(ref.f64(got["lse"]) - lse) <= bound["lse"] + 4 * ref.F * np.abs(lse)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 63, 128])
@pytest.mark.parametrize("which", range(4))
def test_decode_with_a_bias_of_large_magnitude(dtype, dim, which):
    values = _offsets_of(dtype)
    if which >= len(values):
        pytest.skip("fp16 holds two of the values")
    c = Cache(dtype, 4, 2, dim, [3000, 1, 700, 40], 16, 0, 0, [0, 30, 500], seed=54)
    c.append(0, 10 ** 6)
    keep = c.bias
    c.bias = torch.full_like(keep, values[which])
    got = tbe.tbe_attention_decode(c.handle, c.q, c.k_pages, c.v_pages, c.table, c.n, c.bias)
    c.bias = torch.zeros_like(keep)
    want, bound = ref.decode(ref.f64(c.q), [ref.f64(x) for x in c.keys], [ref.f64(x) for x in c.values], 0, 0,
                             c.scale, c.starts, ref.f64(c.bias), dtype)
    ref.close(got, want, bound, "out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("far", [40, 4000])
@pytest.mark.parametrize("histories", [5, 200])
def test_bias_of_large_magnitude_in_some_heads(dtype, dim, far, histories):
    """Beside heads of an ordinary bias, with the table of all distances and
    with tables per block, and where tiles are taken in turn."""
    g = np.random.default_rng(far + histories)
    lengths = g.integers(1, 170, histories)
    lengths[0] = 300
    b = Batch(dtype, 4, 2, dim, lengths.tolist(), 0, 0, [0, 3, far], seed=58)
    b.bias[:, ::2] = -6.0e4 if dtype == torch.float16 else -1.0e9
    bias = ref.f64(b.bias)
    bias[:, ::2] = 0
    got = b.run()
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK
    want, bound = ref.attention(ref.f64(b.q), ref.f64(b.k), ref.f64(b.v), b.off, 0, 0, b.scale, b.starts, bias,
                                ref.f64(b.grad), dtype)
    for x in want:
        if x != "lse":
            ref.close(got[x], want[x], bound[x], x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv_heads,dim,window", [(16, 4, 128, 0), (2, 2, 64, 0), (8, 1, 64, 3000), (12, 1, 200, 0)])
def test_a_decode_workspace_serves_smaller_batches(dtype, heads, kv_heads, dim, window):
    h = tbe.tbe_attention_create(heads, kv_heads, dim, dtype, window, 4 if window else 0)
    for b, n in ((200, 8192), (128, 8192), (37, 65000), (1, 20000), (5, 600)):
        room = tbe.tbe_attention_decode_workspace_bytes(h, b, n)
        table = torch.zeros((b, n), dtype=torch.int32, device="cuda")  # pages of one token, all of them page 0
        page = torch.zeros((1, 1, kv_heads, dim), dtype=dtype, device="cuda")
        q = torch.zeros((b, heads, dim), dtype=dtype, device="cuda")
        space = torch.empty(room, dtype=torch.uint8, device="cuda")
        for few in sorted(x for x in {1, 2, b // 3, b // 2, 3 * b // 4, b - 1, b} if 0 < x <= b):
            for most in sorted({0, 1, 255, 257, 513, n // 7, n // 3, n // 2, 2 * n // 3, n - 1, n} - {n + 1}):
                if most > n:
                    continue
                assert 0 < tbe.tbe_attention_decode_workspace_bytes(h, few, most) <= room, (few, most)
                empty = torch.zeros(few, dtype=torch.int32, device="cuda")
                tbe.tbe_attention_decode(h, q[:few], page, page, table[:few], empty, max_length=most, workspace=space)
    assert tbe.tbe_attention_get_error(h) == tbe.TBE_OK


def test_decode_with_a_most_of_zero_takes_the_table_s_room():
    c = Cache(torch.bfloat16, 4, 2, 64, [3000, 20], 16, seed=55)
    c.append(0, 10 ** 6)
    assert torch.equal(c.check(max_length=0), c.check())


@pytest.mark.parametrize("dim,lengths,window,sinks", [(64, [300, 1, 77], 0, 0), (128, [300, 1, 77], 0, 0),
                                                      (64, [2500, 40], 70, 5), (128, [2500, 40], 70, 5),
                                                      (40, [300, 1, 77], 50, 2)])
def test_fp16_gradients_scale_with_the_upstream_gradient(dim, lengths, window, sinks):
    """Gradients are linear in the upstream gradient: times a power of two,
    they are times that power, bit by bit where fp16 holds them as normal
    numbers.  The logits' gradients on the way may not fit fp16."""
    b = Batch(torch.float16, 4, 2, dim, lengths, window, sinks, [0, 1, 9, 60], seed=56)
    b.v = b.v * 4
    b.grad = torch.where(b.grad.float().abs() < 2.0 ** -6, 2.0 ** -6, b.grad.float()).half()
    base = b.check()
    unit = b.grad.clone()
    for power in (-7, 12):
        b.grad = (unit.float() * 2.0 ** power).half()
        assert torch.equal(b.grad.float() * 2.0 ** -power, unit.float())
        got = b.run()
        for x in ("grad_q", "grad_k", "grad_v", "grad_bias"):
            want = (base[x].double() * 2.0 ** power)
            fits = (base[x].double().abs() < 65504 * 2.0 ** -max(power, 0)) & (base[x].double().abs() < 60000)
            # rounded once more where the smaller result is subnormal (steps of 2^-24), else the same bits
            step = 2.0 ** -24 if power < 0 else 2.0 ** (power - 24)
            assert ((got[x].double() - want).abs() <= step)[fits].all(), (x, power)
            # the bias gradient sums whole diagonals: few of its entries fit times 2^12
            assert x == "grad_bias" or fits.float().mean() > 0.5


@pytest.mark.parametrize("dtype", DTYPES)
def test_caches_without_pages(dtype):
    """Users without events: no page is there, every result is zero."""
    h = tbe.tbe_attention_create(4, 2, 64, dtype)
    none = torch.empty((0, 16, 2, 64), dtype=dtype, device="cuda")
    q = torch.ones((3, 4, 64), dtype=dtype, device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    for width in (0, 2):
        table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
        out = tbe.tbe_attention_decode(h, q, none, none, table, n)
        assert not out.any()
        kv = torch.empty((0, 2, 64), dtype=dtype, device="cuda")
        tbe.tbe_attention_append(h, kv, kv, torch.zeros(4, dtype=torch.int64, device="cuda"), n, none, none, table)
    assert tbe.tbe_attention_get_error(h) == tbe.TBE_OK
    out = tbe.tbe_attention_decode(h, q[:0], none, none, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), n[:0])
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_delta_is_exact(dtype, dim):
    """Short histories, where out's rounding would show in the logits' gradients
    most.  A rounding is off by 0.42 u of a value in the 2-norm (u: the unit
    roundoff).  grad_q carries two, of ds and of the result: 0.6 u, of which 0.7
    is allowed; g . out with the rounded out (and the weights rounded on its way)
    for delta would exceed it, as the same arithmetic in 64 bits shows."""
    g = np.random.default_rng(57)
    b = Batch(dtype, 4, 4, dim, g.integers(2, 9, 400).tolist(), seed=57)
    got = b.check()
    q, k, v, up = (ref.f64(x) for x in (b.q, b.k, b.v, b.grad))
    want = ref.attention(q, k, v, b.off, 0, 0, b.scale, None, None, up, dtype)[0]["grad_q"]

    def rounded(x):
        return ref.f64(torch.from_numpy(x).to(dtype))

    exact, estimate = np.zeros_like(q), np.zeros_like(q)
    for lo, hi in zip(b.off[:-1], b.off[1:]):
        s = np.einsum("ihd,jhd->hij", q[lo:hi], k[lo:hi]) * b.scale
        s = np.where(np.tril(np.ones(s.shape[1:], bool)), s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        total = p.sum(-1, keepdims=True)
        out = np.einsum("hij,jhd->ihd", p / total, v[lo:hi])
        coarse = rounded(np.einsum("hij,jhd->ihd", rounded(p) / total, v[lo:hi]))
        dp = np.einsum("ihd,jhd->hij", up[lo:hi], v[lo:hi])
        for res, o in ((exact, out), (estimate, coarse)):
            ds = rounded(p / total * (dp - (o * up[lo:hi]).sum(-1).T[:, :, None]))
            res[lo:hi] = rounded(b.scale * np.einsum("hij,jhd->ihd", ds, k[lo:hi]))

    def off(x):
        return np.linalg.norm(x - want) / np.linalg.norm(want) / ref.UNIT[dtype]

    assert off(exact) <= 0.7 < off(estimate), (off(exact), off(estimate))
    assert off(ref.f64(got["grad_q"])) <= 0.7, off(ref.f64(got["grad_q"]))


@pytest.mark.parametrize("dim", [64, 128])
def test_many_histories_whose_tokens_see_many_keys(dim):
    """Listed tiles, a CTA each: above the length up to which they are taken in
    turn, one history far longer and one far shorter."""
    g = np.random.default_rng(dim)
    lengths = g.integers(250, 330, 135)
    lengths[7], lengths[90] = 700, 1
    Batch(torch.bfloat16, 2, 1, dim, lengths.tolist(), 0, 0, [0, 2, 60], seed=59).check()
