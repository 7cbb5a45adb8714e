"""How exact the softmax loss is, by the 2-norm of its errors against 64 bits (the element by element bounds of the
other tests have to allow for the worst case of every sum).

Bounds, of the norm of the result.  A result rounded to fp16 is 2.1e-4 off (2^-11 / sqrt(3), values within a factor of
two of each other: times 0.75 on average), and no more comes from d's rounding: together sqrt(2) of that, 3.0e-4; bf16
eight times that, 2.4e-3.  The tensor units cut each sum of 16 products' terms by up to 2^-23 of the sum so far, which
for a sum that grows evenly is 2^-25 of its final value on average (half the cut, half the sum): k products in one
accumulator shrink the result by k 2^-25.
"""

import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe
import rows_reference as ref

pytestmark = pytest.mark.gpu
FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32


class Case:
    def __init__(self, dtype, n, v, d, seed=1, targets_from=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn((n, d), generator=g, device="cuda").to(dtype)
        self.table = (torch.randn((v, d), generator=g, device="cuda") * 1.5 * d ** -0.5).to(dtype)
        self.targets = torch.randint(targets_from, v, (n,), generator=g, device="cuda")
        self.grad = torch.full((n,), 1024.0 if dtype == FP16 else 1.0, device="cuda")
        self.h = tbe.tbe_softmax_loss_create(d, dtype)

    def run(self):
        self.loss, self.lse = tbe.tbe_softmax_loss_forward(self.h, self.x, self.table, self.targets)
        self.grad_x, self.grad_table = tbe.tbe_softmax_loss_backward(self.h, self.x, self.table, self.targets, self.lse,
                                                                     self.grad)
        assert tbe.tbe_softmax_loss_get_error(self.h) == tbe.TBE_OK

    def rows(self, at):
        """loss, lse and grad_x of the rows `at` in 64 bits, and the target's own term of grad_x."""
        w, t = self.table.double(), self.targets[at]
        s = self.x[at].double() @ w.t()
        lse = torch.logsumexp(s, 1)
        hot = w[t] * self.grad[at].double()[:, None]
        return lse - s.gather(1, t[:, None])[:, 0], lse, torch.softmax(s, 1) @ w * self.grad[at].double()[:, None] - hot, hot

    def items(self, at):
        """grad_table of the items `at`, the rows in parts."""
        got = torch.zeros((len(at), self.x.shape[1]), dtype=torch.float64, device="cuda")
        w = self.table[at].double()
        for lo in range(0, self.x.shape[0], 65536):
            x, t = self.x[lo:lo + 65536].double(), self.targets[lo:lo + 65536]
            p = torch.exp(x @ w.t() - self.lse[lo:lo + 65536].double()[:, None]) - (t[:, None] == at[None, :]).double()
            got += (p * self.grad[lo:lo + 65536].double()[:, None]).t() @ x
        return got


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def shrunk(got, want):
    return 1.0 - ((got.double() * want).sum() / (want * want).sum()).item()


@pytest.mark.parametrize("dtype,n,v,d", [(FP16, 10000, 1000000, 128), (FP16, 16384, 400000, 256), (BF16, 10000, 1000000, 40)])
def test_long_sums_over_the_items(dtype, n, v, d):
    """Accumulators take 32,768 items at most: 2^-14, twice that for a cut's size within a power of two (1,000,000 in one
    would be 2e-3).  What is left beside the target's own term, which would cover it, is compared."""
    c = Case(dtype, n, v, d)
    c.run()
    at = torch.arange(0, n, n // 48, device="cuda")
    _, _, want, hot = c.rows(at)
    assert off(c.grad_x[at], want) < (3.0e-4 if dtype == FP16 else 2.4e-3) + 2 ** -13
    if dtype == FP16:  # (bf16's rounding of 48 x 40 results leaves 2e-3 / 44 in the mean, times hot's size beside the rest)
        assert abs(shrunk(c.grad_x[at].double() + hot, want + hot)) < 2 ** -13


@pytest.mark.parametrize("dtype,n,v,d", [(FP16, 262144, 40000, 64), (FP16, 262144, 20000, 256), (FP16, 140000, 30001, 200),
                                         (FP16, 33000, 60000, 64)])
def test_long_sums_over_the_rows(dtype, n, v, d):
    """The same of the table's gradient, of items that are nobody's target and of some that are; 30,001 x 200 columns
    is copied in parts (its rows lie off 16-byte boundaries)."""
    c = Case(dtype, n, v, d, targets_from=64)
    if d == 200:
        c.table = torch.cat([c.table, c.table[:, :1]], 1)[:, :d]
    c.run()
    at = torch.cat([torch.arange(64, device="cuda"), torch.tensor([v - 1, v - 200, v // 2], device="cuda")])
    want = c.items(at)
    assert abs(shrunk(c.grad_table[at[:64]], want[:64])) < 2 ** -13
    assert off(c.grad_table[at], want) < 3.0e-4 + 2 ** -13
    at = torch.arange(0, n, n // 20, device="cuda")
    assert off(c.grad_x[at], c.rows(at)[2]) < 3.0e-4 + 2 ** -13


@pytest.mark.parametrize("copied", [False, True])
def test_long_sums_over_the_rows_of_many_items(copied):
    """More tiles of items than the sums' parts otherwise have room for; copied, in two spans of the table."""
    c = Case(FP16, 33000, 200000, 64)
    if copied:
        c.table = torch.cat([c.table, c.table[:, :1]], 1)[:, :64]
    c.run()
    for at in (0, 65536, 131000, 131072, 199900):
        at = torch.arange(at, at + 100, device="cuda")
        assert off(c.grad_table[at], c.items(at)) < 3.0e-4 + 2 ** -13
    at = torch.arange(0, 33000, 1100, device="cuda")
    assert off(c.grad_x[at], c.rows(at)[2]) < 3.0e-4 + 2 ** -13


def test_long_sums_over_the_rows_of_wide_operands():
    """Above 256 columns d passes through memory in pieces; here of 256 items, whose sums go over 36,864 rows each."""
    c = Case(FP16, 700000, 250, 4096, targets_from=16)
    c.run()
    at = torch.tensor([0, 1, 7, 15, 16, 17, 128, 249], device="cuda")
    got, want = c.grad_table[at], c.items(at)
    # (1024 times a sum of 700,000 rows: results from 65520 on round to an infinity of fp16.  Within 1 % of it, 20 times
    # the errors' norm below, either is right)
    fits, beyond = want.abs() < 64865.0, want.abs() > 66175.0
    assert torch.equal(got[beyond].double(), torch.copysign(torch.full_like(want, float("inf")), want)[beyond])
    assert abs(shrunk(got[:4][fits[:4]], want[:4][fits[:4]])) < 2 ** -13
    assert off(got[fits], want[fits]) < 3.0e-4 + 2 ** -13


# A score of 4096 columns in parts of 512: 32 products each, cut by 32 2^-25 = 1e-6 of the part's size, which grows as a
# random walk's (2/3 of its final value on average) and has a sign of its own: 6e-7 of a score's size, 1.5.  Of a loss
# and lse of about 11 that is 1e-7 by the target's score and, as every score shrinks, E_p[s] 6e-7 / 11 = 1.2e-7 by lse:
# 2e-7 together, and 1e-7 for fp32's roundings and the sum's.  In one accumulator it was 8e-7 to 1e-6.
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("n,v,d", [(300, 30000, 4096), (140, 9000, 2500), (300, 20000, 1000), (200, 5001, 577)])
def test_scores_over_many_columns(dtype, n, v, d):
    c = Case(dtype, n, v, d)
    c.run()
    at = torch.arange(n, device="cuda")
    loss, lse, grad_x, _ = c.rows(at)
    assert off(c.loss, loss) < 3e-7 and off(c.lse, lse) < 3e-7
    # 16 bits: d's and the result's rounding.  fp32: weights off by their scores' 6e-7 times 1.5 and lse's 1e-6, one of
    # which follows the other, and the sums' 32 products 1e-6
    bound = {FP16: 3.0e-4, BF16: 2.4e-3, FP32: 2e-6}[dtype] + 2 ** -13 * (dtype != FP32)
    assert off(c.grad_x, grad_x) < bound
    at = torch.arange(0, v, 97, device="cuda")
    assert off(c.grad_table[at], c.items(at)) < bound


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("n,v,d", [(64, 5000, 64), (300, 700, 250), (2300, 3000, 40)])
def test_rows_of_small_upstream_gradients(dtype, n, v, d):
    """Each row's grad_x is as exact as if it were alone: d enters its sum without g.  The largest g is 2^27 times the
    smallest (they are powers of two, so that scaling them back is exact); fp16's results stay above its smallest
    normal number's neighbourhood by the table's size, and what is below loses half a step of 2^-24."""
    c = Case(dtype, n, v, d)
    c.grad = torch.exp2(-(torch.arange(n, device="cuda") % 28).float() + (10 if dtype == FP16 else 0))
    c.grad[1::2] *= -1.0
    c.run()
    got = c.grad_x.double() / c.grad.double()[:, None]
    want, bound = ref.loss(ref.f64(c.x), ref.f64(c.table), c.targets.cpu().numpy(), 1.0, torch.ones(n).double().numpy(), dtype)
    # (the bound of rows whose g is 1, and what the result's rounding in the subnormals loses)
    half_step = 2.0 ** -25 if dtype == FP16 else 2.0 ** -134
    room = torch.from_numpy(bound["grad_x"]).cuda() + half_step / c.grad.double().abs()[:, None]
    assert bool(((got - torch.from_numpy(want["grad_x"]).cuda()).abs() <= room).all())
    at = torch.arange(v, device="cuda")
    assert off(c.grad_table, c.items(at)) < {FP32: 2e-6, BF16: 2.4e-3, FP16: 3.0e-4}[dtype] + 2 ** -13 * (dtype != FP32)


def check_all(c, tolerance):
    """loss, lse and both gradients of all rows and items, and each element (the norm would not show a single one): none
    is off by more than 16 roundings of the largest, in fp32 64: a weight of 1 is off by lse's error, which may be 3e-7
    of 11, 55 of fp32's roundings of 2^-24, and half a step of an lse of 8 to 16, 8 of them."""
    n, v = c.targets.numel(), c.table.shape[0]
    parts = [c.rows(torch.arange(lo, min(n, lo + 2048), device="cuda")) for lo in range(0, n, 2048)]
    loss, lse, grad_x = (torch.cat([p[i] for p in parts]) for i in range(3))
    # fp32's roundings of sums of up to 40,000 terms in 64 parts or more, one of loss itself, 2^-22 of each exponential
    assert off(c.loss, loss) < 3e-7 and off(c.lse, lse) < 3e-7
    grad_table = torch.cat([c.items(torch.arange(lo, min(v, lo + 2048), device="cuda")) for lo in range(0, v, 2048)])
    for got, want in ((c.grad_x, grad_x), (c.grad_table, grad_table)):
        assert off(got, want) < tolerance
        assert (got.double() - want).abs().max() <= (64 if got.dtype == FP32 else 16) * ref.UNIT[got.dtype] * want.abs().max()


# fp32: 24 to 32 products in an accumulator, 7e-7 to 1e-6 by their cuts, 5e-7 by the scores of up to 264 columns (17
# products, half of their cuts' 5e-7 times 1.5 follows lse's), roundings 1e-7: 1.5e-6 and, above 128 columns, 1.8e-6.
# Two bf16 terms of each operand instead of three are 3.2e-6 off; sums of 313 blocks in one accumulator 2.2e-5.
@pytest.mark.parametrize("dtype,n,v,d,tolerance", [
    (FP32, 2050, 20011, 96, 1.5e-6),     # fused, sums in many parts
    (FP32, 300, 9000, 60, 1.5e-6),
    (FP32, 5000, 8000, 136, 1.8e-6),     # three pieces of d, seven slabs of rows, sums in parts of 8 blocks
    (FP32, 900, 30000, 264, 1.8e-6),     # the table's gradient added to in place
    (BF16, 3000, 40000, 264, 2.4e-3),    # three pieces, the table read in place
    (FP16, 12000, 9001, 264, 3.0e-4),    # three pieces and three slabs of rows: joined two launches later
    (BF16, 12000, 9001, 320, 2.4e-3),
    (FP16, 4096, 20000, 512, 3.0e-4),
    (FP16, 2500, 30000, 128, 3.0e-4),    # fused
    (BF16, 2500, 30000, 250, 2.4e-3)])
def test_all_results(dtype, n, v, d, tolerance):
    c = Case(dtype, n, v, d, seed=n)
    c.run()
    check_all(c, tolerance)


@pytest.mark.parametrize("dtype,n,v,d", [(FP32, 2600, 9000, 192), (BF16, 9000, 6000, 264), (FP16, 9000, 6000, 300)])
def test_pieces_again_alone_in_a_used_workspace_and_in_graphs(dtype, n, v, d):
    """What the fused kernel's tests ask of it, of d in memory: two pieces, several slabs of rows and of items."""
    c, o = Case(dtype, n, v, d, seed=5), Case(FP32 if dtype == BF16 else BF16, 2000, 9001, 264, seed=6)
    c.targets[::7] = -1
    c.run(), o.run()
    want = [c.loss, c.lse, c.grad_x, c.grad_table]
    other = [o.grad_x, o.grad_table]
    assert not c.grad_x[::7].any()
    ws = tbe.make_softmax_loss_workspace(c.h, n, v, True)

    def call(workspace=ws, stream=None, **kw):
        loss, lse = tbe.tbe_softmax_loss_forward(c.h, c.x, c.table, c.targets, workspace=workspace, stream=stream)
        return [loss, lse, *tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, lse, c.grad, workspace=workspace,
                                                          stream=stream, **kw)]

    for byte in (255, 0):
        ws.fill_(byte)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    ws.fill_(255)  # a smaller call in the same workspace, then the large one again
    small = tbe.tbe_softmax_loss_forward(c.h, c.x[:100], c.table[:777], c.targets[:100] % 777, workspace=ws)
    gx, _ = tbe.tbe_softmax_loss_backward(c.h, c.x[:100], c.table[:777], c.targets[:100] % 777, small[1], c.grad[:100],
                                          workspace=ws)
    assert bool(gx.isfinite().all()) and all(torch.equal(a, b) for a, b in zip(call(), want))
    assert torch.equal(call(want=(True, False))[2], want[2]) and torch.equal(call(want=(False, True))[3], want[3])
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(call())
        graphs.append(graph)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    streams = torch.cuda.Stream(), torch.cuda.Stream()  # two handles whose calls overlap
    got = []
    for _ in range(3):
        got.append((call(workspace=None, stream=streams[0]),
                    tbe.tbe_softmax_loss_backward(o.h, o.x, o.table, o.targets, o.lse, o.grad, stream=streams[1])))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, other))
    assert tbe.tbe_softmax_loss_get_error(c.h) == tbe.TBE_OK and tbe.tbe_softmax_loss_get_error(o.h) == tbe.TBE_OK
