"""The softmax loss over a table of items on the GPU against the 64-bit reference."""

import numpy as np
import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe
import rows_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


class Case:
    def __init__(self, dtype, n, v, d, scale=1.0, left_out=0.2, spread=1.5, pad=0, shift=0, table_pad=0,
                 index=torch.int64, seed=0, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.scale = dtype, scale

        def normal(rows, wide, std):
            return (torch.randn((rows, wide), generator=g) * std).to(dtype).cuda()

        self.x = normal(n, d + pad + shift, 1.0)[:, shift:shift + d]
        self.table = normal(v, d + table_pad, spread * d ** -0.5)[:, :d]
        t = torch.randint(0, v, (n,), generator=g)
        t[torch.rand(n, generator=g) < left_out] = -100
        self.targets = t.to(index).cuda()
        self.grad = (torch.rand(n, generator=g) * size).cuda()
        self.h = tbe.tbe_softmax_loss_create(d, dtype, scale)

    def run(self, workspace=None, stream=None):
        loss, lse = tbe.tbe_softmax_loss_forward(self.h, self.x, self.table, self.targets, workspace=workspace,
                                                 stream=stream)
        gx, gw = tbe.tbe_softmax_loss_backward(self.h, self.x, self.table, self.targets, lse, self.grad,
                                               workspace=workspace, stream=stream)
        return {"loss": loss, "lse": lse, "grad_x": gx, "grad_table": gw}

    def want(self):
        return ref.loss(ref.f64(self.x), ref.f64(self.table), self.targets.cpu().numpy(), self.scale,
                        ref.f64(self.grad), self.dtype)

    def check(self, got=None, error=tbe.TBE_OK):
        got = got or self.run()
        assert tbe.tbe_softmax_loss_get_error(self.h) == error
        want, bound = self.want()
        for x in want:
            ref.close(got[x], want[x], bound[x], x)
        return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,d", [(1, 1, 1), (1, 2, 8), (2, 1, 16), (3, 5, 3), (64, 64, 64), (65, 63, 33), (128, 256, 64),
                                   (129, 257, 72), (127, 255, 56), (1, 5000, 64), (300, 1000, 128), (513, 129, 100),
                                   (40, 4097, 16), (130, 700, 256), (70, 300, 264), (33, 600, 520), (20, 100, 1000),
                                   (10, 130, 4096)])
def test_sizes(dtype, n, v, d):
    Case(dtype, n, v, d, seed=n + v + d).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [1, 2, 7, 8, 24, 31, 48, 63, 65, 96, 127, 129, 192, 200, 255, 257, 320, 384, 511, 512, 640])
def test_widths(dtype, d):
    Case(dtype, 150, 290, d, seed=d).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,d", [(700, 9000, 64), (2500, 2100, 40), (260, 20000, 128)])
def test_many_tiles(dtype, n, v, d):
    Case(dtype, n, v, d, seed=v).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,pad,shift,table_pad", [(64, 64, 0, 0), (64, 8, 8, 16), (64, 0, 1, 0), (64, 1, 0, 0),
                                                   (64, 0, 0, 1), (40, 24, 4, 3), (77, 3, 0, 51)])
def test_strided_rows(dtype, d, pad, shift, table_pad):
    Case(dtype, 200, 400, d, pad=pad, shift=shift, table_pad=table_pad, seed=d + pad).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_broadcast_row(dtype):
    c = Case(dtype, 150, 300, 64)
    c.x = c.x[:1].expand(150, 64)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_targets_outside_the_table(dtype, index):
    """Left out and reported; every row of one item, negative ones quietly left out."""
    c = Case(dtype, 140, 270, 48, index=index, left_out=0.5, seed=3)
    c.targets[7], c.targets[130] = 270, 2 ** 31 - 1
    c.check(error=tbe.TBE_ERR_INDEX_OOB)
    c.targets[7] = c.targets[130] = -2 ** 31
    c.check()
    c.targets.fill_(269)
    c.check()


def test_a_64_bit_target_is_read_whole():
    c = Case(torch.bfloat16, 10, 50, 16, left_out=0.0)
    c.targets[3] = 2 ** 32 + 5
    c.check(error=tbe.TBE_ERR_INDEX_OOB)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [40, 64, 65])
def test_rows_left_out_hold_anything(dtype, d):
    """NaN and infinities in rows that are left out, and in their upstream gradients, reach nothing else."""
    c, n = Case(dtype, 300, 500, d, seed=5), Case(dtype, 300, 500, d, seed=5)
    out = c.targets < 0
    n.x[out] = float("nan")
    n.grad[out] = float("inf")
    n.x[299], n.targets[299], c.targets[299] = float("inf"), -1, -1
    out[299] = True
    a, b = c.run(), n.run()
    assert torch.equal(a["lse"][~out], b["lse"][~out])
    for x in ("loss", "grad_x", "grad_table"):
        assert torch.equal(a[x], b[x]), x
    assert not b["grad_x"][out].any() and not b["loss"][out].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_all_rows_left_out(dtype):
    got = Case(dtype, 200, 300, 64, left_out=2.0).check()
    assert not got["loss"].any() and not got["grad_x"].any() and not got["grad_table"].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows_and_no_items(dtype):
    c = Case(dtype, 0, 30, 24)
    got = c.run()
    assert got["loss"].shape == (0,) and not got["grad_table"].any()
    c.table = c.table[:0]
    assert c.run()["grad_table"].shape == (0, 24)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale,spread", [(1e-3, 1.0), (20.0, 3.0), (1.0, 60.0), (0.05, 1.0)])
def test_flat_and_steep_logits(dtype, scale, spread):
    """From logits of 1e-3 to some of several hundred (beyond exp's range in fp32)."""
    Case(dtype, 140, 520, 64, scale=scale, spread=spread, seed=2).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_rising_table(dtype):
    """Each tile of items holds a new maximum, and the first ones nothing beside the last."""
    c = Case(dtype, 140, 1500, 32, spread=0.1, seed=6)
    c.x[:, 0] = 1.0
    c.table[:, 0] = (torch.arange(1500, device="cuda") / 8.0).to(dtype)
    c.check()
    c.table[:, 0] = (-torch.arange(1500, device="cuda") / 8.0).to(dtype)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [0.0, 1e-6, 1.0, 3e4])
def test_sizes_of_the_upstream_gradient(dtype, size):
    """fp16's results are checked where they fit fp16."""
    c = Case(dtype, 150, 300, 64, size=size, seed=4)
    c.grad[::3] *= -1.0
    c.grad[5] = 0.0
    if dtype == torch.float16 and size > 100:
        c.table *= 0.05
    c.check()


def test_small_gradients_of_fp16_beside_many_items():
    """Weights of 1e-4 and upstream gradients of 1e-4: held relative to the largest one, not to 1."""
    c = Case(torch.float16, 400, 10000, 64, left_out=0.0, seed=9)
    c.grad.fill_(65536.0 / 400)
    c.check()
    c.grad.mul_(1e-3)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(150, 64), (2100, 40), (300, 300)])
def test_upstream_gradients_of_all_sizes(dtype, n, d):
    """One row's is far the largest, one is infinite in a row that is left out, some are 0, some are negative; beyond
    2048 rows another launch looks for the largest."""
    c = Case(dtype, n, 200, d, seed=8)
    c.grad = torch.linspace(-1.0, 1.0, n, device="cuda") ** 3
    c.grad[n // 3] = 8.0
    c.targets[n // 3] = 3
    c.grad[5::50] = 0.0
    c.targets[7], c.grad[7] = -1, float("inf")
    got = c.run()
    c.grad[7] = 0.0
    c.check(got)


@pytest.mark.parametrize("dtype", DTYPES)
def test_results_off_16_byte_boundaries(dtype):
    """Results in views that begin anywhere: written element by element."""
    for d in (64, 72, 264):
        c = Case(dtype, 140, 300, d, seed=d)
        want = c.run()
        gx, gw = (torch.full((r * d + 3,), 7.0, dtype=dtype, device="cuda") for r in (140, 300))
        tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, want["lse"], c.grad, grad_x=gx[1:-2].view(140, d),
                                      grad_table=gw[1:-2].view(300, d))
        assert torch.equal(gx[1:-2].view(140, d), want["grad_x"]) and torch.equal(gw[1:-2].view(300, d), want["grad_table"])
        for t in (gx, gw):  # what lies around them is left as it was
            assert t[0] == 7.0 and (t[-2:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 264])
def test_results_in_the_place_of_operands(dtype, d):
    """grad_x may be x; a gradient over the table, or both in one place, are refused before anything is written."""
    c = Case(dtype, 150, 150, d, seed=d)
    want = c.run()
    for kw in (dict(grad_x=c.table), dict(grad_table=c.table), dict(grad_x=c.x, grad_table=c.x),
               dict(grad_x=c.table, want=(True, False)), dict(grad_table=c.table, want=(False, True))):
        with pytest.raises(tbe.TBEError) as e:
            tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, want["lse"], c.grad, **kw)
        assert e.value.code == tbe.TBE_ERR_INVALID_ARG
    both = torch.empty((299, d), dtype=dtype, device="cuda")  # (they share a row)
    with pytest.raises(tbe.TBEError) as e:
        tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, want["lse"], c.grad, both[:150], both[149:])
    assert e.value.code == tbe.TBE_ERR_INVALID_ARG
    gx, gw = tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, want["lse"], c.grad, grad_x=c.x)
    assert gx is c.x and torch.equal(gx, want["grad_x"]) and torch.equal(gw, want["grad_table"])


def test_two_handles_on_two_streams():
    """Calls of two handles whose work overlaps share nothing."""
    a, b = Case(torch.bfloat16, 900, 6000, 128, seed=1), Case(torch.float32, 400, 3001, 96, seed=2)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[c.run(stream=s) for c, s in zip((a, b), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            for x in w:
                assert torch.equal(g[x], w[x]), x


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_gradient_wanted(dtype):
    c = Case(dtype, 200, 700, 72, seed=1)
    both = c.run()
    for want in ((True, False), (False, True), (False, False)):
        gx, gw = tbe.tbe_softmax_loss_backward(c.h, c.x, c.table, c.targets, both["lse"], c.grad, want=want)
        assert (gx is not None) == want[0] and (gw is not None) == want[1]
        assert gx is None or torch.equal(gx, both["grad_x"])
        assert gw is None or torch.equal(gw, both["grad_table"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,d", [(300, 5000, 64), (2000, 9000, 128), (1, 9999, 72)])
def test_the_same_bits_again(dtype, n, v, d):
    c = Case(dtype, n, v, d)
    a, b = c.check(), c.run()
    for x in a:
        assert torch.equal(a[x], b[x]), x


@pytest.mark.parametrize("dtype", DTYPES)
def test_workspace_serves_smaller_calls(dtype):
    big = Case(dtype, 600, 9000, 72)
    for backward in (False, True):
        most = tbe.tbe_softmax_loss_workspace_bytes(big.h, 600, 9000, backward)
        for n, v in ((1, 1), (1, 9000), (600, 1), (37, 8191), (129, 4097), (599, 257)):
            assert tbe.tbe_softmax_loss_workspace_bytes(big.h, n, v, backward) <= most
    ws = tbe.make_softmax_loss_workspace(big.h, 600, 9000, True)
    ws.fill_(255)  # whatever an earlier call left there
    for n, v in ((1, 9000), (37, 8191), (600, 1), (600, 9000)):
        c = Case(dtype, n, v, 72, seed=n)
        c.check(c.run(workspace=ws))


def test_elements_beyond_32_bits():
    """A table of 2.7e9 elements; the rows' items and neighbours lie at its two ends."""
    v, d = 2 ** 24 + 77, 160
    table = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((3, d), generator=g, device="cuda").bfloat16()
    at = torch.tensor([0, 5, v - 300, v - 2, v - 1], device="cuda")
    table[at] = torch.randn((5, d), generator=g, device="cuda").bfloat16()
    targets = torch.tensor([v - 1, 5, v - 300], device="cuda")
    h = tbe.tbe_softmax_loss_create(d, torch.bfloat16)
    loss, lse = tbe.tbe_softmax_loss_forward(h, x, table, targets)
    gx, gw = tbe.tbe_softmax_loss_backward(h, x, table, targets, lse, torch.ones(3, device="cuda"))
    assert tbe.tbe_softmax_loss_get_error(h) == tbe.TBE_OK
    s = x.double() @ table[at].double().t()
    want = torch.log(s.exp().sum(1) + (v - 5))
    assert torch.allclose(lse.double(), want, atol=1e-4, rtol=0)  # 2^24 sums of fp32 in 2^16 parts: 256 steps of 2^-24 each
    p = (s - want[:, None]).exp()
    p[[0, 1, 2], [4, 1, 2]] -= 1.0
    gx_want, gw_want = p @ table[at].double(), p.t() @ x.double()
    assert torch.allclose(loss.double(), want - s[[0, 1, 2], [4, 1, 2]], atol=2e-4, rtol=0)
    # 2^-8 of the rounded weight and of the result, 2^-12 for lse and the products' sums
    assert ((gx.double() - gx_want).abs() <= 2 ** -7 * (p.abs() @ table[at].double().abs()) + 1e-3).all()
    assert ((gw[at].double() - gw_want).abs() <= 2 ** -7 * (p.abs().t() @ x.double().abs()) + 1e-6).all()


def test_streams_and_graphs():
    c = Case(torch.bfloat16, 500, 3001, 64, seed=7)
    want = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = c.run(stream=side)
    side.synchronize()
    for x in want:
        assert torch.equal(got[x], want[x]), x
    ws = tbe.make_softmax_loss_workspace(c.h, 500, 3001, True)
    graphs, results = [], []
    for _ in range(2):  # two graphs that share a workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(c.run(workspace=ws))
        graphs.append(graph)
    c.x.neg_()
    c.targets.fill_(17)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = c.run()
    for got in results:
        for x in want:
            assert torch.equal(got[x], want[x]), x


def test_refusals():
    c = Case(torch.bfloat16, 20, 40, 64)
    _, lse = tbe.tbe_softmax_loss_forward(c.h, c.x, c.table, c.targets)

    def forward(**kw):
        a = dict(x=c.x, table=c.table, targets=c.targets)
        a.update(kw)
        return tbe.tbe_softmax_loss_forward(c.h, **a)

    def backward(**kw):
        a = dict(x=c.x, table=c.table, targets=c.targets, lse=lse, grad_loss=c.grad)
        a.update(kw)
        return tbe.tbe_softmax_loss_backward(c.h, **a)

    for call, kw in ((forward, dict(x=c.x.float())), (forward, dict(x=c.x[:, :32])), (forward, dict(x=c.x[0])),
                     (forward, dict(table=c.table[:, :32])), (forward, dict(targets=c.targets.float())),
                     (forward, dict(targets=c.targets[:5])), (forward, dict(table=c.table.half())),
                     (forward, dict(targets=c.targets.cpu())), (forward, dict(loss=lse[:3])),
                     (forward, dict(table=c.table.t().contiguous().t())),
                     (backward, dict(lse=lse[:3])), (backward, dict(grad_loss=c.grad.double())),
                     (backward, dict(grad_loss=c.grad[:1].expand(20))), (backward, dict(grad_x=c.x.float())),
                     (backward, dict(grad_table=torch.empty((41, 64), dtype=c.dtype, device="cuda"))),
                     (backward, dict(workspace=torch.empty(4096)))):
        with pytest.raises(ValueError):
            call(**kw)
    for call in (forward, backward):
        with pytest.raises(tbe.TBEError) as e:
            call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        assert e.value.code == tbe.TBE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(tbe.TBEError) as e:  # rows over nothing
        forward(table=c.table[:0])
    assert e.value.code == tbe.TBE_ERR_INVALID_ARG
    with pytest.raises(tbe.TBEError) as e:  # rows of the table that overlap
        forward(table=c.table[:1].expand(40, 64))
    assert e.value.code == tbe.TBE_ERR_INVALID_ARG
    c.h.close()
    with pytest.raises(RuntimeError):
        forward()


@pytest.mark.parametrize("dtype,n,v,d", [(torch.float32, 70, 30000, 512), (torch.bfloat16, 130, 150000, 136),
                                         (torch.float16, 20, 40000, 520)])
def test_tables_copied_in_parts(dtype, n, v, d):
    """fp32 and rows off 16-byte boundaries are copied a part of the table at a time; the last part is a short one."""
    c = Case(dtype, n, v, d, seed=3, table_pad=1)
    for x in (c, Case(dtype, n, v - v % 256 - 255, d, seed=4, table_pad=1)):
        x.check()
