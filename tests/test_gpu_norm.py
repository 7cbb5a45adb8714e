"""Layer norm on the GPU against the 64-bit reference."""

import numpy as np
import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe
import rows_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


class Case:
    def __init__(self, dtype, rows, dim, residual=True, weight=True, bias=True, up=True, pad=0, shift=0, eps=1e-5,
                 seed=0, spread=1.0, mean=0.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.eps = dtype, eps

        def normal(*shape, std=1.0, at=0.0):
            return (torch.randn(shape, generator=g) * std + at).to(dtype).cuda()

        def strided(std=1.0, at=0.0):  # rows of a wider buffer, `shift` elements in
            t = normal(rows, dim + pad + shift, std=std, at=at)
            return t[:, shift:shift + dim]

        self.x = strided(spread, mean)
        self.residual = strided() if residual else None
        self.weight = normal(dim, std=0.3, at=1.0) if weight else None
        self.bias = normal(dim, std=0.5) if bias else None
        self.grad = strided()
        self.up = strided() if up else None
        self.h = tbe.tbe_layer_norm_create(dim, dtype, eps, weight, bias)

    def run(self, **kw):
        out, total, stats = tbe.tbe_layer_norm_forward(self.h, self.x, self.weight, self.bias, self.residual, **kw)
        gx, gw, gb = tbe.tbe_layer_norm_backward(self.h, total, stats, self.grad, self.weight, self.up, **kw)
        return {"out": out, "total": total, "mean": stats[0], "rstd": stats[1], "grad_x": gx, "grad_weight": gw,
                "grad_bias": gb}

    def check(self, got=None):
        got = got or self.run()
        if self.residual is not None:
            want = ref.f64(self.x) + ref.f64(self.residual)
            ref.close(got["total"], want, (ref.UNIT[self.dtype] + 2 * ref.F) * np.abs(want) + ref.TINY[self.dtype],
                      "total")
        else:
            assert got["total"] is self.x
        w, b, u = (None if t is None else ref.f64(t) for t in (self.weight, self.bias, self.up))
        want, bound = ref.norm(ref.f64(got["total"]), self.eps, w, b, ref.f64(self.grad), u, self.dtype)
        for x in want:
            if (x == "grad_weight" and w is None) or (x == "grad_bias" and b is None):
                assert got[x] is None
            else:
                ref.close(got[x], want[x], bound[x], x)
        return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 2, 3, 7, 8, 16, 31, 32, 40, 63, 64, 77, 96, 128, 200, 255, 256, 264, 500, 512, 520,
                                 1000, 1024, 1032, 2000, 2048, 2056, 4096, 4104, 5001, 8192, 8200, 16383, 16384])
def test_widths(dtype, dim):
    Case(dtype, 21 if dim < 4000 else 5, dim, seed=dim).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 31, 33, 257, 4099])
@pytest.mark.parametrize("dim", [24, 77, 256, 1100])
def test_rows(dtype, rows, dim):
    Case(dtype, rows, dim, seed=rows).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual,weight,bias,up", [(False, False, False, False), (False, True, False, True),
                                                     (True, False, True, False), (False, True, True, False),
                                                     (True, False, False, True), (True, True, False, True)])
@pytest.mark.parametrize("dim", [64, 77, 640])
def test_what_is_left_out(dtype, residual, weight, bias, up, dim):
    Case(dtype, 67, dim, residual, weight, bias, up, seed=5).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,pad,shift", [(64, 64, 0), (64, 8, 8), (64, 1, 0), (64, 0, 3), (256, 4, 4), (200, 2, 2),
                                           (77, 51, 0), (1024, 129, 1), (1500, 36, 12)])
def test_strided_rows(dtype, dim, pad, shift):
    Case(dtype, 39, dim, pad=pad, shift=shift, seed=dim + pad).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [48, 512])
def test_broadcast_rows(dtype, dim):
    c = Case(dtype, 50, dim, seed=8)
    c.x, c.grad, c.up = (t[:1].expand(50, dim) for t in (c.x, c.grad, c.up))
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 1024, 3000])
def test_mean_far_from_zero(dtype, dim):
    """The variance is that of the differences: no cancellation of squares."""
    Case(dtype, 9, dim, residual=False, spread=0.5, mean=300.0, seed=2).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 40, 512, 2048])
def test_constant_rows_give_the_bias(dtype, dim):
    c = Case(dtype, 6, dim, residual=False, seed=9)
    c.x.fill_(1.5)
    got = c.check()
    assert torch.equal(got["out"], c.bias.expand(6, dim))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [32, 77, 256, 2048])
def test_a_row_of_nan_stays_by_itself(dtype, dim):
    c, n = Case(dtype, 12, dim, seed=4), Case(dtype, 12, dim, seed=4)
    n.x[5] = float("nan")
    a, b = c.run(), n.run()
    keep = torch.arange(12) != 5
    for x in ("out", "total", "grad_x"):
        assert torch.equal(a[x][keep], b[x][keep]) and bool(b[x][5].isnan().all()), x


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows(dtype):
    c = Case(dtype, 0, 72)
    got = c.run()
    assert got["out"].shape == (0, 72) and got["grad_x"].shape == (0, 72)
    assert not got["grad_weight"].any() and not got["grad_bias"].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [77, 256, 5000])
def test_in_place(dtype, dim):
    c = Case(dtype, 130, dim, seed=6)
    want = c.run()
    total, out = c.residual.clone(), c.x.clone()
    tbe.tbe_layer_norm_forward(c.h, out, c.weight, c.bias, total, out=out, total=total)
    assert torch.equal(out, want["out"]) and torch.equal(total, want["total"])
    stats = torch.stack([want["mean"], want["rstd"]])
    for own in ("grad", "up"):
        gx = getattr(c, own).clone()
        args = {"grad": c.grad, "up": c.up, own: gx}
        tbe.tbe_layer_norm_backward(c.h, total, stats, args["grad"], c.weight, args["up"], grad_x=gx)
        assert torch.equal(gx, want["grad_x"]), own


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim", [(70001, 8), (20011, 64), (9001, 512), (3001, 2048)])
def test_many_rows_and_the_same_bits_again(dtype, rows, dim):
    c = Case(dtype, rows, dim, seed=1)
    a = c.check()
    b = c.run()
    for x in a:
        assert torch.equal(a[x], b[x]), x


def test_elements_beyond_32_bits():
    rows, dim = 140000, 16384  # 2.29e9 elements
    h = tbe.tbe_layer_norm_create(dim, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros_like(x)
    last = slice(rows - 3, rows)
    x[last] = torch.randn((3, dim), generator=g, device="cuda").bfloat16()
    up[last] = torch.randn((3, dim), generator=g, device="cuda").bfloat16()
    w, b = torch.randn((2, dim), generator=g, device="cuda").bfloat16()
    out, total, stats = tbe.tbe_layer_norm_forward(h, x, w, b)
    gx, gw, gb = tbe.tbe_layer_norm_backward(h, total, stats, up, w)
    want, bound = ref.norm(ref.f64(x[last]), 1e-5, ref.f64(w), ref.f64(b), ref.f64(up[last]), dtype=torch.bfloat16)
    for name, got in (("out", out[last]), ("grad_x", gx[last]), ("grad_weight", gw), ("grad_bias", gb)):
        ref.close(got, want[name], bound[name], name)


def test_workspace_serves_fewer_rows():
    c = Case(torch.bfloat16, 3000, 256, seed=3)
    ws = tbe.make_layer_norm_workspace(c.h, 3000)
    for n in (1, 40, 700, 3000):
        out, total, stats = tbe.tbe_layer_norm_forward(c.h, c.x[:n], c.weight, c.bias, c.residual[:n])
        got = tbe.tbe_layer_norm_backward(c.h, total, stats, c.grad[:n], c.weight, workspace=ws)
        want = tbe.tbe_layer_norm_backward(c.h, total, stats, c.grad[:n], c.weight)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_and_graphs():
    c = Case(torch.bfloat16, 1000, 256, seed=7)
    want = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = c.run(stream=side)
    side.synchronize()
    for x in want:
        assert torch.equal(got[x], want[x]), x
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.run()
    c.x.neg_()
    c.residual.neg_()
    graph.replay()
    torch.cuda.synchronize()
    want = c.run()
    for x in want:
        assert torch.equal(got[x], want[x]), x


def test_refusals():
    c = Case(torch.bfloat16, 8, 64)
    out, total, stats = tbe.tbe_layer_norm_forward(c.h, c.x, c.weight, c.bias, c.residual)

    def forward(**kw):
        a = dict(x=c.x, weight=c.weight, bias=c.bias, residual=c.residual)
        a.update(kw)
        return tbe.tbe_layer_norm_forward(c.h, **a)

    def backward(**kw):
        a = dict(total=total, stats=stats, grad_out=c.grad, weight=c.weight, grad_total=c.up)
        a.update(kw)
        return tbe.tbe_layer_norm_backward(c.h, **a)

    for call, kw in ((forward, dict(x=c.x.float())), (forward, dict(x=c.x[:, :32])), (forward, dict(x=c.x[0])),
                     (forward, dict(weight=None)), (forward, dict(bias=None)), (forward, dict(residual=c.residual[:4])),
                     (forward, dict(weight=c.weight.float())), (forward, dict(out=torch.empty_like(out)[:4])),
                     (forward, dict(residual=None, total=out)), (forward, dict(stats=stats[:1])),
                     (forward, dict(x=c.x.cpu())), (forward, dict(out=torch.empty((8, 128), dtype=c.dtype,
                                                                                  device="cuda")[:, :64])),
                     (forward, dict(x=torch.empty((64, 8), dtype=c.dtype, device="cuda").t())),
                     (backward, dict(weight=None)), (backward, dict(grad_out=c.grad[:3])), (backward, dict(stats=stats.t())),
                     (backward, dict(grad_total=c.up.half())), (backward, dict(workspace=torch.empty(4096)))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(tbe.TBEError) as e:
        backward(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tbe.TBE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(tbe.TBEError) as e:  # both results in one place
        forward(out=total, total=total)
    assert e.value.code == tbe.TBE_ERR_INVALID_ARG
    for t in (c.x, total):
        with pytest.raises(ValueError):
            tbe.tbe_layer_norm_forward(tbe.tbe_layer_norm_create(32, c.dtype), t, c.weight, c.bias)
    c.h.close()
    with pytest.raises(RuntimeError):
        forward()


def test_handles_without_parameters_refuse_them():
    h = tbe.tbe_layer_norm_create(64, torch.bfloat16, weight=False, bias=False)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    out, total, stats = tbe.tbe_layer_norm_forward(h, x)
    for kw in (dict(weight=x[0]), dict(bias=x[0])):
        with pytest.raises(ValueError):
            tbe.tbe_layer_norm_forward(h, x, **kw)
    for kw in (dict(weight=x[0]), dict(grad_weight=x[0].clone()), dict(grad_bias=x[0].clone())):
        with pytest.raises(ValueError):
            tbe.tbe_layer_norm_backward(h, total, stats, x, **kw)
