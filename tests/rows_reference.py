"""Layer norm and the softmax loss over a table of items in 64 bits, from the
definitions, with error bounds of the operators' results.

Bounds.  u is the unit roundoff of the tensors' type, f = 2^-24, `tiny` half of
the type's smallest step (what a rounding loses in its subnormals).

Layer norm: a thread adds up at most 64 elements of a row, a tree of at most 16
levels joins the threads, so a row's sum is off by n = min(D, 80) roundings.
  mean  (n + 2) f mean|t| =: em
  var   the error of the mean enters squared (the differences' sum vanishes):
        (n + 6) f var + 2 em^2 + 4 f em mean|c|;  rstd: half of that / (var + eps), + 6 f
  xhat  em rstd + |xhat| (that + 4 f) =: eh
  out   u |out| + |w| eh + 4 f (|xhat w| + |b|)
  gradients alike by their formulas; sums over N rows N f of their magnitudes.

Loss: the tensor units may cut instead of round, 2 f a step.
  s     2 (D + 8) f scale |x|.|w| =: es
  lse   sum_v p es + (V + 8) f + 2^-21 + 4 f |lse| =: el  (ex2: 2^-22)
  d     |g| scale (p (es + el + 2^-21) + 8 f (p + [target])) + u |d| =: ed, fp16: and
        its smallest step where the largest |g| stands at 2^14 or more; and 2^-126 (|g| scale + 3):
        ex2 gives 0 below 2^-126, and so may each of the (up to three) bf16 parts of d
  grad_x    sum_v ed |w| + 2 (V + 8) f sum_v |d| |w| + u |grad_x|, grad_table alike
"""

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
F = 2.0 ** -24


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def norm(t, eps, weight=None, bias=None, g=None, up=None, dtype=torch.float32):
    """Rows t (the kept stream) in 64 bits; dicts of values and bounds; `g` (and `up`) add the gradients."""
    u, tiny = UNIT[dtype], TINY[dtype]
    rows, d = t.shape
    n = min(d, 80)
    w = np.ones(d) if weight is None else weight
    b = np.zeros(d) if bias is None else bias
    mean = t.mean(1, keepdims=True)
    c = t - mean
    var = (c * c).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    em = (n + 2) * F * np.abs(t).mean(1, keepdims=True)
    ev = (n + 6) * F * var + 2 * em ** 2 + 4 * F * em * np.abs(c).mean(1, keepdims=True)
    er = ev / (2 * (var + eps)) + 6 * F
    hat = c * rstd
    eh = em * rstd + np.abs(hat) * (er + 4 * F)
    out = hat * w + b
    res = {"out": out, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    bound = {"out": u * np.abs(out) + np.abs(w) * eh + 4 * F * (np.abs(hat * w) + np.abs(b)) + tiny,
             "mean": em[:, 0], "rstd": (er * rstd)[:, 0]}
    if g is None:
        return res, bound
    a = g * w
    s1, s2 = a.mean(1, keepdims=True), (a * hat).mean(1, keepdims=True)
    e1 = (n + 3) * F * np.abs(a).mean(1, keepdims=True)
    e2 = (n + 4) * F * np.abs(a * hat).mean(1, keepdims=True) + (np.abs(a) * eh).mean(1, keepdims=True)
    inner = a - s1 - hat * s2
    e = e1 + np.abs(hat) * e2 + eh * np.abs(s2) + 4 * F * (np.abs(a) + np.abs(s1) + np.abs(hat * s2))
    gx = rstd * inner + (0.0 if up is None else up)
    res["grad_x"] = gx
    bound["grad_x"] = rstd * e + rstd * np.abs(inner) * (er + F) + (u + F) * np.abs(gx) + tiny
    res["grad_weight"], res["grad_bias"] = (g * hat).sum(0), g.sum(0)
    bound["grad_weight"] = (rows + 4) * F * np.abs(g * hat).sum(0) + (np.abs(g) * eh).sum(0) \
        + u * np.abs(res["grad_weight"]) + tiny
    bound["grad_bias"] = (rows + 2) * F * np.abs(g).sum(0) + u * np.abs(res["grad_bias"]) + tiny
    return res, bound


def loss(x, w, targets, scale, g=None, dtype=torch.float32):
    """Rows and table in 64 bits; rows whose target is not in [0, V) are left out."""
    u, tiny = UNIT[dtype], TINY[dtype]
    (n, d), v = x.shape, w.shape[0]
    keep = (targets >= 0) & (targets < v)
    s = scale * x @ w.T
    es = 2 * (d + 8) * F * scale * np.abs(x) @ np.abs(w).T
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    p /= total
    lse = (top + np.log(total))[:, 0]
    el = (p * es).sum(1) + (v + 8) * F + 2.0 ** -21 + 4 * F * np.abs(lse)
    at = np.where(keep, targets, 0)
    row = np.arange(n)
    res = {"lse": lse, "loss": np.where(keep, lse - s[row, at], 0.0)}
    bound = {"lse": el, "loss": np.where(keep, el + es[row, at] + 4 * F * np.abs(s[row, at]), 0.0)}
    if g is None:
        return res, bound
    g = np.where(keep, g, 0.0)
    x = np.where(keep[:, None], x, 0.0)
    hot = np.zeros_like(p)
    hot[row[keep], targets[keep]] = 1.0
    p, es = np.where(keep[:, None], p, 0.0), np.where(keep[:, None], es, 0.0)
    el = np.where(keep, el, 0.0)
    size = (np.abs(g) * scale)[:, None]
    dd = (g * scale)[:, None] * (p - hot)
    ed = size * (p * (es + el[:, None] + 2.0 ** -21) + 8 * F * (p + hot)) + max(u, 4 * F) * np.abs(dd)
    ed = ed + 2.0 ** -126 * (size + 3.0) * keep[:, None]
    if dtype == torch.float16:  # a step of 2^-24 beside a largest value of 2^14 or more
        ed = ed + np.abs(g).max(initial=0.0) * scale * 2.0 ** -38 * keep[:, None]
    ax, aw = np.abs(x), np.abs(w)
    res |= {"grad_x": dd @ w, "grad_table": dd.T @ x}
    bound["grad_x"] = ed @ aw + 2 * (v + 8) * F * np.abs(dd) @ aw + u * np.abs(res["grad_x"]) + tiny
    bound["grad_table"] = ed.T @ ax + 2 * (n + 8) * F * np.abs(dd).T @ ax + u * np.abs(res["grad_table"]) + tiny
    return res, bound


def close(got, want, bound, what):
    dtype, got = got.dtype, f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    top = 65520.0 if dtype == torch.float16 else np.inf  # from here on a value rounds to an infinity of its sign
    with np.errstate(invalid="ignore"):
        over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= top)
        bad = ~((got == want) | (np.abs(got - want) <= bound) | over)
    if bad.any():
        k = [tuple(i) for i in np.argwhere(bad)[:4]]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at {k}: got {[got[i] for i in k]} want "
                             f"{[want[i] for i in k]} bound {[np.broadcast_to(bound, want.shape)[i] for i in k]}")
