"""Attention over ragged histories in 64 bits, from the definitions, one
history and head at a time, with error bounds of the operators' results.

Bounds.  Let u be the unit roundoff of the tensors' type (2^-8 bf16, 2^-11
fp16, 2^-24 fp32) and f = 2^-24.  A logit is an fp32 sum of D products plus
the bias, scaled to base 2 and shifted by the row's maximum: its error is at
most (D + 8) f (scale |q|.|k| + |bias| + |lse|) =: x, and ex2 adds 2^-22, so a
weight p has relative error e = 2 x + 2^-21 (the row's sum doubles it).  The
16-bit kernels round p to the type before the product with v: u more.

  out:    u |out| + (u + e) sum_j p_ij |v_j|
  delta:  g . out with the rounded out: g |out's error| + D f |g| |out| =: t
  ds:     u |ds| + (e + (D + 8) f) p (|dp| + |delta|) + p t  =: E_ij
          (|dp| by the magnitudes' sum |g|.|v|)
  grad_v: u |grad_v| + sum_i (u + e) p_ij |g_i|
  grad_q: u |grad_q| + scale sum_j E_ij |k_j|, grad_k alike, grad_bias: sum E

Sums of n fp32 terms add n f of their magnitudes' sum; fp16's smallest step
(2^-24) bounds what its subnormals lose, per rounding.
"""

import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F = 2.0 ** -24


def visible(i, j, window, sinks):
    d = i[:, None] - j[None, :]
    v = d >= 0
    if window:
        v &= (d < window) | (j[None, :] < sinks)
    return v, d


def bucket_of(starts, d):
    return np.searchsorted(np.asarray(starts), np.maximum(d, 0), side="right") - 1


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def attention(q, k, v, offsets, window, sinks, scale, starts=None, bias=None, grad=None, dtype=None):
    """Arrays in 64 bits in, dict of (value, bound) out; `grad` adds the gradients."""
    u = UNIT[dtype] if dtype is not None else 0.0
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    n, h, d = q.shape
    group = h // k.shape[1]
    res = {"out": np.zeros_like(q), "lse": np.full((h, n), -np.inf)}
    bound = {"out": np.zeros_like(q), "lse": np.zeros((h, n))}
    if grad is not None:
        res |= {"grad_q": np.zeros_like(q), "grad_k": np.zeros_like(k), "grad_v": np.zeros_like(v)}
        bound |= {x: np.zeros_like(res[x]) for x in ("grad_q", "grad_k", "grad_v")}
        if bias is not None:
            res["grad_bias"], bound["grad_bias"] = np.zeros_like(bias), np.zeros_like(bias)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        length = hi - lo
        if length == 0:
            continue
        at = np.arange(length)
        seen, dist = visible(at, at, window, sinks)
        which = bucket_of(starts, dist) if bias is not None else None
        for a in range(h):
            c = a // group
            qa, ka, va = q[lo:hi, a], k[lo:hi, c], v[lo:hi, c]
            s = scale * qa @ ka.T
            size = abs(scale) * np.abs(qa) @ np.abs(ka).T
            if bias is not None:
                s = s + bias[which, a]
                finite_bias = np.where(np.isfinite(bias[which, a]), bias[which, a], 0.0)
                size = size + np.abs(finite_bias)
            s = np.where(seen, s, -np.inf)
            top = s.max(-1)
            safe = np.where(np.isfinite(top), top, 0.0)
            w = np.exp(s - safe[:, None])
            total = w.sum(-1)
            with np.errstate(divide="ignore"):
                lse = safe + np.log(total)
            p = w / np.where(total == 0, 1.0, total)[:, None]
            out = p @ va
            fine = np.where(np.isfinite(lse), lse, 0.0)
            e = 2 * (d + 8) * F * (size + np.abs(fine)[:, None]) + 2.0 ** -21 + length * F
            res["out"][lo:hi, a] = out
            bound["out"][lo:hi, a] = u * np.abs(out) + ((u + e) * p) @ np.abs(va) + tiny * (1 + np.abs(va).sum(0))
            res["lse"][a, lo:hi] = lse / math.log(2.0)
            bound["lse"][a, lo:hi] = 2 * (e * p).sum(-1) + 4 * F * np.abs(fine) + 2.0 ** -20
            if grad is None:
                continue
            ga = grad[lo:hi, a]
            dp = ga @ va.T
            dpsize = np.abs(ga) @ np.abs(va).T
            delta = (ga * out).sum(-1)
            t = (np.abs(ga) * bound["out"][lo:hi, a]).sum(-1) + d * F * (np.abs(ga) * np.abs(out)).sum(-1)
            ds = p * (dp - delta[:, None])
            err = u * np.abs(ds) + (e + (d + 8 + length) * F) * p * (dpsize + np.abs(delta)[:, None]) \
                + p * t[:, None] + tiny * seen
            res["grad_v"][lo:hi, c] += p.T @ ga
            bound["grad_v"][lo:hi, c] += ((u + e) * p + tiny * seen).T @ np.abs(ga)
            res["grad_q"][lo:hi, a] = scale * ds @ ka
            bound["grad_q"][lo:hi, a] = abs(scale) * err @ np.abs(ka)
            res["grad_k"][lo:hi, c] += scale * ds.T @ qa
            bound["grad_k"][lo:hi, c] += abs(scale) * err.T @ np.abs(qa)
            if bias is not None:
                np.add.at(res["grad_bias"][:, a], which[seen], ds[seen])
                np.add.at(bound["grad_bias"][:, a], which[seen], err[seen])
    if grad is not None:
        for x in ("grad_q", "grad_k", "grad_v", "grad_bias"):
            if x in res:
                bound[x] = bound[x] + u * np.abs(res[x]) + tiny
    return res, bound


def decode(q, keys, values, window, sinks, scale, starts=None, bias=None, dtype=None):
    """One new token per history over its cache (lists of [len, Hk, D])."""
    out = np.zeros_like(q)
    bound = np.zeros_like(q)
    for b in range(q.shape[0]):
        n = keys[b].shape[0]
        if n == 0:
            continue
        full = np.zeros((n,) + q.shape[1:])
        full[-1] = q[b]
        r, e = attention(full, keys[b], values[b], [0, n], window, sinks, scale, starts, bias, dtype=dtype)
        out[b], bound[b] = r["out"][-1], e["out"][-1]
    return out, bound


def close(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = got == ref  # infinities too
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - ref) <= bound))
    if bad.any():
        k = np.argwhere(bad)[:4]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at {k.tolist()}: got "
                             f"{[got[tuple(i)] for i in k]} ref {[ref[tuple(i)] for i in k]} "
                             f"bound {[np.broadcast_to(bound, ref.shape)[tuple(i)] for i in k]}")
