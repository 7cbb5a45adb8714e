"""The bounds that the softmax loss's results are held to on the GPU find the mistakes they are there for: these are
planted in the 64-bit reference."""

import numpy as np
import pytest
import torch

import rows_reference as ref

FP32, FP16 = torch.float32, torch.float16


def terms(a, count):
    """a as the sum of `count` bf16 numbers."""
    rest, total = torch.from_numpy(a), torch.zeros(a.shape, dtype=torch.float64)
    for _ in range(count):
        part = rest.to(torch.bfloat16).double()
        total, rest = total + part, rest - part
    return total.numpy()


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("n,v,d,bound", [(300, 4000, 96, 1.5e-6), (150, 3000, 264, 1.8e-6)])
def test_two_terms_of_an_fp32_number_are_too_few(n, v, d, bound):
    g = np.random.default_rng(1)
    x, w = g.standard_normal((n, d)).astype(np.float32).astype(np.float64), (g.standard_normal((v, d)) * 1.5 * d ** -0.5)
    w = w.astype(np.float32).astype(np.float64)
    targets, up = g.integers(0, v, n), np.ones(n)
    want, _ = ref.loss(x, w, targets, 1.0, up, FP32)
    for count, good in ((3, True), (2, False)):
        got, _ = ref.loss(terms(x, count), terms(w, count), targets, 1.0, up, FP32)
        # (d's own terms)
        s = terms(x, count) @ terms(w, count).T
        d_iv = terms(np.exp(s - got["lse"][:, None]) - (targets[:, None] == np.arange(v)), count)
        grads = d_iv @ terms(w, count), d_iv.T @ terms(x, count)
        assert all((off(a, want[k]) < bound) == good for a, k in zip(grads, ("grad_x", "grad_table"))), count


def test_a_shrunk_sum_and_a_wrong_row_are_found():
    g = np.random.default_rng(2)
    a = g.standard_normal((5000, 64))
    for bound in (3.0e-4 + 2 ** -13, 1.5e-6):
        assert off(a * (1 - 1e-3), a) > bound
    wrong = a.copy()
    wrong[77] = a[78]
    assert off(wrong, a) > 2.4e-3
    element = a.copy()
    element[5, 7] += 0.5 * np.abs(a).max()
    for dtype, roundings in ((FP32, 64), (FP16, 16), (torch.bfloat16, 16)):
        assert np.abs(element - a).max() > roundings * ref.UNIT[dtype] * np.abs(a).max()
