"""The bounds of tests/fp32_bounds.py are of a use: the kernel's arithmetic, done
in numpy, keeps to them, and the same with fp32 dot products, or with operands
rounded to TF32 or bf16, does not (CPU)."""
import numpy as np
import pytest

from tests.fp32_bounds import decode_bounds, far_rows

F = np.float32
SIZES = [(1, 64, 128), (4, 100, 64), (8, 257, 128)]


def _rows(G, n, d, level):
    rng = np.random.default_rng([n, d, int(level)])
    if level:
        return far_rows(rng, G, n, d, level)
    q, k, v = (rng.normal(size=s).astype(F) for s in ((G, d), (n, d), (n, d)))
    k[0] *= 3
    return q, k, v


def _attention(q, k, v, dots):
    """Weights, sums and output in fp32 from dot products in `dots`."""
    d = q.shape[1]
    c = 1.0 / np.sqrt(d) * np.log2(np.e)
    x = np.zeros((len(q), len(k)), dots)
    for i in range(d):
        x += np.outer(q[:, i].astype(dots), k[:, i].astype(dots)).astype(dots)
    M = (x.max(1, keepdims=True).astype(F) * F(c)).astype(F)
    p = np.exp2((x * dots(c) - M.astype(dots)).astype(F))
    L, O = np.zeros(len(q), F), np.zeros((len(q), d), F)
    for t in range(len(k)):
        L += p[:, t]
        O += p[:, t:t + 1] * v[t]
    return O / L[:, None], (M[:, 0] + np.log2(L)) * F(np.log(2.0)), p / L[:, None]


def _worst(got, q, k, v):
    ref, tol = decode_bounds(*(x.astype(np.float64) for x in (q, k, v)))
    return [float((np.abs(g.astype(np.float64) - r) / t).max()) for g, r, t in zip(got, ref, tol)]


def _rounded(x, bits):
    """fp32 values to `bits` of mantissa, to nearest even."""
    u = x.view(np.uint32).astype(np.uint64)
    drop = 23 - bits
    u = u + (1 << (drop - 1)) - 1 + ((u >> drop) & 1)
    return (u >> drop << drop).astype(np.uint32).view(F)


@pytest.mark.parametrize("level", [0, 35, 8000])
@pytest.mark.parametrize("G,n,d", SIZES)
def test_the_kernels_arithmetic_is_within_the_bounds(G, n, d, level):
    q, k, v = _rows(G, n, d, level)
    assert max(_worst(_attention(q, k, v, np.float64), q, k, v)) <= 1.0


@pytest.mark.parametrize("G,n,d", SIZES)
def test_fp32_dot_products_are_not(G, n, d):
    q, k, v = _rows(G, n, d, 8000)
    o, lse, w = _worst(_attention(q, k, v, F), q, k, v)
    assert o > 2 and w > 2


@pytest.mark.parametrize("bits", [7, 10])
@pytest.mark.parametrize("G,n,d", SIZES)
def test_rounded_operands_are_not(G, n, d, bits):
    q, k, v = _rows(G, n, d, 0)
    r = [_rounded(x, bits) for x in (q, k, v)]
    o, lse, w = _worst(_attention(*r, np.float64), q, k, v)
    assert min(o, lse, w) > 5
