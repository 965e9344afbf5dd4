"""Error bounds of the fp32 form of dl_decode_attn, from its arithmetic.

u = 2^-24, half an fp32 step; e = 2^-22, the relative error of ex2.approx.ftz.
For a row of n tokens with base-2 exponents a2_t = (x_t c - M), x_t the dot
product in fp64 and M the fp32 reference, nt = ceil(n / 32) tiles at most:
 - x_t: (d + 4) 2^-53 sum_i |q_i k_i|, times the scale;
 - a weight 2^a2: its argument is rounded once, ln 2 u |a2_t|, and e;
 - factors 2^(M' - M) of raised maxima (nt at most), the join of a warp's, a
   run's and a row's states: (nt + 4) e, and u ln 2 of the differences, which add
   up to the spread S of the exponents at most, in three places: 3 ln 2 u S;
 - sums, one rounding an addition: of weights 2 nt + 16 deep (a lane's tiles, five
   and four steps of lanes and warps, the runs), of weighted values n / 4 + nt + 24
   (a warp's keys, one at a time, then warps and runs).
So with g_t the sum of the first three, relative to weight w_t of the row:
  O:    sum_t w_t |v_t| (g_t + (n/4 + nt + 24) u) + |O| (D + 3 u),
        D = sum_t w_t g_t + (2 nt + 16) u   (normaliser; inverse, product, rounding)
  lse:  D + 4 u (|lse| + ln n)   (product, logarithm, sum and product)
  mass: sum_h w_t (g_t + D + 3 u) + (rows + 3) u of the result
Nothing depends on the logits' size beyond their spread: that is what the fp64
dot products are for."""
import numpy as np

U, E, LN2 = 2.0 ** -24, 2.0 ** -22, np.log(2.0)


def decode_bounds(q, K, V):
    """Rows q [R][d] over K, V [n][d] (fp64 arrays): (O, lse, w) exactly, and the
    bounds of O [R][d], of lse [R] and of each weight [R][n]."""
    n, d = K.shape
    s = q @ K.T / np.sqrt(d)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    total = w.sum(1, keepdims=True)
    w = w / total
    O, lse = w @ V, (top + np.log(total))[:, 0]
    nt = -(-n // 32)
    a2 = (top - s) / LN2
    g = (d + 4) * 2.0 ** -53 * (np.abs(q) @ np.abs(K).T) / np.sqrt(d) + LN2 * U * a2 + E
    g = g + (nt + 4) * E + 3 * LN2 * U * a2.max(1, keepdims=True)
    D = (w * g).sum(1) + (2 * nt + 16) * U
    tol_o = (w * (g + (n / 4 + nt + 24) * U)) @ np.abs(V) + np.abs(O) * (D + 3 * U)[:, None]
    tol_l = D + 4 * U * (np.abs(lse) + np.log(n))
    return (O, lse, w), (1.001 * tol_o, 1.001 * tol_l, 1.001 * w * (g + D[:, None] + 3 * U))


def far_rows(rng, G, n, d, level):
    """Queries and keys whose logits lie at `level` with a spread of a few."""
    base = rng.normal(size=d)
    q = base + 0.1 * rng.normal(size=(G, d))
    k = level * np.sqrt(d) / (base @ base) * base + rng.normal(size=(n, d))
    return (x.astype(np.float32) for x in (q, k, rng.normal(size=(n, d))))
