"""The training operators in 64 bits, written from their definitions on the
CPU (numpy), with the error that binary32 arithmetic and one rounding to the
output's type may add to each value.

The bounds. u32 = 2^-24 is half an ulp of binary32 relative to its value, and
an output of bfloat16, whose 8 significant bits leave half an ulp of 2^-8, is
rounded once more by at most that of its value. A
sum of k binary32 terms, however it is split, is off by at most about
(longest chain of additions) * u32 * (sum of the terms' magnitudes); the
chains are those of a row or token sum cut into parts, for which each bound
states the length it takes.
"""
import numpy as np
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126  # the smallest normal number: what rounding near zero may add


def f64(t):
    return t.detach().double().cpu().numpy()


def rounding(dtype):
    return U16 if dtype == torch.bfloat16 else U32


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on arrays of 32-bit words held in uint64."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, np.uint64) for x in (c0, c1, c2, c3)]
    k0, k1 = np.uint64(k0), np.uint64(k1)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k0, b & m, (a >> np.uint64(32)) ^ c[3] ^ k1, a & m]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & m, (k1 + np.uint64(0xBB67AE85)) & m
    return c


def limit(p):
    return int(np.rint((1.0 - p) * 65536))


def mask(rows, cols, p, seed, draw, first_row=0):
    """(rows, cols): 0 where an element is dropped, else what it is multiplied by."""
    blocks = -(-cols // 8)
    r = np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None]
    words = philox(np.arange(blocks, dtype=np.uint64)[None, :] + 0 * r, (r & np.uint64(0xFFFFFFFF)) + np.zeros((1, blocks), np.uint64),
                   (r >> np.uint64(32)) + np.zeros((1, blocks), np.uint64), np.full((rows, blocks), draw, np.uint64),
                   seed & 0xFFFFFFFF, seed >> 32)
    halves = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=-1)
    k = limit(p)
    return np.where(halves.reshape(rows, blocks * 8)[:, :cols] < k, 65536.0 / max(k, 1), 0.0)


def times(x, m):
    """x * m, 0 where m is 0 whatever x is there."""
    return np.where(m == 0, 0.0, np.where(m == 0, 0.0, x) * m)


def embedding(table, ids, scale, first_row, out_dtype):
    """(values, error): one binary32 product by a scale rounded to binary32."""
    t, v = f64(table), np.zeros((ids.numel(), table.shape[1]))
    for i, k in enumerate(ids.reshape(-1).tolist()):
        if first_row <= k < first_row + t.shape[0]:
            v[i] = scale * t[k - first_row]
    return v, np.abs(v) * (2 * U32 + rounding(out_dtype)) + TINY


def embedding_grad(grad, ids, vocab, scale, first_row, out_dtype, before=None):
    """(values, error). A row of k tokens: chains of at most k additions, then
    the scale (rounded itself), what was there, and the rounding."""
    g = f64(grad)
    v, mag, k = (np.zeros((vocab, g.shape[1])) for _ in range(3))
    for i, t in enumerate(ids.reshape(-1).tolist()):
        if first_row <= t < first_row + vocab:
            v[t - first_row] += g[i]
            mag[t - first_row] += np.abs(g[i])
            k[t - first_row] += 1
    v, err = v * scale, (k + 3) * U32 * mag * abs(scale)
    if before is not None:
        b = f64(before)
        v, err = v + b, err + U32 * (np.abs(v) + np.abs(b))
    return v, err + np.abs(v) * rounding(out_dtype) + TINY


def dropout(x, residual, p, seed, draw, first_row=0):
    """(values, error): a product by a rounded scale and one addition."""
    h = times(f64(x), mask(x.shape[0], x.shape[1], p, seed, draw, first_row) if p > 0 else np.ones(x.shape))
    mag = np.abs(h)
    if residual is not None:
        h = h + f64(residual)
        mag = mag + np.abs(f64(residual))
    return h, 4 * U32 * mag + np.abs(h) * rounding(x.dtype) + TINY, 4 * U32 * mag


def layer_norm(x, weight, bias, eps, residual=None, p=0.0, seed=0, draw=0):
    """{name: (values, error)}. Chains of a row's sums: 32 values a thread, the
    warp's and the group's sums, or, for rows too wide for registers, one
    addition a granule on top; CHAIN covers both for the tests' widths. With
    d = h - mean, the error of the mean is M = CHAIN * u32 * mean|h| plus that
    of h; d is off by M and a rounding; the variance, a sum of squares, by
    twice CHAIN roundings relative and by M^2; rstd by half that relative."""
    h, herr, h32 = dropout(x, residual, p, seed, draw)
    n = max(h.shape[1], 1)
    chain = 96 + n // 4096
    mean = h.sum(1, keepdims=True) / n
    d = h - mean
    var = (d * d).sum(1, keepdims=True) / n
    rstd = 1 / np.sqrt(var + eps)
    m_err = chain * U32 * np.abs(h).sum(1, keepdims=True) / n + h32.sum(1, keepdims=True) / n + U32 * np.abs(mean)
    d_err = m_err + h32 + U32 * np.abs(d)
    # var: relative rounding of its sum, and 2 |d| d_err of its terms
    v_err = 2 * chain * U32 * var + (2 * np.abs(d) * d_err + d_err ** 2).sum(1, keepdims=True) / n
    r_rel = 0.5 * v_err / (var + eps) + 4 * U32
    w = np.ones(n) if weight is None else f64(weight)
    b = np.zeros(n) if bias is None else f64(bias)
    y = d * rstd * w + b
    y_err = np.abs(w) * rstd * (d_err * (1 + r_rel) + np.abs(d) * (r_rel + 3 * U32)) + U32 * np.abs(y)
    return {"out": (y, y_err + np.abs(y) * rounding(x.dtype) + TINY), "hidden": (h, herr),
            "mean": (mean[:, 0], m_err[:, 0] + TINY), "rstd": (rstd[:, 0], (rstd * r_rel)[:, 0] + TINY)}


def layer_norm_grad(grad_out, hidden, mean, rstd, weight, param_dtype, grad_hidden=None, p=0.0, seed=0, draw=0,
                    weight_before=None, bias_before=None):
    """{name: (values, error)}. Row sums with CHAIN as in layer_norm; the sums
    over rows go through at most ROWS additions: a group's rows, of which no
    group has more than a 300th share (or 256 rows), and the groups' parts."""
    g, h = f64(grad_out), f64(hidden)
    rows, n = g.shape[0], max(g.shape[1], 1)
    chain, row_chain = 96 + n // 4096, 320 + rows // 64
    m, r = f64(mean)[:, None], f64(rstd)[:, None]
    w = np.ones(g.shape[1]) if weight is None else f64(weight)
    d = h - m
    u, gw = d * r, g * w
    u_err, gw_err = 2 * U32 * np.abs(u), U32 * np.abs(gw)
    c1, c2 = gw.sum(1, keepdims=True) / n, (gw * u).sum(1, keepdims=True) / n
    c1_err = (chain + 3) * U32 * np.abs(gw).sum(1, keepdims=True) / n
    c2_err = (chain + 6) * U32 * np.abs(gw * u).sum(1, keepdims=True) / n
    t = r * (gw - c1 - u * c2)
    mag = np.abs(gw) + np.abs(c1) + np.abs(u * c2)
    t_err = r * (gw_err + c1_err + u_err * np.abs(c2) + np.abs(u) * c2_err + 4 * U32 * mag)
    if grad_hidden is not None:
        t = t + f64(grad_hidden)
        t_err = t_err + U32 * np.abs(t) + U32 * np.abs(f64(grad_hidden))
    k = mask(rows, g.shape[1], p, seed, draw) if p > 0 else np.ones(g.shape)
    ro = rounding(grad_out.dtype)
    out = {"grad_residual": (t, t_err + np.abs(t) * ro + TINY),
           "grad_x": (times(t, k), k * (t_err + 3 * U32 * np.abs(t)) + np.abs(t * k) * ro + TINY)}
    for name, terms, before in (("grad_weight", g * u, weight_before), ("grad_bias", g, bias_before)):
        v = terms.sum(0)
        err = (row_chain + 4) * U32 * np.abs(terms).sum(0)
        if before is not None:
            v = v + f64(before)
            err = err + U32 * (np.abs(v) + np.abs(f64(before)))
        out[name] = (v, err + np.abs(v) * rounding(param_dtype) + TINY)
    return out


def agree(name, got, want):
    """Every value inside its error; infinities and NaN where the definition has them."""
    v, err = want
    g = f64(got).reshape(v.shape)
    fine = np.isfinite(v)
    same = np.where(fine, True, (np.isnan(v) & np.isnan(g)) | (g == v))
    assert same.all(), f"{name}: infinities or NaN differ at {np.argwhere(~same)[:3].tolist()}"
    off = np.where(fine, np.abs(np.where(fine, g - np.where(fine, v, 0), 0)), 0)
    bad = ~(off <= np.where(fine, err, 0)) & fine
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {v.size} outside; first at {at}: got {g[at]!r}, "
                             f"want {v[at]!r}, may be off by {err[at]:.3g}")
