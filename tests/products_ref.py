"""The products' operators in 64 bits, written from their definitions, with the
error that their arithmetic may add to each value.

The bounds. Rounding to bfloat16 is off by at most 2^-8 of the value. A product
of 16-bit values is exact in binary32; the tensor cores add 16 of them at a time
to a sum, aligned to the largest and cut, so a step is off by at most a few
units (taken as 2^-21) of the sum of the magnitudes, and a sum over k by
(k / 16 + 1) of those: ``chain``. Exponentials, error functions and quotients
are off by less than 2^-20 of their values."""
import numpy as np
import torch

U16, FN = 2.0 ** -8, 2.0 ** -20
TINY = 2.0 ** -126


def chain(k):
    return (k / 16 + 1) * 2.0 ** -21


def d(t):
    return t.detach().double().cpu()


def act(name, z):
    """(value, derivative)"""
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    return torch.where(z <= 0, 0.0, z), torch.where(z <= 0, 0.0, torch.ones_like(z))


def gated_ffn(x, w_gate, w_up, w_down, name):
    """{name: (values, error)}. No activation here is steeper than 1.13."""
    x, wg, wu, wd = d(x), d(w_gate), d(w_up), d(w_down)
    k, f = x.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    g_err, u_err = chain(k) * (x.abs() @ wg.abs().T), chain(k) * (x.abs() @ wu.abs().T)
    a, _ = act(name, g)
    a_err = 1.13 * g_err + 4 * FN * (a.abs() + g.abs())
    h = a * u
    h_err = a_err * (u.abs() + u_err) + a.abs() * u_err + U16 * (h.abs() + a_err * u.abs())
    y = h @ wd.T
    y_err = h_err @ wd.abs().T + chain(f) * (h.abs() @ wd.abs().T)
    return {"out": (y, y_err + U16 * (y.abs() + y_err) + TINY), "gate": (g, g_err + U16 * (g.abs() + g_err) + TINY),
            "up": (u, u_err + U16 * (u.abs() + u_err) + TINY)}


def gated_ffn_grad(grad, x, w_gate, w_up, w_down, gate, up, name, param_dtype=torch.bfloat16, before=None):
    """{name: (values, error)}; before: what the weights' gradients are added to."""
    dy, x, wg, wu, wd, g, u = (d(t) for t in (grad, x, w_gate, w_up, w_down, gate, up))
    t, k, f = x.shape[0], x.shape[1], wg.shape[0]
    h_grad = dy @ wd
    e = chain(k) * (dy.abs() @ wd.abs())
    a, slope = act(name, g)
    fn = 4 * FN * (1 + g.abs())  # of the value and the slope
    h, dg, du = a * u, h_grad * u * slope, h_grad * a
    h_err = fn * u.abs() + U16 * h.abs()
    dg_err = (e * slope.abs() + fn * (h_grad.abs() + e)) * u.abs()
    dg_err = dg_err + U16 * (dg.abs() + dg_err)
    du_err = e * (a.abs() + fn) + fn * h_grad.abs()
    du_err = du_err + U16 * (du.abs() + du_err)
    out = {"x": (dg @ wg + du @ wu, dg_err @ wg.abs() + du_err @ wu.abs() + chain(2 * f) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())),
           "w_gate": (dg.T @ x, dg_err.T @ x.abs() + chain(t) * (dg.abs().T @ x.abs())),
           "w_up": (du.T @ x, du_err.T @ x.abs() + chain(t) * (du.abs().T @ x.abs())),
           "w_down": (dy.T @ h, dy.abs().T @ h_err + chain(t) * (dy.abs().T @ h.abs()))}
    for key, (v, err) in out.items():
        if before is not None and key in before:
            v = v + d(before[key])
            err = err + 2.0 ** -24 * (v.abs() + d(before[key]).abs())
        u_out = U16 if key == "x" or param_dtype == torch.bfloat16 else 2.0 ** -24
        out[key] = (v, err + u_out * (v.abs() + err) + TINY)
    return out


def orthogonalize(x, steps=5, coefficients=(3.4445, -4.7750, 2.0315), scale=1.0, eps=1e-7):
    a, b, c = coefficients
    x = d(x)
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            g = x @ x.T
            x = a * x + (b * g + c * g @ g) @ x
        else:
            g = x.T @ x
            x = a * x + x @ (b * g + c * g @ g)
    return scale * x


def agree(name, got, want):
    v, err = want
    g = d(got)
    assert g.shape == v.shape, (name, g.shape, v.shape)
    bad = ~((g - v).abs() <= err)
    if bool(bad.any()):
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {v.numel()} outside; first at {at}: got {g[at]:.6g}, want {v[at]:.6g}, "
                             f"may be off by {err[at]:.3g}")


def distance(got, want):
    """In the 2-norm, relative."""
    n = float(want.norm())
    return float((d(got) - want).norm()) / n if n else float(d(got).norm())
