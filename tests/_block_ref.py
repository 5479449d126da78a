"""Plain 64-bit forms of the block operators, with error bounds for fp32
evaluation, shared by the CPU and GPU tests.

Bounds.  u = 2^-24.  A sum over a row of H runs at most D = H / 64 + 16 deep
(64 lanes at least share a row, then a tree), so its relative error against
the sum of the terms' magnitudes is at most D u.  Every other operation adds
u.  Magnitudes are carried with absolute values, so cancellation (in r', or
in the projections of the gradients) is inside the bound.
"""
import numpy as np
import torch

U = 2.0 ** -24
TINY = np.float32(2.0 ** -100)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def quantize_tokens(x):
    """Codes and scales in the operator's own fp32 operations (each one IEEE)."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(axis=1)
    a = np.maximum(np.abs(np.where(bad[:, None], 0, x)).max(axis=1, initial=0).astype(np.float32), TINY)
    s = a / np.float32(127)
    inv = np.float32(127) / a
    q = np.rint(np.where(bad[:, None], np.float32(0), x) * inv[:, None]).astype(np.int8)
    s[bad] = np.nan
    return q, s


def gemm_int8(xq, sx, wq, sw, bias):
    """The exact sum (integers below 2^31 are exact in float64), then the
    operator's fp32 steps, one rounding each."""
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T
    y = acc.astype(np.float32) * sx[:, None].astype(np.float32)
    y = y * sw[None, :].astype(np.float32)
    return y if bias is None else y + bias[None, :].astype(np.float32)


def gate_rows(T, gate_tokens):
    return np.arange(T) // gate_tokens


def norm_forward(x, r, w_post, w_pre, gate, gate_tokens, post, rho, beta, eps):
    """r', h in float64 and the pieces the bounds and gradients use."""
    T, H = x.shape
    one = np.ones(H)
    wp = one if w_post is None else w_post
    wq = one if w_pre is None else w_pre
    g = np.ones((T, H)) if gate is None else gate[gate_rows(T, gate_tokens)]
    kx = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    z = x * kx * wp if post else x
    rr = np.zeros((T, H)) if r is None else r
    rn = rho * rr + beta * g * z
    kr = 1 / np.sqrt((rn * rn).mean(1, keepdims=True) + eps)
    h = rn * kr * wq
    mag = np.abs(rho * rr) + np.abs(beta * g * z)
    return dict(rn=rn, h=h, kx=kx, kr=kr, z=z, g=g, wp=wp, wq=wq, mag=mag, n_x=x * kx, n_r=rn * kr)


def norm_bounds(f):
    """Elementwise error bounds of r' and h before they are rounded to the output's type."""
    H = f["rn"].shape[1]
    D = H / 64 + 16
    er = f["mag"] * (D / 2 + 8) * U
    norm = np.sqrt((f["rn"] ** 2).sum(1, keepdims=True)) + 1e-300
    rel = np.sqrt((er ** 2).sum(1, keepdims=True)) / norm + (D / 2 + 8) * U
    eh = np.abs(f["kr"] * f["wq"]) * er + np.abs(f["h"]) * rel
    # 1.01: second-order terms; 2^-140: results below the normal range
    return 1.01 * er + 2.0 ** -140, 1.01 * eh + 2.0 ** -140


def outside(got, want, tol):
    """Where a tensor is not the rounding, to its type, of any value within
    tol of want: rounding keeps order, so it has to lie between the roundings
    of both ends."""
    to = lambda v: torch.from_numpy(v.astype(np.float64)).to(got.dtype).double().numpy()  # noqa: E731
    g = f64(got)
    return ~((to(want - tol) <= g) & (g <= to(want + tol)))


def norm_backward(f, x, dh, dr_out, gate, gate_tokens, post, rho, beta):
    """Gradients by the formulas in float64, and the magnitudes their bounds scale with."""
    T, H = x.shape
    dh = np.zeros((T, H)) if dh is None else dh
    up = np.zeros((T, H)) if dr_out is None else dr_out
    n, kr, kx, nx = f["n_r"], f["kr"], f["kx"], f["n_x"]
    N = kr * f["mag"]
    dn = dh * f["wq"]
    d = up + kr * (dn - n * (dn * n).mean(1, keepdims=True))
    A = np.abs(up) + kr * (np.abs(dn) + N * (np.abs(dn) * N).mean(1, keepdims=True))
    got, mag = {}, {}
    got["dr"], mag["dr"] = rho * d, np.abs(rho) * A
    got["dw_pre"], mag["dw_pre"] = (dh * n).sum(0), (np.abs(dh) * N).sum(0)
    if gate is not None:
        G = -(-T // gate_tokens)
        dg, mg = np.zeros((G, H)), np.zeros((G, H))
        idx = gate_rows(T, gate_tokens)
        np.add.at(dg, idx, beta * d * f["z"])
        np.add.at(mg, idx, np.abs(beta * f["z"]) * A)
        got["dgate"], mag["dgate"] = dg, mg
    dz, Az = beta * f["g"] * d, np.abs(beta * f["g"]) * A
    if post:
        got["dw_post"], mag["dw_post"] = (dz * nx).sum(0), (Az * np.abs(nx)).sum(0)
        dn, An = dz * f["wp"], Az * np.abs(f["wp"])
        got["dx"] = kx * (dn - nx * (dn * nx).mean(1, keepdims=True))
        mag["dx"] = kx * (An + np.abs(nx) * (An * np.abs(nx)).mean(1, keepdims=True))
    else:
        got["dx"], mag["dx"] = dz, Az
    return got, mag


def backward_eps(f, H, T=0):
    """Relative error of a gradient against its magnitude: each of the four
    row sums (x^2, r'^2, two projections) runs D deep and enters at most
    twice, r' enters three times with the cancellation factor kappa of its
    row, and a sum over T tokens adds T roundings at most."""
    D = H / 64 + 16
    kappa = np.sqrt((f["mag"] ** 2).sum(1) / ((f["rn"] ** 2).sum(1) + 1e-300)).max(initial=1.0)
    return (8 * D + 3 * kappa * (D / 2 + 8) + 40 + T) * U
