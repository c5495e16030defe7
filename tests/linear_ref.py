"""The dense and grouped products and their gradients in fp64, and elementwise
bounds on how far a kernel may be off, derived from the formats:

  * rounding to type t costs at most eps(t)/2 of the value (plus half the
    smallest subnormal step);
  * the tensor cores add products to a fp32 sum that is cut, not rounded, so
    each of the terms can lose one step (2^-23) of the sum of absolute
    products, S = |a| |b|: K * 2^-23 * S covers any order.  With a fp32 output
    the cut sums span at most 640 terms and are then added with rounding:
    (min(K, 640) + K / 640) * 2^-23 * S;
  * activations and their derivatives are computed in fp32 with errors of a few
    steps of their terms: 2^-20 (1 + |z|) times what multiplies them.
"""
from __future__ import annotations

import math

import torch

CUT = 2.0 ** -23
FN = 2.0 ** -20


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def rounding(v: torch.Tensor, t: torch.dtype) -> torch.Tensor:
    f = torch.finfo(t)
    return half_step(t) * v.abs() + f.tiny * f.eps / 2


def terms(K: int, out: torch.dtype) -> float:
    return (min(K, 640) + K / 640 if out == torch.float32 else K) * CUT + 2 * CUT


def act(name: str, z, u=None):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "swiglu":
        return z * torch.sigmoid(z) * u
    return z


def slope(name: str, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return s + z * s * (1 - s)


def _groups(R, offsets):
    if offsets is None:
        return [(None, 0, R)]
    return [(e, offsets[e], offsets[e + 1]) for e in range(len(offsets) - 1)]


def _pick(t, e):
    return None if t is None else (t if e is None else t[e]).double()


def forward(x, w, w_up=None, bias=None, bias_up=None, name="none", offsets=None, x_rows=None, out=torch.bfloat16):
    """(y without residual, its bound before rounding, z, z_up, bound of z, bound of z_up) in grouped order;
    rows outside the groups are NaN."""
    xg = (x if x_rows is None else x[x_rows.long()]).double()
    R, N, K = xg.shape[0], w.shape[-2], w.shape[-1]
    n = terms(K, out)
    pre = []
    for wt, b in ((w, bias), (w_up, bias_up)):
        if wt is None:
            pre += [None, None]
            continue
        z = torch.full((R, N), math.nan, dtype=torch.float64, device=x.device)
        s = torch.full_like(z, math.nan)
        for e, lo, hi in _groups(R, offsets):
            we, be = _pick(wt, e), _pick(b, e)
            z[lo:hi] = xg[lo:hi] @ we.T + (0 if be is None else be)
            s[lo:hi] = xg[lo:hi].abs() @ we.abs().T + (0 if be is None else be.abs())
        pre += [z, s * n]
    z, dz, u, du = pre
    y = act(name, z, u)
    if name == "none":
        err = dz
    elif name == "swiglu":
        err = 1.2 * dz * u.abs() + (z.abs() + 1) * du + 1.2 * dz * du + FN * (1 + z.abs()) * (1 + u.abs())
    else:
        err = 1.2 * dz + FN * (1 + z.abs())
    return y, err, z, u, dz, du


def backward(dy, x, w, w_up=None, z=None, z_up=None, name="none", offsets=None, x_rows=None, y_rows=None,
             out=torch.bfloat16, t16=None):
    """dx (grouped order), [dw, dw_up], [db, db_up], each with its bound before the output's rounding."""
    t16 = t16 or w.dtype
    d = (dy if y_rows is None else dy[y_rows.long()]).double()
    xg = (x if x_rows is None else x[x_rows.long()]).double()
    R, N, K = xg.shape[0], w.shape[-2], w.shape[-1]
    exact = name == "none" and dy.dtype == t16
    if name == "none":
        parts = [(d, w, torch.zeros_like(d))]
    else:
        zd = z.double()
        fe = FN * (1 + zd.abs())
        if name == "swiglu":
            ud = z_up.double()
            parts = [(d * ud * slope(name, zd), w, (d * ud).abs() * fe),
                     (d * act("silu", zd), w_up, d.abs() * fe)]
        else:
            parts = [(d * slope(name, zd), w, d.abs() * fe)]
    dx = torch.full((R, K), math.nan, dtype=torch.float64, device=x.device)
    dxe = torch.full_like(dx, math.nan)
    dw, db = [], []
    for i, (g, wt, ge) in enumerate(parts):
        off = ge if exact else ge + rounding(g, t16)      # of one dz element, as the products take it
        W = torch.zeros(wt.shape, dtype=torch.float64, device=x.device)
        We, B, Be = torch.zeros_like(W), torch.zeros(wt.shape[:-1], dtype=torch.float64, device=x.device), None
        Be = torch.zeros_like(B)
        for e, lo, hi in _groups(R, offsets):
            we, xe, gg, oo = _pick(wt, e), xg[lo:hi], g[lo:hi], off[lo:hi]
            p = gg @ we
            pe = terms(2 * N, out) * ((gg.abs() + oo) @ we.abs()) + oo @ we.abs()
            if i == 0:
                dx[lo:hi], dxe[lo:hi] = p, pe
            else:
                dx[lo:hi] += p
                dxe[lo:hi] += pe
            at = slice(None) if e is None else e
            W[at] = gg.T @ xe
            We[at] = terms(hi - lo, out) * ((gg.abs() + oo).T @ xe.abs()) + oo.T @ xe.abs()
            B[at] = gg.sum(0)
            Be[at] = (hi - lo + 2) * CUT * gg.abs().sum(0) + ge[lo:hi].sum(0)
        dw.append((W, We))
        db.append((B, Be))
    return (dx, dxe), dw, db


def close(got, want, bound, what=""):
    """Every value within its bound plus the rounding to got's own type."""
    tol = bound + rounding(want.abs() + bound, got.dtype)
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off - tol)[bad].max()):.3e} over its bound"
