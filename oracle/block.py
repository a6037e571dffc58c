"""Float64 oracle of the operators around the sequence layer: root-mean-square norm, short causal convolution and
selective state space scan, with their gradients, written token by token from the formulas.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module; the CUDA library never calls it.

Every function returns, beside each value, a bound on how far an evaluation in float32 may be from it: the rounding
of every step (u = 2^-24 relative), carried through the recursions with absolute values, and the documented or
measured error of the functions used (2^x of the special-function unit: 2^-22 relative; e^x by it: 2 + 1.2 |x|
units of 2^-23; fast division: 2 units; rsqrt: 2 units).  Sums may be taken in any order: their bound counts one
rounding a term.  A test adds half a step of the output's type to it and nothing else.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def wide(t):
    return None if t is None else t.detach().to("cpu", F64)


def _sigmoid_error(x):
    """Relative error of 1 / (1 + e^-x) in float32 by the fast functions."""
    return (2 + 1.2 * x.abs() + 2 + 1) * 2 * U


def _live(B, T, lengths):
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    return n, torch.arange(T)[None, :] < n[:, None]


# ---------------------------------------------------------------- norm
def rmsnorm(x, weight, residual=None, eps=1e-6):
    """y, h and their bounds."""
    x, w, res = wide(x), wide(weight), wide(residual)
    h = x if res is None else x + res
    d = h.shape[-1]
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w
    # h, h w, (h w) r: three roundings; the sum of squares one a term, halved by the root, and h's two; rsqrt two units
    return (y, (3 + (d + 3) / 2 + 4) * U * y.abs()), (h, U * h.abs())


def rmsnorm_backward(h, weight, dy, dh_in=None, eps=1e-6):
    h, w, dy, g = wide(h), wide(weight), wide(dy), wide(dh_in)
    d = h.shape[-1]
    r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    v = dy * w
    dh = r * (v - h * r ** 2 * (v * h).mean(-1, keepdim=True))
    size = r * (v.abs() + h.abs() * r ** 2 * (v * h).abs().mean(-1, keepdim=True))
    if g is not None:
        dh, size = dh + g, size + g.abs()
    rows = h.shape[0] * h.shape[1]
    r_err = ((d + 2) / 2 + 4) * U
    term = dy * h * r
    return ((dh, (3 * r_err + (d + 8) * U) * size),
            (term.sum((0, 1)), ((rows + 4) * U + r_err) * term.abs().sum((0, 1))))


# ---------------------------------------------------------------- convolution
def _window(x, state0, W):
    B, T, C = x.shape
    return torch.cat((torch.zeros(B, W - 1, C, dtype=F64) if state0 is None else state0, x), 1)


def _act(pre, pre_err, silu):
    """act(pre), its bound, act'(pre), its bound."""
    if not silu:
        return pre, pre_err, torch.ones_like(pre), torch.zeros_like(pre)
    s, e = torch.sigmoid(pre), _sigmoid_error(pre)
    y, slope = pre * s, s * (1 + pre * (1 - s))
    size = s * (1 + pre.abs() * (1 - s))
    # |act'| <= 1.1, |act''| <= 0.5; in act' the sigmoid enters as s and as 1 - s (off by s e)
    return y, 1.1 * pre_err + (e + U) * y.abs(), slope, 0.5 * pre_err + (e + 4 * U) * size + pre.abs() * s * s * e


def conv(x, weight, bias=None, state0=None, lengths=None, silu=True):
    """(y, bound), final state."""
    x, w, b, s0 = wide(x), wide(weight), wide(bias), wide(state0)
    B, T, C = x.shape
    W = w.shape[1]
    n, live = _live(B, T, lengths)
    win = torch.where(torch.cat((torch.ones(B, W - 1, dtype=torch.bool), live), 1)[..., None], _window(x, s0, W), 0.0)
    terms = torch.stack([win[:, j:j + T] * w[:, j] for j in range(W)])
    pre, size = terms.sum(0), terms.abs().sum(0)
    if b is not None:
        pre, size = pre + b, size + b.abs()
    y, err, _, _ = _act(pre, (W + 1) * U * size, silu)
    state = torch.stack([win[i, n[i]:n[i] + W - 1] for i in range(B)])
    return (torch.where(live[..., None], y, 0.0), err), state


def conv_backward(x, weight, bias, dy, state0=None, dstate_T=None, lengths=None, silu=True):
    """(value, bound) of dx, dweight, dbias, dstate0."""
    x, w, b, dy, s0, ds = (wide(t) for t in (x, weight, bias, dy, state0, dstate_T))
    B, T, C = x.shape
    W = w.shape[1]
    n, live = _live(B, T, lengths)
    win = torch.where(torch.cat((torch.ones(B, W - 1, dtype=torch.bool), live), 1)[..., None], _window(x, s0, W), 0.0)
    dy = torch.where(live[..., None], dy, 0.0)
    terms = torch.stack([win[:, j:j + T] * w[:, j] for j in range(W)])
    pre, size = terms.sum(0), terms.abs().sum(0)
    if b is not None:
        pre, size = pre + b, size + b.abs()
    _, _, slope, slope_err = _act(pre, (W + 1) * U * size, silu)
    dp, dp_err = dy * slope, dy.abs() * slope_err + U * (dy * slope).abs()
    dwin, dwin_err = torch.zeros_like(win), torch.zeros_like(win)
    for t in range(T):
        for j in range(W):
            dwin[:, t + j] += dp[:, t] * w[:, j]
            dwin_err[:, t + j] += (dp_err[:, t] + (W + 2) * U * dp[:, t].abs()) * w[:, j].abs()
    if ds is not None:
        for i in range(B):
            dwin[i, n[i]:n[i] + W - 1] += ds[i]
            dwin_err[i, n[i]:n[i] + W - 1] += 2 * U * ds[i].abs()
    dw = torch.stack([(dp * win[:, j:j + T]).sum((0, 1)) for j in range(W)], -1)
    many = (B * T + 2) * U
    dw_err = torch.stack([((dp_err + many * dp.abs()) * win[:, j:j + T].abs()).sum((0, 1)) for j in range(W)], -1)
    return ((dwin[:, W - 1:], dwin_err[:, W - 1:]), (dw, dw_err),
            (dp.sum((0, 1)), (dp_err + many * dp.abs()).sum((0, 1))), (dwin[:, :W - 1], dwin_err[:, :W - 1]))


# ---------------------------------------------------------------- selective scan
def _steps(u, dt, A, Bm, dt_bias, softplus, live):
    raw = dt if dt_bias is None else dt + dt_bias
    raw_err = U * raw.abs()
    if softplus:
        step = torch.nn.functional.softplus(raw, threshold=1000.0)
        slope = torch.sigmoid(raw)
        # e^-|raw| by the special-function unit, s = e / (2 + e), the polynomial, the last sum
        step_err = slope * raw_err + step * (2 + 1.2 * raw.abs() + 8) * 2 * U
        slope_err = slope * (_sigmoid_error(raw) + raw_err)
    else:
        step, slope, step_err, slope_err = raw, torch.ones_like(raw), raw_err, torch.zeros_like(raw)
    keep = live[..., None]
    step, step_err, u = (torch.where(keep, v, 0.0) for v in (step, step_err, u))
    x = (step[..., None] * A).abs() / math.log(2)
    a = torch.exp(step[..., None] * A)
    near = torch.where(x < 0.0625, 1.3e-7 * x + 2 * U, 2.0 ** -22 + 2 * U)
    a_err = a * (step_err[..., None] * A.abs() + 3 * U * x + near)
    du, du_err = step * u, (step_err + U * step.abs()) * u.abs()
    Bm = torch.where(keep, Bm, 0.0)
    b = du[..., None] * Bm[:, :, None, :]
    b_err = (du_err + U * du.abs())[..., None] * Bm.abs()[:, :, None, :]
    return raw, step, step_err, slope, slope_err, u, du, du_err, a, a_err, Bm, b, b_err


def _states(a, a_err, b, b_err, h0):
    B, T, C, N = a.shape
    h = torch.zeros(B, C, N, dtype=F64) if h0 is None else h0
    err = torch.zeros_like(h)
    hs, errs = [h], [err]
    for t in range(T):
        new = a[:, t] * h + b[:, t]
        # one rounding for the sum, and as much again for a state put together from two pieces of the sequence
        err = a[:, t] * err + a_err[:, t] * h.abs() + b_err[:, t] + 2 * U * ((a[:, t] * h).abs() + b[:, t].abs())
        h = new
        hs.append(h)
        errs.append(err)
    return torch.stack(hs, 1), torch.stack(errs, 1)


def ssm(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus=True):
    """(y, bound), (final state, bound)."""
    u, dt, A, Bm, Cm, D, z, dt_bias, h0 = (wide(t) for t in (u, dt, A, Bm, Cm, D, z, dt_bias, h0))
    B, T, C = u.shape
    N = A.shape[1]
    _, live = _live(B, T, lengths)
    raw, step, _, _, _, u, _, _, a, a_err, _, b, b_err = _steps(u, dt, A, Bm, dt_bias, softplus, live)
    h, h_err = _states(a, a_err, b, b_err, h0)
    Cm = torch.where(live[..., None], Cm, 0.0)[:, :, None, :]
    y, size = (h[:, 1:] * Cm).sum(-1), (h[:, 1:] * Cm).abs().sum(-1)
    err = (h_err[:, 1:] * Cm.abs()).sum(-1)
    if D is not None:
        y, size = y + D * u, size + (D * u).abs()
    err = err + (N + 2) * U * size
    if z is not None:
        gate = z * torch.sigmoid(z)
        err = err * gate.abs() + (_sigmoid_error(z) + 3 * U) * (y * gate).abs()
        y = y * gate
    return (torch.where(live[..., None], y, 0.0), torch.where(live[..., None], err, 0.0)), (h[:, -1], h_err[:, -1])


def ssm_backward(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, h0=None, dh_T=None, lengths=None, softplus=True):
    """(value, bound) of du, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0."""
    u, dt, A, Bm, Cm, dy, D, z, dt_bias, h0, dh_T = (
        wide(t) for t in (u, dt, A, Bm, Cm, dy, D, z, dt_bias, h0, dh_T))
    B, T, C = u.shape
    N = A.shape[1]
    _, live = _live(B, T, lengths)
    keep = live[..., None]
    raw, step, step_err, slope, slope_err, u, du, du_err, a, a_err, Bm, b, b_err = _steps(
        u, dt, A, Bm, dt_bias, softplus, live)
    h, h_err = _states(a, a_err, b, b_err, h0)
    Cm, dy = torch.where(keep, Cm, 0.0), torch.where(keep, dy, 0.0)
    D = torch.zeros(C, dtype=F64) if D is None else D
    hc = h[:, 1:] * Cm[:, :, None, :]
    y, y_size = hc.sum(-1) + D * u, hc.abs().sum(-1) + (D * u).abs()
    y_err = (h_err[:, 1:] * Cm.abs()[:, :, None, :]).sum(-1) + (N + 2) * U * y_size
    dyg, dyg_err, dz = dy, torch.zeros_like(dy), None
    if z is not None:
        z = torch.where(keep, z, 0.0)
        gate, gate_err, gs, gs_err = _act(z, torch.zeros_like(z), True)
        dyg, dyg_err = dy * gate, dy.abs() * gate_err + U * (dy * gate).abs()
        dz = (dy * gs * y, dy.abs() * (gs_err * y.abs() + gs.abs() * (y_err + 2 * U * y.abs())))
    g = torch.zeros(B, C, N, dtype=F64) if dh_T is None else dh_T
    g_err = torch.zeros_like(g)
    out = {k: torch.zeros_like(u) for k in ("du", "ddt")}
    err = {k: torch.zeros_like(u) for k in out}
    dA, dA_err = torch.zeros_like(A), torch.zeros_like(A)
    dB, dC, dB_err, dC_err = (torch.zeros_like(Bm) for _ in range(4))
    for t in reversed(range(T)):
        c, bt = Cm[:, t, None, :], Bm[:, t, None, :]
        dyt, dyt_err = dyg[:, t, :, None], dyg_err[:, t, :, None]
        dC[:, t] = (dyt * h[:, t + 1]).sum(1)
        dC_err[:, t] = (dyt_err * h[:, t + 1].abs() + dyt.abs() * h_err[:, t + 1]
                        + (C + 1) * U * (dyt * h[:, t + 1]).abs()).sum(1)
        part = c * dyt
        g_err = g_err + c.abs() * dyt_err + 2 * U * (part.abs() + g.abs())
        g = g + part
        d1, d1_err = du[:, t, :, None], du_err[:, t, :, None]
        dB[:, t] = (g * d1).sum(1)
        dB_err[:, t] = (g_err * d1.abs() + g.abs() * d1_err + (C + 1) * U * (g * d1).abs()).sum(1)
        gb, gb_size = (g * bt).sum(-1), (g * bt).abs().sum(-1)
        gb_err = (g_err * bt.abs()).sum(-1) + (N + 1) * U * gb_size
        ga, ga_err = g * a[:, t], g_err * a[:, t] + g.abs() * a_err[:, t] + U * (g * a[:, t]).abs()
        hp, hp_err = h[:, t], h_err[:, t]
        w, w_err = ga * hp, ga_err * hp.abs() + ga.abs() * hp_err + U * (ga * hp).abs()
        wA, wA_size = (w * A).sum(-1), (w * A).abs().sum(-1)
        wA_err = (w_err * A.abs()).sum(-1) + (N + 4) * U * wA_size
        out["du"][:, t] = step[:, t] * gb + D * dyg[:, t]
        err["du"][:, t] = (step_err[:, t] * gb.abs() + step[:, t].abs() * gb_err + D.abs() * dyg_err[:, t]
                           + 2 * U * ((step[:, t] * gb).abs() + (D * dyg[:, t]).abs()))
        d_raw = u[:, t] * gb + wA
        d_err = u[:, t].abs() * gb_err + wA_err + 2 * U * ((u[:, t] * gb).abs() + wA.abs())
        out["ddt"][:, t] = d_raw * slope[:, t]
        err["ddt"][:, t] = d_err * slope[:, t] + d_raw.abs() * slope_err[:, t] + U * (d_raw * slope[:, t]).abs()
        st = step[:, t, :, None]
        dA += (w * st).sum(0)
        dA_err += (w_err * st.abs() + w.abs() * step_err[:, t, :, None] + (T + B) * U * (w * st).abs()).sum(0)
        g, g_err = ga, ga_err
    for k in out:
        out[k], err[k] = torch.where(keep, out[k], 0.0), torch.where(keep, err[k], 0.0)
    many = (B * T + 2) * U
    return {"du": (out["du"], err["du"]), "ddt": (out["ddt"], err["ddt"]), "dA": (dA, dA_err), "dB": (dB, dB_err),
            "dC": (dC, dC_err), "dz": dz, "dh0": (g, g_err),
            "dD": ((dyg * u).sum((0, 1)), ((dyg_err + many * dyg.abs()) * u.abs()).sum((0, 1))),
            "ddt_bias": (out["ddt"].sum((0, 1)), (err["ddt"] + many * out["ddt"].abs()).sum((0, 1)))}
