"""The float64 oracle of the operators around the sequence layer, pinned to torch autograd over the formulas and to
central differences of its own values."""
from __future__ import annotations

import pytest
import torch
import torch.nn.functional as F

import block_cases as bc
from oracle import block as ob

LENGTHS = torch.tensor([12, 0, 5], dtype=torch.int32)


def scan(p, softplus=True, lengths=None):
    T = p["u"].shape[1]
    raw = p["dt"] + p["dt_bias"]
    dt = F.softplus(raw, threshold=1000.0) if softplus else raw
    h, ys = p["h0"], []
    for t in range(T):
        live = torch.ones(len(h), dtype=torch.bool) if lengths is None else t < lengths.long()
        new = (torch.exp(dt[:, t, :, None] * p["A"]) * h
               + (dt[:, t] * p["u"][:, t])[..., None] * p["Bm"][:, t, None, :])
        h = torch.where(live[:, None, None], new, h)
        y = ((h * p["Cm"][:, t, None, :]).sum(-1) + p["D"] * p["u"][:, t]) * F.silu(p["z"][:, t])
        ys.append(torch.where(live[:, None], y, 0.0))
    return torch.stack(ys, 1), h


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, LENGTHS])
def test_scan_and_its_gradient_against_autograd(softplus, lengths):
    i = bc.ssm_inputs(3, 12, 4, 3, "f32", 0, softplus)
    p = {k: v.double().requires_grad_() for k, v in i.items()}
    y, h = scan(p, softplus, lengths)
    g = torch.Generator().manual_seed(1)
    dy, dh = torch.randn(y.shape, generator=g, dtype=torch.float64), torch.randn(h.shape, generator=g, dtype=torch.float64)
    ((y * dy).sum() + (h * dh).sum()).backward()
    (yo, _), (ho, _) = ob.ssm(**i, lengths=lengths, softplus=softplus)
    assert (yo - y).abs().max() < 1e-12 and (ho - h).abs().max() < 1e-12
    out = ob.ssm_backward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], dy, i["D"], i["z"], i["dt_bias"], i["h0"], dh,
                          lengths, softplus)
    for name, leaf in dict(du="u", ddt="dt", dA="A", dB="Bm", dC="Cm", dD="D", dz="z", ddt_bias="dt_bias",
                           dh0="h0").items():
        assert (out[name][0] - p[leaf].grad).abs().max() < 1e-11, name


def test_scan_gradient_against_differences():
    """Central differences of the oracle's own forward values along a random direction of each input."""
    i = {k: v.double() for k, v in bc.ssm_inputs(1, 6, 3, 2, "f32", 3).items()}
    g = torch.Generator().manual_seed(4)
    rnd = lambda s: torch.randn(s, generator=g, dtype=torch.float64)
    dy, dh = rnd((1, 6, 3)), rnd((1, 3, 2))

    def loss(v):
        (y, _), (h, _) = ob.ssm(**v)
        return float((y * dy).sum() + (h * dh).sum())

    out = ob.ssm_backward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], dy, i["D"], i["z"], i["dt_bias"], i["h0"], dh)
    for name, leaf in dict(du="u", ddt="dt", dA="A", dB="Bm", dC="Cm", dD="D", dz="z", ddt_bias="dt_bias",
                           dh0="h0").items():
        e = rnd(i[leaf].shape)
        up, down = (loss({**i, leaf: i[leaf] + s * 1e-5 * e}) for s in (1, -1))
        assert abs((up - down) / 2e-5 - float((out[name][0] * e).sum())) < 1e-7, name


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_convolution_and_its_gradient_against_autograd(W, silu):
    g = torch.Generator().manual_seed(W)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    B, T, C = 3, 12, 4
    x, w, b, s = (t.requires_grad_() for t in (rnd(B, T, C), rnd(C, W), rnd(C), rnd(B, W - 1, C)))
    win = torch.cat((s, x), 1).transpose(1, 2)
    pre = F.conv1d(win, w[:, None, :], b, groups=C).transpose(1, 2)
    live = (torch.arange(T)[None] < LENGTHS[:, None])[..., None]
    y = torch.where(live, F.silu(pre) if silu else pre, 0.0)
    st = torch.stack([win[i, :, n:n + W - 1].t() for i, n in enumerate(LENGTHS.tolist())])
    dy, ds = rnd(*y.shape), rnd(*st.shape)
    ((y * dy).sum() + (st * ds).sum()).backward()
    (yo, _), so = ob.conv(x, w, b, s, LENGTHS, silu)
    assert (yo - y).abs().max() < 1e-12 and torch.equal(so, st.detach())
    for (v, _), leaf in zip(ob.conv_backward(x, w, b, dy, s, ds, LENGTHS, silu), (x, w, b, s)):
        assert (v - leaf.grad).abs().max() < 1e-11


def test_norm_and_its_gradient_against_autograd():
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, r, w = (t.requires_grad_() for t in (rnd(2, 3, 7), rnd(2, 3, 7), rnd(7)))
    h = x + r
    y = F.rms_norm(h, (7,), w, 1e-6)
    dy, dh = rnd(2, 3, 7), rnd(2, 3, 7)
    ((y * dy).sum() + (h * dh).sum()).backward()
    (yo, _), (ho, _) = ob.rmsnorm(x, w, r)
    assert (yo - y).abs().max() < 1e-13 and (ho - h).abs().max() < 1e-13
    (gx, _), (gw, _) = ob.rmsnorm_backward(h, w, dy, dh)
    assert (gx - x.grad).abs().max() < 1e-12 and torch.equal(x.grad, r.grad) and (gw - w.grad).abs().max() < 1e-12


def test_the_bounds_cover_a_float32_evaluation():
    """The formulas evaluated token by token in float32 stay inside the bounds, and the bounds are no blank cheque:
    for the final state, below 1e-3 of its size."""
    i = bc.ssm_inputs(2, 60, 5, 4, "f32", 7)
    y, h = scan(i)
    (yo, ye), (ho, he) = ob.ssm(**i)
    assert ((y.double() - yo).abs() <= ye).all() and ((h.double() - ho).abs() <= he).all()
    assert float(he.norm() / ho.norm()) < 1e-3
