"""The root-mean-square norm kernels against the float64 oracle (oracle/block.py), within the float32 bound that the
oracle carries and half a step of the output's type."""
from __future__ import annotations

import pytest
import torch

import block_cases as bc
from oracle import block as ob

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 7, 31, 32, 64, 100, 255, 256, 264, 768, 1000, 2047, 2048, 4104, 8192, 8200, 16383, 16384]


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


def inputs(B, T, d, kind, residual, seed=0):
    g = torch.Generator().manual_seed(seed + d)
    ty = bc.KINDS[kind]
    x = bc.normal(g, B, T, d).to(ty)
    r = bc.normal(g, B, T, d, std=3.0).to(ty) if residual else None
    return x, r, 1 + bc.normal(g, d, std=0.1)


def up(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(ttt, d, residual, kind):
    x, r, w = inputs(2, 3, d, kind, residual)
    y, h = ttt.ttt_rmsnorm_forward(x.cuda(), w.cuda(), up(r))
    (yo, ye), (ho, he) = ob.rmsnorm(x, w, r)
    bc.close("y", y, yo, ye)
    if residual:
        bc.close("h", h, ho, he)
    else:
        assert h is None


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 7, 64, 768, 1000, 2048, 8200])
def test_q8(ttt, d, kind):
    x, r, w = inputs(2, 3, d, kind, True, seed=1)
    q, scale, h = ttt.ttt_rmsnorm_q8_forward(x.cuda(), w.cuda(), r.cuda())
    (yo, ye), (ho, he) = ob.rmsnorm(x, w, r)
    bc.close("h", h, ho, he)
    so = yo.abs().amax(-1) / 448.0
    s_err = ye.amax(-1) / 448.0 + 4 * ob.U * so
    bc.close("scale", scale, so, s_err)
    v, s = q.cpu().double(), scale.cpu().double()[..., None]
    assert torch.isfinite(v).all() and float(v.abs().amax(-1).min()) == 448.0
    # half a step of e4m3: 2^-4 of the value, or half of its smallest number 2^-9
    bound = s * (yo.abs() / s * 2.0 ** -4 + 2.0 ** -10) + 2 * ye + 4 * ob.U * yo.abs()
    assert ((v * s - yo).abs() <= bound).all()


def test_q8_rows_of_zeros_and_of_tiny_values(ttt):
    x = torch.zeros(1, 3, 256)
    x[0, 1] = 1e-38
    x[0, 2, 5] = 3.0
    q, scale, _ = ttt.ttt_rmsnorm_q8_forward(x.cuda(), torch.ones(256).cuda())
    q, scale = q.float().cpu(), scale.cpu()
    assert not q[0, 0].any() and scale[0, 0] == 2.0 ** -100
    assert torch.isfinite(q).all() and torch.isfinite(scale).all()
    assert q[0, 2, 5] == 448 and q[0, 2].abs().sum() == 448


def test_nan_and_infinity_stay_in_their_row(ttt):
    x, _, w = inputs(1, 4, 300, "f32", False)
    clean, _ = ttt.ttt_rmsnorm_forward(x.cuda(), w.cuda())
    x[0, 1, 7] = float("nan")
    x[0, 2, 9] = float("inf")
    y, _ = ttt.ttt_rmsnorm_forward(x.cuda(), w.cuda())
    q, scale, _ = ttt.ttt_rmsnorm_q8_forward(x.cuda(), w.cuda())
    assert torch.isnan(y[0, 1]).all() and torch.isnan(scale[0, 1]) and torch.isnan(q[0, 1].float()).all()
    for row in (0, 3):
        assert torch.equal(y[0, row], clean[0, row]) and torch.isfinite(q[0, row].float()).all()


@pytest.mark.parametrize("d", [40, 300, 2047, 2048, 9001])
@pytest.mark.parametrize("weight", [1.0, float("nan"), float("inf"), 0.0])
def test_q8_of_values_that_are_not_finite(ttt, d, weight):
    """Scale and q are NaN, or finite, where the formula's are; an infinite weight makes an infinite scale."""
    x, _, w = inputs(1, 6, d, "f32", False)
    w[3] = weight
    x[0, 1, 7], x[0, 2, d - 1], x[0, 3, 3], x[0, 4, 0] = float("nan"), float("inf"), -float("inf"), float("inf")
    q, scale, _ = ttt.ttt_rmsnorm_q8_forward(x.cuda(), w.cuda())
    (y, _), _ = ob.rmsnorm(x, w)
    want = y.abs().amax(-1) / 448.0
    q, scale = q.cpu().double(), scale.cpu().double()
    assert torch.equal(torch.isnan(scale), torch.isnan(want)) and torch.equal(torch.isinf(scale), torch.isinf(want))
    assert torch.equal(torch.isnan(q), torch.isnan(y / want[..., None]))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("past", [True, False])
@pytest.mark.parametrize("B,T,d", [(1, 1, 1), (2, 3, 7), (1, 5, 32), (3, 50, 100), (2, 9, 256), (2, 200, 768),
                                   (1, 17, 2047), (1, 700, 2048), (1, 2, 8200), (1, 3, 16384)])
def test_backward(ttt, B, T, d, past, kind):
    x, r, w = inputs(B, T, d, kind, past, seed=2)
    g = torch.Generator().manual_seed(9)
    dy = bc.normal(g, B, T, d).to(x.dtype)
    dh, dw = ttt.ttt_rmsnorm_backward(x.cuda(), w.cuda(), dy.cuda(), up(r))
    (dho, dhe), (dwo, dwe) = ob.rmsnorm_backward(x, w, dy, r)
    bc.close("dh", dh, dho, dhe)
    bc.close("dweight", dw, dwo, dwe)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [100, 2048, 9001])
def test_backward_of_tiny_and_large_rows(ttt, d, kind):
    """Rows of zeros, of 1e-14 and of 1e14 and 1e17, whose inverse norm's third power is no float."""
    x, r, w = inputs(1, 5, d, kind, True, seed=4)
    x = (x.float() * torch.tensor([0.0, 1e-14, 1.0, 1e14, 1e17])[None, :, None]).to(x.dtype)
    dy = bc.normal(torch.Generator().manual_seed(11), 1, 5, d).to(x.dtype)
    for past in (None, r):
        dh, dw = ttt.ttt_rmsnorm_backward(x.cuda(), w.cuda(), dy.cuda(), up(past), eps=1e-30)
        (dho, dhe), (dwo, dwe) = ob.rmsnorm_backward(x, w, dy, past, eps=float(torch.tensor(1e-30)))
        bc.close("dh", dh, dho, dhe)
        bc.close("dweight", dw, dwo, dwe)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,d", [(64, 300, 5), (8, 1000, 64), (3, 2000, 96), (1, 4000, 200), (1, 400, 9001),
                                   (2, 170, 11000), (1, 300, 13004), (1, 310, 16383)])
def test_many_rows(ttt, B, T, d, kind):
    """Several narrow rows a block, rows that take most of an SM's registers, and more rows than the blocks take at once."""
    x, r, w = inputs(B, T, d, kind, True, seed=3)
    y, h = ttt.ttt_rmsnorm_forward(x.cuda(), w.cuda(), r.cuda())
    (yo, ye), (ho, he) = ob.rmsnorm(x, w, r)
    bc.close("y", y, yo, ye)
    bc.close("h", h, ho, he)
    dy = bc.normal(torch.Generator().manual_seed(10), B, T, d).to(x.dtype)
    dh, dw = ttt.ttt_rmsnorm_backward(x.cuda(), w.cuda(), dy.cuda(), r.cuda())
    (dho, dhe), (dwo, dwe) = ob.rmsnorm_backward(x, w, dy, r)
    bc.close("dh", dh, dho, dhe)
    bc.close("dweight", dw, dwo, dwe)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("B,T,d", [(64, 300, 5), (8, 1000, 64), (3, 2000, 96), (1, 4000, 200), (1, 400, 9001),
                                   (2, 170, 11000), (1, 300, 13004), (1, 310, 16383), (1, 310, 16384)])
def test_q8_of_many_rows(ttt, B, T, d, residual, kind):
    """More rows than the blocks take at once, and rows that take most of an SM's registers."""
    x, r, w = inputs(B, T, d, kind, residual, seed=5)
    q, scale, h = ttt.ttt_rmsnorm_q8_forward(x.cuda(), w.cuda(), up(r))
    (yo, ye), (ho, he) = ob.rmsnorm(x, w, r)
    if residual:
        bc.close("h", h, ho, he)
    so = yo.abs().amax(-1) / 448.0
    bc.close("scale", scale, so, ye.amax(-1) / 448.0 + 4 * ob.U * so)
    v, s = q.cpu().double(), scale.cpu().double()[..., None]
    bound = s * (yo.abs() / s * 2.0 ** -4 + 2.0 ** -10) + 2 * ye + 4 * ob.U * yo.abs()
    assert float(v.abs().amax(-1).min()) == 448.0 and ((v * s - yo).abs() <= bound).all()


def test_backward_twice_is_the_same(ttt):
    x, r, w = (t.cuda() for t in inputs(4, 999, 512, "bf16", True))
    one, two = (ttt.ttt_rmsnorm_backward(x, w, r) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_in_place_on_the_stream(ttt):
    x, r, w = (t.cuda() for t in inputs(2, 5, 768, "bf16", True))
    y0, h0 = ttt.ttt_rmsnorm_forward(x, w, r)
    y, h = ttt.ttt_rmsnorm_forward(x, w, r, y=x, h=r)
    assert y is x and h is r and torch.equal(y, y0) and torch.equal(h, h0)


def test_offsets_past_32_bits(ttt):
    """2.2e9 elements: the last rows equal the same rows on their own."""
    rows, d = 1_080_000, 2048
    x = torch.empty(1, rows, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[0, -7:] = torch.randn(7, d, generator=g, device="cuda").bfloat16()
    w = torch.rand(d, generator=g, device="cuda")
    y, _ = ttt.ttt_rmsnorm_forward(x, w)
    alone, _ = ttt.ttt_rmsnorm_forward(x[:, -7:].contiguous(), w)
    assert torch.equal(y[:, -7:], alone)


def test_gradient_offsets_past_32_bits(ttt):
    """2.2e9 elements, all but the last rows zeros: their gradients equal those of these rows on their own."""
    rows, d = 1_080_000, 2048
    x = torch.zeros(1, rows, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[0, -7:] = torch.randn(7, d, generator=g, device="cuda").bfloat16()
    w = torch.rand(d, generator=g, device="cuda")
    dh, dw = ttt.ttt_rmsnorm_backward(x, w, x, x)
    one, dw1 = ttt.ttt_rmsnorm_backward(*(t[:, -7:].contiguous() if t is x else t for t in (x, w, x, x)))
    assert torch.equal(dh[:, -7:], one) and not dh[0, :1000].any()
    assert torch.allclose(dw, dw1, rtol=1e-5, atol=1e-5 * float(dw1.abs().max()))


def test_refusals_of_the_binding(ttt):
    x = torch.zeros(2, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(TypeError, match="x must be bf16 or fp32"):
        ttt.ttt_rmsnorm_forward(x.half(), w)
    with pytest.raises(ValueError, match="x must be a contiguous"):
        ttt.ttt_rmsnorm_forward(x.transpose(0, 1), w)
    with pytest.raises(ValueError, match="weight must be"):
        ttt.ttt_rmsnorm_forward(x, w[:32].contiguous())
    with pytest.raises(TypeError, match="residual must be"):
        ttt.ttt_rmsnorm_forward(x, w, x.bfloat16())
    with pytest.raises(ttt.TTTError) as e:
        ttt.ttt_rmsnorm_forward(x, w, eps=0.0)
    assert e.value.status == 2
    with pytest.raises(ttt.TTTError) as e:
        ttt.ttt_rmsnorm_backward(x, w, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 9
