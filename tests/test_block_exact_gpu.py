"""Sums of the operators around the sequence layer on inputs that make them exact: small whole numbers, and one value in
every place.  The bounds of the other tests grow with the number of terms; here a term that is lost, or counted twice,
shows whatever their number."""
from __future__ import annotations

import pytest
import torch

import block_cases as bc
from oracle import block as ob

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("kind", ["bf16", "f32"])


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


def whole(g, *shape, most=1, keep=1.0):
    """Whole numbers from -most to most, of which a share of about `keep` is kept and the rest is zero."""
    v = torch.randint(-most, most + 1, shape, generator=g).float()
    return v * (torch.rand(shape, generator=g) < keep)


def same(name, got, want):
    assert torch.equal(got.detach().to("cpu", torch.float64), want), name


# ---------------------------------------------------------------- norm
@KINDS
@pytest.mark.parametrize("d", [1, 7, 32, 100, 264, 1000, 2047, 2048, 4104, 8200, 12289, 16383, 16384])
def test_norm_of_one_value_in_every_place(ttt, d, kind):
    """A row's only value at each place in turn (up to 2048 of them): y is sqrt(d) there, and without the value the sum of
    squares would leave 1 / sqrt(eps).  Its gradient's projection along the row is that one product."""
    g = torch.Generator().manual_seed(d)
    rows = min(d, 2048)
    at = torch.randperm(d, generator=g)[:rows]
    at[0], at[-1] = 0, d - 1
    x = torch.zeros(1, rows, d, dtype=bc.KINDS[kind])
    x[0, torch.arange(rows), at] = 1.0
    w = torch.randint(1, 4, (d,), generator=g).float()
    y, _ = ttt.ttt_rmsnorm_forward(x.cuda(), w.cuda())
    (yo, _), _ = ob.rmsnorm(x, w)
    step = bc.half_step(y.dtype)
    # h w is exact; 1 / d, the sum with eps, the root's two units and the last product: five roundings and the type's own
    assert ((y.cpu().double() - yo).abs() <= (5 * 2 * ob.U + step) * yo.abs()).all()
    # dy is one at the row's place: dh = r w (1 - 1 / (1 + eps d)) there and zero elsewhere, dweight counts rows
    dh, dw = ttt.ttt_rmsnorm_backward(x.cuda(), w.cuda(), x.cuda())
    r = (1.0 / d + 1e-6) ** -0.5
    assert (dh.cpu().double()[x == 0] == 0).all()
    # two terms that cancel, with r's five roundings once and three times and those of the products
    want = r * w[at].double() * (1 - r * r / d)
    assert ((dh[0, torch.arange(rows), at.cuda()].cpu().double() - want).abs() <= 32 * ob.U * r * w[at].double() + step * want).all()
    count = torch.zeros(d, dtype=torch.float64).scatter_add_(0, at, torch.ones(rows, dtype=torch.float64))
    assert ((dw.cpu().double() - r * count).abs() <= 8 * ob.U * r * count).all()


@KINDS
@pytest.mark.parametrize("B,T,d", [(64, 300, 5), (8, 1000, 64), (3, 2000, 96), (1, 4000, 200), (1, 8193, 768), (2, 170, 11000),
                                   (1, 310, 16383)])
def test_norm_weight_gradient_counts_every_row(ttt, B, T, d, kind):
    """Rows of ones and minus ones, dy of small whole numbers: dweight is a whole number times r, which differs from 1 by a
    few 2^-24.  A term is 1 at least and the roundings of all are 8 2^-24 of the terms' sizes, below 0.02."""
    g = torch.Generator().manual_seed(1)
    h = (2.0 * torch.randint(0, 2, (B, T, d), generator=g) - 1).to(bc.KINDS[kind])
    dy = whole(g, B, T, d, most=2).to(h.dtype)
    _, dw = ttt.ttt_rmsnorm_backward(h.cuda(), torch.ones(d).cuda(), dy.cuda(), eps=1e-9)
    want = (dy.double() * h.double()).sum((0, 1))
    assert (dw.cpu().double() - want).abs().max() <= 0.25


# ---------------------------------------------------------------- convolution
@KINDS
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 1, 2), (3, 5, 8, 4), (2, 515, 64, 4), (57, 440, 64, 3), (4, 2048, 70, 4), (1, 9000, 12, 2),
                                     (8, 1000, 520, 4)])
def test_convolution_counts_every_term(ttt, B, T, C, W, padded, kind):
    """Whole numbers throughout and no SiLU: every sum is exact, in any order."""
    g = torch.Generator().manual_seed(T)
    ty = bc.KINDS[kind]
    x, w, b, s0 = whole(g, B, T, C, most=2).to(ty), whole(g, C, W, most=2), whole(g, C), whole(g, B, W - 1, C).to(ty)
    dy, ds = whole(g, B, T, C, most=2).to(ty), whole(g, B, W - 1, C).to(ty)
    n = bc.lengths_for(B, T, g) if padded else None
    up = lambda t: None if t is None else t.cuda()
    y, _ = ttt.ttt_conv_forward(x.cuda(), w.cuda(), b.cuda(), s0.cuda(), lengths=up(n), activation=None)
    same("y", y, ob.conv(x, w, b, s0, n, False)[0][0])
    got = ttt.ttt_conv_backward(x.cuda(), w.cuda(), b.cuda(), dy.cuda(), s0.cuda(), ds.cuda(), lengths=up(n), activation=None)
    for name, a, (want, _) in zip(("dx", "dweight", "dbias", "dstate0"), got, ob.conv_backward(x, w, b, dy, s0, ds, n, False)):
        same(name, a, want)


# ---------------------------------------------------------------- selective scan
@KINDS
@pytest.mark.parametrize("padded", [False, True])
# the kernel for few tokens; few channels, in one block and in a cluster; many channels; more than 16 states; a split time axis
@pytest.mark.parametrize("B,T,C,N", [(3, 8, 40, 16), (3, 70, 9, 16), (1, 2000, 20, 16), (40, 70, 33, 16), (40, 70, 36, 40),
                                     (20, 300, 64, 64), (2, 2641, 64, 16), (8, 200, 300, 8)])
def test_scan_counts_every_term(ttt, B, T, C, N, padded, kind):
    """A = 0, steps of one and few whole numbers: states that only add up.  Every sum stays below 2^24 and is exact in any
    order; what is stored in 16 bits is rounded once."""
    g = torch.Generator().manual_seed(T)
    ty = bc.KINDS[kind]
    few = min(1.0, 16.0 / T)
    i = dict(u=whole(g, B, T, C, keep=few).to(ty), dt=torch.ones(B, T, C).to(ty), A=torch.zeros(C, N), Bm=whole(g, B, T, N).to(ty),
             Cm=whole(g, B, T, N).to(ty), D=whole(g, C, most=2), h0=whole(g, B, C, N))
    dy, dh = whole(g, B, T, C, keep=few).to(ty), whole(g, B, C, N)
    n = bc.lengths_for(B, T, g) if padded else None
    c = bc.cuda(i)
    kw = dict(lengths=None if n is None else n.cuda(), dt_softplus=False)
    y, h = ttt.ttt_ssm_forward(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], c["D"], h0=c["h0"], **kw)
    (yo, _), (ho, _) = ob.ssm(**i, lengths=n, softplus=False)
    same("y", y, yo.to(ty).double())
    same("h_T", h, ho)
    out = ttt.ttt_ssm_backward(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], dy.cuda(), c["D"], None, None, c["h0"], dh.cuda(), **kw)
    want = ob.ssm_backward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], dy, i["D"], None, None, i["h0"], dh, n, False)
    for name, a in zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"), out):
        if a is None:
            continue
        v = want[name][0]
        assert v.abs().max() < 2 ** 24
        same(name, a, v.to(a.dtype).double())
