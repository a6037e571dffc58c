"""The operators around the sequence layer reject bad arguments on the host with the documented status codes, and the
binding's own checks name the argument.  Every call fails a check, so nothing is launched and no pointer is read."""
from __future__ import annotations

import pytest
import torch

b = pytest.importorskip("test_sequence_layers_ttt_b200._binding")

NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUP, WORKSPACE = 1, 2, 3, 4, 5, 6, 9
BASE, STRIDE = 1 << 40, 1 << 34


def fake(n, **at):
    p = [BASE + i * STRIDE for i in range(n)]
    for k, v in at.items():
        p[int(k[1:])] = v
    return p


# ---------------------------------------------------------------- norm: x residual weight y h
def norm(B=2, T=3, d=64, dtype=0, eps=1e-6, **at):
    return b.lib.ttt_rmsnorm_forward(B, T, d, dtype, eps, *fake(5, **at), None)


def norm_q8(B=2, T=3, d=64, dtype=0, eps=1e-6, **at):  # x residual weight q scale h
    return b.lib.ttt_rmsnorm_q8_forward(B, T, d, dtype, eps, *fake(6, **at), None)


def norm_bwd(B=2, T=3, d=64, dtype=0, eps=1e-6, ws=1 << 30, **at):  # h weight dy dh_in dh dweight workspace
    return b.lib.ttt_rmsnorm_backward(B, T, d, dtype, eps, *fake(7, **at), ws, None)


@pytest.mark.parametrize("call", [norm, norm_q8, norm_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(d=0), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(dtype=2), DTYPE), (dict(d=16385), UNSUP),
    (dict(p0=None), NULL), (dict(p2=None), NULL), (dict(p0=BASE + 2), ALIGN),
])
def test_norm_refusals(call, kw, code):
    assert call(**kw) == code


def test_norm_aliases():
    assert norm(p3=BASE + 16) == ALIAS                      # y inside x, but not x
    assert norm(p4=BASE + 3 * STRIDE) == ALIAS              # h is y
    assert norm(p3=BASE + 2 * STRIDE) == ALIAS              # y is the weight
    assert norm_q8(p3=BASE) == ALIAS                        # the 8-bit rows lie otherwise than x's
    assert norm_q8(p4=BASE + 5 * STRIDE) == ALIAS           # scale inside h
    assert norm_bwd(p4=BASE) == ALIAS                       # dh is h
    assert norm_bwd(p5=BASE + 2 * STRIDE) == ALIAS          # dweight inside dy


def test_norm_backward_workspace():
    assert norm_bwd(p6=None) == WORKSPACE
    assert norm_bwd(ws=b.lib.ttt_rmsnorm_backward_workspace_size(2, 3, 64, 0) - 1) == WORKSPACE


# ---------------------------------------------------------------- 8-bit prologue: x sx q sq k sk v sv lr slr blr | Q K V eta
def pro(B=1, T=4, H=4, d=64, dm=128, base=1e4, **at):
    return b.lib.ttt_prologue_q8_forward(B, T, H, d, dm, 0, 1.0, base, 1, *fake(15, **at), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(base=1.0), SHAPE), (dict(H=6), UNSUP), (dict(H=260), UNSUP),
    (dict(d=32), UNSUP), (dict(dm=120), UNSUP), (dict(dm=8), UNSUP), (dict(p1=None), NULL), (dict(p14=None), NULL),
    (dict(p0=BASE + 8), ALIGN), (dict(p11=BASE), ALIAS), (dict(p12=BASE + 11 * STRIDE), ALIAS),
])
def test_prologue_q8_refusals(kw, code):
    assert pro(**kw) == code


def test_prologue_q8_refuses_an_infinite_rope_base():
    """Its first feature's step would be 0 times infinity."""
    assert pro(base=float("inf")) == SHAPE and pro(base=float("nan")) == SHAPE


# ---------------------------------------------------------------- convolution
def conv(B=2, T=5, C=8, W=4, dtype=0, ld=8, **at):  # x weight bias state0 lengths y state_T
    return b.lib.ttt_conv_forward(B, T, C, W, dtype, 1, ld, *fake(7, **at), None)


def conv_dec(B=2, T=1, C=8, W=4, dtype=0, ld=8, **at):  # x weight bias state y
    return b.lib.ttt_conv_decode(B, T, C, W, dtype, 1, ld, *fake(5, **at), None)


def conv_bwd(B=2, T=5, C=8, W=4, dtype=0, ld=8, ws=1 << 30, **at):
    # x weight bias state0 lengths dy dstate_T dx dweight dbias dstate0 workspace
    return b.lib.ttt_conv_backward(B, T, C, W, dtype, 1, ld, *fake(12, **at), ws, None)


@pytest.mark.parametrize("call", [conv, conv_dec, conv_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(C=0), SHAPE), (dict(ld=7), SHAPE), (dict(dtype=5), DTYPE),
    (dict(W=1), UNSUP), (dict(W=5), UNSUP), (dict(p0=None), NULL), (dict(p1=None), NULL), (dict(p0=BASE + 1), ALIGN),
    (dict(p1=BASE + STRIDE + 4), ALIGN),
])
def test_conv_refusals(call, kw, code):
    assert call(**kw) == code


def test_conv_aliases_and_workspace():
    assert conv(p5=BASE) == ALIAS                           # y is x
    assert conv(p6=BASE + 3 * STRIDE + 16) == ALIAS         # the final state inside the first
    assert conv_dec(p3=None) == NULL
    assert conv_dec(p4=BASE + 3 * STRIDE) == ALIAS          # y is the state
    assert conv_bwd(p7=BASE) == ALIAS and conv_bwd(p10=BASE + 3 * STRIDE) == ALIAS
    assert conv_bwd(p11=None) == WORKSPACE
    assert conv_bwd(ws=b.lib.ttt_conv_backward_workspace_size(2, 5, 8, 4) - 1) == WORKSPACE


# ---------------------------------------------------------------- scan
def ssm(B=2, T=5, C=8, N=4, dtype=0, lds=None, **at):  # u dt dt_bias A B C D z h0 lengths y h_T
    return b.lib.ttt_ssm_forward(B, T, C, N, dtype, 1, *(lds or (C, C, N, N, C)), *fake(12, **at), None)


def ssm_dec(B=2, T=1, C=8, N=4, dtype=0, lds=None, **at):  # u dt dt_bias A B C D z h y
    return b.lib.ttt_ssm_decode(B, T, C, N, dtype, 1, *(lds or (C, C, N, N, C)), *fake(10, **at), None)


def ssm_bwd(B=2, T=5, C=8, N=4, dtype=0, lds=None, ws=1 << 40, **at):
    # u dt dt_bias A B C D z h0 lengths | dy dh_T | du ddt dA dB dC dD dz ddt_bias dh0 workspace
    return b.lib.ttt_ssm_backward(B, T, C, N, dtype, 1, *(lds or (C, C, N, N, C)), *fake(22, **at), ws, None)


@pytest.mark.parametrize("call", [ssm, ssm_dec, ssm_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), SHAPE), (dict(B=1, T=(1 << 31) - (1 << 16)), SHAPE), (dict(T=-1), SHAPE), (dict(C=0), SHAPE), (dict(N=0), SHAPE), (dict(N=65), UNSUP),
    (dict(dtype=9), DTYPE), (dict(lds=(7, 8, 4, 4, 8)), SHAPE), (dict(lds=(8, 8, 3, 4, 8)), SHAPE),
    (dict(lds=(8, 8, 4, 4, 7)), SHAPE), (dict(p0=None), NULL), (dict(p3=None), NULL), (dict(p5=None), NULL),
    (dict(p0=BASE + 1), ALIGN), (dict(p3=BASE + 3 * STRIDE + 4), ALIGN),
])
def test_ssm_refusals(call, kw, code):
    assert call(**kw) == code


def test_ssm_aliases_and_workspace():
    assert ssm(p10=BASE) == ALIAS                           # y is u
    assert ssm(p11=BASE + 8 * STRIDE + 16) == ALIAS         # the final state inside the first
    assert ssm(p11=None) == NULL
    assert ssm_dec(p8=None) == NULL and ssm_dec(p9=BASE + 7 * STRIDE) == ALIAS
    assert ssm_bwd(p12=BASE + STRIDE) == ALIAS              # du is dt
    assert ssm_bwd(p7=None) == NULL                         # dz without z
    assert ssm_bwd(p18=None) == NULL                        # z without dz
    assert ssm_bwd(p21=None) == WORKSPACE
    assert ssm_bwd(ws=b.lib.ttt_ssm_backward_workspace_size(2, 5, 8, 4) - 1) == WORKSPACE


def test_workspace_queries_of_bad_shapes_are_zero():
    assert b.lib.ttt_ssm_backward_workspace_size(0, 5, 8, 4) == 0
    assert b.lib.ttt_ssm_backward_workspace_size(1, 5, 8, 65) == 0
    assert b.lib.ttt_conv_backward_workspace_size(1, 5, 8, 9) == 0
    assert b.lib.ttt_rmsnorm_backward_workspace_size(1, 1, 20000, 0) == 0


# ---------------------------------------------------------------- the binding's checks
def test_binding_names_the_argument():
    x, w = torch.zeros(1, 2, 8), torch.ones(8)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        b.ttt_rmsnorm_forward(x, w)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        b.ttt_conv_forward(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="u must be a CUDA tensor"):
        b.ttt_ssm_forward(x, x, torch.zeros(8, 4), x, x)
    with pytest.raises(ValueError, match="state must be"):
        b.ttt_conv_decode(x, torch.zeros(8, 4), None, None)
    with pytest.raises(ValueError, match="activation"):
        b._silu_code("relu")


def test_binding_refuses_sizes_past_31_bits():
    """Sizes that ctypes would cut to the library's 32 bits: the call would work on the first few tokens alone."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    far = 2 ** 32 + 8
    with FakeTensorMode():
        cuda = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda:0")
        f32, f8 = torch.float32, torch.float8_e4m3fn
        x = cuda(1, far, 1)
        w, A = cuda(1, dtype=f32), cuda(1, far, dtype=f32)
        pro = [cuda(1, 4, 16, dtype=f8), cuda(1, 4, dtype=f32)] + [cuda(4, 64, 16, dtype=f8), cuda(4, 64, dtype=f32)] * 3 + [
            cuda(4, 16, dtype=f8), cuda(4, dtype=f32), cuda(4, dtype=f32)]
        u, B = cuda(1, 1, 1), cuda(1, 1, far)
        for call in (lambda: b.ttt_rmsnorm_forward(x, w), lambda: b.ttt_rmsnorm_q8_forward(x, w),
                     lambda: b.ttt_rmsnorm_backward(x, w, x), lambda: b.ttt_conv_forward(x, cuda(1, 4, dtype=f32)),
                     lambda: b.ttt_conv_backward(x, cuda(1, 4, dtype=f32), None, x),
                     lambda: b.ttt_conv_decode(u, cuda(1, far, dtype=f32), None, cuda(1, far - 1, 1)),
                     lambda: b.ttt_ssm_forward(x, x, cuda(1, 1, dtype=f32), x, x),
                     lambda: b.ttt_ssm_forward(u, u, A, B, B), lambda: b.ttt_ssm_backward(u, u, A, B, B, u),
                     lambda: b.ttt_ssm_decode(u, u, A, B, B, cuda(1, 1, far, dtype=f32))):
            with pytest.raises(ValueError, match="past 2\\^31"):
                call()
        with pytest.raises(ValueError, match="pos0"):
            b.ttt_prologue_q8_forward(*pro, pos0=2 ** 31)


def test_q8_weights_layout():
    g = torch.Generator().manual_seed(0)
    theta = torch.randn(3, 32, 64, generator=g)
    q, s = b.prologue_q8_weights(theta)
    assert q.shape == (3, 64, 32) and s.shape == (3, 64) and q.dtype == torch.float8_e4m3fn
    back = (q.float() * s[..., None]).transpose(1, 2)
    assert (back - theta).abs().max() <= theta.abs().max() * 2 ** -4
    assert float(q.float().abs().amax(-1).min()) == 448.0
    ql, sl = b.prologue_q8_weights(theta[:, :, 0])
    assert ql.shape == (3, 32) and sl.shape == (3,)
