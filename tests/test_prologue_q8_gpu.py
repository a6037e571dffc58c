"""The 8-bit prologue (one tcgen05 GEMM of e4m3 operands with a fused epilogue) against the float64 prologue oracle on
the values that the operands stand for.

Products of e4m3 values are exact in float32 and their sums run over d_model terms, so Q, K, V may differ from the
float64 value by half a bf16 step plus the summation error, d_model 2^-24 of the sum of absolute products at most; a
random-sign sum of n terms is about sqrt(n) times smaller than that sum, so the bar is 1e-5 of the tensor's RMS.  eta:
its logit's error, 1e-5 of the logits' RMS, times the sigmoid's slope of at most its own value, and the fast
functions' few 1e-7."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import prologue as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


def make(ttt, B, T, H, dm, seed, d=64):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=g) * std
    x = rnd(B, T, dm)
    scale = x.abs().amax(-1) / 448.0
    ops = [(x / scale[..., None]).to(torch.float8_e4m3fn), scale]
    for shape in ((H, dm, d),) * 3 + ((H, dm),):
        ops += ttt.prologue_q8_weights(rnd(*shape, std=dm ** -0.5))
    return ops + [rnd(H)]


def oracle(ops, window=slice(None), seq=slice(None), **kw):
    x, sx, *rest, b = ops
    w = [q.double() * s.double()[..., None] for q, s in zip(rest[::2], rest[1::2])]
    w = [t.transpose(1, 2) if t.dim() == 3 else t for t in w]
    return op.project((x[seq, window].double() * sx[seq, window].double()[..., None]), *w, b, **kw)


def compare(out, ref, where=""):
    for name, a, r in zip(("Q", "K", "V"), out[:3], ref[:3]):
        a = a.float().cpu().numpy().astype(np.float64)
        err = np.abs(a - r) - (2.0 ** -8) * np.abs(r) - 1e-5 * float(np.sqrt(np.mean(r ** 2)))
        assert err.max() <= 0, f"{name}{where}: worst excess {err.max():.3e}"
    e = out[3].cpu().numpy().astype(np.float64)
    assert float((np.abs(e - ref[3]) / ref[3]).max()) <= 2e-5, f"eta{where}"


@pytest.mark.parametrize("B,T,H,dm,pos0,rotary", [
    (1, 1, 4, 16, 0, True),         # one token, one part of a K step
    (1, 128, 4, 128, 0, True),      # one row tile, one K step
    (2, 100, 4, 144, 0, True),      # rows and d_model end inside a tile
    (1, 300, 8, 256, 37, False),
    (3, 77, 12, 768, 100000, True),  # the 125M-layer width, ragged streams, far positions
    (1, 40, 4, 64, 2 ** 31 - 20, True),  # positions that pass 31 bits: angles 2^-23 of a turn apart at most
    (1, 130, 20, 1040, 5, True),    # 20 heads: the learning-rate tile is padded to 32 columns
])
def test_against_the_oracle(ttt, B, T, H, dm, pos0, rotary):
    ops = make(ttt, B, T, H, dm, T)
    out = ttt.ttt_prologue_q8_forward(*(t.cuda() for t in ops), pos0=pos0, rotary=rotary, eta_base=0.5)
    compare(out, oracle(ops, pos0=pos0, rotary=rotary, eta_base=0.5))


def angles(ttt, pos0, T):
    """How far the rotation's angles are off, at the positions and features whose sine is near zero, where bf16 resolves it:
    Q is -sin in its first 32 features and cos in the others.  Returns (sines near zero, errors of their angles)."""
    H, dm = 4, 16
    x = torch.zeros(1, T, dm)
    x[..., 0] = 1.0
    theta = torch.zeros(H, 64, dm)
    theta[:, 32:, 0] = 1.0
    f8, one = theta.to(torch.float8_e4m3fn).cuda(), torch.ones(H, 64, device="cuda")
    lr = torch.zeros(H, dm, device="cuda").to(torch.float8_e4m3fn)
    Q = ttt.ttt_prologue_q8_forward(x.to(torch.float8_e4m3fn).cuda(), torch.ones(1, T, device="cuda"), f8, one, f8, one, f8, one,
                                    lr, one[:, 0].contiguous(), one[:, 0].contiguous(), pos0=pos0)[0]
    got = -Q[0, 0, :, :32].float().cpu().numpy().astype(np.float64)
    wide = np.longdouble  # 64 bits of mantissa
    pos = np.arange(pos0, pos0 + T).astype(wide)[:, None]
    angle = pos * wide(10000) ** (-np.arange(32).astype(wide) / 32)
    turns = angle / (2 * np.arccos(wide(-1)))
    r = ((turns - np.rint(turns)) * (2 * np.arccos(wide(-1)))).astype(np.float64)
    return np.sin(r), got - np.sin(r), np.cos(r)


def test_rotary_angles_are_rounded_to_both_sides(ttt):
    """Angles in steps of 2^-23 turns (7.5e-7): their errors, 2.2e-7 in the mean square, average out.  With sines below 5e-4
    the outputs' rounding is as small, and the mean of 300 such errors stays below 1.5e-7, five of its deviations and more."""
    s, e, c = angles(ttt, 0, 65536)
    near = (np.abs(s) < 5e-4) & (c > 0)
    assert near.sum() > 300 and abs(e[near].mean()) <= 1.5e-7


def test_rotary_angles_at_far_positions(ttt):
    """Near 2^31: half a step of 2^-23 turns, 3.75e-7; a rounding and a half of a double at that position, 7.2e-7; the sine's
    documented 2^-21.4; and half a step of the output at 5e-5."""
    s, e, _ = angles(ttt, 2 ** 31 - 2 ** 18, 2 ** 18)
    near = np.abs(s) < 5e-5
    assert near.sum() > 100 and np.abs(e[near]).max() <= 3.75e-7 + 7.2e-7 + 2 ** -21.4 + 2.0 ** -9 * 5e-5


@pytest.mark.parametrize("B,T", [(64, 1), (150, 1), (50, 3), (5, 33)])
def test_streams_that_end_within_a_warp(ttt, B, T):
    """One token, or a few, of many streams: a tile's rows belong to as many sequences."""
    ops = make(ttt, B, T, 8, 144, B)
    compare(ttt.ttt_prologue_q8_forward(*(t.cuda() for t in ops), pos0=1971), oracle(ops, pos0=1971))


def test_many_heads(ttt):
    """H = 256: the learning-rate tile is as wide as the others."""
    ops = make(ttt, 1, 40, 256, 64, 1)
    compare(ttt.ttt_prologue_q8_forward(*(t.cuda() for t in ops)), oracle(ops))


def test_full_size_sampled_windows(ttt):
    """The 1.3B layer at 32k tokens in one launch; windows of both sequences against the oracle on each alone."""
    B, T, H, dm, W = 2, 32768, 32, 2048, 32
    ops = make(ttt, B, T, H, dm, 5)
    out = ttt.ttt_prologue_q8_forward(*(t.cuda() for t in ops))
    for b, t0 in ((0, 8128), (0, T - W), (1, 0), (1, 16384 - W // 2)):
        w = slice(t0, t0 + W)
        compare([o[b:b + 1, :, w] for o in out], oracle(ops, w, slice(b, b + 1), pos0=t0), f" ({b}, {t0})")


def test_refusals(ttt):
    ops = [t.cuda() for t in make(ttt, 1, 16, 6, 64, 0)]  # H = 6 is no multiple of 4
    with pytest.raises(ttt.TTTError) as e:
        ttt.ttt_prologue_q8_forward(*ops)
    assert e.value.status == 6
    ops = [t.cuda() for t in make(ttt, 1, 16, 4, 64, 0)]
    with pytest.raises(TypeError, match="x must be"):
        ttt.ttt_prologue_q8_forward(ops[0].bfloat16(), *ops[1:])
    with pytest.raises(ValueError, match="scale_q must be"):
        ttt.ttt_prologue_q8_forward(*ops[:3], ops[3].reshape(-1), *ops[4:])
