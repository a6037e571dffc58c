"""The short causal convolution kernels against the float64 oracle (oracle/block.py), within the float32 bound that
the oracle carries and half a step of the output's type.  Everything that must not be read is NaN."""
from __future__ import annotations

import pytest
import torch

import block_cases as bc
from oracle import block as ob

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


def inputs(B, T, C, W, kind, seed=0, state=True, bias=True):
    g = torch.Generator().manual_seed(seed + 17 * T + C)
    ty = bc.KINDS[kind]
    return (bc.normal(g, B, T, C).to(ty), bc.normal(g, C, W, std=W ** -0.5), bc.normal(g, C, std=0.1) if bias else None,
            bc.normal(g, B, W - 1, C).to(ty) if state else None, g)


def up(t):
    return None if t is None else t.cuda()


SIZES = [(1, 1, 1), (1, 1, 8), (2, 2, 7), (3, 3, 64), (2, 5, 40), (1, 63, 8), (2, 64, 24), (1, 65, 1000), (3, 130, 33),
         (2, 515, 16), (5, 17, 1032)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", SIZES)
def test_forward(ttt, B, T, C, W, kind):
    x, w, b, s, g = inputs(B, T, C, W, kind, state=T % 2 == 1, bias=C % 2 == 0)
    silu = W != 3
    y, st = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s), activation="silu" if silu else None)
    (yo, ye), so = ob.conv(x, w, b, s, None, silu)
    bc.close("y", y, yo, ye)
    assert torch.equal(st.cpu().double(), so)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [(4, 70, 40, 4), (5, 3, 8, 4), (3, 2, 7, 3), (6, 129, 16, 2)])
def test_padded_batch(ttt, B, T, C, W, kind):
    x, w, b, s, g = inputs(B, T, C, W, kind)
    n = bc.lengths_for(B, T, g)
    for i in range(B):
        x[i, n[i]:] = NAN
    y, st = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s), lengths=n.cuda())
    (yo, ye), so = ob.conv(x, w, b, s, n)
    bc.close("y", y, yo, ye)
    assert torch.equal(st.cpu().double(), so)
    for i in range(B):
        assert not y[i, n[i]:].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [(3, 1000, 8, 4), (5, 777, 3, 4), (2, 300, 64, 2), (3, 130, 250, 3), (7, 50, 12, 4)])
def test_narrow_rows(ttt, B, T, C, W, kind):
    """Few channels: a block takes several pieces of the tokens, of several sequences."""
    x, w, b, s, g = inputs(B, T, C, W, kind)
    n = bc.lengths_for(B, T, g)
    dy, ds = bc.normal(g, B, T, C).to(x.dtype), bc.normal(g, B, W - 1, C).to(x.dtype)
    y, st = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s), lengths=n.cuda())
    (yo, ye), so = ob.conv(x, w, b, s, n)
    bc.close("y", y, yo, ye)
    assert torch.equal(st.cpu().double(), so)
    got = ttt.ttt_conv_backward(x.cuda(), w.cuda(), up(b), dy.cuda(), up(s), ds.cuda(), lengths=n.cuda())
    for name, a, (v, e) in zip(("dx", "dweight", "dbias", "dstate0"), got, ob.conv_backward(x, w, b, dy, s, ds, n)):
        bc.close(name, a, v, e)


def test_lengths_outside_the_batch_are_taken_into_it(ttt):
    x, w, b, s, g = inputs(2, 9, 16, 4, "f32")
    y, st = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s), lengths=torch.tensor([-3, 1000], dtype=torch.int32).cuda())
    whole, st1 = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s))
    assert not y[0].any() and torch.equal(st[0].cpu(), s[0]) and torch.equal(y[1], whole[1]) and torch.equal(st[1], st1[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("before,after", [(0, 40), (8, 8), (3, 2), (40, 1)])
def test_slices_of_wider_rows(ttt, before, after, kind):
    """The same result from a slice as from the rows alone, and nothing beside the slice is read."""
    x, w, b, s, g = inputs(2, 33, 40, 4, kind)
    wide, at = bc.slice_of(x, before, after)
    y, st = ttt.ttt_conv_forward(wide.cuda()[at], w.cuda(), up(b), up(s))
    y1, st1 = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), up(s))
    assert torch.equal(y, y1) and torch.equal(st, st1)
    dy = bc.normal(g, 2, 33, 40).to(x.dtype).cuda()
    one = ttt.ttt_conv_backward(wide.cuda()[at], w.cuda(), up(b), dy, up(s))
    (yo, ye), _ = ob.conv(x, w, b, s)
    bc.close("y", y, yo, ye)
    for name, got, (v, e) in zip(("dx", "dweight", "dbias", "dstate0"), one, ob.conv_backward(x, w, b, dy, s)):
        bc.close(name, got, v, e)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_decode_continues_a_prompt_bit_for_bit(ttt, W, kind):
    """A prompt in one call, and the same tokens as a shorter prompt and then in pieces of 1, 2 and 5 in place."""
    x, w, b, s, g = inputs(3, 40, 24, W, kind)
    xg, wg, bg = x.cuda(), w.cuda(), up(b)
    y, st = ttt.ttt_conv_forward(xg, wg, bg, up(s))
    y0, state = ttt.ttt_conv_forward(xg[:, :30].contiguous(), wg, bg, up(s))
    got, t = [y0], 30
    for k in (1, 2, 1, 5, 1):
        got.append(ttt.ttt_conv_decode(xg[:, t:t + k].contiguous(), wg, bg, state))
        t += k
    assert t == 40 and torch.equal(torch.cat(got, 1), y) and torch.equal(state, st)


def test_forward_in_place_state_and_no_tokens(ttt):
    x, w, b, s, g = inputs(2, 200, 64, 4, "bf16")
    sg = s.cuda()
    y1, st1 = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), sg)
    y2, st2 = ttt.ttt_conv_forward(x.cuda(), w.cuda(), up(b), sg, state_T=sg)
    assert st2 is sg and torch.equal(st1, sg) and torch.equal(y1, y2)
    y, st = ttt.ttt_conv_forward(x[:, :0].cuda(), w.cuda(), up(b), s.cuda())
    assert y.numel() == 0 and torch.equal(st.cpu(), s)
    dx, dw, db, ds = ttt.ttt_conv_backward(x[:, :0].cuda(), w.cuda(), up(b), x[:, :0].cuda(), s.cuda(), s.cuda())
    assert dx.numel() == 0 and not dw.any() and not db.any() and torch.equal(ds.cpu(), s)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", SIZES)
def test_backward(ttt, B, T, C, W, kind):
    x, w, b, s, g = inputs(B, T, C, W, kind, seed=3, state=T % 2 == 1, bias=C % 2 == 0)
    silu = W != 3
    dy = bc.normal(g, B, T, C).to(x.dtype)
    ds = bc.normal(g, B, W - 1, C).to(x.dtype) if T % 3 else None
    got = ttt.ttt_conv_backward(x.cuda(), w.cuda(), up(b), dy.cuda(), up(s), up(ds), activation="silu" if silu else None)
    want = ob.conv_backward(x, w, b, dy, s, ds, None, silu)
    for name, a, (v, e) in zip(("dx", "dweight", "dbias", "dstate0"), got, want):
        if a is not None:
            bc.close(name, a, v, e)
    assert (got[2] is None) == (b is None) and (got[3] is None) == (s is None)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [(4, 70, 40, 4), (5, 3, 8, 4), (3, 2, 7, 3), (6, 129, 16, 2)])
def test_backward_of_a_padded_batch(ttt, B, T, C, W, kind):
    x, w, b, s, g = inputs(B, T, C, W, kind, seed=4)
    dy, ds = bc.normal(g, B, T, C).to(x.dtype), bc.normal(g, B, W - 1, C).to(x.dtype)
    n = bc.lengths_for(B, T, g)
    for i in range(B):
        x[i, n[i]:] = dy[i, n[i]:] = NAN
    got = ttt.ttt_conv_backward(x.cuda(), w.cuda(), up(b), dy.cuda(), up(s), up(ds), lengths=n.cuda())
    for name, a, (v, e) in zip(("dx", "dweight", "dbias", "dstate0"), got, ob.conv_backward(x, w, b, dy, s, ds, n)):
        bc.close(name, a, v, e)


def test_backward_twice_is_the_same(ttt):
    x, w, b, s, g = inputs(4, 1500, 96, 4, "bf16")
    args = (x.cuda(), w.cuda(), up(b), x.cuda(), up(s))
    assert all(torch.equal(p, q) for p, q in zip(ttt.ttt_conv_backward(*args), ttt.ttt_conv_backward(*args)))


def test_offsets_past_32_bits(ttt):
    """2.2e9 elements: the last sequence equals itself alone."""
    B, T, C = 33, 8192, 8192
    x = torch.zeros(B, T, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[-1] = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    w = torch.randn(C, 4, generator=g, device="cuda")
    y, st = ttt.ttt_conv_forward(x, w)
    y1, st1 = ttt.ttt_conv_forward(x[-1:].contiguous(), w)
    assert torch.equal(y[-1:], y1) and torch.equal(st[-1:], st1)


def test_gradient_offsets_past_32_bits(ttt):
    """2.2e9 elements, all but the last sequence zeros: its gradients equal those of itself alone."""
    B, T, C = 33, 8192, 8192
    x = torch.zeros(B, T, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[-1] = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    w = torch.randn(C, 4, generator=g, device="cuda")
    dx, dw, _, _ = ttt.ttt_conv_backward(x, w, None, x)
    one, dw1, _, _ = ttt.ttt_conv_backward(x[-1:].contiguous(), w, None, x[-1:].contiguous())
    assert torch.equal(dx[-1:], one) and not dx[0].any()
    assert torch.allclose(dw, dw1, rtol=1e-4, atol=1e-4 * float(dw1.abs().max()))  # 8192 terms, other pieces of the tokens


def test_refusals_of_the_binding(ttt):
    x, w, b, s, g = inputs(2, 6, 16, 4, "f32")
    x, w, s = x.cuda(), w.cuda(), s.cuda()
    with pytest.raises(ValueError, match="rows at one distance"):
        ttt.ttt_conv_forward(x.transpose(1, 2), torch.zeros(6, 4, device="cuda"))
    with pytest.raises(ValueError, match="rows at one distance"):
        ttt.ttt_conv_forward(torch.cat((x, x), 1)[:, :6], w)
    with pytest.raises(TypeError, match="state0 must be"):
        ttt.ttt_conv_forward(x, w, None, s.bfloat16())
    with pytest.raises(ValueError, match="state0 must be"):
        ttt.ttt_conv_forward(x, w, None, s[:, :2].contiguous())
    with pytest.raises(TypeError, match="lengths must be"):
        ttt.ttt_conv_forward(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ttt.TTTError) as e:
        ttt.ttt_conv_forward(x, torch.zeros(16, 5, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(ttt.TTTError) as e:
        ttt.ttt_conv_decode(x, w, None, s, y=x)
    assert e.value.status == 5
