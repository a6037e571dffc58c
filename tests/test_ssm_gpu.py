"""The selective scan kernels against the float64 oracle (oracle/block.py), within the float32 bound that the oracle
carries through the recursion and half a step of the output's type.  Everything that must not be read is NaN."""
from __future__ import annotations

import pytest
import torch

import block_cases as bc
from oracle import block as ob

pytestmark = pytest.mark.gpu
NAN = float("nan")
GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


def forward(ttt, i, **kw):
    return ttt.ttt_ssm_forward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], i.get("D"), i.get("z"), i.get("dt_bias"),
                               i.get("h0"), **kw)


def backward(ttt, i, dy, dh=None, **kw):
    out = ttt.ttt_ssm_backward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], dy, i.get("D"), i.get("z"), i.get("dt_bias"),
                               i.get("h0"), dh, **kw)
    return dict(zip(GRADS, out))


def check_forward(got, i, **kw):
    (yo, ye), (ho, he) = ob.ssm(**i, **kw)
    bc.close("y", got[0], yo, ye)
    bc.close("h_T", got[1], ho, he)


def check_backward(got, i, dy, dh, **kw):
    want = ob.ssm_backward(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], dy, i.get("D"), i.get("z"), i.get("dt_bias"),
                           i.get("h0"), dh, **kw)
    for k, v in got.items():
        if v is not None:
            bc.close(k, v, *want[k])


# states: 1, odd ones, every power of two and one past it; tokens: one, tile borders and their neighbours
SIZES = [(1, 1, 1, 1), (2, 3, 5, 1), (1, 16, 32, 4), (2, 17, 33, 5), (1, 15, 64, 8), (3, 33, 40, 9), (2, 64, 96, 16),
         (1, 100, 31, 16), (1, 65, 130, 17), (2, 48, 20, 32), (1, 50, 36, 33), (1, 31, 70, 64), (2, 200, 12, 16)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", SIZES)
def test_forward(ttt, B, T, C, N, kind):
    i = bc.ssm_inputs(B, T, C, N, kind, seed=T)
    check_forward(forward(ttt, bc.cuda(i)), i)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("missing", [("D",), ("z",), ("dt_bias",), ("h0",), ("D", "z", "h0")])
def test_forward_without_its_options(ttt, missing, kind):
    i = bc.ssm_inputs(2, 21, 36, 16, kind, seed=1)
    if "dt_bias" in missing:
        i["dt"] = (i["dt"].float() - 3.0).to(i["dt"].dtype)
    i = {k: v for k, v in i.items() if k not in missing}
    check_forward(forward(ttt, bc.cuda(i)), i)


def test_forward_without_softplus_and_with_growing_states(ttt):
    i = bc.ssm_inputs(2, 40, 33, 8, "f32", seed=2, softplus=False)
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)
    i["A"] = -0.5 * i["A"]  # states that grow, over decays near 1 and far from it
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)


def test_large_and_small_steps(ttt):
    """Raw steps from -100 (nothing passes, the state stays) to 100 (the state is forgotten at once)."""
    i = bc.ssm_inputs(1, 24, 32, 16, "f32", seed=3)
    i["dt"] = torch.linspace(-100, 100, 24)[None, :, None].expand(1, 24, 32).contiguous()
    check_forward(forward(ttt, bc.cuda(i)), i)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", [(4, 70, 40, 16), (5, 16, 33, 16), (3, 100, 64, 5), (6, 2, 32, 64)])
def test_padded_batch(ttt, B, T, C, N, kind):
    i = bc.ssm_inputs(B, T, C, N, kind, seed=4)
    n = bc.lengths_for(B, T, torch.Generator().manual_seed(5))
    for b in range(B):
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    y, h = forward(ttt, bc.cuda(i), lengths=n.cuda())
    check_forward((y, h), i, lengths=n)
    for b in range(B):
        assert not y[b, n[b]:].any()
    assert torch.equal(h[B // 2].cpu(), i["h0"][B // 2])  # the empty sequence's state


# one sequence of a few tokens, of several tiles, in a cluster; many sequences, with few and many states
@pytest.mark.parametrize("B,T,C,N", [(3, 8, 9, 16), (3, 70, 9, 16), (2, 1100, 8, 5), (40, 70, 33, 16), (40, 70, 9, 20)])
def test_states_that_forget_at_once(ttt, B, T, C, N):
    """A of minus infinity is the limit of large ones: padding and what fills up the last tile still leave the state."""
    i = bc.cuda(bc.ssm_inputs(B, T, C, N, "f32", seed=30))
    n = bc.lengths_for(B, T, torch.Generator().manual_seed(31)).cuda()
    got = []
    for large in (-float("inf"), -1e30):
        i["A"][:, 0] = large
        got.append([*forward(ttt, i, lengths=n), *backward(ttt, i, i["u"], i["h0"], lengths=n).values()])
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_padding_has_zeros_behind_an_infinite_state(ttt):
    i = bc.cuda(bc.ssm_inputs(2, 8, 9, 4, "f32", seed=32))
    i["h0"][:, 3] = float("inf")
    y, _ = forward(ttt, i, lengths=torch.tensor([5, 0], dtype=torch.int32, device="cuda"))
    assert not y[0, 5:].any() and not y[1].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("before,after", [(0, 64), (16, 16), (3, 2)])
def test_slices_of_wider_rows(ttt, before, after, kind):
    i = bc.ssm_inputs(2, 37, 40, 16, kind, seed=6)
    want = forward(ttt, bc.cuda(i))
    c = bc.cuda(i)
    for k in ("u", "dt", "Bm", "Cm", "z"):
        wide, at = bc.slice_of(i[k], before, after)
        c[k] = wide.cuda()[at]
    got = forward(ttt, c)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.Generator().manual_seed(0)
    dy = bc.normal(g, 2, 37, 40).to(i["u"].dtype)
    check_backward(backward(ttt, c, dy.cuda()), i, dy, None)


def test_the_state_goes_in_place(ttt):
    i = bc.cuda(bc.ssm_inputs(3, 300, 64, 16, "bf16", seed=7))
    y, h = forward(ttt, i)
    kept = i["h0"].clone()
    y2, h2 = forward(ttt, i, h_T=i["h0"])
    assert h2 is i["h0"] and torch.equal(h2, h) and torch.equal(y2, y) and not torch.equal(kept, h2)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 6, 16, 40])
def test_decode(ttt, N, kind):
    """Tokens in pieces of 1, 2 and 7 in place, against the oracle over the whole stream."""
    i = bc.ssm_inputs(3, 13, 37, N, kind, seed=8)
    c = bc.cuda(i)
    h, t, ys = c["h0"].clone(), 0, []
    for k in (1, 2, 1, 7, 1, 1):
        p = {n: c[n][:, t:t + k].contiguous() for n in ("u", "dt", "Bm", "Cm", "z")}
        ys.append(ttt.ttt_ssm_decode(p["u"], p["dt"], c["A"], p["Bm"], p["Cm"], h, c["D"], p["z"], c["dt_bias"]))
        t += k
    assert t == 13
    check_forward((torch.cat(ys, 1), h), i)


def test_decode_continues_a_prompt(ttt):
    i = bc.ssm_inputs(2, 80, 64, 16, "f32", seed=9)
    c = bc.cuda(i)
    part = {n: (v[:, :70].contiguous() if n in ("u", "dt", "Bm", "Cm", "z") else v) for n, v in c.items()}
    y, h = forward(ttt, part)
    ys = [y]
    for t in range(70, 80):
        p = {n: c[n][:, t:t + 1].contiguous() for n in ("u", "dt", "Bm", "Cm", "z")}
        ys.append(ttt.ttt_ssm_decode(p["u"], p["dt"], c["A"], p["Bm"], p["Cm"], h, c["D"], p["z"], c["dt_bias"]))
    check_forward((torch.cat(ys, 1), h), i)


def test_no_tokens(ttt):
    i = bc.cuda(bc.ssm_inputs(2, 4, 40, 16, "bf16", seed=10))
    e = {n: (v[:, :0].contiguous() if n in ("u", "dt", "Bm", "Cm", "z") else v) for n, v in i.items()}
    y, h = forward(ttt, e)
    assert y.numel() == 0 and torch.equal(h, i["h0"])
    y, h = forward(ttt, {k: v for k, v in e.items() if k != "h0"})
    assert not h.any()
    out = backward(ttt, e, e["u"], i["h0"])
    assert torch.equal(out["dh0"], i["h0"]) and not out["dA"].any() and not out["dD"].any() and not out["ddt_bias"].any()
    h = i["h0"].clone()
    ttt.ttt_ssm_decode(e["u"], e["dt"], e["A"], e["Bm"], e["Cm"], h)
    assert torch.equal(h, i["h0"])


@pytest.mark.parametrize("B,T,C,N", [(1, 4000, 32, 16), (2, 1111, 70, 16), (1, 1025, 8, 3), (1, 2048, 20, 64)])
def test_few_rows_long(ttt, B, T, C, N):
    """Few channels and a long sequence: the sequence is worked on in pieces."""
    i = bc.ssm_inputs(B, T, C, N, "f32", seed=11)
    check_forward(forward(ttt, bc.cuda(i)), i)


def test_few_rows_long_padded(ttt):
    B, T = 3, 1500
    i = bc.ssm_inputs(B, T, 40, 16, "bf16", seed=12)
    n = torch.tensor([T, 0, 777], dtype=torch.int32)
    for b in range(B):
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    check_forward(forward(ttt, bc.cuda(i), lengths=n.cuda()), i, lengths=n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,C,N", [(1, 3, 16), (3, 40, 16), (2, 100, 5), (3, 33, 40)])
def test_few_rows_in_parts_with_the_state_in_place(ttt, B, C, N, kind):
    """Several parts of the tokens, ragged ones, in a cluster; h_T takes h0's place."""
    T = 1100
    i = bc.ssm_inputs(B, T, C, N, kind, seed=23)
    n = torch.tensor([T, 130, 1000][:B], dtype=torch.int32)
    c = bc.cuda(i)
    y, h = forward(ttt, c, h_T=c["h0"], lengths=n.cuda())
    assert h is c["h0"]
    check_forward((y, h), i, lengths=n)
    again = forward(ttt, bc.cuda(i), lengths=n.cuda())
    assert torch.equal(y, again[0]) and torch.equal(h, again[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", [(3, 1, 40, 16), (4, 8, 37, 5), (4, 9, 37, 5), (40, 24, 40, 16), (40, 25, 40, 16),
                                     (40, 24, 33, 64), (40, 70, 36, 64), (39, 90, 33, 7)])
def test_few_tokens_and_many_rows(ttt, B, T, C, N, kind):
    """On both sides of the sizes at which another kernel takes the call: padded, with the state in place, and from zero."""
    i = bc.ssm_inputs(B, T, C, N, kind, seed=26)
    n = bc.lengths_for(B, T, torch.Generator().manual_seed(27))
    for b in range(B):
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    c = bc.cuda(i)
    y, h = forward(ttt, c, h_T=c["h0"], lengths=n.cuda())
    check_forward((y, h), i, lengths=n)
    for b in range(B):
        assert not y[b, n[b]:].any()
    i.pop("h0")
    check_forward(forward(ttt, bc.cuda(i), lengths=n.cuda()), i, lengths=n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", [(20, 300, 64, 64), (38, 300, 32, 33), (70, 290, 20, 20)])
def test_more_than_16_states_in_parts(ttt, B, T, C, N, kind):
    """32 channels a block and the tokens shared out in clusters of two or four blocks: padded, with the state in place."""
    i = bc.ssm_inputs(B, T, C, N, kind, seed=33)
    n = bc.lengths_for(B, T, torch.Generator().manual_seed(34))
    for b in range(B):
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    c = bc.cuda(i)
    y, h = forward(ttt, c, h_T=c["h0"], lengths=n.cuda())
    assert h is c["h0"]
    check_forward((y, h), i, lengths=n)


def test_few_rows_in_parts_of_growing_states(ttt):
    i = bc.ssm_inputs(1, 600, 20, 8, "f32", seed=24, softplus=False)
    i["A"] = -0.02 * i["A"]
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)
    # a decay that overflows over a part, and nothing for it to carry: zeros, no NaN
    i = {k: torch.zeros_like(v) for k, v in bc.ssm_inputs(1, 8192, 8, 4, "f32", seed=25).items()}
    i["A"], i["dt"] = i["A"] + 1.0, i["dt"] + 1.0
    y, h = forward(ttt, bc.cuda(i), dt_softplus=False)
    assert not y.any() and not h.any()


def growing(B, T, C, N, steps, state=0.0, seed=28):
    """States that grow by e^steps[t] a token, fed by nothing; `state`: the first one's size."""
    i = bc.ssm_inputs(B, T, C, N, "f32", seed=seed, softplus=False)
    i["A"], i["dt_bias"] = torch.ones(C, N), torch.zeros(C)
    i["dt"] = steps[None, :, None].expand(B, T, C).contiguous()
    i["u"], i["h0"] = torch.zeros(B, T, C), state * i["h0"]
    return i


# the kernels for a few tokens, for few channels (one block a row, and a cluster), for more, and for many states
@pytest.mark.parametrize("B,T,C,N", [(1, 8, 9, 16), (1, 60, 9, 16), (1, 700, 8, 5), (40, 60, 9, 16), (40, 60, 9, 20), (20, 300, 9, 33)])
def test_growth_that_overflows_over_tokens_of_an_empty_state(ttt, B, T, C, N):
    """e^6 a token: nothing before the last tokens' inputs, and nothing but zeros without them."""
    i = growing(B, T, C, N, torch.full((T,), 6.0))
    y, h = forward(ttt, bc.cuda(i), dt_softplus=False)
    assert not y.any() and not h.any()
    i["u"][:, -5:] = bc.normal(torch.Generator().manual_seed(29), B, 5, C)
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)


@pytest.mark.parametrize("B,T,C,N,step,at", [(1, 26, 9, 16, 5.6, (0, 26)), (40, 26, 9, 20, 5.6, (0, 26)), (40, 26, 9, 16, 5.6, (0, 26)),
                                             (1, 1024, 8, 5, 0.7, (128, 300))])
def test_growth_that_overflows_over_tokens_of_a_tiny_state(ttt, B, T, C, N, step, at):
    """A state of 1e-30 grows into ordinary numbers, though its decay over a piece of the tokens passes the largest float."""
    steps = torch.zeros(T)
    steps[slice(*at)] = step
    i = growing(B, T, C, N, steps, state=1e-30)
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)


@pytest.mark.parametrize("B,T,C,N", [(1, 8, 9, 16), (1, 60, 9, 16), (1, 700, 8, 5), (40, 60, 9, 16), (40, 60, 9, 20)])
def test_growth_by_a_little_a_token(ttt, B, T, C, N):
    """Growth just inside the decays near 1 (2^(1/16)), the same every token: an error of the decay would add up."""
    i = growing(B, T, C, N, torch.full((T,), 0.043), state=1.0)
    check_forward(forward(ttt, bc.cuda(i), dt_softplus=False), i, softplus=False)
    dy = torch.zeros(B, T, C)
    dy[:, -1] = 1.0
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dt_softplus=False), i, dy, None, softplus=False)


def test_backward_of_growth_that_overflows_over_a_part(ttt):
    """The time axis in parts of 32 tokens: e^3 a token over the first 40, then a state that stays."""
    B, T, C, N = 1, 2048, 8, 4
    steps = torch.zeros(T)
    steps[:40] = 3.0
    i = growing(B, T, C, N, steps, state=1e-30)
    dy = torch.zeros(B, T, C)
    dy[:, -1] = 1e-30
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dt_softplus=False), i, dy, None, softplus=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", SIZES)
def test_backward(ttt, B, T, C, N, kind):
    i = bc.ssm_inputs(B, T, C, N, kind, seed=100 + T)
    g = torch.Generator().manual_seed(T)
    dy, dh = bc.normal(g, B, T, C).to(i["u"].dtype), bc.normal(g, B, C, N)
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dh.cuda()), i, dy, dh)


@pytest.mark.parametrize("missing", [("D",), ("z",), ("dt_bias",), ("h0",), ("D", "z", "h0")])
def test_backward_without_its_options(ttt, missing):
    i = bc.ssm_inputs(2, 21, 36, 16, "f32", seed=13)
    if "dt_bias" in missing:
        i["dt"] -= 3.0
    i = {k: v for k, v in i.items() if k not in missing}
    dy = bc.normal(torch.Generator().manual_seed(1), 2, 21, 36)
    out = backward(ttt, bc.cuda(i), dy.cuda())
    check_backward(out, i, dy, None)
    for leaf, grad in (("D", "dD"), ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        assert (out[grad] is None) == (leaf in missing)


def test_backward_without_softplus(ttt):
    i = bc.ssm_inputs(2, 40, 33, 8, "f32", seed=14, softplus=False)
    dy = bc.normal(torch.Generator().manual_seed(1), 2, 40, 33)
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dt_softplus=False), i, dy, None, softplus=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,N", [(4, 70, 40, 16), (5, 16, 33, 16), (3, 100, 64, 5), (6, 2, 32, 64)])
def test_backward_of_a_padded_batch(ttt, B, T, C, N, kind):
    i = bc.ssm_inputs(B, T, C, N, kind, seed=15)
    g = torch.Generator().manual_seed(5)
    n = bc.lengths_for(B, T, g)
    dy, dh = bc.normal(g, B, T, C).to(i["u"].dtype), bc.normal(g, B, C, N)
    for b in range(B):
        dy[b, n[b]:] = NAN
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    out = backward(ttt, bc.cuda(i), dy.cuda(), dh.cuda(), lengths=n.cuda())
    check_backward(out, i, dy, dh, lengths=n)
    for b in range(B):
        for k in ("du", "ddt", "dz", "dB", "dC"):
            assert not out[k][b, n[b]:].any(), k


@pytest.mark.parametrize("B,T,C,N", [(1, 1500, 40, 16), (1, 700, 20, 33)])
def test_backward_few_rows_long(ttt, B, T, C, N):
    i = bc.ssm_inputs(B, T, C, N, "f32", seed=16)
    g = torch.Generator().manual_seed(6)
    dy, dh = bc.normal(g, B, T, C), bc.normal(g, B, C, N)
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dh.cuda()), i, dy, dh)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("C,N", [(40, 16), (37, 3), (32, 30), (9, 64)])
def test_backward_in_parts_of_a_padded_batch(ttt, C, N, kind):
    """Few channels and hundreds of tokens: the time axis is split; sequences end in its first, a middle and its last part."""
    B, T = 4, 333
    i = bc.ssm_inputs(B, T, C, N, kind, seed=18)
    g = torch.Generator().manual_seed(19)
    n = torch.tensor([T, 0, 5, 170], dtype=torch.int32)
    dy, dh = bc.normal(g, B, T, C).to(i["u"].dtype), bc.normal(g, B, C, N)
    for b in range(B):
        dy[b, n[b]:] = NAN
        for k in ("u", "dt", "Bm", "Cm", "z"):
            i[k][b, n[b]:] = NAN
    out = backward(ttt, bc.cuda(i), dy.cuda(), dh.cuda(), lengths=n.cuda())
    check_backward(out, i, dy, dh, lengths=n)
    for b in range(B):
        for k in ("du", "ddt", "dz", "dB", "dC"):
            assert not out[k][b, n[b]:].any(), k


def test_backward_in_parts_of_growing_states(ttt):
    i = bc.ssm_inputs(1, 200, 33, 8, "f32", seed=20, softplus=False)
    i["A"] = -0.05 * i["A"]
    dy = bc.normal(torch.Generator().manual_seed(21), 1, 200, 33)
    check_backward(backward(ttt, bc.cuda(i), dy.cuda(), dt_softplus=False), i, dy, None, softplus=False)
    # a decay that overflows over a part, and nothing for it to carry: zeros, no NaN
    i = {k: torch.zeros_like(v) for k, v in bc.ssm_inputs(1, 8192, 8, 4, "f32", seed=22).items()}
    i["A"], i["dt"] = i["A"] + 1.0, i["dt"] + 1.0
    out = backward(ttt, bc.cuda(i), torch.zeros(1, 8192, 8, device="cuda"), dt_softplus=False)
    assert all(not v.any() for v in out.values())


def test_backward_twice_is_the_same(ttt):
    i = bc.cuda(bc.ssm_inputs(3, 300, 200, 16, "bf16", seed=17))
    one, two = backward(ttt, i, i["u"]), backward(ttt, i, i["u"])
    assert all(torch.equal(one[k], two[k]) for k in GRADS)


def test_offsets_past_32_bits(ttt):
    """2.2e9 elements: the last sequence equals itself alone."""
    B, T, C, N = 66, 4096, 8192, 2
    u = torch.zeros(B, T, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    u[-1] = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    dt = torch.full_like(u, -2.0)
    Bm = torch.randn(B, T, N, generator=g, device="cuda").bfloat16()
    A = -torch.ones(C, N, device="cuda")
    y, h = ttt.ttt_ssm_forward(u, dt, A, Bm, Bm)
    last = {"u": u[-1:].contiguous(), "dt": dt[-1:].contiguous(), "A": A, "Bm": Bm[-1:].contiguous(), "Cm": Bm[-1:].contiguous()}
    del u, dt
    ya, ha = forward(ttt, last)
    assert torch.allclose(y[-1:].float(), ya.float(), rtol=2 ** -7, atol=1e-5) and torch.allclose(h[-1:], ha, rtol=1e-4, atol=1e-6)


def test_gradient_offsets_past_32_bits(ttt):
    """2.2e9 elements, all but the last sequence zeros: its gradients equal those of itself alone."""
    B, T, C, N = 66, 4096, 8192, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    u = torch.zeros(B, T, C, dtype=torch.bfloat16, device="cuda")
    u[-1] = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    dt = torch.full_like(u, -2.0)
    Bm = torch.randn(B, T, N, generator=g, device="cuda").bfloat16()
    A = -torch.ones(C, N, device="cuda")
    alone = backward(ttt, {"u": u[-1:].contiguous(), "dt": dt[-1:].contiguous(), "A": A, "Bm": Bm[-1:].contiguous(),
                           "Cm": Bm[-1:].contiguous()}, u[-1:].contiguous())
    whole = backward(ttt, {"u": u, "dt": dt, "A": A, "Bm": Bm, "Cm": Bm}, u)
    for k, v in alone.items():
        if v is not None:
            got = whole[k] if k == "dA" else whole[k][-1:]
            # rows are rounded to bf16 once each; sums go by other parts of the time axis
            assert torch.allclose(got.float(), v.float(), rtol=2 ** -7, atol=1e-4 * float(v.float().abs().max())), k
            assert k == "dA" or not whole[k][0].any(), k


def test_refusals_of_the_binding(ttt):
    i = bc.cuda(bc.ssm_inputs(2, 6, 16, 4, "f32", seed=18))
    with pytest.raises(TypeError, match="Bm must be"):
        forward(ttt, {**i, "Bm": i["Bm"].bfloat16()})
    with pytest.raises(ValueError, match="Cm must be"):
        forward(ttt, {**i, "Cm": i["Cm"][:, :, :3]})
    with pytest.raises(ValueError, match="A must be"):
        forward(ttt, {**i, "A": i["A"][:8]})
    with pytest.raises(ValueError, match="rows at one distance"):
        forward(ttt, {**i, "u": torch.cat((i["u"], i["u"]), 1)[:, :6]})
    with pytest.raises(ValueError, match="dy must be"):
        backward(ttt, i, i["u"][:, :5])
    with pytest.raises(ttt.TTTError) as e:
        forward(ttt, i, y=i["z"])
    assert e.value.status == 5
    with pytest.raises(ttt.TTTError) as e:
        backward(ttt, i, i["u"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 9
