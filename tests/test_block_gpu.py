"""The operators around the sequence layer as a block runs them together, under graph capture and on other streams.

Two blocks: norm (8 bits) -> 8-bit prologue -> TTT-Linear scan; and norm -> joint projection -> convolution ->
selective scan -> projection out, whole, then as a prompt followed by single tokens, and backwards."""
from __future__ import annotations

import pytest
import torch
import torch.nn.functional as F

import block_cases as bc
import oracle
from oracle import prologue as oracle_prologue

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt(cuda_device):
    from test_sequence_layers_ttt_b200 import _binding
    return _binding


class Block:
    """A selective-scan block in float32: weights, and its pass over the tokens with the state it carries."""

    def __init__(self, ttt, dm=96, C=160, N=16, rank=8, W=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, std: torch.randn(s, generator=g, device="cuda") * std
        self.ttt, self.C, self.N, self.rank, self.W = ttt, C, N, rank, W
        self.p = dict(norm=1 + rnd(dm, std=0.1), inp=rnd(dm, 2 * C, std=dm ** -0.5), cw=rnd(C, W, std=0.5),
                      cb=rnd(C, std=0.1), xp=rnd(C, rank + 2 * N, std=C ** -0.5), dtp=rnd(rank, C, std=rank ** -0.5),
                      dtb=rnd(C, std=0.5) - 3.0, A=-torch.arange(1, N + 1, device="cuda").float().expand(C, N).contiguous(),
                      D=1 + rnd(C, std=0.1), out=rnd(C, dm, std=C ** -0.5))

    def state(self, B):
        return (torch.zeros(B, self.W - 1, self.C, device="cuda"), torch.zeros(B, self.C, self.N, device="cuda"))

    def forward(self, x, res, state, lengths=None):
        p, t = self.p, self.ttt
        y, h = t.ttt_rmsnorm_forward(x, p["norm"], res)
        xz = y @ p["inp"]
        c, s1 = t.ttt_conv_forward(xz[..., :self.C], p["cw"], p["cb"], state[0], lengths=lengths)
        d = c @ p["xp"]
        dt = d[..., :self.rank] @ p["dtp"]
        Bm, Cm = d[..., self.rank:self.rank + self.N], d[..., self.rank + self.N:]
        o, s2 = t.ttt_ssm_forward(c, dt, p["A"], Bm, Cm, p["D"], xz[..., self.C:], p["dtb"], state[1], lengths=lengths)
        self.kept = (h, y, xz, c, dt, d, o)
        return o @ p["out"], h, (s1, s2)

    def token(self, x, res, state):
        p, t = self.p, self.ttt
        y, h = t.ttt_rmsnorm_forward(x, p["norm"], res)
        xz = y @ p["inp"]
        c = t.ttt_conv_decode(xz[..., :self.C], p["cw"], p["cb"], state[0])
        d = c @ p["xp"]
        o = t.ttt_ssm_decode(c, d[..., :self.rank] @ p["dtp"], p["A"], d[..., self.rank:self.rank + self.N],
                             d[..., self.rank + self.N:], state[1], p["D"], xz[..., self.C:], p["dtb"])
        return o @ p["out"], h

    def plain(self, x, res, p):
        """The same block in torch, for autograd in 64 bits."""
        h = x + res
        y = F.rms_norm(h, (h.shape[-1],), p["norm"], 1e-6)
        xz = y @ p["inp"]
        c = F.conv1d(F.pad(xz[..., :self.C].transpose(1, 2), (self.W - 1, 0)), p["cw"][:, None], p["cb"], groups=self.C)
        c = F.silu(c.transpose(1, 2))
        d = c @ p["xp"]
        dt = F.softplus(d[..., :self.rank] @ p["dtp"] + p["dtb"], threshold=1000.0)
        Bm, Cm = d[..., self.rank:self.rank + self.N], d[..., self.rank + self.N:]
        s, ys = torch.zeros(x.shape[0], self.C, self.N, dtype=x.dtype, device=x.device), []
        for t in range(x.shape[1]):
            s = torch.exp(dt[:, t, :, None] * p["A"]) * s + (dt[:, t] * c[:, t])[..., None] * Bm[:, t, None, :]
            ys.append((s * Cm[:, t, None, :]).sum(-1) + p["D"] * c[:, t])
        return (torch.stack(ys, 1) * F.silu(xz[..., self.C:])) @ p["out"], h

    def backward(self, dout, dh):
        """Gradients of sum(out dout) + sum(h dh) after forward, by the library's backward calls."""
        p, t, C, r, N = self.p, self.ttt, self.C, self.rank, self.N
        h, y, xz, c, dt, d, o = self.kept
        g = {"out": o.flatten(0, 1).t() @ dout.flatten(0, 1)}
        s0 = self.state(h.shape[0])
        du, ddt, g["A"], dB, dC, g["D"], dz, g["dtb"], _ = t.ttt_ssm_backward(
            c, dt, p["A"], d[..., r:r + N], d[..., r + N:], dout @ p["out"].t(), p["D"], xz[..., C:], p["dtb"], s0[1])
        g["dtp"] = d[..., :r].flatten(0, 1).t() @ ddt.flatten(0, 1)
        dd = torch.cat((ddt @ p["dtp"].t(), dB, dC), -1)
        g["xp"] = c.flatten(0, 1).t() @ dd.flatten(0, 1)
        dc = du + dd @ p["xp"].t()
        dx, g["cw"], g["cb"], _ = t.ttt_conv_backward(xz[..., :C], p["cw"], p["cb"], dc, s0[0])
        dxz = torch.cat((dx, dz), -1)
        g["inp"] = y.flatten(0, 1).t() @ dxz.flatten(0, 1)
        g["x"], g["norm"] = t.ttt_rmsnorm_backward(h, p["norm"], dxz @ p["inp"].t(), dh)
        return g


def io(B, T, dm=96, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(B, T, dm, generator=g, device="cuda") for _ in range(2))


def near(a, b, tol, name=""):
    """Relative 2-norm error.  The block chains about ten float32 steps of 1e-6 or better each."""
    r = float((a.double() - b.double()).norm() / b.double().norm())
    assert r <= tol, f"{name}: {r:.2e}"


def test_a_prompt_then_single_tokens_equal_the_whole(ttt):
    blk = Block(ttt)
    x, res = io(3, 50)
    whole, hw, sw = blk.forward(x, res, blk.state(3))
    part, h, state = blk.forward(x[:, :40].contiguous(), res[:, :40].contiguous(), blk.state(3))
    outs, hs = [part], [h]
    for t in range(40, 50):
        o, h = blk.token(x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous(), state)
        outs.append(o)
        hs.append(h)
    near(torch.cat(outs, 1), whole, 1e-5, "out")
    near(torch.cat(hs, 1), hw, 1e-7, "h")
    near(state[0], sw[0], 1e-5, "conv state")
    near(state[1], sw[1], 1e-5, "scan state")


def test_a_padded_batch_equals_its_sequences_alone(ttt):
    blk = Block(ttt)
    x, res = io(3, 45)
    n = torch.tensor([45, 0, 19], dtype=torch.int32, device="cuda")
    out, h, (s1, s2) = blk.forward(x, res, blk.state(3), n)
    for b, k in ((0, 45), (2, 19)):
        o, _, (a1, a2) = blk.forward(x[b:b + 1, :k].contiguous(), res[b:b + 1, :k].contiguous(), blk.state(1))
        near(out[b:b + 1, :k], o, 1e-5)
        near(s1[b:b + 1], a1, 1e-5)
        near(s2[b:b + 1], a2, 1e-5)
        assert not out[b, k:].any()
    assert not out[1].any() and not s1[1].any() and not s2[1].any()


def test_gradients_through_the_block(ttt):
    blk = Block(ttt, dm=40, C=48, N=8)
    x, res = io(2, 30, 40)
    out, h, _ = blk.forward(x, res, blk.state(2))
    dout, dh = io(2, 30, 40, seed=2)
    got = blk.backward(dout, dh)
    p = {k: v.double().requires_grad_() for k, v in blk.p.items()}
    xd, rd = x.double().requires_grad_(), res.double()
    o, hd = blk.plain(xd, rd, p)
    ((o * dout).sum() + (hd * dh).sum()).backward()
    near(out, o.detach(), 1e-5, "out")
    for k, v in got.items():
        near(v, xd.grad if k == "x" else p[k].grad, 5e-5, k)


def test_the_ttt_layer_from_8_bits(ttt):
    """norm in 8 bits -> 8-bit prologue -> scan, against the 16-bit path on the values that the 8 bits stand for."""
    B, T, H, dm = 2, 64, 4, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std
    x, res = rnd(B, T, dm).bfloat16(), rnd(B, T, dm).bfloat16()
    q, scale, h = ttt.ttt_rmsnorm_q8_forward(x, torch.ones(dm, device="cuda"), res)
    ws = [ttt.prologue_q8_weights(rnd(H, dm, 64, std=dm ** -0.5)) for _ in range(3)] + [
        ttt.prologue_q8_weights(rnd(H, dm, std=dm ** -0.5))]
    b = rnd(H)
    Q, K, V, eta = ttt.ttt_prologue_q8_forward(q, scale, *(t for w in ws for t in w), b)
    W0, b0 = rnd(1, H, 64, 64, std=0.02).expand(B, -1, -1, -1).contiguous(), torch.zeros(B, H, 64, device="cuda")
    gam, bet = torch.ones(H, 64, device="cuda"), torch.zeros(H, 64, device="cuda")
    Z, W_T, b_T = ttt.ttt_linear_forward(Q, K, V, eta, W0, b0, gam, bet)
    xs = q.float() * scale[..., None]
    y, _ = ttt.ttt_rmsnorm_forward(x, torch.ones(dm, device="cuda"), res)
    near(xs, y, 2.0 ** -4, "8 bits against 16")
    th = [(w.float() * s[..., None]).transpose(1, 2) for w, s in ws[:3]]
    want = [torch.einsum("btm,hmn->bhtn", xs.double(), t.double()) for t in th]
    near(V, want[2], 2.0 ** -8, "V")
    assert torch.isfinite(Z).all() and torch.isfinite(W_T).all()
    again = ttt.ttt_linear_forward(Q, K, V, eta, W0, b0, gam, bet)
    assert torch.equal(Z, again[0])


def test_the_ttt_layer_from_8_bits_against_the_oracles(ttt):
    """The same chain, each link against its float64 oracle on the values that the link before has left: 8 bits to Q, K, V
    within half a bf16 step and the 1e-5 of the prologue's own test, and those to the scan's outputs at its bar for bf16
    inputs, 3e-3 of the RMS."""
    B, T, H, dm = 2, 75, 4, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std
    x, res = rnd(B, T, dm).bfloat16(), rnd(B, T, dm).bfloat16()
    q, scale, _ = ttt.ttt_rmsnorm_q8_forward(x, 1 + rnd(dm, std=0.1), res)
    ws = [ttt.prologue_q8_weights(rnd(H, dm, 64, std=dm ** -0.5)) for _ in range(3)] + [
        ttt.prologue_q8_weights(rnd(H, dm, std=dm ** -0.5))]
    b = rnd(H)
    out = ttt.ttt_prologue_q8_forward(q, scale, *(t for w in ws for t in w), b, pos0=9)
    wide = [(w.cpu().double() * s.cpu().double()[..., None]) for w, s in ws]
    ref = oracle_prologue.project((q.cpu().double() * scale.cpu().double()[..., None]), *(t.transpose(1, 2) for t in wide[:3]), wide[3],
                                  b.cpu(), pos0=9)
    for got, want in zip(out[:3], ref[:3]):
        got, want = got.cpu().double(), torch.as_tensor(want)
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * want.square().mean().sqrt()).all()
    eta = torch.as_tensor(ref[3])
    assert ((out[3].cpu().double() - eta).abs() <= 2e-5 * eta).all()
    W0, b0 = rnd(B, H, 64, 64, std=0.02), rnd(B, H, 64, std=0.02)
    gam, bet = 1 + rnd(H, 64, std=0.1), rnd(H, 64, std=0.1)
    scan = ttt.ttt_linear_forward(*out, W0, b0, gam, bet)
    for got, want in zip(scan, oracle.ttt_linear(*(t.cpu().double().numpy() for t in (*out, W0, b0, gam, bet)), 16)):
        want = torch.as_tensor(want)
        assert (got.cpu().double() - want).abs().max() <= 3e-3 * want.square().mean().sqrt()


def every_call(ttt, i, x, w, cw, q8):
    """One call of every entry point; the outputs in a flat list."""
    h, s = i["h0"].clone(), torch.zeros(x.shape[0], 3, x.shape[2], device="cuda", dtype=x.dtype)
    y, r = ttt.ttt_rmsnorm_forward(x, w, x)
    out = [y, r, *ttt.ttt_rmsnorm_backward(x, w, x), *ttt.ttt_conv_forward(x, cw), *ttt.ttt_conv_backward(x, cw, None, x)]
    q, sc, _ = ttt.ttt_rmsnorm_q8_forward(x, w)
    out += [q.float(), sc, ttt.ttt_conv_decode(x, cw, None, s), s, *ttt.ttt_prologue_q8_forward(*q8)]
    a = (i["u"], i["dt"], i["A"], i["Bm"], i["Cm"])
    out += [*ttt.ttt_ssm_forward(*a, i["D"], i["z"], i["dt_bias"], i["h0"]),
            ttt.ttt_ssm_decode(*a, h, i["D"], i["z"], i["dt_bias"]), h,
            *ttt.ttt_ssm_backward(*a, i["u"], i["D"], i["z"], i["dt_bias"], i["h0"])]
    return [t for t in out if t is not None]


@pytest.fixture(scope="module")
def operands(ttt):
    g = torch.Generator(device="cuda").manual_seed(3)
    i = bc.cuda(bc.ssm_inputs(2, 600, 40, 16, "bf16", seed=1))
    q8 = [t.cuda() for t in _q8(ttt)]
    return i, i["u"], torch.rand(40, generator=g, device="cuda"), torch.randn(40, 4, generator=g, device="cuda"), q8


def _q8(ttt):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(1, 50, 128, generator=g)
    s = x.abs().amax(-1) / 448.0
    ops = [(x / s[..., None]).to(torch.float8_e4m3fn), s]
    for shape in ((4, 128, 64),) * 3 + ((4, 128),):
        ops += ttt.prologue_q8_weights(torch.randn(shape, generator=g))
    return ops + [torch.randn(4, generator=g)]


def test_capture_and_replay_on_new_inputs(ttt, operands):
    """Every call captured into one graph; the graph replayed on other inputs equals plain calls on them."""
    i, x, w, cw, q8 = operands
    i, x = {k: v.clone() for k, v in i.items()}, x.clone()
    i["u"] = x
    every_call(ttt, i, x, w, cw, q8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = every_call(ttt, i, x, w, cw, q8)
    for seed in (5, 6):
        new = bc.cuda(bc.ssm_inputs(2, 600, 40, 16, "bf16", seed=seed))
        for k in i:
            i[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = every_call(ttt, i, x, w, cw, q8)
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_two_streams_at_once(ttt, operands):
    """The calls on two streams at the same time equal the calls one after the other."""
    i, x, w, cw, q8 = operands
    j = bc.cuda(bc.ssm_inputs(2, 600, 40, 16, "bf16", seed=9))
    want = [every_call(ttt, i, x, w, cw, q8), every_call(ttt, j, j["u"], w, cw, q8)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for k, (s, a) in enumerate(zip(streams, ((i, x), (j, j["u"])))):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[k] = every_call(ttt, *a, w, cw, q8)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_stream_given_by_hand(ttt, operands):
    """stream=: the call waits for what that stream holds, and its buffers belong to it."""
    i, x, w, cw, q8 = operands
    s = torch.cuda.Stream()
    a = (i["u"], i["dt"], i["A"], i["Bm"], i["Cm"])
    want = ttt.ttt_ssm_forward(*a, h0=i["h0"]), ttt.ttt_conv_forward(x, cw), ttt.ttt_rmsnorm_forward(x, w)
    torch.cuda.synchronize()
    got = (ttt.ttt_ssm_forward(*a, h0=i["h0"], stream=s), ttt.ttt_conv_forward(x, cw, stream=s),
           ttt.ttt_rmsnorm_forward(x, w, stream=s.cuda_stream))
    s.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(m, n) for m, n in zip(p, q) if m is not None)
