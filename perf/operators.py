"""The operators around the sequence layer, case by case: their inputs, their plain form, their definition in 64 bits.

Four operators of a layer's block, in the order in which a block runs them:

norm      h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight, with y in the input's type, or in 8 bits
          (e4m3) with one scale a token; and its gradient
prologue  the layer's projections, learning-rate gate and rotary embedding from such an 8-bit y and 8-bit weights
conv      the short causal depthwise convolution with its SiLU, for prompts (padded batches, a carried state),
          for single tokens, and its gradient
ssm       the selective state space scan  h_t = exp(dt_t A) h_{t-1} + dt_t B_t u_t,  y_t = C_t h_t + D u_t, gated
          by silu(z_t), for prompts, for single tokens, and its gradient

`run` computes a pass in elementary torch operations in 32 bits, or, where `own` is true, by the library's calls.
`exact` gives the definition in 64 bits, one token after the other.
"""
import math

import torch

own = False

EPS = 1e-6
ROPE = 10000.0
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100  # the scale of a token of zeros
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # The input norm of the 1.3B-class layer over two sequences of 32k tokens, with the residual stream, its output
        # in 8 bits for the projections.
        {"name": "norm_q8_32k", "op": "norm", "way": "q8", "B": 2, "T": 32768, "d": 2048, "type": "bf16", "residual": True},
        # One token for each of eight streams of the 125M-class layer: launch latency is all there is.
        {"name": "norm_token", "op": "norm", "way": "forward", "B": 8, "T": 1, "d": 768, "type": "bf16", "residual": True},
        # The norm's gradient in a training step in 32 bits at a width that is no multiple of eight.
        {"name": "norm_backward_f32", "op": "norm", "way": "backward", "B": 3, "T": 2731, "d": 2047, "type": "f32", "residual": True},
        # The projections of the 1.3B-class layer over two sequences of 32k tokens, 8-bit operands.
        {"name": "prologue_q8_32k", "op": "prologue", "way": "q8", "B": 2, "T": 32768, "H": 32, "dm": 2048, "pos0": 0},
        # A continued piece of eight ragged streams at the 125M-class width: row tiles that end inside a stream.
        {"name": "prologue_q8_piece", "op": "prologue", "way": "q8", "B": 8, "T": 77, "H": 12, "dm": 768, "pos0": 1971},
        # The convolution of a 32k prompt; x is half of the joint projection's output.
        {"name": "conv_32k", "op": "conv", "way": "forward", "B": 2, "T": 32768, "C": 2048, "W": 4, "type": "bf16", "padded": False},
        # Its gradient in a training step of the 125M-class layer, expanded twice.
        {"name": "conv_backward_2k", "op": "conv", "way": "backward", "B": 8, "T": 2048, "C": 1536, "W": 4, "type": "bf16", "padded": False},
        # One token of 64 streams through the convolution, its state updated in place.
        {"name": "conv_token", "op": "conv", "way": "decode", "B": 64, "T": 1, "C": 2048, "W": 4, "type": "bf16", "padded": False},
        # The scan over a 32k prompt of the 1.3B-class width, gated; B and C are slices of one projection.
        {"name": "ssm_32k", "op": "ssm", "way": "forward", "B": 2, "T": 32768, "C": 2048, "N": 16, "type": "bf16", "padded": False},
        # A padded batch of prompts of a small model in 32 bits: few channels, so few rows to share out, an odd width.
        {"name": "ssm_padded_f32", "op": "ssm", "way": "forward", "B": 5, "T": 3001, "C": 203, "N": 16, "type": "f32", "padded": True},
        # The scan's gradient in a training step of the 125M-class layer, expanded twice.
        {"name": "ssm_backward_2k", "op": "ssm", "way": "backward", "B": 8, "T": 2048, "C": 1536, "N": 16, "type": "bf16", "padded": False},
        # One token of 64 streams through the scan, its state updated in place.
        {"name": "ssm_token", "op": "ssm", "way": "decode", "B": 64, "T": 1, "C": 2048, "N": 16, "type": "bf16", "padded": False},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "prologue", "conv", "ssm", "ssm"))
    kind = rng.choice(("bf16", "f32"))
    B = _between(rng, 1, 64)
    if op == "norm":
        way = rng.choice(("forward", "q8", "backward"))
        d = _between(rng, 1, 16384)
        if rng.random() < 0.5:
            d = (d + 63) // 64 * 64
        T = _between(rng, 1, max(1, min(32768, (1 << 26) // (B * d))))
        return {"op": op, "way": way, "B": B, "T": T, "d": d, "type": kind, "residual": rng.random() < 0.7}
    if op == "prologue":
        H, dm = 4 * _between(rng, 1, 16), 16 * _between(rng, 4, 160)
        T = _between(rng, 1, max(1, min(32768, (1 << 34) // (B * H * 64 * dm))))
        return {"op": op, "way": "q8", "B": B, "T": T, "H": H, "dm": dm, "pos0": rng.choice((0, _between(rng, 1, 100000)))}
    way = rng.choice(("forward", "backward", "decode"))
    C = _between(rng, 1, 8192)
    if rng.random() < 0.5:
        C = (C + 63) // 64 * 64
    if op == "conv":
        T = rng.choice((1, _between(rng, 1, 8))) if way == "decode" else _between(rng, 1, max(1, min(32768, (1 << 26) // (B * C))))
        return {"op": op, "way": way, "B": B, "T": T, "C": C, "W": rng.choice((2, 3, 4)), "type": kind, "padded": way != "decode" and rng.random() < 0.5}
    N = rng.choice((16, 16, _between(rng, 1, 64)))
    T = rng.choice((1, _between(rng, 1, 8))) if way == "decode" else _between(rng, 1, max(1, min(4096, (1 << 28) // (B * C * N))))
    return {"op": op, "way": way, "B": B, "T": T, "C": C, "N": N, "type": kind, "padded": way != "decode" and rng.random() < 0.5}


def work(case):
    """Bytes: every input once, every output once. flops: multiplications, additions and functions of the formulas."""
    B, T = case["B"], case["T"]
    if case["op"] == "prologue":
        H, dm = case["H"], case["dm"]
        cols = 3 * H * 64 + H
        return {"bytes": B * T * (dm + 4 + H * (3 * 64 * 2 + 4)) + cols * (dm + 4), "flops": 2 * B * T * dm * cols}
    e = 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        n, d, r = B * T * case["d"], case["d"], case["residual"]
        if case["way"] == "backward":
            return {"bytes": n * e * (4 if r else 3) + 8 * d, "flops": 12 * n}
        return {"bytes": n * e * (3 if r else 1) + n * (1 if case["way"] == "q8" else e) + 4 * d + (4 * B * T if case["way"] == "q8" else 0), "flops": 6 * n}
    n, C, way = B * T * case["C"], case["C"], case["way"]
    if case["op"] == "conv":
        W = case["W"]
        state = 2 * B * (W - 1) * C * e
        if way == "backward":
            return {"bytes": 3 * n * e + 2 * state + 8 * C * (W + 1), "flops": n * (6 * W + 12)}
        return {"bytes": 2 * n * e + state + 4 * C * (W + 1), "flops": n * (2 * W + 5)}
    N = case["N"]
    small = 4 * C * (N + 2) + 8 * B * C * N  # A, D, dt_bias; the state read and written
    if way == "backward":
        return {"bytes": n * e * 7 + 2 * B * T * N * (e + 4) + 2 * small, "flops": n * (20 * N + 40)}
    return {"bytes": n * e * 4 + 2 * B * T * N * e + small, "flops": n * (7 * N + 20)}


# ---------------------------------------------------------------- what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    B, T = case["B"], case["T"]
    s = dict(case)
    if case["op"] == "prologue":
        H, dm = case["H"], case["dm"]
        s["x"], s["x_scale"] = _q8(normal(B, T, dm))
        for name in ("q", "k", "v"):
            s["theta_" + name], s["scale_" + name] = _q8(normal(H, 64, dm, std=dm ** -0.5))
        s["theta_lr"], s["scale_lr"] = _q8(normal(H, dm, std=dm ** -0.5))
        s["b_lr"] = normal(H)
        s["out"] = [torch.empty((B, H, T, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3)] + [
            torch.empty((B, H, T), device="cuda")]
        return s
    kind = TYPES[case["type"]]
    if case["op"] == "norm":
        d = case["d"]
        s["weight"] = 1.0 + normal(d, std=0.1)
        s["x"] = normal(B, T, d).to(kind)
        s["residual"] = (normal(B, T, d, std=3.0)).to(kind) if case["residual"] else None
        if case["way"] == "backward":
            s["dy"] = normal(B, T, d, std=0.01).to(kind)
        return s
    C = case["C"]
    s["lengths"] = None
    if case["padded"]:  # one sequence fills the batch's length, one is empty where there are more than two
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        if B > 2:
            n[B // 2] = 0
        s["lengths"] = n
    joint = normal(B, T, 2 * C).to(kind)  # the joint projection: its first half goes on, its second half gates
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = joint[..., :C]
        s["weight"], s["bias"] = normal(C, W, std=W ** -0.5), normal(C, std=0.1)
        s["state"] = normal(B, W - 1, C).to(kind)
        if case["way"] == "backward":
            s["dy"] = normal(B, T, C, std=0.01).to(kind)
            s["dstate"] = normal(B, W - 1, C, std=0.01).to(kind)
        return s
    N = case["N"]
    u = normal(B, T, C)
    s["u"] = (u * torch.sigmoid(u)).to(kind)  # what the convolution's SiLU leaves
    s["dt"] = normal(B, T, C, std=0.5).to(kind)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(C, N, std=0.1))
    rank = 8 * ((C // 16 + 7) // 8)  # the low-rank part of the projection that B and C are slices of
    both = normal(B, T, rank + 2 * N).to(kind)
    s["Bm"], s["Cm"] = both[..., rank:rank + N], both[..., rank + N:]
    s["D"] = 1.0 + normal(C, std=0.1)
    s["z"] = joint[..., C:]
    s["h0"] = normal(B, C, N)
    if case["way"] == "backward":
        s["dy"] = normal(B, T, C, std=0.01).to(kind)
        s["dhT"] = normal(B, C, N, std=0.01)
    return s


def _q8(x):
    """Rows of x in e4m3 with a scale each."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from test_sequence_layers_ttt_b200 import _binding as ttt

    op, way = s["op"], s["way"]
    if op == "norm":
        if way == "q8":
            q, scale, h = ttt.ttt_rmsnorm_q8_forward(s["x"], s["weight"], s["residual"], eps=EPS)
            return {"q": q, "scale": scale, "h": h}
        if way == "forward":
            y, h = ttt.ttt_rmsnorm_forward(s["x"], s["weight"], s["residual"], eps=EPS)
            return {"y": y, "h": h}
        dx, dw = ttt.ttt_rmsnorm_backward(s["x"], s["weight"], s["dy"], s["residual"], eps=EPS)
        return {"dx": dx, "dweight": dw}
    if op == "prologue":
        Q, K, V, eta = ttt.ttt_prologue_q8_forward(
            s["x"], s["x_scale"], s["theta_q"], s["scale_q"], s["theta_k"], s["scale_k"], s["theta_v"], s["scale_v"],
            s["theta_lr"], s["scale_lr"], s["b_lr"], pos0=s["pos0"], rope_base=ROPE, out=s["out"])
        return {"Q": Q, "K": K, "V": V, "eta": eta}
    if op == "conv":
        if way == "forward":
            y, state = ttt.ttt_conv_forward(s["x"], s["weight"], s["bias"], s["state"], lengths=s["lengths"])
            return {"y": y, "state": state}
        if way == "decode":
            state = s["state"].clone()  # the same state at every pass; a program decodes on in place
            return {"y": ttt.ttt_conv_decode(s["x"], s["weight"], s["bias"], state), "state": state}
        dx, dw, db, d0 = ttt.ttt_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], s["state"], s["dstate"],
                                               lengths=s["lengths"])
        return {"dx": dx, "dweight": dw, "dbias": db, "dstate0": d0}
    if way == "forward":
        y, hT = ttt.ttt_ssm_forward(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["h0"],
                                    lengths=s["lengths"])
        return {"y": y, "hT": hT}
    if way == "decode":
        h = s["h0"].clone()
        y = ttt.ttt_ssm_decode(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], h, s["D"], s["z"], s["dt_bias"])
        return {"y": y, "hT": h}
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
    return dict(zip(names, ttt.ttt_ssm_backward(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], s["D"], s["z"],
                                                s["dt_bias"], s["h0"], s["dhT"], lengths=s["lengths"])))


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm_backward(s) if s["way"] == "backward" else _plain_norm(s)
    if s["op"] == "prologue":
        return _plain_prologue(s)
    if s["op"] == "conv":
        return _plain_conv_backward(s) if s["way"] == "backward" else _plain_conv(s)
    return _plain_ssm_backward(s) if s["way"] == "backward" else _plain_ssm(s)


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    stream = None if s["residual"] is None else h.to(s["x"].dtype)
    if s["way"] == "forward":
        return {"y": y.to(s["x"].dtype), "h": stream}
    q, scale = _q8(y)
    return {"q": q, "scale": scale, "h": stream}


def _plain_norm_backward(s):
    """x is the normed stream h; the residual is the gradient that comes to h past the norm."""
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    xhat, wdy = h * r, dy * s["weight"]
    dx = r * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum((0, 1))}


def _rotate(x, pos0):
    """Features i and i + 32 of each head turn together by position * base^(-i / 32), the angle in 64 bits."""
    T = x.shape[-2]
    pos = torch.arange(pos0, pos0 + T, device=x.device, dtype=torch.float64)
    angle = pos[:, None] * ROPE ** (-torch.arange(32, device=x.device, dtype=torch.float64) / 32)
    c, n = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * c - b * n, b * c + a * n), -1)


def _plain_prologue(s):
    B, T, H = s["B"], s["T"], s["H"]
    x = (s["x"].float() * s["x_scale"][..., None]).reshape(B * T, -1)

    def heads(name):
        w = (s["theta_" + name].float() * s["scale_" + name][..., None]).reshape(H * 64, -1)
        return (x @ w.t()).reshape(B, T, H, 64).transpose(1, 2)

    logit = x @ (s["theta_lr"].float() * s["scale_lr"][:, None]).t() + s["b_lr"]
    eta = (1.0 / (1.0 + torch.exp(-logit)) / 64).reshape(B, T, H).transpose(1, 2).contiguous()
    Q, K, V = (t.to(torch.bfloat16).contiguous() for t in (_rotate(heads("q"), s["pos0"]), _rotate(heads("k"), s["pos0"]), heads("v")))
    return {"Q": Q, "K": K, "V": V, "eta": eta}


def _padding(s, T):
    """[B, T, 1]: which tokens are padding."""
    t = torch.arange(T, device=s["lengths"].device)
    return (t[None, :] >= s["lengths"][:, None])[..., None]


def _last_rows(s, window, W):
    """The W - 1 rows before each sequence's end, of the window's rows (the state, then x)."""
    n = torch.full((s["B"],), s["T"], device=window.device) if s["lengths"] is None else s["lengths"].long()
    at = n[:, None] + torch.arange(W - 1, device=window.device)
    return window[torch.arange(s["B"], device=window.device)[:, None], at]


def _plain_conv(s):
    W, T = s["W"], s["T"]
    window = torch.cat((s["state"], s["x"]), 1)
    pre = s["bias"] + sum(window[:, j:j + T].float() * s["weight"][:, j] for j in range(W))
    y = pre / (1.0 + torch.exp(-pre))
    if s["lengths"] is not None:
        y = torch.where(_padding(s, T), 0.0, y)
    return {"y": y.to(s["x"].dtype), "state": _last_rows(s, window, W)}


def _plain_conv_backward(s):
    W, T, B = s["W"], s["T"], s["B"]
    window = torch.cat((s["state"], s["x"]), 1).float()
    pre = s["bias"] + sum(window[:, j:j + T] * s["weight"][:, j] for j in range(W))
    sig = 1.0 / (1.0 + torch.exp(-pre))
    dpre = s["dy"].float() * sig * (1.0 + pre * (1.0 - sig))
    if s["lengths"] is not None:
        dpre = torch.where(_padding(s, T), 0.0, dpre)
    dwindow = torch.zeros_like(window)
    for j in range(W):
        dwindow[:, j:j + T] += dpre * s["weight"][:, j]
    n = torch.full((B,), T, device=window.device) if s["lengths"] is None else s["lengths"].long()
    at = n[:, None] + torch.arange(W - 1, device=window.device)
    dwindow[torch.arange(B, device=window.device)[:, None], at] += s["dstate"].float()
    dweight = torch.stack([(dpre * window[:, j:j + T]).sum((0, 1)) for j in range(W)], -1)
    kind = s["x"].dtype
    return {"dx": dwindow[:, W - 1:].to(kind), "dweight": dweight, "dbias": dpre.sum((0, 1)), "dstate0": dwindow[:, :W - 1].to(kind)}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 with h before it zero, by doubling the span that each place has taken in."""
    T, step = a.shape[1], 1
    while step < T:
        b = torch.cat((b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]), 1)
        if 2 * step < T:
            a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return b


def _ssm_parts(s):
    """The step (zero at padding, so that the state passes it unchanged), u, the decay and the state after every token.
    For the gradient in 64 bits: dA and ddt_bias are sums over all tokens of products of two such recursions, whose
    terms nearly cancel, and the roundings of a thousand decays close to one show in them."""
    wide = torch.float64 if s["way"] == "backward" else torch.float32
    raw = s["dt"].to(wide) + s["dt_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    u, Bm, Cm = s["u"].to(wide), s["Bm"].to(wide), s["Cm"].to(wide)
    if s["lengths"] is not None:
        pad = _padding(s, s["T"])
        dt, u, Bm, Cm = (torch.where(pad, 0.0, t) for t in (dt, u, Bm, Cm))
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * u)[..., None] * Bm[:, :, None, :]
    b[:, 0] += a[:, 0] * s["h0"]
    return raw, dt, u, Bm, Cm, a, _scan(a, b)


def _plain_ssm(s):
    raw, dt, u, Bm, Cm, a, h = _ssm_parts(s)
    z = s["z"].float()
    y = ((h * Cm[:, :, None, :]).sum(-1) + u * s["D"]) * z / (1.0 + torch.exp(-z))
    if s["lengths"] is not None:
        y = torch.where(_padding(s, s["T"]), 0.0, y)
    return {"y": y.to(s["u"].dtype), "hT": h[:, -1].contiguous()}


def _plain_ssm_backward(s):
    raw, dt, u, Bm, Cm, a, h = _ssm_parts(s)
    kind, z, dy = s["u"].dtype, s["z"].double(), s["dy"].double()
    if s["lengths"] is not None:
        pad = _padding(s, s["T"])
        z, dy, raw = (torch.where(pad, 0.0, t) for t in (z, dy, raw))
    sig = 1.0 / (1.0 + torch.exp(-z))
    y = (h * Cm[:, :, None, :]).sum(-1) + u * s["D"]
    dz = dy * y * sig * (1.0 + z * (1.0 - sig))
    dy = dy * z * sig
    dC = (h * dy[..., None]).sum(2)
    before = torch.cat((s["h0"][:, None], h[:, :-1]), 1)
    del h
    # the gradient of h_t, from the last token back: g_t = C_t dy_t + a_{t+1} g_{t+1}
    own_part = Cm[:, :, None, :] * dy[..., None]
    own_part[:, -1] += s["dhT"]
    later = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    g = _scan(later.flip(1), own_part.flip(1)).flip(1)
    del later, own_part
    dh0 = a[:, 0] * g[:, 0]
    gB = (g * Bm[:, :, None, :]).sum(-1)
    dB = (g * (dt * u)[..., None]).sum(2)
    ga = g * before * a
    del g, before, a
    ddt = u * gB + (ga * s["A"]).sum(-1)
    dA = (ga * dt[..., None]).sum((0, 1))
    ddt = ddt / (1.0 + torch.exp(-raw))
    du = dt * gB + dy * s["D"]
    dD = (dy * u).sum((0, 1))
    if s["lengths"] is not None:
        ddt = torch.where(pad, 0.0, ddt)
    return {"du": du.to(kind), "ddt": ddt.to(kind), "dA": dA.float(), "dB": dB.float(), "dC": dC.float(), "dD": dD.float(),
            "dz": dz.to(kind), "ddt_bias": ddt.sum((0, 1)).float(), "dh0": dh0.float()}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    steps = case["T"] if case["op"] == "ssm" else 1
    if steps * (3 if case["way"] == "backward" else 1) > 50000 or (case["way"] == "backward" and case["op"] == "ssm" and case["B"] * case["C"] * case["N"] * case["T"] > 1 << 30):
        return None  # too long a recursion, or too many states to keep
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm": _exact_norm, "prologue": _exact_prologue, "conv": _exact_conv, "ssm": _exact_ssm}[case["op"]](s)


def _exact_norm(s):
    x, w, d = s["x"], s["weight"], s["d"]
    if s["way"] == "backward":
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
        v = s["dy"] * w
        dx = v / norm - x * (v * x).sum(-1, keepdim=True) / (d * norm ** 3)
        return {"dx": dx if s["residual"] is None else dx + s["residual"], "dweight": torch.einsum("btd,btd->d", s["dy"], x / norm)}
    h = x if s["residual"] is None else x + s["residual"]
    y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / d + EPS) * w
    stream = None if s["residual"] is None else h
    if s["way"] == "forward":
        return {"y": y, "h": stream}
    scale = torch.clamp(torch.amax(torch.abs(y), -1) / E4M3_MAX, min=SCALE_MIN)
    v = y / scale[..., None]
    # the nearest of the type's values: steps of 2^(e - 3), with e >= -6, ties to the even one
    e = torch.floor(torch.log2(torch.clamp(torch.abs(v), min=2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return {"q": torch.clamp(torch.round(v / unit) * unit, -E4M3_MAX, E4M3_MAX), "scale": scale, "h": stream}


def _exact_prologue(s):
    x = s["x"] * s["x_scale"].unsqueeze(-1)
    out = {}
    for name in ("q", "k", "v"):
        p = torch.einsum("btm,hnm->bhtn", x, s["theta_" + name] * s["scale_" + name].unsqueeze(-1))
        if name != "v":
            pos = s["pos0"] + torch.arange(s["T"], device=x.device).double()
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos[:, None] / ROPE ** (torch.arange(32, device=x.device).double() / 32))
            pair = torch.complex(p[..., :32], p[..., 32:]) * turn
            p = torch.cat((pair.real, pair.imag), -1)
        out[name.upper()] = p
    logit = torch.einsum("btm,hm->bht", x, s["theta_lr"] * s["scale_lr"].unsqueeze(-1)) + s["b_lr"][None, :, None]
    out["eta"] = torch.sigmoid(logit) / 64
    return out


def _exact_conv(s):
    B, T, C, W = s["B"], s["T"], s["C"], s["W"]
    x, w = s["x"], s["weight"]
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    out = {k: torch.zeros_like(x) for k in (("dx",) if s["way"] == "backward" else ("y",))}
    out["dstate0" if s["way"] == "backward" else "state"] = torch.zeros_like(s["state"])
    dw, db = torch.zeros_like(w), torch.zeros_like(s["bias"])
    for b in range(B):
        rows = torch.cat((s["state"][b], x[b, :n[b]]))
        pieces = torch.stack([rows[j:j + n[b]] for j in range(W)], -1)  # [n, C, W]
        pre = torch.einsum("tcw,cw->tc", pieces, w) + s["bias"]
        if s["way"] != "backward":
            out["y"][b, :n[b]] = pre * torch.sigmoid(pre)
            out["state"][b] = rows[n[b]:]
            continue
        sig = torch.sigmoid(pre)
        dpre = s["dy"][b, :n[b]] * (sig + pre * sig * (1 - sig))
        dw += torch.einsum("tcw,tc->cw", pieces, dpre)
        db += dpre.sum(0)
        drows = torch.zeros_like(rows)
        drows[n[b]:] += s["dstate"][b]
        for j in range(W):
            drows[j:j + n[b]] += dpre * w[:, j]
        out["dx"][b, :n[b]], out["dstate0"][b] = drows[W - 1:], drows[:W - 1]
    return out | {"dweight": dw, "dbias": db} if s["way"] == "backward" else out


def _exact_ssm(s):
    B, T = s["B"], s["T"]
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"]
    dt = torch.nn.functional.softplus(s["dt"] + s["dt_bias"], threshold=100.0)
    h, back, states, y = s["h0"], s["way"] == "backward", [], torch.zeros_like(s["u"])
    live = [(t < n).tolist() for t in range(T)] if s["lengths"] is not None else [None] * T
    where = [None if k is None or all(k) else torch.tensor(k, device="cuda")[:, None, None] for k in live]
    for t in range(T):
        states.append(h if back else None)
        new = torch.exp(dt[:, t, :, None] * s["A"]) * h + (dt[:, t] * s["u"][:, t])[..., None] * s["Bm"][:, t, None, :]
        h = new if where[t] is None else torch.where(where[t], new, h)
        y[:, t] = (h @ s["Cm"][:, t, :, None])[..., 0] + s["D"] * s["u"][:, t]
    pad = (torch.arange(T, device="cuda")[None, :] >= n[:, None])[..., None]
    gate = s["z"] * torch.sigmoid(s["z"])
    if not back:
        return {"y": (y * gate).masked_fill(pad, 0.0), "hT": h}
    sig = torch.sigmoid(s["z"])
    dz = (s["dy"] * y * (sig + s["z"] * sig * (1 - sig))).masked_fill(pad, 0.0)
    dy = (s["dy"] * gate).masked_fill(pad, 0.0)
    g, dA = s["dhT"], torch.zeros_like(s["A"])
    du, ddt, dB, dC = (torch.zeros_like(v) for v in (s["u"], s["dt"], s["Bm"], s["Cm"]))
    for t in reversed(range(T)):
        after = states[t + 1] if t + 1 < T else h
        decay = torch.exp(dt[:, t, :, None] * s["A"])
        dC[:, t] = torch.einsum("bcn,bc->bn", after, dy[:, t])
        g_t = g + dy[:, t, :, None] * s["Cm"][:, t, None, :]
        g_dt = g_t * decay * states[t]
        if where[t] is not None:
            g_t_live, g_dt = (torch.where(where[t], v, 0.0) for v in (g_t, g_dt))
        else:
            g_t_live = g_t
        gB = torch.einsum("bcn,bn->bc", g_t_live, s["Bm"][:, t])
        dB[:, t] = torch.einsum("bcn,bc->bn", g_t_live, dt[:, t] * s["u"][:, t])
        du[:, t] = dt[:, t] * gB + s["D"] * dy[:, t]
        ddt[:, t] = s["u"][:, t] * gB + (g_dt * s["A"]).sum(-1)
        dA += torch.einsum("bcn,bc->cn", g_dt, dt[:, t])
        g = g_t * decay if where[t] is None else torch.where(where[t], g_t * decay, g)
    ddt = (ddt * torch.sigmoid(s["dt"] + s["dt_bias"])).masked_fill(pad, 0.0)
    return {"du": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (dy * s["u"]).sum((0, 1)), "dz": dz,
            "ddt_bias": ddt.sum((0, 1)), "dh0": g}
