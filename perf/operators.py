"""The cases that the state space and block norm operators are measured on.

Four operators, each in plain torch form and through the library's entry points:

* ``conv``  the short causal depthwise convolution in front of a selective scan, along one of
  the four scan directions of the token grid, for whole prompts and for single tokens;
* ``scan``  the selective state space scan over a prompt;
* ``step``  the selective scan of one token per sequence, from and to a stored state;
* ``norm``  the norms after one block and before the next, fused with the block's gate, its
  residual scale and the residual stream.

Widths and grids are those of the workloads in ``gtr_inputs`` (model width 384, hidden width
1536, stride-16 grids of 640^2 to 2048^2 images, a batch of eight 1280x768 images) and sizes
next to them.
"""
import math

import torch

own = False

L2R, R2L, T2B, B2T = 0, 1, 2, 3
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the mixer's convolution on one 640^2 image: width 2 x 384, a few microseconds
        dict(name="conv_640", op="conv", dtype="f16", B=1, H=40, W=40, C=768, K=4, direction=R2L,
             half=False, state=False, ragged=False),
        # eight 1280x768 images by columns; x is one half of the input projection's rows; the
        # carried inputs come from and go to a cache
        dict(name="conv_stack", op="conv", dtype="bf16", B=8, H=48, W=80, C=1152, K=4, direction=T2B,
             half=True, state=True, ragged=True),
        # one new token for each of 64 streams
        dict(name="conv_token", op="conv", dtype="bf16", B=64, H=1, W=1, C=1536, K=4, direction=L2R,
             half=False, state=True, ragged=False),
        # one 640^2 image, width 2 x 384: few channels, so the time axis has to give the work
        dict(name="scan_640", op="scan", dtype="f16", B=1, H=40, W=40, D=768, N=16, G=1, direction=R2L,
             half=True, gate=True, state=False, ragged=False),
        # one 2048^2 image: a long sequence on few channels
        dict(name="scan_2048", op="scan", dtype="bf16", B=1, H=128, W=128, D=768, N=16, G=1, direction=B2T,
             half=True, gate=True, state=False, ragged=False),
        # eight 1280x768 images, hidden width: the throughput case
        dict(name="scan_stack", op="scan", dtype="bf16", B=8, H=48, W=80, D=1536, N=16, G=1, direction=T2B,
             half=False, gate=True, state=True, ragged=False),
        # odd grid, padded batch of sequences of different lengths, two groups, no gate, fp32
        dict(name="scan_ragged", op="scan", dtype="f32", B=3, H=37, W=53, D=416, N=8, G=2, direction=L2R,
             half=False, gate=False, state=True, ragged=True),
        # one token for each of four streams: latency
        dict(name="step_4", op="step", dtype="f16", B=4, D=768, N=16, G=1, half=True, gate=True),
        # one token for each of 512 streams: the state's traffic
        dict(name="step_512", op="step", dtype="bf16", B=512, D=1536, N=16, G=1, half=False, gate=True),
        # between two blocks of one 640^2 image at model width 384
        dict(name="norm_640", op="norm", dtype="f16", B=1, L=1600, C=384, residual="f16", post=True, pre=True,
             gate="token", silu=True, scale=True),
        # between two blocks of a batch of 1280x768 images, fp32 residual stream, a gate for each image
        dict(name="norm_stack", op="norm", dtype="bf16", B=8, L=3840, C=1536, residual="f32", post=True, pre=True,
             gate="batch", silu=False, scale=True),
        # fp32, an odd number of rows of an uncommon width, no norm after the block
        dict(name="norm_odd", op="norm", dtype="f32", B=3, L=1961, C=1060, residual="f32", post=False, pre=True,
             gate="none", silu=False, scale=True),
    ]


def _spread(rng, low, high, of=1):
    """A multiple of `of` between low and high, uniform over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / of)) * of))


def _grid(rng, most):
    """A grid of 1 to `most` cells."""
    cells = _spread(rng, 1, most)
    h = _spread(rng, 1, cells)
    return h, max(1, cells // h)


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "step", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "conv":
        C = _spread(rng, 64, 2048, 8)
        B = _spread(rng, 1, 64)
        H, W = _grid(rng, max(1, min(16384, 16_000_000 // (B * C))))
        return dict(op=op, dtype=dtype, B=B, H=H, W=W, C=C, K=rng.choice([2, 3, 4]), direction=rng.randrange(4),
                    half=rng.random() < 0.5, state=rng.random() < 0.5, ragged=rng.random() < 0.3)
    if op == "scan":
        G = rng.choice([1, 1, 1, 2, 4])
        D = G * _spread(rng, 32, 1536 // G, 16)
        N = rng.choice([8, 16, 16, 24, 32, 64])
        B = _spread(rng, 1, 16)
        H, W = _grid(rng, max(1, min(16384, 500_000_000 // (B * D * N))))
        return dict(op=op, dtype=dtype, B=B, H=H, W=W, D=D, N=N, G=G, direction=rng.randrange(4),
                    half=rng.random() < 0.5, gate=rng.random() < 0.7, state=rng.random() < 0.5,
                    ragged=rng.random() < 0.3)
    if op == "step":
        G = rng.choice([1, 1, 2])
        D, N = G * _spread(rng, 32, 2048 // G, 16), rng.choice([8, 16, 16, 24, 32, 64])
        return dict(op=op, dtype=dtype, B=_spread(rng, 1, min(512, 12_000_000 // (D * N))), D=D, N=N, G=G, half=rng.random() < 0.5, gate=rng.random() < 0.7)
    C = _spread(rng, 64, 8192, 8)
    B = _spread(rng, 1, 16)
    post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
    gate = rng.choice(["none", "batch", "token"])
    return dict(op=op, dtype=dtype, B=B, L=_spread(rng, 1, max(1, min(16384, 25_000_000 // (B * C)))), C=C,
                residual=rng.choice([dtype, "f32"]), post=post, pre=pre, gate=gate,
                silu=gate != "none" and rng.random() < 0.5, scale=rng.random() < 0.7)


def _share(case):
    """The share of a padded batch's tokens that is expected to be there, as _lengths draws them."""
    B = case["B"]
    return (1 + 0.5 * (B - 1 - (B > 2))) / B if case["ragged"] else 1.0


def _lengths(g, case):
    """How many tokens each sequence of a padded batch has: some, all, and in the last one none."""
    B, L = case["B"], case["H"] * case["W"]
    n = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = L
    if B > 2:
        n[B - 1] = 0
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, of=None):
        return torch.randn(*shape, generator=g, device="cuda").to(dt if of is None else of)

    op, B = case["op"], case["B"]
    s = {"case": case}
    if op == "conv":
        C, K, L = case["C"], case["K"], case["H"] * case["W"]
        s["x"] = normal(B, L, 2 * C)[..., :C] if case["half"] else normal(B, L, C)
        s["w"] = normal(C, K, of=torch.float32) / math.sqrt(K)
        s["bias"] = 0.1 * normal(C, of=torch.float32)
        s["state"] = normal(B, K - 1, C) if case["state"] else None
        s["state_out"] = torch.empty(B, K - 1, C, device="cuda", dtype=dt)
        s["lengths"] = _lengths(g, case) if case["ragged"] else None
        s["out"] = torch.zeros(B, L, C, device="cuda", dtype=dt)
    elif op in ("scan", "step"):
        D, N, G = case["D"], case["N"], case["G"]
        shape = (B, case["H"] * case["W"]) if op == "scan" else (B,)
        # u follows the convolution's SiLU, z is the other half of the input projection
        u = normal(*shape, D, of=torch.float32)
        s["u"] = (u / (1 + torch.exp(-u))).to(dt)
        s["dt"] = normal(*shape, D)
        # B and C are neighbouring columns of one projection's rows
        bc = normal(*shape, 2, G, N)
        s["Bm"], s["Cm"] = (bc[..., 0, :, :], bc[..., 1, :, :]) if case["half"] else (
            bc[..., 0, :, :].contiguous(), bc[..., 1, :, :].contiguous())
        s["z"] = None
        if case["gate"]:
            s["z"] = normal(*shape, 2 * D)[..., D:] if case["half"] else normal(*shape, D)
        # decay rates near -1 .. -N, step sizes spread over 0.001 .. 0.1 before the tokens' own part
        rate = torch.arange(1, N + 1, device="cuda", dtype=torch.float32).repeat(D, 1)
        s["A"] = -rate * torch.exp(0.1 * normal(D, N, of=torch.float32))
        step = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=g))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["skip"] = 1 + 0.1 * normal(D, of=torch.float32)
        s["state"] = normal(B, D, N, of=torch.float32) if op == "step" or case["state"] else None
        s["state_out"] = torch.empty(B, D, N, device="cuda")
        s["lengths"] = _lengths(g, case) if op == "scan" and case["ragged"] else None
        s["out"] = torch.zeros(*shape, D, device="cuda", dtype=dt)
    else:
        L, C = case["L"], case["C"]
        res = TYPES[case["residual"]]
        s["y"] = normal(B, L, C)
        s["h"] = normal(B, L, C, of=torch.float32).mul_(3).to(res)
        s["post_w"] = 1 + 0.1 * normal(C, of=torch.float32) if case["post"] else None
        s["pre_w"] = 1 + 0.1 * normal(C, of=torch.float32) if case["pre"] else None
        s["gate"] = {"none": None, "batch": normal(B, C), "token": normal(B, L, C) if case["gate"] == "token" else None}[
            case["gate"]]
        s["scale"] = 0.5 + 0.1 * normal(C, of=torch.float32) if case["scale"] else None
        s["h_out"] = torch.empty(B, L, C, device="cuda", dtype=res)
        s["n_out"] = torch.empty(B, L, C, device="cuda", dtype=dt) if case["pre"] else None
    return s


def _order(direction, H, W):
    """Token index y * W + x of each position of the scan."""
    m = torch.arange(H * W, device="cuda").view(H, W)
    m = m if direction in (L2R, T2B) else m.flip(1 if direction == R2L else 0)
    return (m if direction in (L2R, R2L) else m.t()).reshape(-1)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _valid(lengths, B, L):
    """[B, L] truth values: which positions of the scan each sequence has."""
    if lengths is None:
        return torch.ones(B, L, device="cuda", dtype=torch.bool)
    return torch.arange(L, device="cuda") < lengths[:, None]


def _prefix(decay, value, reach):
    """value_t <- sum over s <= t of value_s times the decays of s+1 .. t, in place along axis 1,
    by doubling the reach: each pass joins every position with the one `reach` before it."""
    if reach >= value.shape[1]:
        return value
    value[:, reach:] += decay[:, reach:] * value[:, :-reach]
    decay[:, reach:] = decay[:, reach:] * decay[:, :-reach]
    return _prefix(decay, value, 2 * reach)


def _plain_conv(s):
    case = s["case"]
    B, C, K, H, W = case["B"], case["C"], case["K"], case["H"], case["W"]
    order = _order(case["direction"], H, W)
    x = s["x"][:, order].float()
    before = torch.zeros(B, K - 1, C, device="cuda") if s["state"] is None else s["state"].float()
    line = torch.cat([before, x], 1)
    y = _silu((line.unfold(1, K, 1) * s["w"]).sum(-1) + s["bias"])
    valid = _valid(s["lengths"], B, H * W)
    out = torch.empty_like(y)
    out[:, order] = torch.where(valid[..., None], y, 0.0)
    last = valid.sum(1)[:, None] + torch.arange(K - 1, device="cuda")
    state = torch.gather(line, 1, last[..., None].expand(B, K - 1, C))
    return out.to(s["x"].dtype), state.to(s["x"].dtype)


def _by_group(x, m):
    """x [..., D] or [..., D, N] times m [..., G, N], each group's row for each of its D / G channels: [..., D, N]."""
    G = m.shape[-2]
    x = x[..., None] if x.dim() < m.dim() else x
    return (x.unflatten(-2, (G, -1)) * m.float()[..., None, :]).flatten(-3, -2)


def _plain_scan(s):
    case = s["case"]
    B, H, W = case["B"], case["H"], case["W"]
    order = _order(case["direction"], H, W)
    valid = _valid(s["lengths"], B, H * W)
    u = s["u"][:, order].float()
    dt = _softplus(s["dt"][:, order].float() + s["dt_bias"]) * valid[..., None]
    decay = torch.exp(dt[..., None] * s["A"])
    h = _by_group(dt * u, s["Bm"][:, order])
    if s["state"] is not None:
        h[:, 0] += decay[:, 0] * s["state"]
    h = _prefix(decay, h, 1)
    y = _by_group(h, s["Cm"][:, order]).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"][:, order].float())
    out = torch.empty_like(y)
    out[:, order] = torch.where(valid[..., None], y, 0.0)
    return out.to(s["u"].dtype), h[:, -1].clone()


def _plain_step(s):
    u = s["u"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + _by_group(dt * u, s["Bm"])
    y = _by_group(h, s["Cm"]).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["u"].dtype), h


EPS = 1e-6


def _plain_norm(s):
    p = s["y"].float()
    if s["post_w"] is not None:
        p = p * torch.rsqrt((p * p).mean(-1, keepdim=True) + EPS) * s["post_w"]
    if s["gate"] is not None:
        g = s["gate"].float() if s["gate"].dim() == 3 else s["gate"].float()[:, None]
        p = p * (_silu(g) if s["case"]["silu"] else g)
    if s["scale"] is not None:
        p = p * s["scale"]
    h = s["h"].float() + p
    if s["pre_w"] is None:
        return (h.to(s["h"].dtype),)
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["pre_w"]
    return h.to(s["h"].dtype), n.to(s["y"].dtype)


def _own(s):
    import gated_token_recurrence_b200 as gtr
    case = s["case"]
    op = case["op"]
    if op == "conv":
        out = gtr.ssm_conv(s["x"], s["w"], s["bias"], grid=(case["H"], case["W"]), direction=case["direction"], silu=True,
                           state=s["state"], state_out=s["state_out"], lengths=s["lengths"], out=s["out"])
        return out, s["state_out"]
    if op == "scan":
        out = gtr.ssm_scan(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], grid=(case["H"], case["W"]),
                           direction=case["direction"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], softplus=True,
                           state=s["state"], state_out=s["state_out"], lengths=s["lengths"], out=s["out"])
        return out, s["state_out"]
    if op == "step":
        out = gtr.ssm_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], skip=s["skip"], z=s["z"],
                           dt_bias=s["dt_bias"], softplus=True, state_out=s["state_out"], out=s["out"])
        return out, s["state_out"]
    h, n = gtr.block_norm(s["y"], s["h"], post_w=s["post_w"], pre_w=s["pre_w"], gate=s["gate"], gate_silu=case["silu"],
                          scale=s["scale"], eps=EPS, h_out=s["h_out"], n_out=s["n_out"])
    return (h,) if n is None else (h, n)


def run(state):
    if own:
        return _own(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    op, B = case["op"], case["B"]
    es = 4 if case["dtype"] == "f32" else 2
    if op == "conv":
        C, K = case["C"], case["K"]
        L = case["H"] * case["W"] * _share(case)
        states = (2 if case["state"] else 1) * B * (K - 1) * C
        return {"bytes": int(es * (2 * B * L * C + states) + 4 * C * (K + 1)), "flops": int(B * L * C * (2 * K + 5))}
    if op in ("scan", "step"):
        D, N, G = case["D"], case["N"], case["G"]
        L = case["H"] * case["W"] * _share(case) if op == "scan" else 1
        rows = B * L * ((4 if case["gate"] else 3) * D + 2 * G * N)
        states = (2 if op == "step" or case["state"] else 1) * B * D * N
        # per token, channel and state: the decay's product and exponential, the input's product,
        # one multiply-add for the state and one for the output; about 20 per token and channel besides
        return {"bytes": int(es * rows + 4 * (states + D * N + 2 * D)), "flops": int(B * L * D * (7 * N + 20))}
    L, C = case["L"], case["C"]
    er = 4 if case["residual"] == "f32" else 2
    gate = {"none": 0, "batch": B * C, "token": B * L * C}[case["gate"]]
    rows = B * L * C
    per_channel = 4 * C * (case["post"] + case["pre"] + case["scale"])
    return {"bytes": rows * (es * (2 if case["pre"] else 1) + 2 * er) + es * gate + per_channel, "flops": 14 * rows}


def _silu64(x):
    return x * torch.sigmoid(x)


def exact(case, seed):
    """The definitions in 64 bits: token by token along the scan, tap by tap, row by row."""
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op, B = case["op"], case["B"]
    if op == "norm":
        p = s["y"]
        if s["post_w"] is not None:
            p = p / p.square().mean(-1, keepdim=True).add(EPS).sqrt() * s["post_w"]
        if s["gate"] is not None:
            g = _silu64(s["gate"]) if case["silu"] else s["gate"]
            p = p * (g if g.dim() == 3 else g.unsqueeze(1))
        h = s["h"] + (p if s["scale"] is None else p * s["scale"])
        return (h,) if s["pre_w"] is None else (h, h / h.square().mean(-1, keepdim=True).add(EPS).sqrt() * s["pre_w"])
    if op == "step":
        H = W = 1
        s = {k: v.unsqueeze(1) if k in ("u", "dt", "Bm", "Cm", "z", "out") and v is not None else v for k, v in s.items()}
    else:
        H, W = case["H"], case["W"]
    cells = [(y, x) for y in range(H) for x in range(W)] if case.get("direction", L2R) in (L2R, R2L) else [
        (y, x) for x in range(W) for y in range(H)]
    mirror = {R2L: lambda y, x: (y, W - 1 - x), B2T: lambda y, x: (H - 1 - y, x)}.get(case.get("direction"), lambda y, x: (y, x))
    tokens = [y * W + x for y, x in (mirror(*c) for c in cells)]
    lengths = [len(tokens)] * B if s.get("lengths") is None else s["lengths"].tolist()
    out = torch.zeros_like(s["out"])
    if op == "conv":
        K = case["K"]
        index = torch.tensor(tokens, device="cuda")
        state = torch.empty_like(s["state_out"])
        for b in range(B):
            n = lengths[b]
            start = torch.zeros_like(s["state_out"][b]) if s["state"] is None else s["state"][b]
            line = torch.cat([start, s["x"][b, index[:n]]])
            acc = s["bias"].expand(n, -1).clone()
            for k in range(K):
                acc += line[k:k + n] * s["w"][:, k]
            out[b, index[:n]] = _silu64(acc)
            state[b] = line[n:]
        return out, state
    D, G = case["D"], case["G"]
    h = torch.zeros_like(s["state_out"]) if s["state"] is None else s["state"].clone()
    live = torch.tensor(lengths, device="cuda").view(B, 1, 1)
    for i, m in enumerate(tokens):
        dt = torch.logaddexp(s["dt"][:, m] + s["dt_bias"], torch.zeros((), device="cuda", dtype=torch.float64)).unsqueeze(-1)
        bm, cm = (s[k][:, m].unsqueeze(2).expand(B, G, D // G, -1).reshape(B, D, -1) for k in ("Bm", "Cm"))
        new = torch.exp(dt * s["A"]) * h + dt * s["u"][:, m].unsqueeze(-1) * bm
        h = torch.where(live > i, new, h)
        y = torch.einsum("bdn,bdn->bd", h, cm) + s["skip"] * s["u"][:, m]
        if s["z"] is not None:
            y = y * _silu64(s["z"][:, m])
        out[:, m] = torch.where(live[..., 0] > i, y, 0.0)
    return (out.squeeze(1) if op == "step" else out), h
