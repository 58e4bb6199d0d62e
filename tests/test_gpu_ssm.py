"""The selective SSM calls against the float64 oracle: the short convolution, the scan over a
prompt, the step of one token, and the three run together.

Bounds.  Convolution: the K + 1 terms are exact products of the inputs rounded at most K + 2
times in fp32, SiLU (Lipschitz constant below 1.1) adds its own relative error, the output is
rounded once:
    |out - ref| <= half_step(ref) + 1.1 (K + 2) 2^-24 mag + (2^-20 + 2^-21 |v|) |ref|,
mag the sum of the terms' magnitudes (|v| <= mag), the last term SiLU's exponential (a few
ulp, plus half an ulp of its argument) and quotient.

Scan and step: oracle.ssm_scan carries the errors of a rounded evaluation along the recurrence.
An exponential costs 2^-21 (its approximation, 2^-22.5, and roundings) and 2^-19 of its
argument's size: the argument is a product of delta (softplus with its argument's rounding,
|dt + bias| 2^-24 <= 12 2^-24, and about 8 roundings) and A log2(e) (two), and sums of up to 16
deltas; 2^-19 = 32 2^-24 covers them.  The input delta u B costs the same 2^-19.  The output is
rounded once to its type.

half_step: a rounding is off by half the spacing of the type's values, u |v| for a normal number
and, below the smallest one, half the spacing there: fp16's is 2^-24 under 2^-14, so 2^-25."""
import numpy as np
import pytest
import torch

import gated_token_recurrence_b200 as gtr
import oracle

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
ROUNDING = (2.0 ** -21, 2.0 ** -19, 2.0 ** -19, 2.0 ** -24)
SENTINEL = 123.0


def half_step(dtype, ref):
    return np.maximum(U[dtype] * np.abs(ref), SUBNORMAL[dtype])


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float32)


def wide(t, lead, pad_left, pad_right):
    """The same values as columns of wider rows, the rest NaN."""
    full = torch.full((*t.shape[:lead], t[(0,) * lead].numel() + pad_left + pad_right), float("nan"), dtype=t.dtype)
    full[..., pad_left:full.shape[-1] - pad_right] = t.reshape(*t.shape[:lead], -1)
    full = full.cuda()
    return full[..., pad_left:full.shape[-1] - pad_right].unflatten(-1, t.shape[lead:])


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def within(got, ref, bound, what):
    got = f64(got)
    valid = ~np.isnan(ref)
    assert (got[~valid] == SENTINEL).all(), f"{what}: a value behind a sequence's end was written"
    err = np.abs(got - ref)[valid] / np.maximum(bound[valid], 1e-300)
    assert np.isfinite(got[valid]).all() and (err.size == 0 or err.max() <= 1.0), f"{what}: error / bound = {err.max():.3g}"


# ------------------------------------------------------------------------------------ convolution
def check_conv(dtype, B, H, W, C, K, direction, silu=True, bias=True, state=True, lengths=None, strided=False,
               in_place=False, seed=0):
    gen = torch.Generator().manual_seed(seed + 17 * K + C)
    dt = DT[dtype]
    x, w = rnd(gen, B, H * W, C).to(dt), rnd(gen, C, K) / K ** 0.5
    b = rnd(gen, C) if bias else None
    st = rnd(gen, B, K - 1, C).to(dt) if state else None
    ref, last, mag = oracle.ssm_conv(x, w, b, H, W, direction, silu, st, lengths)
    xd = wide(x, 2, 16, 8) if strided else x.cuda()
    if lengths is not None:  # what is behind a sequence's end must not matter
        order = oracle.scan_order(direction, H, W)
        for i, n in enumerate(lengths):
            xd[i, torch.from_numpy(order[max(n, 0):].copy()).cuda()] = float("nan")
    sd = None if st is None else st.cuda()
    so = sd if in_place else torch.full((B, K - 1, C), SENTINEL, dtype=dt, device="cuda")
    out = torch.full((B, H * W, C), SENTINEL, dtype=dt, device="cuda")
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    gtr.ssm_conv(xd, w.cuda(), None if b is None else b.cuda(), grid=(H, W), direction=direction, silu=silu, state=sd,
                 state_out=so, lengths=ln, out=out)
    torch.cuda.synchronize()
    bound = half_step(dtype, ref) + 1.1 * (K + 2) * 2.0 ** -24 * mag + (2.0 ** -20 + 2.0 ** -21 * mag) * np.abs(ref)
    within(out, ref, bound, "out")
    np.testing.assert_array_equal(f64(so), last)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("grid,C", [((1, 1), 64), ((1, 2), 8), ((1, 3), 24), ((5, 7), 72), ((40, 40), 96), ((3, 333), 40)])
def test_conv(dtype, K, grid, C):
    check_conv(dtype, 2, *grid, C, K, direction=(K + grid[1]) % 4)


@pytest.mark.parametrize("direction", [0, 1, 2, 3])
@pytest.mark.parametrize("kw", [dict(), dict(strided=True), dict(silu=False, bias=False), dict(state=False),
                                dict(in_place=True), dict(lengths=[91, 0, 2]), dict(lengths=[1, 200, -5], in_place=True)])
def test_conv_forms(direction, kw):
    check_conv("bf16", 3, 7, 13, 136, 4, direction, **kw)


def test_conv_large_takes_long_strips():
    check_conv("f16", 8, 48, 80, 512, 4, 2, lengths=[3840, 3839, 3833, 1, 0, 3, 1000, 9])


# ------------------------------------------------------------------------------------------- scan
def scan_case(dtype, B, H, W, D, N, G, direction=0, skip=True, z=True, bias=True, softplus=True, state=True, seed=0,
              step=(1e-3, 1e-1)):
    gen = torch.Generator().manual_seed(seed + 31 * N + D)
    dt = DT[dtype]
    L = H * W
    c = dict(u=rnd(gen, B, L, D).to(dt), dt=rnd(gen, B, L, D).to(dt),
             A=-torch.arange(1, N + 1).float().repeat(D, 1) * torch.exp(0.1 * rnd(gen, D, N)),
             Bm=rnd(gen, B, L, G, N).to(dt), Cm=rnd(gen, B, L, G, N).to(dt))
    s = torch.exp(torch.empty(D).uniform_(np.log(step[0]), np.log(step[1]), generator=gen))
    c["dt_bias"] = s + torch.log(-torch.expm1(-s)) if bias else None
    c["skip"] = 1 + 0.1 * rnd(gen, D) if skip else None
    c["z"] = rnd(gen, B, L, D).to(dt) if z else None
    c["state"] = rnd(gen, B, D, N) if state else None
    if not softplus:
        c["dt"] = c["dt"].abs()
        if bias:
            c["dt_bias"] = c["dt_bias"].abs()
    return c


def on_gpu(c, strided=False):
    g = {k: None if v is None else v.cuda() for k, v in c.items()}
    if strided:
        for k, (a, b) in dict(u=(32, 0), dt=(0, 16), Bm=(8, 40), Cm=(48, 8), z=(8, 8)).items():
            if c[k] is not None:
                g[k] = wide(c[k], 2, a, b)
    return g


def check_scan(dtype, B, H, W, D, N, G, direction=0, softplus=True, lengths=None, strided=False, in_place=False, **kw):
    c = scan_case(dtype, B, H, W, D, N, G, softplus=softplus, **kw)
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=H, W=W, direction=direction, softplus=softplus, lengths=lengths,
                                          rounding=ROUNDING)
    g = on_gpu(c, strided)
    if lengths is not None:
        order = oracle.scan_order(direction, H, W)
        for i, n in enumerate(lengths):
            for k in ("u", "dt", "Bm", "Cm", "z"):
                if g[k] is not None:
                    g[k][i, torch.from_numpy(order[max(n, 0):].copy()).cuda()] = float("nan")
    out = torch.full((B, H * W, D), SENTINEL, dtype=DT[dtype], device="cuda")
    so = g["state"] if in_place else torch.full((B, D, N), SENTINEL, device="cuda")
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    gtr.ssm_scan(**g, grid=(H, W), direction=direction, softplus=softplus, lengths=ln, out=out, state_out=so)
    torch.cuda.synchronize()
    within(out, ref, oerr + half_step(dtype, ref), "out")
    within(so, st, serr + half_step("f32", st), "state")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 24, 32, 40, 48, 56, 64])
def test_scan_states(dtype, N):
    check_scan(dtype, 2, 11, 13, 32, N, 1, direction=N // 8 % 4)


@pytest.mark.parametrize("grid", [(1, 1), (1, 2), (3, 5), (4, 4), (1, 17), (8, 16), (3, 43), (16, 16), (1, 257),
                                  (27, 19), (2, 520)])
@pytest.mark.parametrize("direction", [0, 3])
def test_scan_lengths_of_the_sequence(grid, direction):
    check_scan("f16", 1, *grid, 48, 16, 1, direction=direction)


@pytest.mark.parametrize("direction", [0, 1, 2, 3])
@pytest.mark.parametrize("kw", [dict(), dict(strided=True), dict(skip=False, z=False, bias=False, state=False),
                                dict(softplus=False), dict(in_place=True), dict(lengths=[131, 0, 300, 17]),
                                dict(lengths=[0, -3, 1, 273], in_place=True), dict(G=3, strided=True)])
def test_scan_forms(direction, kw):
    check_scan("bf16", 4, 13, 21, 96, 16, direction=direction, **{"G": 2, **kw})


@pytest.mark.parametrize("B,D", [(1, 16), (1, 176), (2, 1040), (1, 4096), (5, 1200), (40, 272)])
def test_scan_widths(B, D):
    """From one tile of channels to more than the GPU holds at once: every plan of the scan."""
    check_scan("f16", B, 5, 53, D, 8, 1, direction=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,D,N,G,grid", [(16, 1024, 16, 1, (1, 1)), (17, 1024, 8, 2, (4, 6)), (33, 512, 24, 1, (3, 5)),
                                          (5, 1024, 64, 2, (2, 4)), (16, 1024, 40, 1, (5, 5)), (64, 272, 32, 1, (24, 1))])
def test_scan_of_a_few_tokens(dtype, B, D, N, G, grid):
    """Short prompts on many channels walk token by token up to 24 (8) positions."""
    L = grid[0] * grid[1]
    for kw in (dict(), dict(strided=True, lengths=[(3 * i) % (L + 2) - 1 for i in range(B)], in_place=True)):
        check_scan(dtype, B, *grid, D, N, G, direction=3, **kw)


@pytest.mark.parametrize("dtype,B,D,N,G", [("bf16", 12, 1056, 16, 1), ("f16", 8, 1024, 16, 2),
                                           ("f32", 8, 1024, 48, 1), ("f32", 11, 1056, 16, 3), ("bf16", 2, 768, 64, 2),
                                           ("f32", 1, 800, 64, 1), ("f32", 5, 1040, 64, 1), ("f16", 1, 768, 48, 1)])
def test_scan_plans_with_more_states(dtype, B, D, N, G):
    check_scan(dtype, B, 3, 50, D, N, G, direction=2, lengths=[150, 77] + [149] * (B - 2) if B > 1 else None)


def test_scan_slow_and_fast_decays():
    check_scan("f32", 1, 1, 2100, 32, 16, 1, step=(1e-5, 1e-4))     # remembers everything
    check_scan("f32", 1, 1, 300, 32, 64, 2, step=(5.0, 9.0))        # forgets at once: decays underflow
    check_scan("f16", 2, 9, 40, 64, 8, 1, step=(1e-3, 3.0))


def test_scan_extreme_steps_and_gates():
    """delta of 0 (dt far below 0) keeps the state as it is; a closed gate gives 0."""
    B, L, D, N = 1, 40, 32, 16
    c = scan_case("f32", B, 1, L, D, N, 1)
    c["dt"][:] = -200.0
    c["z"][:] = -200.0
    g = on_gpu(c)
    so = torch.empty(B, D, N, device="cuda")
    out = gtr.ssm_scan(**g, grid=(1, L), state_out=so)
    assert torch.equal(so, g["state"]) and (out == 0).all()
    c["dt"][:] = 60.0  # softplus is the identity there, and exp(-60) is gone in fp32
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=1, W=L, rounding=ROUNDING)
    out = gtr.ssm_scan(**on_gpu(c), grid=(1, L), state_out=so)
    within(so, st, serr + half_step("f32", st), "state")


def test_scan_carries_infinities_and_nans_forward_only():
    c = scan_case("f32", 1, 1, 300, 32, 16, 1, z=False)
    c["u"][0, 150, 3] = float("nan")
    c["u"][0, 150, 9] = float("inf")
    out = gtr.ssm_scan(**on_gpu(c), grid=(1, 300)).cpu()
    bad = ~torch.isfinite(out[0])
    assert not bad[:150].any() and bad[150:160, 3].all() and bad[150:160, 9].all()
    bad[:, [3, 9]] = False
    assert not bad.any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,D,N,G", [(1, 16, 8, 1), (3, 96, 16, 2), (70, 48, 24, 3), (2, 528, 64, 1), (9, 32, 40, 2)])
@pytest.mark.parametrize("form", ["plain", "strided", "bare", "in_place"])
def test_step(dtype, B, D, N, G, form):
    kw = dict(skip=False, z=False, bias=False) if form == "bare" else {}
    c = scan_case(dtype, B, 1, 1, D, N, G, **kw)
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=1, W=1, rounding=ROUNDING)
    g = on_gpu(c, form == "strided")
    g = {k: v[:, 0] if k in ("u", "dt", "Bm", "Cm", "z") and v is not None else v for k, v in g.items()}
    old = g["state"].clone()
    so = None if form == "in_place" else torch.empty_like(old)
    out = gtr.ssm_step(**g, state_out=so)
    torch.cuda.synchronize()
    within(out, ref[:, 0], (oerr + half_step(dtype, ref))[:, 0], "out")
    within(g["state"] if so is None else so, st, serr + half_step("f32", st), "state")
    if so is not None:
        assert torch.equal(g["state"], old)


# --------------------------------------------------------------------------------------- together
def test_prompt_then_tokens_equals_one_prompt():
    """Convolution and scan over a padded batch of prompts, then token by token from the carried
    states, against the oracle on each whole sequence."""
    B, L, T, D, N, K = 3, 37, 6, 64, 16, 4
    lens = [37, 5, 0]
    gen = torch.Generator().manual_seed(5)
    c = scan_case("f32", B, 1, L + T, D, N, 1, state=False)
    x, w, cb = rnd(gen, B, L + T, D), rnd(gen, D, K) / 2, rnd(gen, D)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = on_gpu(c)
    seq = {k: g[k] for k in ("dt", "Bm", "Cm", "z")}
    whole = {k: g[k] for k in ("A", "skip", "dt_bias")}
    conv_st, ssm_st = torch.zeros(B, K - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda")
    xd, wd, bd = x.cuda(), w.cuda(), cb.cuda()
    first = {k: v[:, :L].contiguous() for k, v in seq.items()}
    u = gtr.ssm_conv(xd[:, :L].contiguous(), wd, bd, grid=(1, L), state=conv_st, state_out=conv_st, lengths=ln)
    y = gtr.ssm_scan(u, **first, **whole, grid=(1, L), state=ssm_st, state_out=ssm_st, lengths=ln)
    got = [[y[b, :lens[b]]] for b in range(B)]
    for t in range(T):
        at = torch.tensor([n + t for n in lens], device="cuda")
        row = lambda v: v[torch.arange(B, device="cuda"), at].contiguous()
        u = gtr.ssm_conv(row(xd)[:, None], wd, bd, grid=(1, 1), state=conv_st, state_out=conv_st)
        y = gtr.ssm_step(u[:, 0], **{k: row(v) for k, v in seq.items()}, **whole, state=ssm_st)
        for b in range(B):
            got[b].append(y[b:b + 1])
    for b in range(B):
        n = lens[b] + T
        cut = lambda v: None if v is None else v[b:b + 1, :n]
        uref, _, mag = oracle.ssm_conv(x[b:b + 1, :n], w, cb, 1, n)
        args = {k: cut(c[k]) for k in ("dt", "Bm", "Cm", "z")}
        ref, st, oerr, serr = oracle.ssm_scan(uref, **args, A=c["A"], skip=c["skip"], dt_bias=c["dt_bias"], H=1, W=n,
                                              rounding=ROUNDING)
        # u itself is off by the convolution's bound, relative to the magnitudes the scan adds up
        extra = 2.0 ** -19 * np.abs(ref).max() + 2.0 ** -19 * mag.max() * np.abs(ref).max()
        assert np.abs(f64(torch.cat(got[b])) - ref[0]).max() <= oerr.max() + extra
        assert np.abs(f64(ssm_st[b]) - st[0]).max() <= serr.max() + 2.0 ** -19 * (1 + mag.max()) * np.abs(st).max()


def test_other_stream_and_captured_replays():
    """On a side stream, and captured: two graphs of the same calls replayed in turn give what
    the eager calls give, bit for bit, and follow new inputs."""
    c = scan_case("bf16", 2, 9, 33, 80, 16, 1)
    g = on_gpu(c)
    gen = torch.Generator().manual_seed(1)
    w, x = rnd(gen, 80, 4).cuda(), rnd(gen, 2, 297, 80).to(torch.bfloat16).cuda()
    rest = {k: v for k, v in g.items() if k not in ("u", "state")}

    def run(bufs):
        gtr.ssm_conv(x, w, None, grid=(9, 33), direction=3, state_out=bufs["conv"], out=bufs["u"])
        gtr.ssm_scan(bufs["u"], **rest, grid=(9, 33), direction=3, state=g["state"], state_out=bufs["h"], out=bufs["y"])

    def new():
        return dict(conv=torch.empty(2, 3, 80, dtype=torch.bfloat16, device="cuda"), u=torch.empty_like(x),
                    y=torch.empty_like(x), h=torch.empty(2, 80, 16, device="cuda"))

    eager, side = new(), new()
    run(eager)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        bufs = new()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(bufs)
        graphs.append((graph, bufs))
    for graph, _ in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for other in (side, graphs[0][1], graphs[1][1]):
        assert all(torch.equal(eager[k], other[k]) for k in eager)
    x.mul_(0.5)
    run(eager)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(eager[k], graphs[0][1][k]) for k in eager)


def test_calls_are_bitwise_repeatable():
    c = scan_case("f16", 2, 16, 40, 160, 16, 1)
    g = on_gpu(c)
    a = gtr.ssm_scan(**g, grid=(16, 40))
    assert all(torch.equal(a, gtr.ssm_scan(**g, grid=(16, 40))) for _ in range(3))


def test_two_streams_at_once():
    """Calls of every kind on two streams at the same time give what they give alone."""
    def work(seed):
        c = scan_case("bf16", 2, 16, 40, 160, 16, 1, seed=seed)
        g = on_gpu(c)
        gen = torch.Generator().manual_seed(seed)
        w = rnd(gen, 160, 4).cuda()

        def run():
            u = gtr.ssm_conv(g["z"], w, None, grid=(16, 40), direction=1)
            h = torch.empty_like(g["state"])
            rest = {k: v for k, v in g.items() if k != "u"}
            y = gtr.ssm_scan(u, **rest, grid=(16, 40), direction=1, state_out=h)
            one = {k: g[k][:, 0] for k in ("dt", "Bm", "Cm", "z")}
            s = gtr.ssm_step(u[:, 0], A=g["A"], state=h, skip=g["skip"], dt_bias=g["dt_bias"], **one)
            return u, y, h, s, *gtr.block_norm(y, u, pre_w=g["skip"])
        return run
    runs = [work(1), work(2)]
    alone = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                both.append(r())
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_stream_argument():
    c = scan_case("f32", 1, 1, 40, 32, 8, 1)
    g = on_gpu(c)
    ref = gtr.ssm_scan(**g, grid=(1, 40))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    gtr.ssm_scan(**g, grid=(1, 40), out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)


def test_refusals_on_the_gpu():
    """Wrong types, shapes, spacings and overlaps are errors that leave nothing enqueued."""
    c = scan_case("f16", 1, 2, 4, 32, 8, 1)
    g = on_gpu(c)
    for bad in (dict(u=g["u"].float()), dict(A=g["A"].half()), dict(Bm=g["Bm"][:, :4]), dict(z=g["z"].cpu()),
                dict(state=g["state"][:, :16]), dict(lengths=torch.ones(1, device="cuda")),
                dict(out=torch.empty(1, 8, 64, dtype=torch.float16, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            gtr.ssm_scan(**{**g, **bad}, grid=(2, 4))
    for bad in (dict(out=g["u"]), dict(state_out=g["A"].view(1, 32, 8)), dict(direction=4)):
        with pytest.raises(gtr.GTRError):
            gtr.ssm_scan(**{**g, **bad}, grid=(2, 4))
    with pytest.raises(ValueError):
        gtr.ssm_scan(**g, grid=(2, 5))
    with pytest.raises(ValueError):
        gtr.block_norm(g["u"], g["u"], gate=g["z"][:, :3])
    with pytest.raises(gtr.GTRError):
        gtr.block_norm(g["u"], g["u"], n_out=torch.empty_like(g["u"]))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------- rates beyond fp32
@pytest.mark.parametrize("rate", [float("-inf"), -3e38])
@pytest.mark.parametrize("B,D,L,lengths", [(1, 32, 1, None), (1, 32, 130, None), (2, 768, 130, [77, 130]),
                                           (5, 1200, 130, None), (40, 272, 70, None), (16, 1024, 8, None)])
def test_scan_with_rates_at_the_end_of_the_range(rate, B, D, L, lengths):
    """A state whose rate is -inf, or leaves fp32's range once multiplied by log2(e), forgets at
    once; the positions behind a sequence's end, which lie in its last tile, leave it alone.  Every
    exp(delta A) is 0 here, as for the rate -1e30 that the oracle gets."""
    c = scan_case("f32", B, 1, L, D, 16, 1)
    c["A"][:, 3] = -1e30
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=1, W=L, lengths=lengths, rounding=ROUNDING)
    c["A"][:, 3] = rate
    out = torch.full((B, L, D), SENTINEL, device="cuda")
    so = torch.full((B, D, 16), SENTINEL, device="cuda")
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    gtr.ssm_scan(**on_gpu(c), grid=(1, L), lengths=ln, out=out, state_out=so)
    within(out, ref, oerr + half_step("f32", ref), "out")
    within(so, st, serr + half_step("f32", st), "state")


@pytest.mark.parametrize("B,L", [(2, 1), (2, 40), (16, 8)])
def test_a_step_of_zero_keeps_the_state_at_any_rate(B, L):
    c = scan_case("f32", B, 1, L, 1024, 16, 1, bias=False)
    c["dt"][:] = -200.0
    c["A"][:, 5] = -3e38
    g = on_gpu(c)
    so = torch.empty_like(g["state"])
    gtr.ssm_scan(**g, grid=(1, L), state_out=so)
    assert torch.equal(so, g["state"])
    one = {k: g[k][:, 0] for k in ("u", "dt", "Bm", "Cm", "z")}
    gtr.ssm_step(**one, A=g["A"], state=g["state"], skip=g["skip"], state_out=so.zero_())
    assert torch.equal(so, g["state"])


def test_a_refused_launch_leaves_no_error_behind():
    """Calls on a stream whose capture has become invalid are errors; the next call elsewhere is
    not, whichever it is: the split GLA path looks at the runtime's last error."""
    q, lg = torch.randn(1, 64, 1, 64, device="cuda"), -torch.rand(1, 64, 1, 64, device="cuda")
    ws = gtr.new_workspace(1, 1, 8, 8, 64, 64, gtr.F32, "split", device="cuda")
    split = lambda: gtr.gla_fwd(q, q, q, lg, grid=(8, 8), path="split", workspace=ws)
    ref = split()
    c = scan_case("f32", 1, 1, 40, 32, 8, 1)
    g = on_gpu(c)
    w, ones, buf, so = torch.ones(32, 4, device="cuda"), torch.ones(32, device="cuda"), torch.empty_like(g["u"]), \
        torch.empty_like(g["state"])
    one = {k: g[k][:, 0] for k in ("u", "dt", "Bm", "Cm", "z")}
    rest = {k: g[k] for k in ("A", "skip", "dt_bias")}
    calls = [lambda: gtr.ssm_conv(g["u"], w, None, grid=(1, 40), out=buf),
             lambda: gtr.ssm_scan(**g, grid=(1, 40), out=buf, state_out=so),
             lambda: gtr.ssm_step(**one, **rest, state=g["state"], state_out=so, out=buf[:, 0]),
             lambda: gtr.block_norm(g["u"], g["z"], pre_w=ones, h_out=buf, n_out=torch.empty_like(buf))]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in calls:
        refused = False
        with pytest.raises(RuntimeError):  # the capture itself ends with an error
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
                with pytest.raises(RuntimeError):
                    torch.cuda.synchronize()  # not permitted while capturing
                try:
                    call()
                except gtr.GTRError as e:
                    refused = e.status == 3
        assert refused
        assert torch.equal(split(), ref)


# ----------------------------------------------------------------------------------- long memories
TILES = {"deep4": (16, 8), "deep8": (16, 8), "deep8short": (8, 8), "wide32x8": (32, 8), "wide16x16": (16, 16),
         "wide16x8": (16, 8), "wide8x16": (8, 16), "wide8x8": (8, 8)}  # time lanes, positions a lane


def long_memory(B, L, D, N, delta):
    """Constant steps and no input: h = h0 exp(L delta A), and every exponential repeats its error."""
    c = scan_case("f32", B, 1, L, D, N, 1, skip=False, z=False, bias=False, softplus=False)
    c["dt"][:], c["u"][:] = delta, 0.0
    arg = L * float(torch.tensor(delta)) * c["A"].double().numpy()
    return c, c["state"].double().numpy() * np.exp(arg), np.abs(arg)


@pytest.mark.parametrize("delta", [1e-6, 1e-5, 1e-4])
@pytest.mark.parametrize("B,D,N", [(1, 48, 16), (1, 768, 16), (1, 1200, 16), (3, 1584, 16), (5, 1440, 8), (9, 1056, 8)])
def test_long_memory_of_the_scan(B, D, N, delta):
    """Per tile of TL TS positions a state meets TL - 1 lane products and TS decays, each an
    exponential (2^-22.5) and two roundings of fp32, besides 2^-19 of its argument: far fewer than
    one a position (16,384 at the 1e-7 that was measured for each would exceed the bound)."""
    L = 128 * 128
    TL, TS = TILES[gtr.ssm_scan_plan(B, 1, L, D, N, 1, gtr.F32)]
    c, ref, arg = long_memory(B, L, D, N, delta)
    g = on_gpu(c)
    so = torch.empty_like(g["state"])
    gtr.ssm_scan(**g, grid=(1, L), softplus=False, state_out=so)
    factors = -(-L // (TL * TS)) * (TL - 1 + TS)
    assert (np.abs(f64(so) - ref) <= (factors * (2.0 ** -22.5 + 2 * 2.0 ** -24) + 2.0 ** -19 * arg) * np.abs(ref)).all()


@pytest.mark.parametrize("delta", [1e-6, 1e-4])
def test_long_memory_of_the_step(delta):
    """One exponential and one rounding a token."""
    T = 4096
    c, ref, arg = long_memory(2, T, 96, 16, delta)
    g = on_gpu(c)
    one = {k: g[k][:, 0] for k in ("u", "dt", "Bm", "Cm")}
    for _ in range(T):
        gtr.ssm_step(**one, A=g["A"], state=g["state"], softplus=False)
    assert (np.abs(f64(g["state"]) - ref) <= (T * (2.0 ** -22.5 + 2.0 ** -24) + 2.0 ** -19 * arg) * np.abs(ref)).all()


def test_scan_outputs_of_large_steps():
    """softplus is the identity at 60, exp(-60) is gone in fp32; with open gates the outputs say so."""
    B, L, D, N = 1, 40, 32, 16
    c = scan_case("f32", B, 1, L, D, N, 1)
    c["dt"][:] = 60.0
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=1, W=L, rounding=ROUNDING)
    so = torch.empty(B, D, N, device="cuda")
    out = gtr.ssm_scan(**on_gpu(c), grid=(1, L), state_out=so)
    within(out, ref, oerr + half_step("f32", ref), "out")
    within(so, st, serr + half_step("f32", st), "state")
    assert np.abs(ref).max() > 100.0


@pytest.mark.parametrize("B,D,L,N", [(1, 48, 137, 1), (16, 1024, 8, 4)])
def test_fewer_states_are_served_by_eight(B, D, L, N):
    """Bm, Cm and A of 0 behind the model's own states, as the header says."""
    c = scan_case("bf16", B, 1, L, D, N, 1)
    ref, st, oerr, serr = oracle.ssm_scan(**c, H=1, W=L, rounding=ROUNDING)
    pad = lambda t: torch.nn.functional.pad(t, (0, 8 - N))
    c.update({k: pad(c[k]) for k in ("A", "Bm", "Cm", "state")})
    so = torch.empty(B, D, 8, device="cuda")
    out = gtr.ssm_scan(**on_gpu(c), grid=(1, L), state_out=so)
    # the added terms are zeros: adding them rounds nothing
    within(out, ref, oerr + half_step("bf16", ref), "out")
    within(so[..., :N].contiguous(), st, serr + half_step("f32", st), "state")
    assert (so[..., N:] == 0).all()
