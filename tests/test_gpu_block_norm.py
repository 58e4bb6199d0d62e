"""The norms around a block (gtr_block_norm) against the float64 oracle.

Bounds.  A sum of squares of C values, each thread adding at most 32 of them before the tree, is
off by at most 40 half-ulps, so its root's reciprocal by 20, and the two or three factors and the
quotient bring the block's part p to 64 2^-24 relative at most, plus SiLU's error where the gate
has one (2^-20 + 2^-21 |g|).  h' is one more addition: e_h = that + 2^-24 (|h| + |p|).  n divides
by the root mean square of h', whose relative error is at most that of the errors e_h:
    e_n = |pre_w| (e_h + |h'| rms(e_h) / rms(h')) / rms(h') + 64 2^-24 |n|.
Outputs are rounded once to their types: half the spacing of the type's values, u |v|, and for
fp16 below 2^-14, where that spacing stays 2^-24, 2^-25."""
import numpy as np
import pytest
import torch

import gated_token_recurrence_b200 as gtr
import oracle

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def half_step(dtype, ref):
    return np.maximum(U[dtype] * np.abs(ref), SUBNORMAL[dtype])


def check(dtype, residual, B, L, C, post=True, pre=True, gate="token", silu=False, scale=True, eps=1e-6, in_place=False,
          size=1.0):
    gen = torch.Generator().manual_seed(B * L + C)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float32)
    y, h = (size * rnd(B, L, C)).to(DT[dtype]), (3 * size * rnd(B, L, C)).to(DT[residual])
    wa, wb = (1 + 0.1 * rnd(C) if on else None for on in (post, pre))
    sc = 0.5 + 0.1 * rnd(C) if scale else None
    g = {"none": None, "batch": rnd(B, C).to(DT[dtype]), "token": rnd(B, L, C).to(DT[dtype])}[gate]
    r, n, mag = oracle.block_norm(y, h, wa, wb, g, silu, sc, eps)
    d = lambda t: None if t is None else t.cuda()
    yd, hd = d(y), d(h)
    ho, no = gtr.block_norm(yd, hd, post_w=d(wa), pre_w=d(wb), gate=d(g), gate_silu=silu, scale=d(sc), eps=eps,
                            h_out=hd if in_place else None, n_out=yd if in_place and pre else None)
    torch.cuda.synchronize()
    p = np.abs(r - h.double().numpy())
    gg = 0.0 if g is None or not silu else np.abs(g.double().numpy()).reshape(B, -1, C)
    eh = 2.0 ** -24 * (mag + 64 * p) + (0.0 if not silu else (2.0 ** -20 + 2.0 ** -21 * gg) * p)
    got = ho.to("cpu", torch.float64).numpy()
    worst = (np.abs(got - r) / (eh + half_step(residual, r))).max()
    assert np.isfinite(got).all() and worst <= 1.0, f"h': error / bound = {worst:.3g}"
    if not pre:
        assert no is None
        return
    rms = lambda v: np.sqrt((v * v).mean(-1, keepdims=True))
    root = np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    en = np.abs(wb.double().numpy()) * (eh + np.abs(r) * rms(eh) / root) / root + 64 * 2.0 ** -24 * np.abs(n)
    got = no.to("cpu", torch.float64).numpy()
    worst = (np.abs(got - n) / (en + half_step(dtype, n))).max()
    assert np.isfinite(got).all() and worst <= 1.0, f"n: error / bound = {worst:.3g}"


@pytest.mark.parametrize("dtype,residual", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("C", [8, 64, 200, 384, 520, 1024, 1032, 1536, 2048, 4104, 8192])
def test_widths(dtype, residual, C):
    check(dtype, residual, 2, 7, C)


@pytest.mark.parametrize("dtype,C", [("f32", 4), ("f32", 1060), ("f16", 16384), ("bf16", 12296)])
def test_smallest_odd_and_largest_widths(dtype, C):
    check(dtype, "f32", 1, 3, C)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "batch", "token"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("scale", [True, False])
def test_forms(post, pre, gate, silu, scale):
    if gate == "none" and silu:
        silu = False
    check("bf16", "f32", 3, 11, 384, post=post, pre=pre, gate=gate, silu=silu, scale=scale, in_place=scale)
    check("f16", "f16", 1, 5, 1160, post=post, pre=pre, gate=gate, silu=silu, scale=scale, in_place=not scale)


def test_many_rows_and_one():
    check("f16", "f16", 5, 1601, 384, gate="batch")
    check("bf16", "f32", 1, 1, 768)


def test_zero_rows_and_small_values():
    check("f32", "f32", 1, 3, 256, size=1e-12)   # eps decides
    check("f32", "f32", 1, 3, 256, size=1e15, eps=0.0)
    z = torch.zeros(1, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, n = gtr.block_norm(z, z, post_w=w, pre_w=w)
    assert (h == 0).all() and (n == 0).all()


def test_run_with_the_mixers_of_a_block():
    """A block of the library's own calls, twice: GLA with its output gate, the norms around it,
    a selective scan with its convolution, the norms again; eager and captured agree, and the
    last norms agree with the oracle on their own inputs."""
    B, H, W, C, heads, N = 1, 12, 11, 128, 2, 16
    L = H * W
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float32).cuda()
    h0 = rnd(B, L, C)
    q, k, v = (rnd(B, L, heads, 64).half() for _ in range(3))
    lg = torch.nn.functional.logsigmoid(rnd(B, L, heads, 64)) / 16
    og, nw = rnd(B, L, heads, 64).half(), torch.ones(64, device="cuda")
    cw, cb, wa, wb, gate = rnd(C, 4) / 2, rnd(C), torch.ones(C, device="cuda"), torch.ones(C, device="cuda"), rnd(B, C).half()
    dt, A = rnd(B, L, C).half(), -torch.arange(1, N + 1, device="cuda").float().repeat(C, 1)
    bm, cm = rnd(B, L, 1, N).half(), rnd(B, L, 1, N).half()
    ws = gtr.new_workspace(B, heads, H, W, 64, 64, gtr.F16, device="cuda")

    def run():
        y = gtr.gla_block_fwd(q, k, v, grid=(H, W), direction=gtr.T2B, log_gamma=lg, out_gate=og, norm_w=nw, workspace=ws)
        h, n = gtr.block_norm(y.view(B, L, C), h0, post_w=wa, pre_w=wb, gate=gate)
        u = gtr.ssm_conv(n, cw, cb, grid=(H, W), direction=gtr.R2L)
        s = gtr.ssm_scan(u, dt, A, bm, cm, grid=(H, W), direction=gtr.R2L, z=n)
        return (h, s, *gtr.block_norm(s, h, post_w=wa, pre_w=wb, gate=gate))

    eager = run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, kept))
    r, n, _ = oracle.block_norm(eager[1], eager[0], wa, wb, gate)
    assert np.abs(eager[2].double().cpu().numpy() - r).max() <= 2.0 ** -18 * np.abs(r).max()
    assert np.abs(eager[3].double().cpu().numpy() - n).max() <= 2.0 ** -10 * np.abs(n).max()
