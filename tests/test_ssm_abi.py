"""Host-side refusals of the selective SSM calls and the block norm: every case is decided
before anything reaches CUDA, so the pointers are never dereferenced.  Runs without a GPU."""
import pytest
import torch

import gated_token_recurrence_b200 as gtr

P = [1 << 20 | i << 32 for i in range(1, 16)]  # far apart: nothing overlaps


def _conv(**kw):
    a = dict(x=P[0], ld=64, w=P[1], bias=P[2], si=P[3], so=P[3], len=None, out=P[4], B=2, H=3, W=5, C=64, K=4, dir=0,
             silu=1, dt=gtr.F16)
    a.update(kw)
    return gtr.lib.gtr_ssm_conv(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(x=P[0] + 8), 1), (dict(out=P[4] + 8), 1),
    (dict(si=P[3] + 8), 1), (dict(so=P[3] + 8), 1), (dict(w=P[1] + 8), 1), (dict(bias=P[2] + 4), 1), (dict(len=P[5] + 2), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(W=-1), 1), (dict(C=0), 1), (dict(K=0), 1), (dict(dir=4), 1),
    (dict(dir=-1), 1), (dict(dt=3), 1), (dict(ld=56), 1), (dict(ld=68), 1), (dict(ld=66, dt=gtr.F32), 1),
    (dict(K=1), 2), (dict(K=5), 2), (dict(C=60), 2), (dict(C=62, dt=gtr.F32), 2),
    (dict(H=1 << 15, W=1 << 14), 2), (dict(B=1 << 30, H=1 << 10, W=1 << 10), 2),
    (dict(out=P[0]), 1),                                         # output over the input
    (dict(out=P[0] + 29 * 64 * 2), 1), (dict(out=P[3]), 1),      # over its last row, over the state
    (dict(so=P[3] + 64), 1), (dict(so=P[0] + 128), 1),           # shifted onto the old state; over the input
])
def test_conv_arguments_rejected_on_host(kw, code):
    assert _conv(**kw) == code


def _scan(step=False, **kw):
    a = dict(u=P[0], ul=64, dt=P[1], dl=64, A=P[2], Bm=P[3], bl=32, Cm=P[4], cl=32, z=P[5], zl=64, skip=P[6],
             bias=P[7], sp=1, si=P[8], so=P[8])
    tail = dict(out=P[9], B=2, D=64, N=16, G=2, ty=gtr.F16) if step else dict(
        len=None, out=P[9], B=2, H=3, W=5, D=64, N=16, G=2, dir=0, ty=gtr.F16)
    a.update(tail)
    a.update(kw)
    return (gtr.lib.gtr_ssm_step if step else gtr.lib.gtr_ssm_scan)(*a.values(), None)


COMMON = [
    (dict(u=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(Bm=None), 1), (dict(Cm=None), 1),
    (dict(out=None), 1), (dict(u=P[0] + 8), 1), (dict(Bm=P[3] + 8), 1), (dict(A=P[2] + 4), 1), (dict(so=P[8] + 4), 1),
    (dict(skip=P[6] + 2), 1), (dict(ul=56), 1), (dict(ul=68), 1), (dict(bl=24), 1), (dict(zl=8), 1), (dict(cl=36), 1),
    (dict(B=0), 1), (dict(D=0), 1), (dict(N=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(ty=4), 1),
    (dict(N=12), 2), (dict(N=72, bl=144, cl=144), 2), (dict(G=8, bl=128, cl=128), 2), (dict(B=65536), 2),
    (dict(out=P[0]), 1), (dict(out=P[5]), 1), (dict(out=P[8]), 1), (dict(so=P[8] + 64), 1), (dict(so=P[2]), 1),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(H=0), 1), (dict(dir=4), 1), (dict(len=P[10] + 1), 1), (dict(H=1 << 15, W=1 << 14), 2)])
def test_scan_arguments_rejected_on_host(kw, code):
    assert _scan(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(si=None), 1), (dict(so=None), 1)])
def test_step_arguments_rejected_on_host(kw, code):
    assert _scan(step=True, **kw) == code


def _norm(**kw):
    a = dict(y=P[0], h=P[1], wa=P[2], wb=P[3], gate=P[4], per_token=0, silu=0, scale=P[5], eps=1e-6, ho=P[1], no=P[6],
             B=2, L=3, C=64, dt=gtr.F16, rt=gtr.F32)
    a.update(kw)
    return gtr.lib.gtr_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), 1), (dict(h=None), 1), (dict(ho=None), 1), (dict(no=None), 1), (dict(wb=None), 1),
    (dict(y=P[0] + 8), 1), (dict(wa=P[2] + 4), 1), (dict(gate=P[4] + 2), 1), (dict(B=0), 1), (dict(L=0), 1),
    (dict(C=-8), 1), (dict(dt=7), 1), (dict(rt=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(rt=gtr.BF16), 2), (dict(dt=gtr.F32, rt=gtr.F16), 2), (dict(C=60), 2),
    (dict(C=16392), 2), (dict(C=8196, dt=gtr.F32), 2), (dict(L=1 << 29), 2),
    (dict(ho=P[1] + 64), 1), (dict(no=P[0] + 128), 1), (dict(ho=P[0]), 1), (dict(no=P[1]), 1), (dict(no=P[4]), 1),
    (dict(ho=P[2]), 1), (dict(no=P[5]), 1),
])
def test_norm_arguments_rejected_on_host(kw, code):
    assert _norm(**kw) == code


def test_row_distances_of_strided_inputs():
    rows = lambda t, tokens=2: gtr._marshal().distance(t, tokens)
    x = torch.zeros(3, 5, 64, dtype=torch.float16)
    assert rows(x) == 64 and rows(x[..., 8:40]) == 64 and rows(x[:1, :, :32]) == 64
    assert rows(x[:, :1]) == 5 * 64 and rows(x[:1, :1, :24]) == 24 and rows(x[:1, :1, :20]) == 24
    bc = torch.zeros(3, 5, 2, 2, 16)
    assert rows(bc[:, :, 1]) == 64 and rows(bc[:, 0, 1], 1) == 5 * 64
    for bad in (x[:, :4], x.transpose(0, 1), x[..., ::2], bc.transpose(-1, -2)[:, :, 0]):
        with pytest.raises(ValueError):
            rows(bad)


def test_marshalling_refuses_what_it_cannot_pass():
    """Each refusal is a ValueError that names the argument; nothing reaches the library."""
    m = gtr._marshal()
    x, w = torch.zeros(1, 4, 64), torch.zeros(64, 4)
    args = lambda **kw: tuple({**dict(x=x, w=w, bias=None, H=2, W=2, d=0, silu=True, st=None, so=None, ln=None, out=x, dev=0,
                                      stream=0), **kw}.values())
    for kw, word in ((dict(), "x: expected a CUDA tensor"), (dict(x=None), "x: expected a tensor"),
                     (dict(x=torch.zeros(4, 64)), "x: expected 3 axes"), (dict(w=torch.zeros(64)), "w: expected 2 axes"),
                     (dict(x=x.double()), "x: must be float32, float16 or bfloat16")):
        with pytest.raises(ValueError, match=word):
            m.conv(*args(**kw))
    with pytest.raises(ValueError):
        m.conv(x)
    with pytest.raises(TypeError):
        m.conv(*args(dev="0"))


def test_host_tensors_are_refused():
    x = torch.zeros(1, 4, 64)
    v = torch.zeros(64)
    with pytest.raises((ValueError, RuntimeError)):
        gtr.ssm_conv(x, torch.zeros(64, 4), v, grid=(2, 2))
    with pytest.raises((ValueError, RuntimeError)):
        gtr.block_norm(x, x)
    with pytest.raises(ValueError):
        gtr.ssm_conv(x, torch.zeros(64, 4), v, grid=(2, 3))


@pytest.mark.parametrize("kw", [
    dict(out=P[1]), dict(out=P[1] + 64 * 4 * 4 - 16), dict(out=P[2]), dict(out=P[2] + 64 * 4 - 16), dict(len=P[4]),
    dict(len=P[4] + 2 * 3 * 5 * 64 * 2 - 4), dict(len=P[4] - 4), dict(so=P[1]), dict(so=P[1] + 64 * 4 * 4 - 16),
    dict(so=P[2]), dict(so=P[2] + 64 * 4 - 16), dict(si=P[5], len=P[3]), dict(si=P[5], len=P[3] + 2 * 3 * 64 * 2 - 4)])
def test_conv_outputs_over_weights_or_lengths_are_rejected(kw):
    """The first and the last bytes of the taps, the bias and the lengths under an output."""
    assert _conv(**kw) == 1


def test_conv_outputs_next_to_weights_or_lengths_pass_the_overlap_checks():
    """So many tokens that the call ends with GTR_ERR_UNSUPPORTED after the overlap checks."""
    x, out, B, H = 1 << 44, 1 << 45, 50, 1 << 14
    behind = out + B * H * H * 64 * 2
    many = dict(B=B, H=H, W=H, x=x, out=out)
    for kw in (dict(w=behind), dict(w=out - 64 * 4 * 4), dict(bias=behind), dict(bias=out - 64 * 4), dict(len=behind),
               dict(len=out - B * 4)):
        assert _conv(**many, **kw) == 2
    for kw in (dict(w=behind - 16), dict(w=out - 64 * 4 * 4 + 16), dict(bias=behind - 16), dict(bias=out - 64 * 4 + 16),
               dict(len=behind - 4), dict(len=out - B * 4 + 4)):
        assert _conv(**many, **kw) == 1
