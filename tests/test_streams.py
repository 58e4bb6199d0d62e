"""Results and scratch that a call allocates belong to the stream it runs on: memory of the
current stream's pool could still be in use there, or be handed out again while the call runs."""
import contextlib

import pytest
import torch

import gated_token_recurrence_b200 as gtr


class Fake:
    """What the binding asks of a CUDA tensor; each allocation notes the stream that it is made under."""
    is_cuda, device = True, torch.device("cpu")
    made = []
    under = [None]

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype = shape, dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1

    def new_empty(self, shape, dtype=None):
        Fake.made.append(Fake.under[-1])
        return Fake(*shape, dtype=dtype or self.dtype)

    def new_zeros(self, shape, dtype=None):
        return self.new_empty(shape, dtype)


class Marshal:
    conv = scan = step = norm = staticmethod(lambda *a: 0)


def calls():
    x, g, q = Fake(2, 12, 64), Fake(2, 12, 1, 16), Fake(2, 12, 1, 64)
    lg = Fake(2, 12, 1, 64, dtype=torch.float32)
    one, gone = Fake(2, 64), Fake(2, 1, 16)
    return {
        "ssm_conv": lambda **kw: gtr.ssm_conv(x, Fake(64, 4), None, grid=(3, 4), **kw),
        "ssm_scan": lambda **kw: gtr.ssm_scan(x, x, Fake(64, 16), g, g, grid=(3, 4), **kw),
        "ssm_step": lambda **kw: gtr.ssm_step(one, one, Fake(64, 16), gone, gone, Fake(2, 64, 16), **kw),
        "block_norm": lambda **kw: gtr.block_norm(x, x, pre_w=Fake(64), **kw),
        "gla_fwd": lambda **kw: gtr.gla_fwd(q, q, q, lg, grid=(3, 4), **kw),
        "gla_fwd_split": lambda **kw: gtr.gla_fwd(q, q, q, lg, grid=(3, 4), path="split", **kw),
        "gla_block_fwd": lambda **kw: gtr.gla_block_fwd(q, q, q, grid=(3, 4), log_gamma=lg, **kw),
        "sswiglu_dwconv": lambda **kw: gtr.sswiglu_dwconv(x, x, Fake(64, 3, 3, dtype=torch.float32), None, grid=(3, 4), **kw),
    }


NAMES = ["ssm_conv", "ssm_scan", "ssm_step", "block_norm", "gla_fwd", "gla_fwd_split", "gla_block_fwd", "sswiglu_dwconv"]
ALLOCATIONS = {"block_norm": 2, "gla_fwd_split": 2}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", [True, False])
def test_allocations_are_made_under_the_calls_stream(monkeypatch, name, given):
    class Lib:
        gtr_gla_workspace_bytes = staticmethod(lambda *a: 1024)

        def __getattr__(self, f):
            return lambda *a: 0

    class Stream:
        cuda_stream = 7

    @contextlib.contextmanager
    def under(s):
        Fake.under.append(s)
        yield
        Fake.under.pop()

    monkeypatch.setattr(gtr, "lib", Lib())
    monkeypatch.setattr(gtr, "_native", Marshal)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "stream", under)
    Fake.made.clear()
    s = Stream() if given else None
    calls()[name](stream=s)
    assert Fake.made == [s] * ALLOCATIONS.get(name, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["ssm_conv", "ssm_scan", "ssm_step", "block_norm", "gla_fwd", "gla_fwd_split",
                                  "sswiglu_dwconv"])
def test_results_on_another_stream_without_out(name):
    """The result is right, and lies neither in memory just freed on the current stream, nor is
    handed out to the current stream once it is dropped."""
    B, H, W, C, N = 4, 16, 40, 256, 16
    L = H * W
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, dt=torch.float32: torch.randn(*s, generator=gen, device="cuda").to(dt)
    x, bm, A, w = rnd(B, L, C), rnd(B, L, 1, N), -rnd(C, N).abs(), rnd(C, 4)
    wide, state = rnd(4096, C), rnd(4096, C, N)
    q, lg = rnd(B, L, 4, 64, dt=torch.float16), -rnd(B, L, 4, 64).abs()
    call = {
        "ssm_conv": lambda **kw: gtr.ssm_conv(x, w, None, grid=(H, W), **kw),
        "ssm_scan": lambda **kw: gtr.ssm_scan(x, x, A, bm, bm, grid=(H, W), **kw),
        "ssm_step": lambda **kw: gtr.ssm_step(wide, wide, A, rnd_one, rnd_one, state, state_out=other, **kw),
        "block_norm": lambda **kw: gtr.block_norm(x, x, post_w=post, **kw)[0],
        "gla_fwd": lambda **kw: gtr.gla_fwd(q, q, q, lg, grid=(H, W), **kw),
        "gla_fwd_split": lambda **kw: gtr.gla_fwd(q, q, q, lg, grid=(H, W), path="split", **kw),
        "sswiglu_dwconv": lambda **kw: gtr.sswiglu_dwconv(x, x, conv, None, grid=(H, W), **kw),
    }[name]
    rnd_one, other, conv, post = rnd(4096, 1, N), torch.empty_like(state), rnd(C, 3, 3), rnd(C)
    ref = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = torch.empty_like(ref)
    place = freed.data_ptr()
    del freed
    got = call(stream=s)
    s.synchronize()
    assert got.data_ptr() != place and torch.equal(got, ref)
    place = got.data_ptr()
    del got
    assert torch.empty_like(ref).data_ptr() != place
