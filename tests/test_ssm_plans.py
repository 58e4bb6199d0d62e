"""Every kernel of the selective scan, in every form: shapes of several tiles, the last one not
full, that the plan query says they take, each in a 16-bit type and fp32.  The bounds are those of
test_gpu_ssm."""
import ctypes

import pytest

import gated_token_recurrence_b200 as gtr

# plan: (B, grid, D, N) without and with lengths
SHAPES = {
    "walk": ((12, (2, 11), 1440, 16), (12, (2, 11), 1440, 16)),
    "deep4": ((1, (9, 56), 48, 16), (2, (9, 56), 48, 16)),
    "deep8": ((1, (3, 85), 624, 16), (5, (3, 85), 240, 16)),
    "deep8short": ((1, (7, 55), 624, 16), (5, (7, 55), 240, 16)),
    "wide32x8": ((1, (9, 56), 1200, 16), (2, (9, 56), 1200, 16)),
    "wide16x16": ((3, (9, 56), 1200, 8), (6, (9, 56), 1200, 8)),
    "wide16x8": ((3, (3, 85), 1584, 16), (6, (3, 85), 1584, 8)),
    "wide8x16": ((5, (3, 85), 1440, 8), (10, (3, 85), 1440, 8)),
    "wide8x8": ((9, (3, 85), 1056, 8), (18, (3, 85), 1056, 8)),
}
DTYPES = {"f32": gtr.F32, "f16": gtr.F16, "bf16": gtr.BF16}


def test_every_plan_has_its_shapes():
    assert set(SHAPES) == set(gtr.SSM_PLANS)
    for name, both in SHAPES.items():
        for padded, (B, (H, W), D, N) in enumerate(both):
            for G in (1, 3):
                for dtype in DTYPES.values():
                    assert gtr.ssm_scan_plan(B, H, W, D, N, G, dtype, bool(padded)) == name


def test_plans_of_the_measured_workloads():
    """What the comments at the plan table say is taken (2048 positions, 16 states, bf16)."""
    for W, name in ((144, "deep8"), (288, "wide32x8"), (432, "wide32x8"), (576, "wide16x16"), (880, "wide16x8"),
                    (1152, "wide8x16"), (1728, "wide8x8")):
        assert gtr.ssm_scan_plan(4, 32, 64, 2 * W, 16, 1, gtr.BF16) == name


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(W=-1), 1), (dict(D=0), 1), (dict(N=0), 1), (dict(G=0), 1), (dict(G=3), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(plan=None), 1), (dict(N=12), 2), (dict(N=72), 2), (dict(D=40), 2),
    (dict(B=65536), 2), (dict(H=1 << 15, W=1 << 14), 2)])
def test_plan_query_refuses_what_the_scan_refuses(kw, code):
    a = dict(B=2, H=3, W=5, D=64, N=16, G=1, dtype=gtr.F16, padded=0, plan=ctypes.byref(ctypes.c_int(0)))
    assert gtr.lib.gtr_ssm_scan_plan(*a.values()) == 0
    a.update(kw)
    assert gtr.lib.gtr_ssm_scan_plan(*a.values()) == code


FORMS = {
    "bare": dict(skip=False, z=False, bias=False, state=False, G=1, direction=1),
    "strided_in_place_groups": dict(strided=True, in_place=True, G=3, direction=0),
    "no_softplus": dict(softplus=False, G=1, direction=2),
    "padded": dict(G=1, direction=3),
    "padded_strided_in_place_groups_no_gate": dict(strided=True, in_place=True, z=False, G=3, direction=2),
}


@pytest.mark.gpu
@pytest.mark.parametrize("plan", list(SHAPES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
def test_forms_on_every_plan(plan, dtype, form):
    from test_gpu_ssm import check_scan
    padded = form.startswith("padded")
    B, (H, W), D, N = SHAPES[plan][padded]
    L = H * W
    lengths = [L, 0, L - 1, 1, L // 2, 67, 130, -4][:B] + [(97 * i) % (L + 3) for i in range(B - 8)] if padded else None
    kw = dict(FORMS[form])
    assert gtr.ssm_scan_plan(B, H, W, D, N, kw["G"], DTYPES[dtype], padded) == plan
    check_scan(dtype, B, H, W, D, N, kw.pop("G"), lengths=lengths, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("plan", [p for p in SHAPES if p != "walk"])
def test_half_precision_on_every_plan(plan):
    from test_gpu_ssm import check_scan
    B, (H, W), D, N = SHAPES[plan][0]
    check_scan("f16", B, H, W, D, N, 1, direction=3)
