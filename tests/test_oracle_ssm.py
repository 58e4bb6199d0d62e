"""Pins for the oracle's selective SSM block: the short causal convolution, the selective scan
and the norms around a block, against library routines, closed forms and hand-worked values.
CPU only."""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("direction", [0, 1, 2, 3])
def test_conv_against_torch_conv1d(K, direction):
    rng = np.random.default_rng(K)
    B, H, W, C = 2, 3, 5, 6
    x, w, b = rng.standard_normal((B, H * W, C)), rng.standard_normal((C, K)), rng.standard_normal(C)
    st = rng.standard_normal((B, K - 1, C))
    out, last, mag = oracle.ssm_conv(x, w, b, H, W, direction, True, st)
    order = oracle.scan_order(direction, H, W)
    line = torch.from_numpy(np.concatenate([st, x[:, order]], 1)).transpose(1, 2)
    ref = F.silu(F.conv1d(line, torch.from_numpy(w)[:, None], torch.from_numpy(b), groups=C)).transpose(1, 2).numpy()
    np.testing.assert_allclose(out[:, order], ref, rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(last, x[:, order][:, -(K - 1):])
    assert (mag > 0).all()


def test_conv_hand_worked_and_short_sequences():
    x = np.array([[[1.0], [2.0]], [[3.0], [4.0]]])
    w = np.array([[10.0, 100.0, 1000.0]])
    st = np.array([[[5.0], [6.0]], [[7.0], [8.0]]])
    out, last, _ = oracle.ssm_conv(x, w, None, 1, 2, 0, False, st, lengths=[2, 0])
    assert out[0, :, 0].tolist() == [50 + 600 + 1000, 60 + 100 + 2000]
    assert np.isnan(out[1]).all() and last[1, :, 0].tolist() == [7.0, 8.0]
    _, last, _ = oracle.ssm_conv(x, w, None, 1, 2, 0, False, st, lengths=[1, 1])
    assert last[0, :, 0].tolist() == [6.0, 1.0] and last[1, :, 0].tolist() == [8.0, 3.0]


def _scan_inputs(rng, B, L, D, N, G):
    return dict(u=rng.standard_normal((B, L, D)), dt=rng.standard_normal((B, L, D)) - 2.0,
                A=-np.exp(rng.standard_normal((D, N))), Bm=rng.standard_normal((B, L, G, N)),
                Cm=rng.standard_normal((B, L, G, N)))


def test_scan_against_explicit_sums():
    """out_t = sum_{s <= t} u_s delta_s sum_n C_t B_s exp(A sum of delta over s+1 .. t), written out
    per channel; groups: channels 0-1 use row 0 of Bm and Cm, channels 2-3 row 1."""
    rng = np.random.default_rng(1)
    B, H, W, D, N, G = 2, 2, 4, 4, 3, 2
    i = _scan_inputs(rng, B, H * W, D, N, G)
    h0, skip, bias = rng.standard_normal((B, D, N)), rng.standard_normal(D), rng.standard_normal(D)
    z = rng.standard_normal((B, H * W, D))
    for direction in range(4):
        out, st = oracle.ssm_scan(**i, H=H, W=W, direction=direction, skip=skip, z=z, dt_bias=bias, state=h0)
        order = oracle.scan_order(direction, H, W)
        for b in range(B):
            for d in range(D):
                g = d // 2
                dl = np.logaddexp(i["dt"][b, order, d] + bias[d], 0.0)
                cum = np.cumsum(dl)
                for t, m in enumerate(order):
                    h = np.exp(i["A"][d] * cum[t]) * h0[b, d]
                    for s in range(t + 1):
                        h = h + np.exp(i["A"][d] * (cum[t] - cum[s])) * dl[s] * i["u"][b, order[s], d] * i["Bm"][b, order[s], g]
                    y = (h @ i["Cm"][b, m, g] + skip[d] * i["u"][b, m, d]) * F.silu(torch.tensor(z[b, m, d])).item()
                    np.testing.assert_allclose(out[b, m, d], y, rtol=1e-10, atol=1e-12)
                np.testing.assert_allclose(st[b, d], h, rtol=1e-10, atol=1e-12)


def test_scan_geometric_series_and_prefix_sums():
    """Constant inputs without softplus: delta = 1, A = ln a: h = B (1 + a + ... + a^t); A = 0: sums."""
    L, a = 6, 0.5
    one = np.ones((1, L, 1))
    bc = np.ones((1, L, 1, 2))
    out, st = oracle.ssm_scan(one, one, np.array([[math.log(a), 0.0]]), 3 * bc, bc, 1, L, softplus=False)
    t = np.arange(1, L + 1)
    np.testing.assert_allclose(out[0, :, 0], 3 * ((1 - a ** t) / (1 - a) + t), rtol=1e-13)
    np.testing.assert_allclose(st[0, 0], [3 * (1 - a ** L) / (1 - a), 3 * L], rtol=1e-13)


def test_scan_cut_in_two_equals_one_scan_and_lengths():
    rng = np.random.default_rng(2)
    B, L, D, N, G = 2, 9, 4, 3, 1
    i = _scan_inputs(rng, B, L, D, N, G)
    whole, last = oracle.ssm_scan(**i, H=1, W=L)
    cut = lambda s: {k: (v if k == "A" else v[:, s]) for k, v in i.items()}
    a, h = oracle.ssm_scan(**cut(slice(0, 4)), H=1, W=4)
    b, h = oracle.ssm_scan(**cut(slice(4, L)), H=1, W=L - 4, state=h)
    np.testing.assert_allclose(np.concatenate([a, b], 1), whole, rtol=1e-13)
    np.testing.assert_allclose(h, last, rtol=1e-13)
    ragged, hr = oracle.ssm_scan(**i, H=1, W=L, lengths=[4, 0])
    np.testing.assert_array_equal(ragged[0, :4], a[0])
    assert np.isnan(ragged[0, 4:]).all() and np.isnan(ragged[1]).all() and (hr[1] == 0).all()


def test_scan_error_bounds_hold_for_single_precision():
    """The bounds that the GPU tests use contain the error of a float32 evaluation of the loop,
    and reject planted mistakes."""
    rng = np.random.default_rng(3)
    B, L, D, N, G = 1, 60, 8, 4, 1
    i = _scan_inputs(rng, B, L, D, N, G)
    i = {k: v.astype(np.float32) for k, v in i.items()}
    out, st, oerr, serr = oracle.ssm_scan(**i, H=1, W=L, rounding=(2 ** -21, 2 ** -19, 2 ** -19, 2 ** -24))

    def single(late_decay=False, no_dt=False):
        h, ys = np.zeros((B, D, N), np.float32), []
        for t in range(L):
            dl = np.logaddexp(i["dt"][:, t], np.float32(0))[..., None]
            add = (np.float32(1) if no_dt else dl) * i["u"][:, t, :, None] * i["Bm"][:, t]
            a = np.exp(dl * i["A"])
            h = a * (h + add) if late_decay else a * h + add
            ys.append((h * i["Cm"][:, t]).sum(-1))
        return np.stack(ys, 1), h

    y, h = single()
    assert (np.abs(y - out) <= oerr).all() and (np.abs(h - st) <= serr).all()
    assert oerr.max() < 1e-3 * np.abs(out).max()
    for wrong in (dict(late_decay=True), dict(no_dt=True)):
        y, h = single(**wrong)
        assert not (np.abs(y - out) <= oerr).all() and not (np.abs(h - st) <= serr).all()


def test_block_norm_against_torch_and_by_hand():
    rng = np.random.default_rng(4)
    B, L, C = 2, 3, 10
    y, h = rng.standard_normal((B, L, C)), rng.standard_normal((B, L, C))
    wa, wb, sc = rng.standard_normal(C), rng.standard_normal(C), rng.standard_normal(C)
    g = rng.standard_normal((B, C))
    T = torch.from_numpy
    r, n, _ = oracle.block_norm(y, h, wa, wb, g, True, sc, 1e-3)
    p = F.rms_norm(T(y), (C,), T(wa), 1e-3) * F.silu(T(g))[:, None] * T(sc)
    np.testing.assert_allclose(r, (T(h) + p).numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(n, F.rms_norm(T(h) + p, (C,), T(wb), 1e-3).numpy(), rtol=1e-12, atol=1e-13)
    r, n, mag = oracle.block_norm(np.array([[[3.0, 4.0]]]), np.array([[[1.0, -4.0]]]), None, [1.0, 2.0], eps=0.0)
    np.testing.assert_allclose(r[0, 0], [4.0, 0.0])
    np.testing.assert_allclose(n[0, 0], [math.sqrt(2.0), 0.0])
    assert mag[0, 0].tolist() == [4.0, 8.0]
