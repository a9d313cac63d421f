"""Pins of the oracles of the selective scan, the causal convolution and the 8-bit copies (CPU): the scan
against its closed sum over earlier tokens, the convolution against numpy's, packing against its
definition, and every gradient against central differences."""
import numpy as np
import pytest

import oracle as O


def _scan(seed, B=2, T=6, E=4, G=2, N=3):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(size=s)  # noqa: E731
    return dict(u=n(B, T, E), dt=n(B, T, E), A=-r.exponential(1.0, size=(E, N)), B=n(B, T, G, N), C=n(B, T, G, N),
                D=n(E), z=n(B, T, E), bias=n(E), state=n(B, E, N)), r


@pytest.mark.parametrize("softplus", [True, False])
def test_the_scan_is_the_decayed_sum_over_earlier_tokens(softplus):
    p, _ = _scan(1)
    lens = np.array([6, 4])
    y, S = O.selective_scan(**p, softplus=softplus, lens=lens)
    raw = p["dt"] + p["bias"]
    delta = np.log(1 + np.exp(raw)) if softplus else raw
    for b in range(2):
        for e in range(4):
            g = e // 2
            for t in range(6):
                want = (np.exp(p["A"][e] * delta[b, :t + 1, e].sum()) * p["state"][b, e]) @ p["C"][b, t, g]
                for j in range(t + 1):
                    w = np.exp(p["A"][e] * delta[b, j + 1:t + 1, e].sum()) * delta[b, j, e] * p["u"][b, j, e]
                    want += (w * p["B"][b, j, g]) @ p["C"][b, t, g]
                zt = p["z"][b, t, e]
                want = (want + p["D"][e] * p["u"][b, t, e]) * zt / (1 + np.exp(-zt))
                assert np.allclose(y[b, t, e], want if t < lens[b] else 0.0, rtol=1e-12, atol=1e-12)
    # the state after row 1's four tokens continues like the whole sequence
    tail = {k: v[:, 4:] if k in ("u", "dt", "B", "C", "z") else v for k, v in p.items() if k != "state"}
    y2, _ = O.selective_scan(**tail, softplus=softplus, state=S)
    full, _ = O.selective_scan(**p, softplus=softplus)
    assert np.allclose(y2[1], full[1, 4:], rtol=1e-12, atol=1e-12)


def _differences(f, x, eps=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + eps
        hi = f()
        x[i] = keep - eps
        d[i] = (hi - f()) / (2 * eps)
        x[i] = keep
    return d


@pytest.mark.parametrize("lens", [None, [6, 0], [3, 1]], ids=str)
@pytest.mark.parametrize("softplus", [True, False])
def test_gradients_of_the_scan(lens, softplus):
    p, r = _scan(2)
    gy, gs = r.normal(size=p["u"].shape), r.normal(size=p["state"].shape)

    def loss():
        y, S = O.selective_scan(**p, softplus=softplus, lens=lens)
        return (y * gy).sum() + (S * gs).sum()
    got = O.selective_scan_grad(gy=gy, gstate=gs, softplus=softplus, lens=lens, **p)
    # a difference over 2e-6 does not resolve the rounding of the loss itself: its terms, some 64
    # roundings deep, are known to 64 * 2^-53 of their size (which grows where delta < 0)
    y, S = O.selective_scan(**p, softplus=softplus, lens=lens)
    blur = 64 * 2.0 ** -53 * (np.abs(y * gy).sum() + np.abs(S * gs).sum()) / 1e-6
    for name in got:
        want = _differences(loss, p["bias" if name == "dt_bias" else name])
        assert np.abs(got[name] - want).max() <= 1e-7 * max(1.0, np.abs(want).max()) + blur, name


@pytest.mark.parametrize("W", [1, 2, 4])
def test_the_convolution_is_numpys(W):
    r = np.random.default_rng(3)
    x, w, b, s = r.normal(size=(2, 7, 3)), r.normal(size=(3, W)), r.normal(size=3), r.normal(size=(2, W - 1, 3))
    y, S = O.causal_conv(x, w, b, "none", s, [7, 2])
    for e in range(3):
        full = np.concatenate([s[0, :, e], x[0, :, e]])
        assert np.allclose(y[0, :, e], np.convolve(full, w[e, ::-1], "valid") + b[e])
        assert np.allclose(S[0, :, e], full[7:])
        short = np.concatenate([s[1, :, e], x[1, :2, e]])
        assert np.allclose(y[1, :2, e], np.convolve(short, w[e, ::-1], "valid") + b[e]) and not y[1, 2:].any()
        assert np.allclose(S[1, :, e], short[2:])


@pytest.mark.parametrize("lens", [None, [6, 0], [2, 1]], ids=str)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_of_the_convolution(lens, act):
    r = np.random.default_rng(4)
    p = dict(x=r.normal(size=(2, 6, 3)), weight=r.normal(size=(3, 4)), bias=r.normal(size=3), state=r.normal(size=(2, 3, 3)))
    gy, gs = r.normal(size=p["x"].shape), r.normal(size=p["state"].shape)

    def loss():
        y, S = O.causal_conv(act=act, lens=lens, **p)
        return (y * gy).sum() + (S * gs).sum()
    got = O.causal_conv_grad(gy=gy, gstate=gs, act=act, lens=lens, **p)
    for name in got:
        want = _differences(loss, p[name])
        assert np.abs(got[name] - want).max() <= 1e-7 * max(1.0, np.abs(want).max()), name


def test_packing_keeps_half_a_step():
    r = np.random.default_rng(5)
    x = r.normal(size=(3, 70)) * np.exp(r.normal(size=(3, 1)) * 20)
    x[0, :32], x[1, 5], x[2, 40] = 0.0, np.inf, np.nan
    codes, exps, v = O.packed(x)
    assert codes.shape == (3, 70) and exps.shape == (3, 3) and (np.abs(codes.astype(int)) <= 127).all()
    for i in range(3):
        for k in range(3):
            at = slice(32 * k, min(32 * k + 32, 70))
            if (i, k) in ((1, 0), (2, 1)):
                assert exps[i, k] == 255 and np.isnan(v[i, at]).all()
                continue
            step = 2.0 ** (int(exps[i, k]) - 127)
            assert (np.abs(v[i, at] - x[i, at]) <= step / 2).all()
            if x[i, at].any():       # the least power of two: half of it would not reach
                assert np.abs(x[i, at]).max() > 127 * step / 2
            else:
                assert exps[i, k] == 1
