"""Pins of the sequence-mixing oracles (CPU): linear attention against its closed sum over
earlier tokens, group norm against torch, and every gradient against central differences."""
import numpy as np
import pytest
import torch

import oracle as O


def _attention(seed, B=2, T=7, H=4, Hkv=2, Dk=3, Dv=2, token=True):
    r = np.random.default_rng(seed)
    q, k, v = r.normal(size=(B, T, H, Dk)), r.normal(size=(B, T, Hkv, Dk)), r.normal(size=(B, T, Hkv, Dv))
    g = -r.exponential(0.4, size=(B, T, Hkv) if token else (Hkv,))
    return dict(q=q, k=k, v=v, g=g, state=r.normal(size=(B, Hkv, Dk, Dv))), r


@pytest.mark.parametrize("token", [True, False])
def test_linear_attention_is_the_decayed_sum_over_earlier_tokens(token):
    p, _ = _attention(1, token=token)
    lens = np.array([7, 4])
    o, S = O.linear_attention(p["q"], p["k"], p["v"], p["g"], 0.7, p["state"], lens)
    for b in range(2):
        for h in range(4):
            g = np.full(7, p["g"][h // 2]) if not token else p["g"][b, :, h // 2]
            for t in range(7):
                want = np.exp(g[:t + 1].sum()) * p["q"][b, t, h] @ p["state"][b, h // 2]
                for j in range(t + 1):
                    want = want + np.exp(g[j + 1:t + 1].sum()) * (p["q"][b, t, h] @ p["k"][b, j, h // 2]) * p["v"][b, j, h // 2]
                want = 0.7 * want if t < lens[b] else np.zeros(2)
                assert np.allclose(o[b, t, h], want, rtol=1e-12, atol=1e-12)
    # the state after row 1's four tokens continues like the whole sequence
    o2, _ = O.linear_attention(p["q"][:, 4:], p["k"][:, 4:], p["v"][:, 4:], p["g"][:, 4:] if token else p["g"], 0.7, S)
    full, _ = O.linear_attention(p["q"], p["k"], p["v"], p["g"], 0.7, p["state"])
    assert np.allclose(o2[1], full[1, 4:], rtol=1e-12, atol=1e-12)


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


@pytest.mark.parametrize("token", [True, False])
@pytest.mark.parametrize("lens", [None, [7, 0], [3, 1]])
def test_linear_attention_gradients_match_central_differences(token, lens):
    p, r = _attention(2, token=token)
    lens = None if lens is None else np.array(lens)
    go, gs = r.normal(size=(2, 7, 4, 2)), r.normal(size=p["state"].shape)

    def loss():
        o, S = O.linear_attention(p["q"], p["k"], p["v"], p["g"], 0.7, p["state"], lens)
        return (o * go).sum() + (S * gs).sum()
    d = O.linear_attention_grad(p["q"], p["k"], p["v"], p["g"], 0.7, go, p["state"], lens, gs)
    for name, key in (("q", "q"), ("k", "k"), ("v", "v"), ("state", "state"),
                      ("g", "log_decay" if token else "log_decay_head")):
        assert np.allclose(d[key], _differences(loss, p[name]), rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated,lens", [(False, None), (True, None), (False, [3, 0, 1]), (True, [2, 5, 9])])
def test_group_norm_gradients_match_central_differences(activation, gated, lens):
    r = np.random.default_rng(3)
    x, gate = r.normal(size=(3, 5, 6)) * 2 + 0.5, r.normal(size=(3, 5, 6)) if gated else None
    w, b, gy = r.normal(size=6), r.normal(size=6), r.normal(size=x.shape)

    def loss():
        return (O.group_norm(x, 2, w, b, gate, activation, 1e-3, lens)[0] * gy).sum()
    d = O.group_norm_grad(gy, x, 2, w, b, gate, activation, 1e-3, lens)
    for name, a in (("x", x), ("weight", w), ("bias", b), ("gate", gate)):
        if a is not None:
            assert np.allclose(d[name], _differences(loss, a), rtol=1e-5, atol=1e-7), name


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
def test_group_norm_matches_torch(activation):
    r = np.random.default_rng(4)
    x, w, b = r.normal(size=(3, 5, 12)) * 2 + 1, r.normal(size=12), r.normal(size=12)
    y, mean, rstd = O.group_norm(x, 3, w, b, None, activation, 1e-5)
    z = torch.nn.functional.group_norm(torch.from_numpy(x).transpose(1, 2), 3, torch.from_numpy(w), torch.from_numpy(b))
    z = {"none": lambda u: u, "silu": torch.nn.functional.silu,
         "gelu": lambda u: torch.nn.functional.gelu(u, approximate="tanh")}[activation](z).transpose(1, 2).numpy()
    assert np.allclose(y, z, rtol=1e-12, atol=1e-12)
    assert np.allclose(mean, x.reshape(3, 5, 3, 4).mean((1, 3)))
    assert np.allclose(rstd, (x.reshape(3, 5, 3, 4).var((1, 3)) + 1e-5) ** -0.5)
