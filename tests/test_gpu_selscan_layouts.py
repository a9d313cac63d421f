"""The selective scan, the convolution and the 8-bit copies on layouts, sizes and devices that choose other code:
slices off any alignment, pools and batches large enough for the wide forms, many rows, many groups, tensors of
a device that is not the current one, two streams at once.

References are the same calls on plain layouts or parts (equal to the bit where sums have one order), or the
fp64 oracles with the tolerances of test_gpu_selscan.py and test_gpu_conv.py.
"""
import contextlib

import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr
from test_gpu_selscan import BF16, F32, GRADS, TOL, _case, _check, _f64, _near, _split


def _offset(t, by):
    """The same values, `by` elements into a wider row."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + by + 3, dtype=t.dtype, device=t.device)
    wide[..., by:by + t.shape[-1]] = t
    return wide[..., by:by + t.shape[-1]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("by", [1, 2, 4])
def test_slices_off_alignment(by, dtype):
    c, gy, gs = _case(40, 2, 90, 68, 16, 1, dtype)
    args, kw = _split(c)
    ref, dref = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    args = [a if a.dim() == 2 else _offset(a, by) for a in args]
    kw["z"] = _offset(kw["z"], by)
    got, d = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    assert torch.equal(ref["y"], got["y"]) and torch.equal(ref["state"], got["state"])
    for n in GRADS:
        assert torch.equal(dref[n], d[n]), n
    step = [a if a.dim() == 2 else a[:, 3] for a in args]
    one = pnr.selective_scan_step(*step, kw["state"].clone(), z=kw["z"][:, 3], D=kw["D"], dt_bias=kw["dt_bias"])
    two = pnr.selective_scan_step(*[a.contiguous() for a in step], kw["state"].clone(), z=kw["z"][:, 3].contiguous(), D=kw["D"],
                                  dt_bias=kw["dt_bias"])
    assert torch.equal(one["y"], two["y"]) and torch.equal(one["state"], two["state"])
    x, w = _offset(c["u"], by), torch.randn(68, 4, generator=torch.Generator().manual_seed(1)).cuda()
    a, b = pnr.causal_conv(x, w), pnr.causal_conv(c["u"], w)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["state"], b["state"])
    a, b = pnr.causal_conv_backward(x, w, gy), pnr.causal_conv_backward(c["u"], w, gy)
    assert torch.equal(a["x"], b["x"]) and torch.equal(a["weight"], b["weight"])
    p, q = pnr.checkpoint_pack(x), pnr.checkpoint_pack(c["u"])
    assert torch.equal(p.codes, q.codes) and torch.equal(p.exponents, q.exponents)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 1000, 16, 2), (130, 2050, 33, 1), (1030, 260, 8, 1)], ids=str)
def test_a_full_serving_batch_of_tokens(shape):
    """One token of many requests against the whole-sequence call over one token."""
    B, E, N, G = shape
    c, _, _ = _case(41, B, 1, E, N, G, BF16)
    args, kw = _split(c)
    ref = pnr.selective_scan(*args, **kw)
    pool = torch.zeros(B + 5, E, N, device="cuda")
    slots = torch.randperm(B + 5, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32).cuda()
    pool[slots.long()] = c["state"]
    r = pnr.selective_scan_step(*[a if a.dim() == 2 else a[:, 0] for a in args], pool, slots=slots, z=kw["z"][:, 0], D=kw["D"],
                                dt_bias=kw["dt_bias"])
    _near("y", r["y"], _f64(ref["y"][:, 0]), 2 * TOL[BF16])
    _near("state", r["state"][slots.long()], _f64(ref["state"]), 2 * TOL[F32])


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [True, False])
def test_rows_enough_for_one_segment(gated):
    """48 x 4096 channels fill the device, forwards and backwards, in one piece along time: against the
    same row alone, which is cut."""
    c, gy, gs = _case(42, 1, 100, 64, 16, 1, F32, gated=gated)
    args, kw = _split(c)
    a, da = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    B, rep = 48, 64
    big = {k: None if c[k] is None else c[k].repeat(B, 1, rep) for k in ("u", "dt", "z")}
    big.update({k: c[k].expand(B, -1, -1, -1) for k in ("B", "C")})
    kw = dict(D=c["D"].repeat(rep), z=big["z"], dt_bias=c["dt_bias"].repeat(rep), state=c["state"].repeat(B, rep, 1))
    args = [big["u"], big["dt"], c["A"].repeat(rep, 1), big["B"], big["C"]]
    b = pnr.selective_scan(*args, **kw)
    db = pnr.selective_scan_backward(*args, gy.repeat(B, 1, rep), grad_state=gs.repeat(B, rep, 1), **kw)
    _near("y", b["y"], _f64(a["y"].repeat(B, 1, rep)), 2 * TOL[F32])
    _near("state", b["state"], _f64(a["state"].repeat(B, rep, 1)), 2 * TOL[F32])
    for n in ("u", "dt") + (("z",) if gated else ()):
        _near(n, db[n], _f64(da[n].repeat(B, 1, rep)), 2 * TOL[F32])
    for n in ("B", "C"):
        _near(n, db[n], rep * _f64(da[n].repeat(B, 1, 1, 1)), 2 * TOL[F32])
    _near("A", db["A"], B * _f64(da["A"].repeat(rep, 1)), 2 * TOL[F32])
    _near("state", db["state"], _f64(da["state"].repeat(B, rep, 1)), 2 * TOL[F32])


@pytest.mark.gpu
@pytest.mark.parametrize("E,G", [(130, 130), (96, 32), (640, 5)], ids=str)
def test_many_groups(E, G):
    _check(*_case(43, 2, 70, E, 8, G, F32, lens=[70, 41]))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [None, [4999, 2500]], ids=["whole", "ragged"])
def test_few_channels_over_many_tokens(lens):
    """Long enough that the number of segments follows from the tokens alone.  Roundings of 2^-24 over 5000 tokens
    add like sqrt(5000) = 2^6.2, which is below the bound of 2^-17 too."""
    c, gy, gs = _case(47, 2, 5000, 5, 4, 1, F32, lens=lens)
    _check(c, gy, gs)


@pytest.mark.gpu
def test_a_single_token_has_no_stride():
    """Strides of a dimension of one element mean nothing, however large."""
    c, gy, gs = _case(44, 2, 1, 40, 16, 1, F32)
    args, kw = _split(c)
    ref = pnr.selective_scan(*args, **kw)
    odd = lambda t: t.as_strided(t.shape, (t.stride(0), 1 << 40, *t.stride()[2:]))  # noqa: E731
    kw["z"] = odd(kw["z"])
    args = [a if a.dim() == 2 else odd(a) for a in args]
    got, d = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    assert torch.equal(ref["y"], got["y"]) and torch.isfinite(d["u"]).all()
    c["u"], c["dt"], c["B"], c["C"], c["z"] = args[0], args[1], args[3], args[4], kw["z"]
    _check(c, gy, gs)


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [(1 << 24) + 1, (1 << 31) - 1, (1 << 31) + 5, (1 << 40) + (1 << 26) + 3])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_single_tokens_stride_is_in_no_offset(dtype, stride):
    """Strides whose lower 32 bits are large too."""
    c, gy, gs = _case(46, 2, 1, 40, 16, 1, dtype)
    args, kw = _split(c)
    ref, dref = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    odd = lambda t: t.as_strided(t.shape, (t.stride(0), stride, *t.stride()[2:]))  # noqa: E731
    kw["z"] = odd(kw["z"])
    args = [a if a.dim() == 2 else odd(a) for a in args]
    got, d = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    assert torch.equal(ref["y"], got["y"]) and torch.equal(ref["state"], got["state"])
    for n in GRADS:
        assert torch.equal(dref[n], d[n]), n


@pytest.mark.gpu
def test_a_large_batch_of_convolutions_is_its_rows():
    """Long runs of tokens a thread against short ones: outputs and input gradients have one order of sums."""
    g = torch.Generator().manual_seed(45)
    x = torch.randn(8, 1700, 4096, generator=g).to(BF16).cuda()
    gy = torch.randn(8, 1700, 4096, generator=g).to(BF16).cuda()
    w, bias = torch.randn(4096, 4, generator=g).cuda(), torch.randn(4096, generator=g).cuda()
    lens = torch.tensor([1700, 0, 1, 31, 32, 33, 1699, 800], dtype=torch.int32).cuda()
    a, da = pnr.causal_conv(x, w, bias=bias, lens=lens), pnr.causal_conv_backward(x, w, gy, bias=bias, lens=lens)
    gw = torch.zeros_like(w, dtype=torch.float64)
    for i in range(8):
        one = dict(bias=bias, lens=lens[i:i + 1])
        b, db = pnr.causal_conv(x[i:i + 1], w, **one), pnr.causal_conv_backward(x[i:i + 1], w, gy[i:i + 1], **one)
        assert torch.equal(a["y"][i], b["y"][0]) and torch.equal(a["state"][i], b["state"][0])
        assert torch.equal(da["x"][i], db["x"][0])
        gw += db["weight"].double()
    _near("weight", da["weight"], _f64(gw), 2.0 ** -18)


@pytest.mark.gpu
def test_calls_select_their_tensors_device(monkeypatch):
    c, gy, gs = _case(46, 2, 8, 32, 16, 1, F32)
    args, kw = _split(c)
    w = torch.randn(32, 4).cuda()
    dev = c["u"].get_device()

    def calls():
        a, b = pnr.selective_scan(*args, **kw), pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
        s = pnr.selective_scan_step(*[t if t.dim() == 2 else t[:, 0] for t in args], a["state"].clone(), dt_bias=c["dt_bias"])
        k = pnr.checkpoint_pack(c["u"])
        x = pnr.checkpoint_unpack(k, F32)
        f, d = pnr.causal_conv(c["u"], w), pnr.causal_conv_backward(k, w, gy)
        t = pnr.causal_conv_step(c["u"][:, 0], w, f["state"].clone())
        return [a["y"], b["A"], s["y"], k.codes, x, f["y"], d["x"], t["state"]]
    ref, seen = calls(), []

    @contextlib.contextmanager
    def select(device):
        seen.append(device)
        yield
    monkeypatch.setattr(torch.cuda, "device", select)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: dev + 1)
    for p, q in zip(ref, calls()):
        assert torch.equal(p, q)
    assert seen == [dev] * 8


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two calls in flight with workspaces of their own."""
    cases = [_case(47 + i, 2, 700, 256, 16, 1, BF16) for i in range(2)]
    calls = [(_split(c), gy, gs) for c, gy, gs in cases]
    ref = [pnr.selective_scan_backward(*a, gy, grad_state=gs, **kw) for (a, kw), gy, gs in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in calls], []
    for s, ((a, kw), gy, gs) in zip(streams, calls):
        with torch.cuda.stream(s):
            got.append(pnr.selective_scan_backward(*a, gy, grad_state=gs, **kw))
    for s in streams:
        s.synchronize()
    for r, g in zip(ref, got):
        for n in GRADS:
            assert torch.equal(r[n], g[n]), n


@pytest.mark.gpu
def test_a_workspace_of_the_callers_is_used_and_checked():
    c, gy, gs = _case(49, 1, 300, 64, 16, 1, F32)
    args, kw = _split(c)
    r = pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    dirty = torch.full_like(r["workspace"], 0xff)              # NaN all over: nothing is read that was not written
    again = pnr.selective_scan_backward(*args, gy, grad_state=gs, workspace=dirty, **kw)
    assert again["workspace"].data_ptr() == dirty.data_ptr()
    for n in GRADS:
        assert torch.equal(r[n], again[n]), n
    f = pnr.selective_scan(*args, **kw)
    dirty = torch.full_like(f["workspace"], 0xff)
    assert torch.equal(f["y"], pnr.selective_scan(*args, workspace=dirty, **kw)["y"])
    d = pnr.causal_conv_backward(c["u"], torch.ones(64, 4, device="cuda"), gy)
    dirty = torch.full_like(d["workspace"], 0xff)
    assert torch.equal(d["weight"], pnr.causal_conv_backward(c["u"], torch.ones(64, 4, device="cuda"), gy, workspace=dirty)["weight"])
    lens = torch.tensor([5], dtype=torch.int32).cuda()
    dirty = torch.full_like(r["workspace"], 0xff)
    short = pnr.selective_scan_backward(*args, gy, grad_state=gs, workspace=dirty, **{**kw, "lens": lens})
    assert all(torch.isfinite(short[n]).all() for n in GRADS)
