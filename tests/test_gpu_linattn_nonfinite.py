"""Infinities and NaNs in the linear attention: which results they reach."""
import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@pytest.mark.gpu
@DTYPES
@pytest.mark.parametrize("B,Dk", [(1, 1), (2, 16), (3, 100), (70, 24), (2, 128)])
def test_a_single_token_with_an_infinite_value(B, Dk, dtype):
    """Keys and queries of one sign: the state's column and the output are that infinity, as the formula says."""
    gen = torch.Generator().manual_seed(Dk)
    q, k = (torch.rand(B, 4, Dk, generator=gen).add(0.5).to(dtype).cuda() for _ in range(2))
    v = torch.randn(B, 4, 12, generator=gen).to(dtype).cuda()
    v[0, 1, 5], v[B - 1, 2, 0] = float("inf"), float("-inf")
    g = torch.full((4,), -0.5, device="cuda")
    r = pnr.linear_attention_step(q, k, v, g, torch.zeros(B, 4, Dk, 12, device="cuda"))
    bad = torch.zeros(B, 4, 12, dtype=torch.bool, device="cuda")
    bad[0, 1, 5] = bad[B - 1, 2, 0] = True
    assert r["o"][0, 1, 5] == float("inf") and r["o"][B - 1, 2, 0] == float("-inf")
    assert torch.isfinite(r["o"][~bad]).all()
    assert (r["state"][0, 1, :, 5] == float("inf")).all() and (r["state"][B - 1, 2, :, 0] == float("-inf")).all()
    assert torch.isfinite(r["state"].transpose(2, 3)[~bad]).all()


# rows that are cut into segments of a chunk, and many rows whose blocks walk all chunks
REACH = pytest.mark.parametrize("shape", [(2, 200, 4, 2, 64, 64), (80, 200, 8, 4, 24, 40)],
                                ids=lambda s: "x".join(map(str, s)))


@pytest.mark.gpu
@REACH
@DTYPES
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "grad_o"])
def test_what_a_token_reaches(where, junk, dtype, shape):
    """Token t of one row, in one head: everything that the formula computes without it stays finite.
    o_i and dq_i follow the state S_i (tokens up to i), dk_i and dv_i the state's gradient D_i (q and grad_o
    from i on, decays behind i), and each its own row besides."""
    B, T, H, Hkv, Dk, Dv = shape
    G, t, h = H // Hkv, 100, 1
    gen = torch.Generator().manual_seed(5)
    draw = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    a = dict(q=draw(B, T, H, Dk).to(dtype).cuda(), k=draw(B, T, Hkv, Dk).to(dtype).cuda(),
             v=draw(B, T, Hkv, Dv).to(dtype).cuda(), grad_o=draw(B, T, H, Dv).to(dtype).cuda(),
             log_decay=-torch.empty(B, T, Hkv).exponential_(10.0, generator=gen).cuda())
    a[where][(0, t, h * G if where in ("q", "grad_o") else h) + (() if where == "log_decay" else (3,))] = junk
    x, state, gs = [a[n] for n in ("q", "k", "v", "log_decay")], draw(B, Hkv, Dk, Dv).cuda(), draw(B, Hkv, Dk, Dv).cuda()
    f = pnr.linear_attention(*x, state=state)
    d = pnr.linear_attention_backward(*x, a["grad_o"], state=state, grad_state=gs)
    tok, past = torch.arange(T).cuda(), torch.zeros(T, dtype=torch.bool).cuda()
    later, earlier, own = tok >= t, tok < t, tok == t
    state_moved = where in ("k", "v", "log_decay")
    grad_moved = {"q": earlier | own, "grad_o": earlier | own, "log_decay": earlier}.get(where, past)
    may = dict(o=later if state_moved else own if where == "q" else past,
               dq=later if state_moved else own if where == "grad_o" else past,
               dk=grad_moved | (own if where == "v" else past), dv=grad_moved | (own if where == "k" else past))
    for n, got, heads in (("o", f["o"], range(h * G, h * G + G)), ("dq", d["q"], range(h * G, h * G + G)),
                          ("dk", d["k"], [h]), ("dv", d["v"], [h])):
        bad = ~torch.isfinite(got).all(-1)                    # [B, T, heads]
        for i in heads:
            # q and grad_o belong to one of the query heads that share the state
            allowed = past if where in ("q", "grad_o") and n in ("o", "dq") and i != h * G else may[n]
            assert not (bad[0, :, i] & ~allowed).any(), (n, i, bad[0, :, i].nonzero().flatten().tolist())
            bad[0, :, i] = False
        assert not bad.any(), n
    others = torch.ones(B, Hkv, dtype=torch.bool).cuda()
    others[0, h] = False
    for n, got, moved in (("state", f["state"], state_moved), ("dstate", d["state"], where in ("q", "grad_o", "log_decay"))):
        fine = torch.isfinite(got).all(-1).all(-1)
        assert fine[others].all() and (moved or fine.all()), n
    # the decay's gradient adds up along the row: a NaN may reach all of its row and head
    assert torch.isfinite(d["log_decay"]).all(1)[others].all()
