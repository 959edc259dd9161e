"""Values that are not finite stay where they are: nothing past a row's end
takes them up, and a row without tokens gives nothing to the parameters."""
import pytest
import torch

import seq_ref as sr
from test_gpu_sequence import DEV, TYPES, say, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_spd_selected_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ty,T,C,W", [("bf16", 21, 64, 4), ("f32", 21, 5, 3), ("f16", 40, 24, 7),
                                      ("f32", 9, 8, 2), ("bf16", 1031, 4096, 4)])
def test_short_conv_gradient(ssa, ty, T, C, W, bad, silu):
    say("short_conv_vjp", ty, T, C, W, bad, silu)
    B = 4  # a whole row, one that ends inside a run, one that ends at four tokens, an empty one
    lengths = [T, T - 5, 4, 0]
    r = sr.rng(C + T)
    x, yb = (up(sr.normal(r, B, T, C), TYPES[ty]) for _ in range(2))
    st, sob = (up(sr.normal(r, B, W - 1, C), TYPES[ty]) for _ in range(2))
    w, b = up(sr.normal(r, C, W)), up(sr.normal(r, C))
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)

    def vjp(x, st):
        return ssa.short_conv_vjp(x, w, b, yb, sob, silu=silu, state=st, lengths=ln)

    want = vjp(x, st)
    # the empty row's past: its own gradient is the output's, and no sum sees it
    odd = st.clone()
    odd[3] = bad
    for got, ref in zip(vjp(x, odd), want):
        assert torch.equal(got, ref)
    # a row's last token: nothing past the end, nothing of another row
    odd = x.clone()
    odd[1, T - 6], odd[2, 3] = bad, bad
    got = vjp(odd, st)
    for i, n in enumerate(lengths):
        assert not got[0][i, n:].any(), i
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][3], want[0][3])
    # ... nor of the tokens that do not meet it
    assert torch.equal(got[0][1, :T - 5 - W], want[0][1, :T - 5 - W])
    if not silu:  # linear: the inputs' gradients do not depend on the inputs
        assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])


@pytest.mark.parametrize("ty,H,P,G,N", [("bf16", 4, 64, 2, 128), ("bf16", 3, 20, 1, 7),
                                        ("f32", 2, 64, 1, 32), ("f16", 2, 33, 2, 20)])
def test_selective_scan_gradient(ssa, ty, H, P, G, N):
    """States and their cotangents that are not finite spoil their row's tokens
    alone, not the padding behind them; an empty row's spoil no sum."""
    say("selective_scan_vjp", ty, H, P, G, N)
    B, T, lengths = 3, 100, [100, 37, 0]
    r = sr.rng(P)
    x, yb = (up(sr.normal(r, B, T, H, P), TYPES[ty]) for _ in range(2))
    Bm, Cm = (up(sr.normal(r, B, T, G, N), TYPES[ty]) for _ in range(2))
    dt, st, sob = up(sr.normal(r, B, T, H), TYPES[ty]), up(sr.normal(r, B, H, P, N)), up(
        sr.normal(r, B, H, P, N))
    A, D, bias = -up(sr.normal(r, H).abs()) - 0.1, up(sr.normal(r, H)), up(sr.normal(r, H) - 1)
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)

    def vjp(st, sob):
        return ssa.selective_scan_vjp(x, dt, A, Bm, Cm, yb, sob, D, bias, state=st, lengths=ln)

    want = vjp(st, sob)
    for bad in (float("nan"), float("inf")):
        for row in (1, 2):
            s, o = st.clone(), sob.clone()
            s[row], o[row] = bad, bad
            got = vjp(s, o)
            for k in (0, 1, 3, 4):  # the tokens' gradients: x, dt, B, C
                for i, n in enumerate(lengths):
                    assert not got[k][i, n:].any(), (bad, row, k, i)
                    if i != row:
                        assert torch.equal(got[k][i], want[k][i])
            if row == 2:
                for k in (2, 5, 6):
                    assert torch.equal(got[k], want[k])
