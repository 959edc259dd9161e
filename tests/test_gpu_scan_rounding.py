"""The selective scan in bfloat16 loses nothing but its outputs' own rounding.

An error e, relative to a value, moves the value's rounding to bfloat16 (whose
steps are 2^-8 of it at least) with a chance of 2 |e| / 2^-8 at most.  Sums held
in float32 throughout are off by a few of its roundings: eight of 2^-24 on
average, for the sums of up to two chunks taken here, move 2^9 2^-21 = 2^-12 of the outputs.  An
operand cut to two bfloat16 terms is off by up to 2^-18 of itself, 2^-19.3 at
random, and moves three times as many.
"""
import pytest
import torch

import seq_ref as sr
from test_gpu_scan import ref_inputs, scan_case
from test_gpu_sequence import say

pytestmark = pytest.mark.gpu
CASE = ("bf16", 16, 64, 4, 64, 2, 64, True, True, True, True, None, 0)


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_spd_selected_amd as m
    m.lib()
    return m


def moved(got, ref):
    return float((got.cpu() != ref.to(got.dtype)).double().mean())


def test_outputs_are_rounded_once(ssa):
    say("selective_scan", CASE)
    c = scan_case(*CASE)
    x, dt, A, Bm, Cm, Dv, bias, st = c[:8]
    y, _ = ssa.selective_scan(x, dt, A, Bm, Cm, Dv, bias, state=st)
    ry, _ = sr.selective_scan(softplus=True, lengths=None, **ref_inputs(c, None))
    assert moved(y, ry) <= 2.0 ** -12


def test_gradients_are_rounded_once(ssa):
    say("selective_scan_vjp", CASE)
    c = scan_case(*CASE)
    x, dt, A, Bm, Cm, Dv, bias, st, _, yb, sob = c
    got = ssa.selective_scan_vjp(x, dt, A, Bm, Cm, yb, sob, Dv, bias, state=st)
    ref = sr.grads(lambda **k: sr.selective_scan(softplus=True, lengths=None, **k),
                   ref_inputs(c, None), (sr.wide(yb), sr.wide(sob)))
    for g, name in ((got[0], "x"), (got[3], "Bm"), (got[4], "Cm")):
        assert moved(g, ref[name]) <= 2.0 ** -12, name
