"""The sequence kernels where a call's sizes choose another way through them:
long runs of the convolution, many heads of a workgroup and many segments of a
row in the scan.  References and tolerances are those of the operators' tests."""
import pytest
import torch

import test_gpu_scan as scan
import test_gpu_sequence as sequence
from test_gpu_sequence import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_spd_selected_amd as m
    m.lib()
    return m


# Sixteen tokens a thread: 1024 wavefronts or more with those.
@pytest.mark.parametrize("case", sequence.CONV_LONG + [
    ("bf16", 2, 2060, 2064, 2, True, False, True, (2060, 17), 0)], ids=str)
def test_short_conv_long_runs(ssa, case):
    sequence.test_short_conv(ssa, case)


# A workgroup of the gradient takes heads in turn.  Its heads are split up while
# rows x chunks x groups x parts < 256 and a part has a head or two at least, so
# these have
HEADS = [
    # 8 rows x 9 chunks of 64 x 4 groups: five heads in turn
    ("bf16", 8, 520, 20, 16, 4, 16, True, True, True, True, None, 0),
    # 10 x 5 x 2, four parts of fourteen heads: 4, 4, 4 and 2, in two tiles of P
    ("bf16", 10, 300, 28, 66, 2, 8, True, True, True, True,
     (300, 0, 299, 64, 65, 1, 128, 200, 300, 30), 0),
    # 16 x 9 chunks of 32 x 2 groups: five heads, no whole vectors
    ("f32", 16, 257, 10, 5, 2, 6, True, True, True, True, None, 0),
    # 20 x 7 x 2: seven heads, two tiles of P
    ("f16", 20, 200, 14, 96, 2, 20, True, False, True, False, None, 0),
]


@pytest.mark.parametrize("case", HEADS, ids=str)
def test_scan_gradient_of_many_heads(ssa, case):
    scan.test_selective_scan_vjp(ssa, case)


# (segments of the forward call, of the gradient's sweeps), case
SEGMENTS = [
    # two heads a workgroup, the state's columns shared out, rows that end inside
    # a segment and before the last one
    ((6, 6), ("bf16", 2, 1700, 2, 64, 1, 128, True, True, True, True, (1700, 777), 0)),
    # more than the ten segments that one batch of the chain takes
    ((13, 13), ("bf16", 1, 3300, 2, 16, 1, 128, True, True, True, True, None, 0)),
    ((14, 14), ("f32", 1, 2100, 2, 20, 1, 33, True, True, True, True, None, 0)),
    # one head a workgroup, no whole vectors
    ((4, 4), ("f16", 2, 600, 3, 40, 3, 50, True, True, True, True, (600, 411), 0)),
    ((8, 8), ("f16", 1, 1200, 4, 64, 2, 128, True, True, True, True, None, 0)),
]


def padded(P, N):
    return (P + 63) // 64 * 64 * (32 if N <= 32 else 64 if N <= 64 else 128) * 4


@pytest.mark.parametrize("want,case", SEGMENTS, ids=str)
def test_scan_in_segments(ssa, want, case):
    ty, B, T, H, P, G, N = case[:7]
    room = ssa.lib().selinv_scan_workspace_bytes(4 if ty == "f32" else 2, B, T, H, P, N)
    assert room >= want[0] * B * H * padded(P, N)
    scan.test_selective_scan(ssa, case)


@pytest.mark.parametrize("want,case", SEGMENTS, ids=str)
def test_scan_gradient_in_segments(ssa, want, case):
    ty, B, T, H, P, G, N = case[:7]
    if ty == "bf16":
        room = ssa.lib().selinv_scan_vjp_bf16_workspace_bytes(B, T, H, P, G, N)
    else:
        room = ssa.lib().selinv_scan_vjp_workspace_bytes(4 if ty == "f32" else 2, B, T, H, P, G, N)
    chunks = -(-T // (64 if ty == "bf16" else 32))
    states = 2 * B * H * chunks * padded(P, N)
    # at most: B's and C's where a group's heads are split, and the sums' places
    parts = (2 * H // G * B * T * G * N * 4 if H > G else 0) + 4096
    assert room - states - parts >= (2 * want[1] - 1) * B * H * padded(P, N)
    scan.test_selective_scan_vjp(ssa, case)


def test_same_bits_in_segments(ssa):
    case = SEGMENTS[0][1]
    say("selective_scan", case)
    x, dt, A, Bm, Cm, Dv, bias, st, ln, yb, sob = scan.scan_case(*case)
    runs = [ssa.selective_scan(x, dt, A, Bm, Cm, Dv, bias, state=st, lengths=ln) +
            ssa.selective_scan_vjp(x, dt, A, Bm, Cm, yb, sob, Dv, bias, state=st, lengths=ln)
            for _ in range(3)]
    for other in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], other))
