"""The sequence operators where a size or an offset passes 32 bits."""
import pytest
import torch

from test_gpu_sequence import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_spd_selected_amd as m
    m.lib()
    return m


def test_a_row_of_four_gib(ssa):
    """A row's outputs are 2^32 bytes: all of them are written, and the first
    ones are those of the row's beginning alone."""
    B, T, H, P, N = 1, 32768, 256, 256, 4
    say("selective_scan", B, T, H, P, N)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).bfloat16()

    x = normal(B, T, 1, P).expand(B, T, H, P)  # the heads share their input
    dt, Bm, Cm = normal(B, T, H), normal(B, T, 1, N), normal(B, T, 1, N)
    A = -torch.rand(H, generator=gen, device=DEV) - 0.5
    # memory that y is likely to get: an output that is not written shows
    torch.full((B * T * H * P,), float("nan"), dtype=torch.bfloat16, device=DEV)
    y, out = ssa.selective_scan(x, dt, A, Bm, Cm)
    assert y.numel() * y.element_size() == 2 ** 32
    assert all(torch.isfinite(v).all() for v in y.view(64, -1)) and torch.isfinite(out).all()
    head, _ = ssa.selective_scan(x[:, :256], dt[:, :256], A, Bm[:, :256], Cm[:, :256])
    assert torch.equal(y[:, :256], head)
    # and the last ones those of the end, from the state before it
    _, st = ssa.selective_scan(x[:, :-256], dt[:, :-256], A, Bm[:, :-256], Cm[:, :-256])
    tail, last = ssa.selective_scan(x[:, -256:], dt[:, -256:], A, Bm[:, -256:], Cm[:, -256:],
                                    state=st)
    assert torch.equal(y[:, -256:], tail) and torch.equal(out, last)


def test_sizes_past_32_bits_are_refused(ssa):
    """Not taken for what their lower halves say.  Without rows nothing is
    allocated."""
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=DEV)

    many, f32 = 2 ** 32 + 8, torch.float32
    for call in (
            lambda: ssa.short_conv(z(0, 1, many), z(1, 1, dtype=f32).expand(many, 1)),
            lambda: ssa.short_conv_step(z(0, many), z(0, 0, many), z(1, 1, dtype=f32).expand(many, 1)),
            lambda: ssa.qk_norm_rotate(z(0, 1, many, 8), None, z(8, dtype=f32), None),
            lambda: ssa.qk_norm_rotate(z(0, 1, 1, 8), z(0, 1, many, 8), z(8, dtype=f32),
                                       z(8, dtype=f32)),
            lambda: ssa.selective_scan(z(0, 1, many, 4), z(0, 1, many), z(1, dtype=f32).expand(many),
                                       z(0, 1, 1, 4), z(0, 1, 1, 4))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_scan_gradient_takes_what_it_needs(ssa):
    """bfloat16: two states a head and chunk of 64 tokens, the outputs, and the
    sums of the heads and of the shared B and C."""
    B, T, H, P, G, N = 2, 4096, 16, 64, 1, 128
    x, yb = (torch.ones(B, T, H, P, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Bm = torch.ones(B, T, G, N, dtype=torch.bfloat16, device=DEV)
    dt = torch.zeros(B, T, H, dtype=torch.bfloat16, device=DEV)
    A = -torch.ones(H, device=DEV)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = ssa.selective_scan_vjp(x, dt, A, Bm, Bm, yb)
    peak = torch.cuda.max_memory_allocated() - before
    states = 2 * B * H * (T // 64) * P * N * 4
    outputs = sum(g.numel() * g.element_size() for g in got if g is not None)
    # beside the states, an eighth of them each for the segments and for the slices of B and C
    assert peak <= 1.5 * states + outputs, (peak, states, outputs)
