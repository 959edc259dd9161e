"""Calls whose launch would have 2^32 threads or more are refused on the host
(the addresses are never used)."""
import os

import pytest

import sparse_spd_selected_amd as ssa
from test_sequence_abi import P, conv, qk, scan

ROOM = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssa.LIB_PATH):
        ssa.build()
    return ssa.lib()


def test_scan_gradient(lib):
    """512 threads a chunk and group."""
    for sfx, Q in (("f32", 32), ("f16", 32), ("bf16", 64)):
        for B, T, G in ((1, (1 << 23) * Q, 1), (1, (1 << 17) * Q, 64), (8, (1 << 20) * Q - Q + 1, 1)):
            a = scan(B=B, T=T, H=G, G=G, P=1, N=1)
            assert getattr(lib, "selinv_scan_vjp_" + sfx)(a, P, ROOM, None) == ssa.INVALID_ARG


def test_head_norm(lib):
    for T in range((1 << 26) - 3, (1 << 26) + 1):
        a = qk(B=1, T=T)
        assert lib.selinv_qkrot_bf16(a, None) == ssa.INVALID_ARG
        assert lib.selinv_qkrot_vjp_bf16(a, P, ROOM, None) == ssa.INVALID_ARG


def test_convolution_without_rows(lib):
    """The parameters' gradients of an empty batch: a thread a channel and tap."""
    a = conv(B=0, C=1 << 28)
    assert lib.selinv_conv_vjp_bf16(a, P, ROOM, None) == ssa.INVALID_ARG
