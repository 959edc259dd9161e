"""The scan gradient's workspace query of each type (the addresses are never
used)."""
import os

import pytest

import sparse_spd_selected_amd as ssa
from test_sequence_abi import P, scan


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssa.LIB_PATH):
        ssa.build()
    return ssa.lib()


def test_scan_gradient(lib):
    sizes = (4, 4096, 32, 64, 2, 128)
    own = lib.selinv_scan_vjp_bf16_workspace_bytes(*sizes)
    states = 2 * 4 * 64 * 32 * 64 * 128 * 4  # of 64 chunks a row
    assert states <= own <= 1.01 * states
    assert lib.selinv_scan_vjp_workspace_bytes(2, *sizes) >= own
    a = scan(**dict(zip("BTHPGN", sizes)))
    assert lib.selinv_scan_vjp_bf16(a, P, own - 1, None) == ssa.INVALID_ARG
    assert lib.selinv_scan_vjp_f16(a, P, own, None) == ssa.INVALID_ARG
    assert lib.selinv_scan_vjp_bf16_workspace_bytes(4, 4096, 32, 64, 3, 128) == 0
