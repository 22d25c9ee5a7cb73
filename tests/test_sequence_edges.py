"""Edges of the sequence operators that need no GPU: buffer sizes, refusals and the arithmetic of rows at the limits."""
import pytest
import torch

from sparse_spd_selected_b200 import build, selinv
from tests.test_sequence_abi import FAKE, scan_inputs


@pytest.fixture(scope="module")
def lib():
    build.build()
    return selinv.lib()


def test_backward_workspace_of_sequences_without_rows(lib):
    """The size that the query gives is the one that the call asks for: the parameters' partial sums, zero."""
    empty = scan_inputs(lines=1, rows=0, table=FAKE, live=0, sequences=2)
    size = lib.selinv_selective_scan_backward_workspace_size
    assert size(empty) >= 6 * 4 * 4 + 2 * 6 * 4
    assert size(scan_inputs(rows=0)) == 0 and lib.selinv_selective_scan_workspace_size(empty) == 0
    v = [FAKE] + [0] * 3 + [0] + [0] * 15 + [0, 0] + [FAKE, 0, 0, 0]
    assert lib.selinv_selective_scan_backward(empty, selinv._SCAN_GRADS.pack(*v), FAKE, size(empty) - 1, 0) == \
        selinv.ERR_WORKSPACE
