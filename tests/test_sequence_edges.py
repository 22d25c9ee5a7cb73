"""Edges of the sequence operators that need no GPU: buffer sizes, refusals and the arithmetic of rows at the limits."""
import subprocess

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


def test_pieces_end_within_the_line(tmp_path):
    """Segments and chunks cover a line up to the most rows that one may have, whatever their length."""
    src = tmp_path / "pieces.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#include "pieces.h"
int main()
{
    long long bad = 0;
    for (int rows : {0x7fffffff - 64, 0x7fffffff - 65, 0x7fffffff - 200, 0x7fffffff - 2600, 1000, 1})
        for (int pieces = 1; pieces <= 160; ++pieces)
            for (int round : {4, 16, 128}) {
                const long long step = ((1LL * rows + pieces - 1) / pieces + round - 1) / round * round;
                long long at = 0;
                for (long long r0 = 0; r0 < rows; r0 += step) {
                    const int end = selinv::piece_end((int)r0, (int)(step < 0x7fffffff ? step : 0x7fffffff), rows);
                    bad += r0 != at || end <= r0 || end - r0 > step;
                    at = end;
                }
                bad += at != rows;
            }
    printf("%lld\\n", bad);
}
""")
    exe = tmp_path / "pieces"
    subprocess.check_call(["g++", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover", "-I",
                           build.CSRC, str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)]).decode().strip() == "0"


def test_steps_refuse_arrays_in_the_cache_that_is_written(lib):
    """Addresses alone decide; what passes them is not called here."""
    from tests.test_sequence_abi import step
    cache = FAKE + (1 << 20)                # 3 slots x 6 channels x 4 states: 288 bytes
    apart = dict(cache=cache, out=cache)
    for at in (cache, cache + 284, cache - 4):
        for key in ("x", "dt", "z", "B", "C", "y", "A", "D", "bias", "index", "info"):
            assert lib.selinv_selective_scan_step(step(**{**apart, key: at}), 0) == selinv.ERR_INVALID_ARG, key
    for at in (cache + 4, cache - 284):
        assert lib.selinv_selective_scan_step(step(cache=at, out=cache), 0) == selinv.ERR_INVALID_ARG

    def conv(**change):
        v = dict(dtype=selinv.F32, flags=0, batch=3, slots=3, d=6, k=4, x=FAKE, weight=FAKE, bias=0, cache=cache, xr=6, yr=6,
                 out=cache, y=FAKE, index=0, info=0)        # 3 slots x 3 rows x 6 channels: 216 bytes
        v.update(change)
        return lib.selinv_causal_conv_step(selinv._CONV_STEP.pack(*v.values()), 0)

    for at in (cache, cache + 212, cache - 4):
        for key in ("x", "weight", "bias", "y", "index", "info"):
            assert conv(**{key: at}) == selinv.ERR_INVALID_ARG, key
    assert conv(cache=cache + 4) == selinv.ERR_INVALID_ARG
