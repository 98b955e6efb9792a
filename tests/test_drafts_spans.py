"""Arrays that lie between each other's rows: refused by their spans, as the header says, before
any HIP call."""
import pytest

from test_drafts_refusals import BAD, FORK, MiB, changed, no_gpu_only
from vocab_wide_add_amd import native


@no_gpu_only
@pytest.mark.parametrize("at", [
    {3: 16, 12: 16, 11: 2 * MiB + 32},                   # both tables in one of twice the width
    {12: 64, 13: 6 * MiB + 32},                          # copies, written, behind the new table's first row
    {12: 64, 4: 6 * MiB + 32},
])
def test_fork_tables_between_rows(at):
    assert native.load().xpress_kv_fork(*changed(FORK, at), None) == BAD


@no_gpu_only
def test_states_between_rows():
    def go(states):
        return native.load().xpress_beam_reorder(b"".join(native._STATE.pack(*s) for s in states), len(states), MiB, 4, 6,
                                                 None)
    # two halves of one buffer's rows, written; read and written
    assert go([(2 * MiB, 4 * MiB, 64, 128, 64), (3 * MiB, 4 * MiB + 64, 64, 128, 64)]) == BAD
    assert go([(2 * MiB, 2 * MiB + 64, 128, 128, 64)]) == BAD
    # src between the rows that are written
    assert go([(2 * MiB, MiB - 64, 64, 256, 64)]) == BAD
