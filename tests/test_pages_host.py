"""Fork and compact refuse outputs that lie over what the call still reads (no GPU)."""
import pytest

from paged_kv_cache_448_b200 import _native

P = 1 << 20                     # addresses 1 MiB apart; never touched


@pytest.mark.parametrize("out", ["nbt", "ncl"])
@pytest.mark.parametrize("over", ["bt", "cl", "par", "fr", "nbt", "ncl"])
def test_fork_outputs_over_inputs(out, over):
    at = {n: (i + 2) * P for i, n in enumerate(("bt", "cl", "par", "fr", "nbt", "ncl"))}
    if out == over:
        return
    size = {"bt": 3 * 4 * 4, "cl": 3 * 4, "par": 5 * 4, "fr": 5 * 4, "nbt": 5 * 4 * 4, "ncl": 5 * 4}
    plane = (_native.Plane * 1)(_native.Plane(P, 4096))
    for shift in (0, size[over] - 4, 4 - size[out]):
        a = dict(at)
        a[out] = at[over] + shift
        assert _native.lib().pa_fork_sequences(plane, 1, 8, 16, a["bt"], 3, 4, a["cl"], a["par"],
                                               a["fr"], 5, a["nbt"], a["ncl"], None,
                                               None) == _native.PA_ERR_INVALID_ARG, shift


def test_compact_table_over_moves():
    plane = (_native.Plane * 1)(_native.Plane(P, 4096))
    for table in (2 * P, 2 * P + 8, 2 * P - 28):
        assert _native.lib().pa_compact_blocks(plane, 1, 8, 2 * P, 2, table, 8, None,
                                               None) == _native.PA_ERR_INVALID_ARG
