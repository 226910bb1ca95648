"""How many samples group norm takes, as its header says; the size queries need no device."""

import pytest

import sparse_addressed_delta_gb300 as sdm

QUERIES = ["sdm_group_norm_workspace_bytes", "sdm_group_norm_backward_workspace_bytes"]


@pytest.mark.parametrize("query", QUERIES)
def test_samples(query):
    ask = getattr(sdm.library(), query)
    for N, L, C, G in ((1 << 24, 1, 4, 1), ((1 << 31) - (1 << 20), 1, 1, 1), (1 << 26, 1, 32, 16), (1 << 23, 9, 64, 4), (1 << 23, 1, 16384, 1)):
        assert ask(N, L, C, G) > 0, (N, L, C, G)
    for N, L, C, G in (((1 << 31) - (1 << 20) + 1, 1, 1, 1), (1 << 27, 1, 32, 16), ((1 << 23) + 1, 2, 64, 4), ((1 << 23) + 1, 1, 16384, 1),
                       (1 << 62, 1, 4, 4), (1, 1 << 31, 4, 4)):
        assert ask(N, L, C, G) == 0 and b"must be below 2^31" in sdm.library().sdm_last_error(), (N, L, C, G)


@pytest.mark.parametrize("query", QUERIES)
def test_nothing_needs_no_room(query):
    ask = getattr(sdm.library(), query)
    for N, L in ((0, 1), (0, 7), (1 << 23, 0), (1 << 40, 0), (0, 1 << 40)):
        assert ask(N, L, 16384, 4) == 256
