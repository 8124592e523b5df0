"""Host-side tests (no GPU) of the paged operators' arguments and index arithmetic where they go to their limits."""

import ctypes

import pytest

from test_paged import fake, index, tq2  # noqa: F401 (fixtures)


@pytest.mark.parametrize("window", [1, 5, 2 ** 62, 2 ** 63 - 2 ** 31, 2 ** 63 - 3, 2 ** 63 - 1])
def test_windows_up_to_64_bits(index, window):  # noqa: F811
    """Tokens before the first key (negative positions) and the widest windows that the call takes."""
    for n, kv, group in ((7, 2, 1), (9, 0, 2), (40, 33, 3), (3, 300, 1)):
        for causal in (0, 1):
            see = [{j for j in range(kv) if (j <= kv - n + i or not causal) and j > kv - n + i - window} for i in range(n)]
            for i in range(n):
                out = (ctypes.c_int * 2)()
                index.keys(n, kv, i, ctypes.c_longlong(window), causal, out)
                assert set(range(out[0], out[1])) == see[i] and out[0] >= 0
            out = (ctypes.c_int * 7)()
            index.item(n, kv, group, 0, 256, ctypes.c_longlong(window), causal, 128, out)
            some = set().union(*see)
            assert out[0] == n * group and out[2] == len({j // 128 for j in some}) and min(out[3:7]) >= 0
            assert set(range(out[3], out[4])) == some or not some
