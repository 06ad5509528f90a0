"""Sizes at the ends of what the gated projection and the adapters take, without a GPU: refused before anything else."""
import ctypes

import pytest

from nvfp4_bit_microscaled_b200 import _lib, build as libbuild

FAKE, BIG = 1 << 20, 1 << 50   # an address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.lib()


def _t(rows, cols):
    return ctypes.byref(_lib.Nvfp4Tensor(4096, 8192, 16384, rows, cols))


@pytest.mark.parametrize("C,want", [(1 << 24, 2), (1 << 28, 2), ((1 << 31) - 64, 2), ((1 << 24) - 64, 7)])
@pytest.mark.parametrize("T", [1, 128, 129])
def test_gated_apply_counts_blocks_in_32_bits(L, T, C, want):
    # 128 rows of 2^28 columns have 2^31 blocks of 16
    assert L.nvfp4_gated_apply(FAKE, T, C, _t(256, C), 0, FAKE, 128, FAKE, 0, None) == want
    assert (L.nvfp4_gated_apply_workspace_bytes(T, C) == 0) == (want == 2)
