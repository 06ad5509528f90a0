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


@pytest.mark.parametrize("T,F,want", [(1 << 20, 1 << 15, 2), (1 << 21, (1 << 14) + 128, 2), (1 << 30, 1 << 23, 2), ((1 << 20) - 64, 1 << 15, 7)])
def test_gated_training_counts_gradients_below_2_36(L, T, F, want):
    # G | U of 2^36 elements and dH are more than a GPU holds; the gradients' blocks are counted in 32 bits
    assert L.nvfp4_gated_fwd(FAKE, FAKE, T, 64, F, 0, FAKE, FAKE, FAKE, 0, None) == want
    assert L.nvfp4_gated_bwd(FAKE, FAKE, T, 64, F, 0, 1, FAKE, FAKE, 0, FAKE, 0, None) == want
    assert (L.nvfp4_gated_workspace_bytes(T, 64, F) == 0) == (want == 2)
