"""Host-side checks (no GPU) of sizes at the edge of 32 bits in the paged-cache operators."""
import ctypes

import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import build as fabuild

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def _decode(lib, Hq, Sq):
    return lib.fa_decode_paged_fp8(P(16), P(16), P(16), P(4), P(4), P(4), P(4), None, None, P(16),
                                   None, 1, Hq, 1, Sq, 4, 8, 0, 16, 64, ctypes.c_float(0.1), P(256),
                                   1 << 40, None)


def _select(lib, Hq, Sq):
    return lib.fa_select_blocks(P(16), P(16), P(4), P(4), P(4), P(4), P(4), 1, Hq, 1, Sq, 4, 8, 16, 64,
                                4, 1, 1, P(256), 1 << 40, None)


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 9, (1 << 31) - 32])
def test_rows_that_overflow_when_rounded_up_are_refused(lib, rows):
    """Row tiles of up to 32 are counted in 32 bits."""
    for call in (_decode, _select):
        assert call(lib, 1, rows) == fa.FA_ERR_INVALID_ARG
        assert b"32-bit row indices" in lib.fa_last_error_detail()
    assert lib.fa_decode_paged_fp8_workspace_size(1, 1, 1, rows, 64) == 0


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 4), ((1 << 31), 3)])
def test_tensor_sizes_past_32_bits_are_refused(shape):
    """ctypes would pass their low 32 bits: a table of 2^32 + 4 blocks as one of 4."""
    table = torch.empty(shape, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="block_table.*32 bits"):
        fa._dims(table, "block_table", 2)


def test_workspace_sizes_of_arguments_past_32_bits_are_refused(lib):
    with pytest.raises(ValueError, match="32 bits"):
        fa.fa_select_blocks_workspace_size(1, 2, (1 << 32) + 16)
    for at in range(5):
        args = [1, 8, 2, 1, 64]
        args[at] += 1 << 32
        with pytest.raises(ValueError, match="32 bits"):
            fa.fa_decode_paged_fp8_workspace_size(*args)
