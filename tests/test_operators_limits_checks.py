"""CPU checks of the operators around the GEMMs at the top of their sizes: what is refused on the host."""
from __future__ import annotations

import pytest

import moe_grouped_gemm_08_b200 as fg

P = 0x10000  # a fake aligned address: these calls fail before any dereference


@pytest.mark.parametrize("M", [2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1])
def test_dispatch_refuses_rows_whose_scales_have_no_leading_dimension(M):
    assert fg.lib.fg_moe_dispatch_fp8(P, P, P, P, 4, 2, 1, M, 16, 0, None) == 3
