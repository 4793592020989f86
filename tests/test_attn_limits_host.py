"""Host-side limits of the attention sublayer (no GPU): sizes whose indices
would leave the kernels' integers are refused before any launch."""

import pytest

from mhc_pre_gb300 import binding as B
from mhc_pre_gb300 import build as mbuild

A = 0x7F0000000000          # never dereferenced, 16-byte aligned


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return B.lib()


def _sizes(B_, Hk, T=1 << 20):
    return (T, B_, Hk, Hk, 64, 16)          # T, B, Hq, Hk, Dh, page_size


@pytest.mark.parametrize("dt", [B.MHC_BF16, B.MHC_F32])
@pytest.mark.parametrize("seqs,Hk", [(1 << 24, 16), (1 << 24, 64), (1 << 19, 1024)])
def test_more_join_counters_than_32_bits_number(L, seqs, Hk, dt):
    """8 counters for each tile and key head; every sequence may have a tile."""
    sizes = _sizes(seqs, Hk)
    assert seqs * Hk * 8 >= 2 ** 31
    assert L.mhc_paged_attn_workspace_bytes(dt, *sizes, 1) == 0
    assert L.mhc_paged_attn_plan(dt, A, A, *sizes, 1, 64, 0, A, 1 << 60, None) == B.MHC_ERR_UNSUPPORTED
    T, _, Hq, _, Dh, page = sizes
    assert L.mhc_paged_attn(dt, A, Hq * Dh, A, page * Hk * Dh, Hk * Dh, Dh, A, page * Hk * Dh, Hk * Dh, Dh, 100, page,
                            A, 4, A, A, T, seqs, Hq, Hk, Dh, 1, 64, 0, 0.125, 0.0, A, A, A, 1 << 60,
                            None) == B.MHC_ERR_UNSUPPORTED


@pytest.mark.parametrize("seqs,Hk", [(1 << 24, 8), (1 << 18, 512)])
def test_join_counters_that_fit(L, seqs, Hk):
    assert (seqs + 4096) * Hk * 8 < 2 ** 31
    assert L.mhc_paged_attn_workspace_bytes(B.MHC_BF16, *_sizes(seqs, Hk, 1 << 10), 1) > seqs * Hk * 32
