"""Refusals of the rotating append that need no GPU: nothing is launched."""

import pytest

from tests.test_page_scales_abi import append_params


def test_batches_whose_search_would_pass_32_bits(dflash_lib):
    """The device looks tokens up in cu_tokens with 32-bit places, which hold
    for up to 2^30 requests."""
    d = dflash_lib
    #        q, k, v, cos_sin, k_pages, v_pages, ks, vs, table, lens, cu, q_out, workspace, stream
    ptrs = [0] + [1 << 20] * 5 + [0, 0] + [1 << 20] * 3 + [0, 0, 0]
    for batch in ((1 << 30) + 1, (1 << 31) - 1):
        for total in (1, 28, 1 << 30):
            p = append_params(d, batch=batch, total_tokens=total, max_new_tokens=1)
            assert d.rope_append_kv_raw(p, *ptrs) == d.DFLASH_ERR_INVALID
