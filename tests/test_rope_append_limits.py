"""Refusals of the rotating append that need no GPU: nothing is launched."""

import pytest
import torch

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


@pytest.fixture
def unlaunched(dflash_lib, monkeypatch):
    """The Python layer with CPU tensors taken for the current device's, and
    the library's call replaced: the arguments it would get."""
    calls = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(dflash_lib, "rope_append_kv_raw", lambda *args: calls.append(args) or 0)
    types = dflash_lib._types()
    monkeypatch.setattr(dflash_lib, "_types", lambda: types[:-1] + (lambda device: 0,))
    return calls


def cache(rows, B=2):
    pages = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    return dict(args=(None, rows, rows, None, pages, pages.clone(), torch.zeros(B, 4, dtype=torch.int32),
                      torch.zeros(B, dtype=torch.int32)), kw=dict(max_ctx_len=32))


def test_workspaces_that_do_not_hold_the_status_word(dflash_lib, unlaunched):
    d = dflash_lib
    c = cache(torch.zeros(2, 2, 64, dtype=torch.bfloat16))
    good = torch.zeros(256, dtype=torch.uint8)
    d.rope_append_kv(*c["args"], **c["kw"], workspace=good)
    d.rope_append_kv(*c["args"], **c["kw"], workspace=good[:4])
    assert [args[13] for args in unlaunched] == [good.data_ptr()] * 2
    for bad in (good[:0], good[:3], torch.zeros(1, dtype=torch.uint8).expand(256), good[::2]):
        with pytest.raises(ValueError, match="workspace"):
            d.rope_append_kv(*c["args"], **c["kw"], workspace=bad)
    assert len(unlaunched) == 2


def test_rows_by_request_name_the_batch(dflash_lib, unlaunched):
    """[B, K, H, D] rows carry their batch: one that is not ctx_lens' would be
    split among the requests in another way."""
    d = dflash_lib
    rows = torch.zeros(6, 4, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(6, 4, 3, 64, dtype=torch.bfloat16)
    c = cache(rows, B=6)
    assert d.rope_append_kv(q, *c["args"][1:], **c["kw"]).shape == q.shape
    p = unlaunched[0][0]
    assert (p.batch, p.total_tokens, p.max_new_tokens) == (6, 24, 4)
    for B in (2, 3, 8, 12):
        c = cache(rows, B=B)
        with pytest.raises(ValueError, match="requests"):
            d.rope_append_kv(*c["args"], **c["kw"])
    c = cache(rows.view(24, 2, 64), B=6)
    for wrong in (q.view(4, 6, 3, 64), q.view(3, 8, 3, 64)):
        with pytest.raises(ValueError, match="requests"):
            d.rope_append_kv(wrong, *c["args"][1:], **c["kw"])
    # With cu_tokens the rows are packed, whatever their first two sizes.
    cu = torch.tensor([0, 5, 24], dtype=torch.int32)
    c = cache(rows, B=2)
    d.rope_append_kv(*c["args"], **c["kw"], cu_tokens=cu, max_new_tokens=19)
    p = unlaunched[1][0]
    assert (p.batch, p.total_tokens, p.max_new_tokens) == (2, 24, 19)
    assert len(unlaunched) == 2


def test_rows_of_other_ranks(dflash_lib, unlaunched):
    d = dflash_lib
    rows = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = cache(rows)
    for q in (torch.zeros(64, dtype=torch.bfloat16), torch.zeros((), dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="q"):
            d.rope_append_kv(q, *c["args"][1:], **c["kw"])
    assert not unlaunched
