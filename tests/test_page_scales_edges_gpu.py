"""Page-scale attention at the ends of its arguments' ranges: windows near
2^31, pages of zeros and value scales far apart."""

import pytest
import torch

import speculative_decoding_draft_paged_gb300 as dflash
from tests._page8 import make_attn
from tests.test_page_scales_gpu import call, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 100, 2 ** 30 + 1, 308])
@pytest.mark.parametrize("future_keys,right_window", [(1, 0), (0, 0), (0, 2)])
@pytest.mark.parametrize("D,Hq", [(128, 16), (64, 4)])
def test_windows_that_reach_every_key(cuda_device, window, future_keys, right_window, D, Hq):
    """A window as long as the context or longer masks nothing, up to the
    largest number its field holds."""
    inp = make_attn(lens=[0, 1, 100, 120, 128, 300], Hq=Hq, Hkv=1, D=D, K=7, P=32, seed=21)
    kw = dict(W=window, future_keys=future_keys, right_window=right_window)
    got = call(inp, cuda_device, **kw)
    assert got[2] == 0
    compare(inp, got, **kw)


@pytest.mark.parametrize("D,K,Hq", [(64, 1, 4), (64, 7, 4), (64, 7, 6), (128, 7, 16)])
@pytest.mark.parametrize("zero", ["first", "middle", "last", "all", "all but one"])
def test_appended_pages_of_zeros(cuda_device, D, K, Hq, zero):
    """Value rows of zeros (a slot's scale is then 2^-100, the least that the
    append writes) beside slots of ordinary values, then attention over them."""
    dev, P, n = cuda_device, 32, 700
    g = torch.Generator().manual_seed(23)
    pages = (n + P - 1) // P
    rows = torch.randn((2, n, 1, D), generator=g).bfloat16()
    slots = {"first": [0, 1], "middle": [9, 10], "last": [pages - 1], "all": list(range(pages)),
             "all but one": [s for s in range(pages) if s != 12]}[zero]
    for s in slots:
        rows[1, s * P:(s + 1) * P] = 0
    kp, vp = (torch.zeros(pages, 1, P, D, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(pages, 1, device=dev) for _ in range(2))
    table = torch.randperm(pages, generator=g).int()[None].to(dev)
    zero_len = torch.zeros(1, dtype=torch.int32, device=dev)
    dflash.rope_append_kv(None, rows[0].to(dev), rows[1].to(dev), None, kp, vp, table, zero_len, max_ctx_len=0, k_scales=ks, v_scales=vs)
    assert {float(vs[table[0, s].item(), 0]) for s in slots} == {2.0 ** -100}
    inp = {"q": torch.randn((1, K, Hq, D), generator=g).bfloat16(), "k": kp.cpu(), "v": vp.cpu(), "ks": ks.cpu(), "vs": vs.cpu(),
           "table": table.cpu(), "ctx": torch.tensor([n - K], dtype=torch.int32)}
    for split in (0, 1, 6):
        got = call(inp, dev, split=split)
        assert got[2] == 0
        ro = compare(inp, got)
        assert (ro == 0).all() == (zero == "all")


def test_value_scales_over_the_whole_range(cuda_device):
    """Scales of 2^-100 with codes that are not zero, alone and beside
    ordinary ones, in either order; a dominant key on either kind of page."""
    for low, high in ((2.0 ** -100, 2.0 ** -100), (2.0 ** -100, 2.0 ** -8), (2.0 ** -70, 2.0 ** -8)):
        for first_low in (True, False):
            for loud in (None, 0, 20):
                inp = make_attn(lens=[1000], Hq=6, Hkv=1, D=64, K=7, P=32, seed=24)
                ids = inp["table"][0, :32].long()
                quiet = (torch.arange(32) < 16) == first_low
                inp["vs"][ids, 0] = torch.where(quiet, torch.tensor(low), torch.tensor(high))
                if loud is not None:
                    inp["ks"][ids[loud], 0] *= 12
                got = call(inp, cuda_device)
                assert got[2] == 0
                compare(inp, got)
