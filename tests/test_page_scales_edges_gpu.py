"""Page-scale attention at the ends of its arguments' ranges: windows near
2^31, query rows of far different size, pages of zeros."""

import math

import pytest
import torch

import speculative_decoding_draft_paged_gb300 as dflash
from tests._page8 import make_attn, ref_attn
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


@pytest.mark.parametrize("power", [-100, -30, -20, -10, -4, 4, 10, 20, 100])
@pytest.mark.parametrize("Hq,K,D", [(4, 1, 128), (4, 7, 64), (6, 7, 64), (16, 7, 128), (16, 8, 64)])
def test_a_row_far_from_the_others_in_size(cuda_device, power, Hq, K, D):
    """One query row of 2^power times the others' size.  Far from it the others
    are those of a call without it, and a quiet row is that of its own softmax;
    near, all are within the tolerance of their tile."""
    scale = float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32))
    for split in (0, 1):
        inp = make_attn(lens=[300, 40, 1100], Hq=Hq, Hkv=1, D=D, K=K, P=32, seed=22)
        plain = inp["q"].clone()
        odd = (plain[:, K // 2, 1].double() * 2.0 ** power).bfloat16()
        inp["q"][:, K // 2, 1] = odd
        got = call(inp, cuda_device, split=split)
        assert got[2] == 0
        if abs(power) <= 4:
            compare(inp, got)
            continue
        rest = torch.ones(K, Hq, dtype=torch.bool)
        rest[K // 2, 1] = False
        plain[:, K // 2, 1] = 0
        alone = torch.zeros_like(plain)
        alone[:, K // 2, 1] = odd
        for q, rows in ((plain, rest), (alone, ~rest)):
            if power > 0 and rows is not rest:
                continue  # scores of thousands and more
            ro, rl, to, tl = ref_attn(dict(inp, q=q), W=0, future_keys=1, right_window=0, scale=scale)
            assert ((got[0].double() - ro).abs() <= to)[:, rows].all()
            assert ((got[1].double() - rl).abs() <= tl)[:, rows].all()


@pytest.mark.parametrize("Hq,K,D,W", [(4, 7, 64, 0), (6, 7, 64, 90), (16, 7, 128, 0), (8, 1, 64, 0)])
def test_rows_of_every_size(cuda_device, Hq, K, D, W):
    """Rows from 2^-120 to 2^20, rows of zeros and one with a NaN in one tile,
    written over the queries' own memory or elsewhere."""
    inp = make_attn(lens=[200, 900, 0], Hq=Hq, Hkv=1, D=D, K=K, P=16, W=W, seed=26)
    plain = inp["q"].clone()
    power = torch.tensor([-120.0, -40.0, -25.0, 0.0, 0.0, 9.0, 20.0, 0.0])[torch.arange(K * Hq) % 8].view(1, K, Hq, 1)
    inp["q"] = (plain.double() * 2.0 ** power).bfloat16()
    inp["q"][:, -1, 0] = 0
    inp["q"][1, K // 2, 2, 5] = float("nan")
    got = call(inp, cuda_device, W=W)
    assert got[2] == 0
    scale = float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32))
    ok = torch.ones(3, K, Hq, dtype=torch.bool)
    ok[1, K // 2, 2] = False
    assert got[0][1, K // 2, 2].isnan().all() and got[1][1, K // 2, 2] == -math.inf
    for e in (-120.0, -40.0, -25.0, 0.0):
        rows = (power[0, :, :, 0] == e).expand(3, K, Hq) & ok
        q = torch.where(rows[..., None], inp["q"].float(), 0.0).bfloat16()
        ro, rl, to, tl = ref_attn(dict(inp, q=q), W=W, future_keys=1, right_window=0, scale=scale)
        assert ((got[0].double() - ro).abs() <= to)[rows].all(), e
        assert ((got[1].double() - rl).abs() <= tl)[rows].all(), e
    d = {n: t.to(cuda_device) for n, t in inp.items()}
    kw = dict(block_size=K, window=W, future_keys=1, scale=1.0 / math.sqrt(D), max_ctx_len=900)
    for split in (0, 100):
        want = call(inp, cuda_device, W=W, split=split)
        q = d["q"].clone()
        out, lse = dflash.block_attn_fp8_page_scales(q, *[d[n] for n in ("k", "v", "ks", "vs", "table", "ctx")], **kw, out=q,
                                                     force_split_tiles=split)
        assert torch.equal(out.view(torch.int16).cpu()[ok], want[0].view(torch.int16)[ok]) and torch.equal(lse.cpu(), want[1])


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
