"""Page-scale attention where few keys hold most of a row's weight: the long
tail behind them must keep its share of the output.

References are plain 64-bit torch on the device.  Tolerances: an output element
is rounded to bf16 (at most 2^-8 of it, 2^-8 / sqrt(3) in the mean square), a
probability to two E4M3 terms and f16 (relative 2^-8.7 at most), and the keys of
a tile that a far louder key shares are dropped below 2^-19 of that key.  With
values of mean zero the probabilities' errors average out: relative L2 of 5e-3
holds with room, and so does 1e-2 absolute, beside the rounding of the output,
at values of about 1.  With equal scores and equal values they add up: 2^-8 +
2^-8.6 relative.  The LSE's sums are fp32 over up to 1024 tiles: 1024 2^-24
log2(e), less than 2^-13.
"""

import math

import pytest
import torch

import speculative_decoding_draft_paged_gb300 as dflash

pytestmark = pytest.mark.gpu

REL_L2, ABS, LSE = 5e-3, 1e-2, 2.0 ** -13
COHERENT = 2.0 ** -8 + 2.0 ** -8.6


def reference(d, scale):
    """(out, lse2) of one request, every key seen by every row."""
    K, Hq, D = d["q"].shape[1:]
    Hkv, P = d["k"].shape[1:3]
    n = int(d["ctx"][0]) + K
    ids = d["table"][0, :(n + P - 1) // P].long()
    out = torch.empty(K, Hq, D, dtype=torch.float64, device=d["q"].device)
    lse = torch.empty(K, Hq, dtype=torch.float64, device=d["q"].device)
    G = Hq // Hkv
    for h in range(Hkv):
        def rows(codes, scales):
            x = codes.view(torch.float8_e4m3fn)[ids, h].double() * scales[ids, h].double()[:, None, None]
            return x.reshape(-1, D)[:n]

        kd, vd = rows(d["k"], d["ks"]), rows(d["v"], d["vs"])
        s = d["q"][0, :, h * G:(h + 1) * G].double().reshape(K * G, D) @ kd.T * scale
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - m)
        t = p.sum(1, keepdim=True)
        out[:, h * G:(h + 1) * G] = ((p / t) @ vd).reshape(K, G, D)
        lse[:, h * G:(h + 1) * G] = ((m + t.log()) / math.log(2.0)).reshape(K, G)
    return out, lse


def attend(d, scale, split=0, window=0, copies=1, unit=0):
    """``copies`` requests alike over the same pages, so that the planner gives
    each at least ``unit`` tiles in one unit."""
    K = d["q"].shape[1]
    n = int(d["ctx"][0])
    q, table, ctx = (d[x].repeat(copies, *[1] * (d[x].dim() - 1)) for x in ("q", "table", "ctx"))
    p = dflash.params_for(q, d["k"], table, block_size=K, window=window, future_keys=1, scale=scale, max_ctx_len=n,
                          force_split_tiles=split, kv_dtype=dflash.KV_FP8_E4M3)
    assert dflash.fp8_page_scales_plan(p)["split_tiles"] >= unit
    ws = torch.zeros(dflash.fp8_page_scales_workspace_size(p), dtype=torch.uint8, device=q.device)
    out, lse = dflash.block_attn_fp8_page_scales(
        q, d["k"], d["v"], d["ks"], d["vs"], table, ctx, block_size=K, window=window, future_keys=1,
        scale=scale, max_ctx_len=n, workspace=ws, force_split_tiles=split)
    assert dflash.read_device_status(ws) == 0
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    return out[0].double(), lse[0].double()


def codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def cache(device, *, n, Hq, K, D, P, sigma, seed, equal_values=False):
    """One kv head; n keys, the block's among them, in shuffled pages.  Column
    0 of the keys is zero, so that a key with a code there alone has a score
    set by column 0 of the queries; the other scores have deviation sigma (in
    nats).  Values are random of deviation 1, or all 1."""
    g = torch.Generator(device=device).manual_seed(seed)
    pages = (n + P - 1) // P
    q = torch.randn((1, K, Hq, D), generator=g, device=device).bfloat16()
    k = torch.randn((pages, 1, P, D), generator=g, device=device) * 100
    k[..., 0] = 0
    v = torch.ones_like(k) * 128 if equal_values else torch.randn(k.shape, generator=g, device=device) * 128
    d = {"q": q, "k": codes(k), "v": codes(v), "table": torch.randperm(pages, generator=g, device=device).int()[None],
         "ctx": torch.tensor([n - K], dtype=torch.int32, device=device)}
    d["ks"] = torch.full((pages, 1), max(sigma, 1e-6) / 100, device=device)
    d["vs"] = torch.full((pages, 1), 1 / 128, device=device)
    return d


def place(d, pos):
    P = d["k"].shape[2]
    return int(d["table"][0, pos // P]), pos % P


def dominate(d, positions, weight, *, zero_values, scale):
    """Makes the keys at ``positions`` hold ``weight`` of every row together."""
    P = d["k"].shape[2]
    d["q"][..., 0] = 0
    for pos in positions:
        page, off = place(d, pos)
        d["k"][page, 0, off] = 0
        if zero_values:
            d["v"][page, 0, off] = 0
    _, lse = reference(d, scale)  # the tail, and exp(0) for each of the keys
    tail = torch.log(torch.exp(lse * math.log(2.0)) - len(positions))
    want = tail + math.log(weight / (1 - weight) / len(positions))
    top = 256.0
    for pos in positions:
        page, off = place(d, pos)
        d["k"][page, 0, off, 0] = codes(torch.tensor([top], device=d["k"].device))[0]
    assert len({float(d["ks"][place(d, pos)[0], 0]) for pos in positions}) == 1
    d["q"][0, :, :, 0] = (want / (scale * top * float(d["ks"][place(d, positions[0])[0], 0]))).bfloat16()


def compare(d, scale, **kw):
    ro, rl = reference(d, scale)
    out, lse = attend(d, scale, **kw)
    rel = float((out - ro).norm() / ro.norm())
    assert rel <= REL_L2, f"relative L2 {rel:.3g}"
    assert float(((out - ro).abs() - ro.abs() * 2.0 ** -8).max()) <= ABS
    assert float((lse - rl).abs().max()) <= LSE + float(rl.abs().max()) * 2.0 ** -20
    return ro, out


# Padded rows 16, 32, 48, 64, 112 and 128; heads of 64 and 128.
SHAPES = [(4, 1, 64), (4, 7, 64), (6, 7, 64), (8, 7, 128), (16, 7, 128), (16, 7, 64), (16, 8, 128), (2, 5, 128)]


@pytest.mark.parametrize("Hq,K,D", SHAPES)
@pytest.mark.parametrize("weight", [0.5, 0.9])
@pytest.mark.parametrize("split", [0, 256])
def test_one_key_and_its_tail(cuda_device, Hq, K, D, weight, split):
    """In the first, a middle and the last tile, its value row zero or not;
    4296 keys, planned and in one unit."""
    n, scale = 4296, 1.0 / math.sqrt(D)
    for where in (0, 2000, 4290 - K):
        for zero in (True, False):
            d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=32, sigma=0.7, seed=where + K)
            dominate(d, [where], weight, zero_values=zero, scale=scale)
            compare(d, scale, split=split)


@pytest.mark.parametrize("Hq,K,D,copies,unit", [(4, 7, 64, 256, 64), (6, 7, 64, 152, 1024), (16, 7, 128, 152, 1024)])
@pytest.mark.parametrize("weight", [0.5, 0.9])
@pytest.mark.parametrize("where", [0, 65000])
def test_one_key_and_a_long_tail(cuda_device, Hq, K, D, copies, unit, weight, where):
    """131072 keys: as planned for one request, in units of 256 tiles, and as
    planned for a batch that fills the card (one unit where the rows allow)."""
    n, scale = 131072, 1.0 / math.sqrt(D)
    d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=64, sigma=0.7, seed=3)
    dominate(d, [where], weight, zero_values=True, scale=scale)
    compare(d, scale)
    compare(d, scale, split=256)
    compare(d, scale, copies=copies, unit=unit)


@pytest.mark.parametrize("Hq,K,D", [(1, 1, 64), (4, 7, 64), (6, 7, 64), (16, 7, 128)])
@pytest.mark.parametrize("nats", [10.0, 11.5, 12.0, 12.5, 14.0])
def test_equal_keys_behind_a_louder_one(cuda_device, Hq, K, D, nats):
    """65536 keys of one score and value behind a first key that lies ``nats``
    above them, in one unit.  With its value equal to theirs the output is that
    value; with its value zero it is their share, which a kernel that dropped
    them, or took them 1 % off, would miss."""
    n, scale = 65536, 1.0 / math.sqrt(D)
    d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=64, sigma=0.0, seed=1, equal_values=True)
    d["k"][:] = 0
    d["q"][:] = 0
    page, off = place(d, 0)
    d["ks"][:] = 1.0
    d["k"][page, 0, off, 0] = codes(torch.tensor([1.0], device=cuda_device))[0]
    d["q"][..., 0] = nats / scale
    out, _ = attend(d, scale, split=256)
    assert float((out - 1.0).abs().max()) <= COHERENT + 127 / n
    d["v"][page, 0, off] = 0
    ro, _ = reference(d, scale)
    share = (n - 1) / (n - 1 + math.exp(float(d["q"][0, 0, 0, 0]) * scale))
    assert abs(float(ro.min()) / share - 1) < 1e-9 and share > 0.05
    for split in (256, 0):
        out, _ = attend(d, scale, split=split)
        # 127 keys share the loud key's tile: 2^-9 of the tail at most.
        assert float((out / ro - 1).abs().max()) <= COHERENT + 127 / n, split


@pytest.mark.parametrize("Hq,K,D", [(4, 7, 64), (6, 7, 64), (16, 7, 128)])
def test_several_loud_keys(cuda_device, Hq, K, D):
    """Sinks beside each other, spread over a tile, one every few tiles, and
    in the last tile too."""
    n, scale = 20000, 1.0 / math.sqrt(D)
    for positions in ([0, 1, 2, 3], [0, 40, 70, 100], list(range(10000, 10128, 16)), list(range(5, n - 200, 1000)),
                      [0, n - 20]):
        for weight in (0.5, 0.9):
            d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=64, sigma=0.7, seed=len(positions))
            dominate(d, positions, weight, zero_values=True, scale=scale)
            compare(d, scale, split=256)


@pytest.mark.parametrize("Hq,K,D", [(4, 7, 64), (6, 7, 64), (16, 7, 128)])
@pytest.mark.parametrize("first", [700, 5000])
def test_quiet_keys_behind_loud_ones(cuda_device, Hq, K, D, first):
    """The scores fall by 6 nats after ``first`` keys and stay there: no key
    stands alone.  The loud keys' values are zero, so the output is the quiet
    keys' alone."""
    n, scale = 60000, 1.0 / math.sqrt(D)
    d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=64, sigma=0.7, seed=first)
    d["q"][..., 0] = 32.0
    keys = d["k"].view(torch.float8_e4m3fn).float()
    values = d["v"].clone()
    for page in range(first // 64):
        at = int(d["table"][0, page])
        keys[at, 0, :, 0] = 6.0 / (scale * 32.0 * float(d["ks"][0, 0]))
        values[at] = 0
    d["k"], d["v"] = codes(keys), values
    compare(d, scale, split=256)
    compare(d, scale)


@pytest.mark.parametrize("sigma", [0.3, 1.5, 3.0, 6.0])
@pytest.mark.parametrize("Hq,K,D", [(4, 1, 128), (4, 7, 64), (6, 7, 64), (16, 7, 128)])
def test_peaked_scores(cuda_device, sigma, Hq, K, D):
    scale = 1.0 / math.sqrt(D)
    for n, split in ((200, 0), (9000, 0), (9000, 256)):
        d = cache(cuda_device, n=n, Hq=Hq, K=K, D=D, P=16, sigma=sigma, seed=7)
        compare(d, scale, split=split)


def test_a_window_over_loud_keys(cuda_device):
    """A dominant key that only the first rows' windows reach."""
    scale, n, W = 1.0 / math.sqrt(64), 6000, 1500
    d = cache(cuda_device, n=n, Hq=6, K=7, D=64, P=32, sigma=0.7, seed=9)
    L = n - 7
    dominate(d, [L - W + 3], 0.9, zero_values=False, scale=scale)  # rows 0 .. 2 see it
    out, lse = attend(d, scale, split=256, window=W)
    P, D = 32, 64
    ids = d["table"][0].long()
    kd = (d["k"].view(torch.float8_e4m3fn)[ids, 0].double() * d["ks"][ids, 0].double()[:, None, None]).reshape(-1, D)[:n]
    vd = (d["v"].view(torch.float8_e4m3fn)[ids, 0].double() * d["vs"][ids, 0].double()[:, None, None]).reshape(-1, D)[:n]
    for i in range(7):
        lo = L + i - W + 1
        s = d["q"][0, i].double() @ kd[lo:].T * scale
        p = torch.softmax(s, 1)
        ro = p @ vd[lo:]
        assert float((out[i] - ro).norm() / ro.norm()) <= REL_L2, i
        assert float((lse[i] - torch.logsumexp(s, 1) / math.log(2.0)).abs().max()) <= LSE
