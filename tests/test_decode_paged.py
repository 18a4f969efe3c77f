"""Attention of one new token over a paged cache (fa_decode_paged) against the
64-bit form: head layouts, cache types and orders, lengths around the tiles and
pages, hidden keys, values that must not be read, cuts of the batch's work."""
import math

import numpy as np
import pytest

from . import serve_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


def make(lens, hq, hkv, d, page, e4m3=False, order="token", seed=0, extra=2, width=None):
    """Inputs on the CPU generator (the same on every machine), pages scattered."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-max(n, 0) // page) for n in lens]
    blocks = sum(pages) + extra
    perm = torch.randperm(blocks, generator=g).int()
    width = width or max(1, max(pages))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16

    def values():
        return torch.randn(blocks, page, hkv, d, generator=g).to(t).cuda()

    if order == "token":
        k, v = values(), values()
    elif order == "head":
        k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if not e4m3 else
                x.view(torch.uint8).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(t)
                for x in (values(), values()))
    else:  # keys and values side by side in one tensor
        kv = torch.empty(blocks, 2, page, hkv, d, dtype=t, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
        k.copy_(values())
        v.copy_(values())
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16().cuda()
    ks = vs = None
    if e4m3:
        ks, vs = ((0.3 + torch.rand(hkv, generator=g)).cuda() for _ in range(2))
    return dict(q=q, k=k, v=v, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(), ks=ks, vs=vs)


def small_form(fa, x):
    """Whether the call is done by clusters, one per request and key head (it
    then needs no workspace), and not cut into equal runs."""
    B, hq, d = x["q"].shape
    _, page, hkv, _ = x["k"].shape
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    kind = fa.CACHE_E4M3 if x["k"].dtype == torch.float8_e4m3fn else fa.CACHE_BF16
    return fa.fa_decode_paged_workspace(B, hq, hkv, d, kind, page, x["table"].shape[1], sms) == 0


def call(fa, x, **kw):
    return fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], k_scale=x["ks"], v_scale=x["vs"],
                                     **kw)


def want(x, scale=None):
    ks, vs = (None if s is None else so.f64(s) for s in (x["ks"], x["vs"]))
    scale = scale or 1.0 / math.sqrt(x["q"].shape[-1])
    return so.decode(so.f64(x["q"]), so.f64(x["k"]), so.f64(x["v"]), x["table"].cpu().numpy(),
                     x["lens"].cpu().numpy(), scale, ks, vs)


def check(fa, x, **kw):
    o, lse = call(fa, x, **kw)
    torch.cuda.synchronize()
    one_p = x["ks"] is not None and x["q"].shape[1] > 8 * x["k"].shape[2]
    so.assert_decode(so.f64(o), so.f64(lse), want(x, kw.get("scale")), one_p)
    return o, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 1), (6, 2), (16, 2), (18, 2), (16, 1), (40, 1)])
def test_lengths_around_tiles_and_pages(d, e4m3, hq, hkv):
    """Both forms: the table's width alone decides which."""
    fa = _fa()
    x = make(EDGES, hq, hkv, d, 16, e4m3, seed=hq * 100 + hkv)
    assert small_form(fa, x)
    check(fa, x)
    x = make(EDGES, hq, hkv, d, 16, e4m3, seed=hq * 100 + hkv, width=5000)
    assert not small_form(fa, x)
    check(fa, x)


@pytest.mark.parametrize("d,e4m3,hq,hkv", [(128, False, 4, 1), (64, True, 24, 2), (128, True, 3, 3), (64, False, 20, 1)])
@pytest.mark.parametrize("tiles", [3, 8, 9, 16, 17, 32, 33, 100, 256, 257])
def test_cluster_sizes(d, e4m3, hq, hkv, tiles):
    """Tables of 1 to 256 tiles (clusters of 1 to 8 blocks, shares with and
    without tiles) and the first past them."""
    fa = _fa()
    keys = 4096 // (d if e4m3 else 2 * d)
    n = tiles * keys
    x = make([n, n - 1, 1, 0, keys + 1, n // 2], hq, hkv, d, 16, e4m3, seed=tiles)
    assert small_form(fa, x) == (tiles <= 256)
    check(fa, x)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("order", ["token", "head", "side"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_page_sizes_and_orders_in_memory(page, order, e4m3):
    fa = _fa()
    check(fa, make([1, 300, 77, 513], 8, 2, 128, page, e4m3, order, seed=page))


@pytest.mark.parametrize("d,e4m3,hq,hkv", [(128, False, 8, 1), (128, True, 8, 1), (64, False, 12, 12), (64, True, 32, 2)])
@pytest.mark.parametrize("lens", [[5000], [20011], [3, 9000, 0, 1, 4097], [700] * 40])
def test_requests_cut_across_blocks(d, e4m3, hq, hkv, lens):
    fa = _fa()
    check(fa, make(lens, hq, hkv, d, 32, e4m3, seed=len(lens)))


@pytest.mark.parametrize("d,e4m3,hq,hkv", [(64, False, 4, 4), (128, True, 32, 8), (128, False, 64, 4), (64, True, 48, 4),
                                           (128, False, 80, 4), (64, True, 12, 12)])
def test_one_head_per_warp(d, e4m3, hq, hkv):
    """Enough work that each warp takes a key head (or a row group of one) of
    its own: cut and whole units, no keys, hidden pages, NaN in unfilled places."""
    fa = _fa()
    keys = 4096 // (d if e4m3 else 2 * d)
    heads = hkv * -(-(hq // hkv) // 16)
    lens = [0, 1, keys, keys + 1, 9000, 3 * keys - 1] + [(i * 61) % 700 for i in range(90)] + [5003]
    workers = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    while sum(max(1, -(-n // keys)) for n in lens) * (heads // 4) < 20 * workers:
        lens += [4001, 0, 777, 2500]
    x = make(lens, hq, hkv, d, 16, e4m3, seed=hq)
    x["table"][4, 7] = -1
    x["table"][4, 100:140] = x["k"].shape[0]
    table = x["table"].cpu()
    for b in (1, 3, 5, 9):                                 # behind the last key of these requests
        n = lens[b]
        if n % 16:
            for name in ("k", "v"):
                t = x[name][table[b, n // 16].item()].float()
                t[n % 16:] = float("nan")
                x[name][table[b, n // 16].item()] = t.to(x[name].dtype)
    check(fa, x)
    o1, l1 = call(fa, x)
    o2, l2 = call(fa, x)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_many_requests():
    """More requests than a block has threads, and more units than blocks."""
    fa = _fa()
    lens = [(i * 37) % 90 for i in range(700)]
    check(fa, make(lens, 4, 2, 64, 16, seed=4))


def test_scale_and_large_scores():
    """Scores in the hundreds: the running maximum moves, weights are spiky."""
    fa = _fa()
    for e4m3 in (False, True):
        x = make([1500, 64, 333], 8, 2, 128, 16, e4m3, seed=11)
        x["q"] = (x["q"].float() * 6).bfloat16()
        check(fa, x, scale=0.5)
        check(fa, x, scale=0.01)


@pytest.mark.parametrize("e4m3,hq", [(False, 4), (False, 16), (True, 4), (True, 16)])
@pytest.mark.parametrize("width", [None, 3001])
def test_negative_and_zero_scales_of_the_cache(e4m3, hq, width):
    """A key scale below zero turns the order of the scores round, one of zero
    makes them equal; hidden keys stay hidden."""
    fa = _fa()
    x = make([700, 33, 0, 129], hq, 1, 64, 16, e4m3, seed=15, width=width)
    x["table"][0, 5] = -1
    for value in (-0.7, 0.0):
        x["ks"] = torch.full((1,), value, device="cuda")
        x["vs"] = torch.full((1,), -1.5, device="cuda")
        check(fa, x)


def test_rising_scores_rescale_every_tile():
    """Keys ordered so that the row maximum rises by more than the kernel's
    threshold from tile to tile."""
    fa = _fa()
    x = make([640], 2, 1, 64, 16, seed=12)
    x["q"][:] = 1.0
    ramp = (torch.arange(640).float() * 0.25).cuda()
    k = torch.zeros_like(x["k"])
    pages = x["table"][0].long()
    for i in range(40):
        k[pages[i], :, 0, :] = ramp[i * 16:(i + 1) * 16, None].bfloat16()
    x["k"] = k
    check(fa, x, scale=1.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_dominant_key_and_many_small_ones(e4m3):
    """One key 20 (natural) above 30000 others: their weights are each below
    fp16's smallest step, their sum is not."""
    fa = _fa()
    x = make([30000], 1, 1, 64, 64, e4m3, seed=13)
    x["q"][:] = 0.0
    x["q"][:, :, 0] = 1.0
    k = torch.zeros(x["k"].shape, device="cuda")
    k[x["table"][0, 0].item(), 5, 0, 0] = 12.0
    x["k"] = k.to(x["k"].dtype)
    x["ks"] = None
    v = torch.ones(x["v"].shape, device="cuda") * 2
    v[x["table"][0, 0].item(), 5] = 0.0
    x["v"] = v.to(x["v"].dtype)
    check(fa, x, scale=1.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_unfilled_places_have_no_effect(e4m3):
    """NaN and infinities behind each request's last key, in its last page and in
    the pages that no request has."""
    fa = _fa()
    lens = [1, 40, 0, 129, 63]
    x = make(lens, 8, 2, 128, 32, e4m3, seed=21)
    o1, l1 = check(fa, x)
    used = torch.zeros(x["k"].shape[:2], dtype=torch.bool)
    table = x["table"].cpu()
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // 32], j % 32] = True
    for name, bad in (("k", float("nan")), ("v", float("nan"))):
        t = x[name].float()
        t[~used.cuda()] = bad
        x[name] = t.to(x[name].dtype)
    o2, l2 = call(fa, x)
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)
    if not e4m3:
        for name in ("k", "v"):
            t = x[name].float()
            t[~used.cuda()] = float("inf")
            x[name] = t.to(x[name].dtype)
        o2, l2 = call(fa, x)
        assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)


def test_nan_in_a_visible_place_is_passed_on():
    fa = _fa()
    x = make([100, 100], 2, 1, 64, 16, seed=22)
    x["k"][x["table"][0, 2].item(), 3, 0, 7] = float("nan")
    o, lse = call(fa, x)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(o[1].float()).all() and torch.isfinite(lse[1]).all()
    x["q"][1] = float("nan")
    o, lse = call(fa, x)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_blocks_outside_the_cache_hide_their_keys(e4m3):
    fa = _fa()
    x = make([300, 300, 48, 17], 8, 2, 64, 16, e4m3, seed=23)
    blocks = x["k"].shape[0]
    x["table"][0, 3] = -1
    x["table"][0, 7] = blocks
    x["table"][0, 18] = 2 ** 31 - 1
    x["table"][1, 0] = -2 ** 31
    x["table"][2, :] = -1                  # nothing left to see
    x["table"][3, 1] = -7                  # the last page
    _, lse = check(fa, x)
    assert torch.isneginf(lse[2]).all()


def test_lengths_past_the_table_and_below_zero():
    fa = _fa()
    x = make([64, 64, 30], 2, 1, 128, 16, seed=24)
    x["lens"] = torch.tensor([1000, -5, 2 ** 31 - 1], dtype=torch.int32).cuda()
    x["table"][2, 2:] = x["table"][0, 2:]
    check(fa, x)


def test_table_wider_than_needed_and_strided():
    fa = _fa()
    x = make([50, 700], 4, 2, 128, 16, seed=25)
    wide = torch.full((2, 4000), 12345678, dtype=torch.int32, device="cuda")
    w = x["table"].shape[1]
    wide[:, :w] = x["table"]
    o1, l1 = check(fa, x)
    x["table"] = wide[:, :2999]
    o2, l2 = check(fa, x)
    x["table"] = wide[:, :w]
    o3, l3 = call(fa, x)
    assert torch.equal(o1, o3) and torch.equal(l1, l3)


def test_large_block_offsets():
    """Blocks whose first value lies past 2^31 elements and 2^32 bytes."""
    fa = _fa()
    blocks, page, d = 34000, 16, 128
    need = blocks * page * 32 * d
    assert need > 2 ** 31
    store = torch.empty(need, dtype=torch.bfloat16, device="cuda").view(blocks, page, 32, d)
    x = make([70, 33], 4, 4, d, page, seed=26)
    count = x["k"].shape[0]
    small = x["table"].clone()
    for name, view in (("k", store[:, :, :4]), ("v", store[:, :, 16:20])):
        view[-count:] = x[name]
        x[name] = view
    x["table"] = torch.where(small >= 0, small + blocks - count, small)  # the last blocks of the large cache
    o, lse = call(fa, x)
    part = dict(x)
    part["k"], part["v"], part["table"] = x["k"][-count:], x["v"][-count:], small
    so.assert_decode(so.f64(o), so.f64(lse), want(part))


def test_outputs_given_and_nothing_else_written():
    fa = _fa()
    x = make([100, 0, 3], 6, 3, 64, 16, seed=27)
    big = torch.full((5, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 6), 7.0, device="cuda")
    o1, l1 = call(fa, x)
    o2, l2 = call(fa, x, out=big[1:4], lse=lse[1:4])
    assert o2.data_ptr() == big[1:4].data_ptr()
    assert torch.equal(o1, big[1:4]) and torch.equal(l1, lse[1:4])
    assert (big[0] == 7).all() and (big[4] == 7).all() and (lse[0] == 7).all() and (lse[4] == 7).all()
    o3 = call(fa, x, return_lse=False)
    assert torch.equal(o1, o3)
    n = fa.fa_decode_paged_workspace(3, 6, 3, 64, 0, 16, x["table"].shape[1],
                                     torch.cuda.get_device_properties(0).multi_processor_count)
    ws = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
    o4, l4 = call(fa, x, workspace=ws[:n])
    assert torch.equal(o1, o4) and torch.equal(l1, l4) and (ws[n:] == 171).all()


def test_same_call_gives_the_same_bits():
    fa = _fa()
    x = make([4000, 1, 900, 2222], 8, 2, 128, 16, seed=28)
    o1, l1 = call(fa, x)
    for _ in range(5):
        o, lse = call(fa, x)
        assert torch.equal(o, o1) and torch.equal(lse, l1)


def test_empty_batch():
    fa = _fa()
    x = make([5], 2, 1, 64, 16, seed=29)
    x["q"], x["table"], x["lens"] = x["q"][:0], x["table"][:0], x["lens"][:0]
    o, lse = call(fa, x)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
