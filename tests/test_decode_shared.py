"""Decode behind shared prefixes (fa_decode_shared) against the 64-bit form of paged decode: groups, rows per key head
around the tiles, prefixes around the tiles and pages, cache types and orders, hidden pages, requests shorter than their
prefix, values that must not be read."""
import shutil

import numpy as np
import pytest

import exact_attention_91_gb300 as fa
from exact_attention_91_gb300 import build as fa_build

from . import serve_oracle as so

torch = pytest.importorskip("torch")
P = 1 << 26  # an aligned fake address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not fa_build.up_to_date():
        if shutil.which(fa_build.nvcc_path()) is None:
            pytest.skip("nvcc not available to build libfa.so")
        fa_build.build()
    return fa.load_library()


# ---- without a GPU ----------------------------------------------------------


def cache(k=P, v=2 * P, ks=0, vs=0, page=16, heads=2, d=64, blocks=4, kind=fa.CACHE_BF16, **st):
    s = dict(k_block=page * heads * d, k_token=heads * d, k_head=d, v_block=page * heads * d, v_token=heads * d, v_head=d)
    s.update(st)
    return fa.FaPagedCache(k, v, ks, vs, s["k_block"], s["k_token"], s["k_head"], s["v_block"], s["v_token"], s["v_head"],
                           kind, blocks, page, heads, d)


def shared(c=None, q=3 * P, table=4 * P, lens=5 * P, prefix=12 * P, o=6 * P, lse=7 * P, B=4, Hq=4, groups=2, width=8,
           stride=8, scale=0.125, ws=8 * P, ws_bytes=1 << 24):
    return fa.fa_decode_shared(q, c or cache(), table, lens, prefix, o, lse, B, Hq, groups, width, stride, scale, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(table=0), -1), (dict(lens=0), -1), (dict(o=0), -1), (dict(prefix=0), -1),
    (dict(B=-1), -2), (dict(B=5), -2), (dict(groups=0), -2), (dict(groups=-1), -2), (dict(Hq=3), -2), (dict(width=0), -2),
    (dict(stride=7), -2), (dict(q=3 * P + 8), -4), (dict(prefix=12 * P + 2), -4), (dict(ws=8 * P + 8), -4),
    (dict(scale=0.0), -9), (dict(scale=float("nan")), -9), (dict(o=12 * P), -10), (dict(ws=12 * P - 64), -10),
    (dict(o=3 * P), -10), (dict(ws=6 * P), -10), (dict(c=cache(k=0)), -1), (dict(c=cache(d=80)), -3),
    (dict(c=cache(kind=5)), -12), (dict(c=cache(page=24)), -2),
])
def test_bad_calls_are_rejected(kw, code):
    assert shared(**kw) == code


def test_no_request_and_no_device():
    assert shared(B=0, q=0, o=0, table=0, lens=0, prefix=0, ws=0, ws_bytes=0) == 0
    if not torch.cuda.is_available():
        assert shared() == -5


def test_workspace_sizes():
    f = fa.fa_decode_shared_workspace
    #                B  Hq  Hkv d  type page width groups SMs
    small, large = f(4, 32, 8, 128, 0, 16, 4096, 1, 152), f(64, 32, 8, 128, 0, 16, 4096, 1, 152)
    assert 0 < small < large < 128 << 20
    assert f(64, 32, 8, 128, 0, 16, 10 ** 6, 1, 152) == large      # bounded by the requests and the GPU
    assert f(4, 32, 8, 128, 0, 16, 64, 1, 152) == 0                 # read as fa_decode_paged reads it
    assert f(0, 32, 8, 128, 0, 16, 64, 1, 152) == 0
    for bad, code in ((dict(B=5, groups=2), -2), (dict(groups=0), -2), (dict(Hq=9), -2), (dict(d=80), -3), (dict(sms=0), -2),
                      (dict(page=20), -2), (dict(width=0), -2), (dict(kind=3), -12)):
        kw = dict(B=4, Hq=8, Hkv=8, d=64, kind=0, page=16, width=9, groups=2, sms=152) | bad
        assert f(*kw.values()) == code, bad


# ---- on the GPU -------------------------------------------------------------


def make(prefixes, own, hq, hkv, d, page, e4m3=False, order="token", seed=0, width=None, share=None):
    """Groups of len(own) requests; own: tokens of a request behind its group's prefix (negative: how much it falls
    short of it; None: an empty request). `share`: the lengths given as shared (the prefixes)."""
    g = torch.Generator().manual_seed(seed)
    n, lens, rows = len(own), [], []
    fresh = iter(torch.randperm(100000, generator=g).tolist())
    pool = []

    def new():
        pool.append(None)
        return len(pool) - 1

    for p in prefixes:
        common = [new() for _ in range(p // page)]
        for m in own:
            total = 0 if m is None else max(p + m, 0)
            lens.append(total)
            rows.append(common + [new() for _ in range(max(0, -(-total // page) - len(common)))])
    del fresh
    blocks = len(pool) + 2
    perm = torch.randperm(blocks, generator=g).int()
    # (a table too small for 128 MB would be read as fa_decode_paged reads it)
    room = (1 << 27) // (len(rows) * hkv * d * (2 if e4m3 else 4) * page) + 1
    width = width or max(room, max(len(r) for r in rows))
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = perm[torch.tensor(r, dtype=torch.long)] if r else table[b, :0]
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16

    def values():
        return torch.randn(blocks, page, hkv, d, generator=g).to(t).cuda()

    if order == "token":
        k, v = values(), values()
    elif order == "head":
        k, v = (x.view(torch.uint8 if e4m3 else t).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(t)
                for x in (values(), values()))
    else:  # keys and values side by side in one tensor
        kv = torch.empty(blocks, 2, page, hkv, d, dtype=t, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
        k.copy_(values())
        v.copy_(values())
    q = torch.randn(len(rows), hq, d, generator=g).bfloat16().cuda()
    ks = vs = None
    if e4m3:
        ks, vs = ((0.3 + torch.rand(hkv, generator=g)).cuda() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    return dict(q=q, k=k, v=v, table=table.cuda(), lens=i32(lens), prefix=i32(share or list(prefixes)), ks=ks, vs=vs)


def call(x, **kw):
    return fa.attention_decode_shared(x["q"], x["k"], x["v"], x["table"], x["lens"], x["prefix"], k_scale=x["ks"],
                                      v_scale=x["vs"], **kw)


def want(x, scale=None):
    ks, vs = (None if s is None else so.f64(s) for s in (x["ks"], x["vs"]))
    return so.decode(so.f64(x["q"]), so.f64(x["k"]), so.f64(x["v"]), x["table"].cpu().numpy(), x["lens"].cpu().numpy(),
                     scale or x["q"].shape[-1] ** -0.5, ks, vs)


def check(got, ref):
    """As of paged decode (a score off by big·2^-19, fp32 sums and the joins of partial results below 2^-14 of A), and
    each weight of a shared key rounded to bf16: 2^-8 of A at most."""
    o, lse = (so.f64(t) for t in got)
    o_ref, lse_ref, a, big = ref
    none = np.isneginf(lse_ref)
    np.testing.assert_array_equal(np.isneginf(lse), none)
    assert np.all(o[none] == 0.0)
    off = np.abs(big) * 2.0 ** -19
    bound = so.BF16_HALF * np.abs(o_ref) + a * (2 * off[..., None] + 2.0 ** -14 + 2.0 ** -8) * (1 + so.BF16_HALF) + 1e-38
    d = np.abs(o - o_ref)
    assert np.all(d <= bound), (float((d / bound).max()), np.unravel_index((d / bound).argmax(), d.shape))
    with np.errstate(invalid="ignore"):
        dl = np.where(none, 0.0, np.abs(lse - lse_ref))
    lb = off + 2.0 ** -18 + np.where(none, 0.0, np.abs(lse_ref)) * 2.0 ** -22
    assert np.all(dl <= lb), float((dl / lb).max())
    assert fa.fa_device_status() == (0, 0)


LAYOUTS = [(4, 1, 64), (8, 2, 128), (12, 12, 64), (7, 1, 128), (32, 2, 64), (20, 1, 128), (3, 3, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
def test_head_layouts(hq, hkv, d, e4m3):
    x = make([300, 16, 1000], [5, 130, 1], hq, hkv, d, 16, e4m3=e4m3, seed=hq + d)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (16, 8, 1), (17, 8, 1), (32, 8, 1), (33, 8, 1), (40, 7, 1), (70, 8, 1)])
def test_rows_around_the_tiles(n, hq, hkv, e4m3):
    """1 to 560 rows to a key head: one tile shared out over two chains, two tiles, more row blocks."""
    x = make([700, 257], [1 + i % 9 for i in range(n)], hq, hkv, 64 if n % 2 else 128, 32, e4m3=e4m3, seed=n)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 112, 127, 128, 129, 255, 256, 400, 2049])
def test_prefixes_around_tiles_and_pages(prefix, page):
    x = make([prefix], [0, 1, 40, 300], 8, 2, 128, page, seed=prefix + page)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["token", "head", "side"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_orders_in_memory(order, e4m3, d):
    x = make([333, 64], [9, 70], 8, 4, d, 32, e4m3=e4m3, order=order, seed=d)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_short_and_empty_requests_and_values_behind_them(e4m3):
    """Requests shorter than their group's prefix, empty ones, and infinities and NaN in keys and values that only the
    other requests see, and in unfilled places."""
    x = make([200, 320], [5, -60, None, 0, -199, 17], 8, 2, 64, 16, e4m3=e4m3, seed=4)
    # the prefix's last page (tokens 176 to 191 of group 0) holds infinities: the two short requests do not see them
    bad = float("nan")
    page = int(x["table"][0, 11])
    v, k = x["v"].clone(), x["k"].clone()
    v[page], k[page] = bad, bad
    for b in range(12):  # unfilled places behind each request's last key
        n = int(x["lens"][b])
        if n % 16:
            last = int(x["table"][b, n // 16])
            v[last, n % 16:], k[last, n % 16:] = bad, bad
    got, ref = call(dict(x, k=k, v=v)), want(dict(x, k=k, v=v))
    # the 64-bit form reads what a request sees and nothing else: NaN there (also where a short request's unfilled
    # places are others' prefix), and nowhere else
    lost = np.isnan(ref[0]).any((1, 2))
    assert lost[0] and not lost[[2, 4, 8, 10]].any()
    assert torch.isnan(got[0][torch.from_numpy(lost).cuda()].float()).all()
    rest = np.flatnonzero(~lost)
    check(tuple(t[torch.from_numpy(rest).cuda()] for t in got), tuple(t[rest] for t in ref))


@pytest.mark.gpu
def test_hidden_pages():
    x = make([512, 300], [40, 3], 8, 2, 128, 16, seed=11)
    table = x["table"].clone()
    table[0, 3] = table[1, 3] = -1          # of the prefix: in all rows
    table[2, 0] = table[3, 0] = 10 ** 6
    table[1, 33] = -5                       # of a request's own
    x["table"] = table
    check(call(x), want(x))
    table[:, :] = -1
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("share", [[0, 0], [-7, 5], [64, 10 ** 9], [15, 128]])
def test_shared_lengths_that_are_less_or_more_than_the_prefix(share):
    """What is given as shared may be any part of what the rows have in common; past the table it counts as the table."""
    x = make([256, 256], [0, 0], 8, 2, 64, 16, seed=12, share=share)
    check(call(x), want(x))


@pytest.mark.gpu
def test_negative_and_zero_key_scales():
    x = make([300], [4, 90], 8, 4, 64, 16, e4m3=True, seed=13)
    x["ks"] = torch.tensor([0.7, -0.4, 0.0, 1.3], device="cuda")
    check(call(x), want(x))


@pytest.mark.gpu
def test_rising_scores_and_a_large_scale():
    """Row maxima that move at every tile: O is rescaled each time."""
    x = make([1500], [7, 200, 30], 4, 1, 128, 16, seed=14)
    order = torch.arange(x["k"].shape[0], device="cuda")
    x["k"][x["table"][0, :90].long()] *= torch.linspace(0.1, 3.0, 90, device="cuda")[:, None, None, None].bfloat16()
    del order
    for scale in (None, 1.0):
        check(call(x, scale=scale), want(x, scale))


@pytest.mark.gpu
def test_many_groups_and_long_prefixes():
    x = make([16 * (i % 7) for i in range(40)], [1, 20], 4, 2, 64, 16, seed=15)   # more groups than a warp has lanes
    check(call(x), want(x))
    x = make([20000], [1, 333], 2, 1, 128, 64, seed=16)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d,lens", [
    (8, 8, 64, "short"), (16, 8, 128, "short"), (16, 8, 128, "long"), (5, 5, 64, "long"), (30, 10, 128, "mixed"),
    (80, 8, 64, "mixed"), (40, 1, 128, "none"),
])
def test_many_requests(hq, hkv, d, lens, e4m3):
    """More units than one wave of clusters: own keys in equal runs, ahead of the prefixes."""
    n = 40 if hkv >= 5 else 160
    own = {"short": [i % 5 for i in range(n)], "long": [900 if i == 7 else 30 + i for i in range(n)],
           "mixed": [(None, -3, 0, 1, 64, 257)[i % 6] for i in range(n)], "none": [0] * n}[lens]
    x = make([208, 33], own, hq, hkv, d, 16, e4m3=e4m3, seed=hq + n)
    got = call(x)
    check(got, want(x))
    for a, b in zip(call(x), got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(40, 8, 128), (96, 12, 64)])
def test_many_rows(hq, hkv, d):
    """More rows than one wave of the joining kernel's blocks, own keys cut between runs, several groups."""
    x = make([208, 0, 1009], [700 if i == 5 else (i * 37) % 90 for i in range(28)], hq, hkv, d, 16, seed=hq)
    check(call(x), want(x))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_repeats_streams_buffers_and_agreement_with_paged_decode(e4m3):
    x = make([640, 1024], [50, 3, 200], 16, 4, 128, 16, e4m3=e4m3, seed=17)
    ref = call(x)
    check(ref, want(x))
    side = torch.cuda.Stream()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    room = fa.fa_decode_shared_workspace(6, 16, 4, 128, fa.CACHE_E4M3 if e4m3 else fa.CACHE_BF16, 16, x["table"].shape[1],
                                         2, sms)
    ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(ref[0], float("nan")), torch.full_like(ref[1], float("nan"))
    for kw in ({}, dict(stream=side), dict(out=out, lse=lse, workspace=ws)):
        got = call(x, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert got[0] is out
    assert torch.equal(call(x, return_lse=False), ref[0])
    o, l = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], k_scale=x["ks"], v_scale=x["vs"])
    # (both are within their bounds of the same value: LSE of fp32's rounding, O of two roundings to bf16 and P's)
    assert (l - ref[1]).abs().max() <= 2.0 ** -15
    assert (o.float() - ref[0].float()).abs().max() <= 2 * 2.0 ** -8 * o.float().abs().max() + 2.0 ** -8


@pytest.mark.gpu
def test_a_small_batch_is_read_as_by_paged_decode():
    x = make([64, 64], [1, 20], 4, 2, 64, 16, seed=19, width=8)
    want_o, want_l = fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"])
    got = call(x)
    assert torch.equal(got[0], want_o) and torch.equal(got[1], want_l)


@pytest.mark.gpu
def test_refusals_of_the_python_function():
    x = make([64], [1, 2], 4, 2, 64, 16, seed=18)
    with pytest.raises(TypeError):
        call(dict(x, prefix=x["prefix"].long()))
    for bad in (dict(prefix=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(prefix=x["prefix"].cpu()),
                dict(prefix=x["prefix"].view(1, 1)), dict(prefix=x["prefix"][:0])):
        with pytest.raises(ValueError):
            call(dict(x, **bad))
    with pytest.raises(fa.FaError):
        call(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError):
        call(x, out=x["q"])
