"""The serving entry points without a GPU: argument checks of the C ABI (made
before CUDA is touched), of the Python functions, and the host-only sizes."""
import ctypes
import shutil

import pytest

import exact_attention_91_gb300 as fa
from exact_attention_91_gb300 import build as fa_build

torch = pytest.importorskip("torch")

P = 1 << 24  # an aligned fake address; never dereferenced by these calls


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not fa_build.up_to_date():
        if shutil.which(fa_build.nvcc_path()) is None:
            pytest.skip("nvcc not available to build libfa.so")
        fa_build.build()
    return fa.load_library()


def test_new_codes_have_texts():
    for code in (-11, -12):
        assert "unknown" not in fa.fa_strerror(code)


def cache(k=P, v=2 * P, ks=0, vs=0, page=16, heads=2, d=64, blocks=4, kind=fa.CACHE_BF16, **st):
    s = dict(k_block=page * heads * d, k_token=heads * d, k_head=d, v_block=page * heads * d, v_token=heads * d, v_head=d)
    s.update(st)
    return fa.FaPagedCache(k, v, ks, vs, s["k_block"], s["k_token"], s["k_head"], s["v_block"], s["v_token"], s["v_head"],
                           kind, blocks, page, heads, d)


BAD_CACHES = [
    (dict(k=0), -1), (dict(v=0), -1), (dict(kind=2), -12), (dict(kind=-1), -12),
    (dict(page=0), -2), (dict(page=8), -2), (dict(page=17), -2), (dict(page=48), -2), (dict(page=131072), -2),
    (dict(page=-16), -2), (dict(heads=0), -2), (dict(blocks=0), -2), (dict(blocks=-1), -2),
    (dict(d=32), -3), (dict(d=96), -3), (dict(d=256), -3),
    (dict(k_token=32), -2), (dict(v_head=0), -2), (dict(k_block=-2048), -2), (dict(v_block=1 << 41), -2),
    (dict(k_token=132), -4), (dict(v_block=2049), -4), (dict(k=P + 8), -4), (dict(v=2 * P + 2), -4),
    (dict(ks=P + 2), -4), (dict(vs=P + 1), -4),
    (dict(kind=fa.CACHE_E4M3, k_token=136), -4),   # 136 bytes: no multiple of 16
]


def decode(c=None, q=3 * P, table=4 * P, lens=5 * P, o=6 * P, lse=7 * P, B=2, Hq=4, width=8, stride=8, scale=0.125,
           ws=8 * P, ws_bytes=1 << 23):
    return fa.fa_decode_paged(q, c or cache(), table, lens, o, lse, B, Hq, width, stride, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_rejected(kw, code):
    assert decode(cache(**kw)) == code
    assert append(cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(table=0), -1), (dict(lens=0), -1), (dict(o=0), -1),
    (dict(B=-1), -2), (dict(Hq=0), -2), (dict(Hq=3), -2), (dict(width=0), -2), (dict(stride=7), -2),
    (dict(width=1 << 28, stride=1 << 28), -2), (dict(B=1 << 20, Hq=1 << 12), -2),
    (dict(q=3 * P + 8), -4), (dict(o=6 * P + 2), -4), (dict(lse=7 * P + 2), -4), (dict(table=4 * P + 2), -4),
    (dict(lens=5 * P + 1), -4), (dict(ws=8 * P + 8), -4),
    (dict(scale=0.0), -9), (dict(scale=-1.0), -9), (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9),
    (dict(o=3 * P), -10), (dict(o=P), -10), (dict(lse=6 * P + 16), -10), (dict(o=2 * P + 64), -10),
    (dict(o=4 * P), -10), (dict(lse=5 * P), -10), (dict(ws=3 * P - (1 << 23) + 16), -10), (dict(ws=6 * P), -10),
])
def test_bad_decode_calls_are_rejected(kw, code):
    assert decode(**kw) == code


def test_decode_of_no_request_and_without_a_device():
    assert decode(B=0, q=0, o=0, table=0, lens=0, ws=0, ws_bytes=0) == 0
    if not torch.cuda.is_available():
        assert decode() == -5


def test_decode_workspace_sizes():
    f = fa.fa_decode_paged_workspace
    #        B   Hq Hkv d   type page width SMs
    assert f(1, 32, 8, 128, 0, 16, 64, 152) == 0           # 1024 keys at most: one cluster per key head
    n = f(64, 32, 8, 128, 0, 16, 512, 152)
    assert 0 < n < 16 << 20
    assert f(64, 32, 8, 128, 0, 16, 100000, 152) == n      # bounded by the GPU, not by the lengths
    assert f(10 ** 6, 32, 8, 128, 0, 16, 512, 152) == n
    assert f(64, 128, 8, 128, 0, 16, 512, 152) > n         # 16 query heads per key head
    assert f(0, 32, 8, 128, 0, 16, 512, 152) == 0
    for bad, code in ((dict(B=-1), -2), (dict(Hq=9), -2), (dict(Hkv=0), -2), (dict(d=80), -3), (dict(kind=7), -12),
                      (dict(page=24), -2), (dict(width=0), -2), (dict(sms=0), -2)):
        kw = dict(B=4, Hq=8, Hkv=8, d=64, kind=0, page=16, width=9, sms=152) | bad
        assert f(*kw.values()) == code, bad


def rotary(x=P, y=2 * P, pos=3 * P, freq=4 * P, B=2, H=3, N=4, d=64, xs=(768, 256, 64), ys=(768, 256, 64), ps=0, r=64,
           factor=1.0):
    return fa.fa_rotary(x, y, pos, freq, B, H, N, d, xs, ys, ps, r, False, False, factor, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), -1), (dict(y=0), -1), (dict(pos=0), -1), (dict(freq=0), -1),
    (dict(B=-1), -2), (dict(H=-1), -2), (dict(N=-1), -2), (dict(H=40000), -2), (dict(B=1 << 16, N=1 << 16), -2),
    (dict(r=8), -2), (dict(r=80), -2), (dict(r=-16), -2), (dict(d=80), -3),
    (dict(xs=(768, 256, 60)), -4), (dict(ys=(768, 260, 64)), -4), (dict(xs=(-768, 256, 64)), -2),
    (dict(ys=(0, 256, 64)), -2), (dict(ys=(768, 256, 32)), -2),
    (dict(x=P + 8), -4), (dict(y=2 * P + 4), -4), (dict(pos=3 * P + 2), -4), (dict(freq=4 * P + 4), -4),
    (dict(factor=float("nan")), -9), (dict(factor=float("inf")), -9),
    (dict(y=P + 64), -10), (dict(y=P, ys=(768, 64, 192)), -10),
    (dict(pos=2 * P + 64), -10), (dict(freq=2 * P + 128), -10), (dict(ps=-4), -2),
    (dict(ys=(768, 64, 64)), -10), (dict(ys=(512, 256, 64)), -10),   # rows of y on one another
])
def test_bad_rotary_calls_are_rejected(kw, code):
    assert rotary(**kw) == code


def test_rotary_calls_that_pass_the_checks():
    ok = 0 if torch.cuda.is_available() else -5
    assert rotary(B=0) == 0 and rotary(H=0, x=0) == 0 and rotary(N=0) == 0
    if ok:
        assert rotary() == ok
        assert rotary(y=P) == ok                                 # in place
        assert rotary(xs=(0, 0, 64)) == ok                       # broadcast input
        assert rotary(r=0, freq=0) == ok
        assert rotary(B=1, ys=(0, 256, 64)) == ok                # the stride of a dimension of size 1


def append(c=None, q=3 * P, k=4 * P, v=5 * P, qs=256, ks=128, vs=128, pos=6 * P, slots=7 * P, freq=8 * P, q_out=9 * P,
           k_out=10 * P, qos=256, kos=128, T=5, Hq=4, r=64, factor=1.0):
    return fa.fa_cache_append(q, k, v, qs, ks, vs, pos, slots, freq, c or cache(), q_out, k_out, qos, kos, T, Hq, r, False,
                              factor, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(q_out=0), -1), (dict(pos=0), -1), (dict(slots=0), -1),
    (dict(freq=0), -1), (dict(T=-1), -2), (dict(Hq=0), -2), (dict(Hq=40000), -2), (dict(qs=255), -2), (dict(ks=64), -2),
    (dict(qos=128), -2), (dict(kos=0), -2), (dict(r=24), -2), (dict(r=128), -2),
    (dict(qs=257), -4), (dict(vs=129), -4), (dict(q=3 * P + 8), -4), (dict(k_out=10 * P + 2), -4), (dict(pos=6 * P + 1), -4),
    (dict(slots=7 * P + 2), -4), (dict(freq=8 * P + 4), -4), (dict(factor=float("inf")), -9),
    (dict(q_out=4 * P), -10), (dict(q_out=3 * P + 64), -10), (dict(q_out=3 * P, qos=512), -10), (dict(k_out=3 * P), -10),
    (dict(pos=9 * P), -10), (dict(slots=10 * P), -10), (dict(freq=P), -10), (dict(slots=2 * P), -10),
    (dict(k_out=9 * P), -10), (dict(q_out=P), -10), (dict(v=2 * P), -10), (dict(k_out=5 * P), -10),
])
def test_bad_append_calls_are_rejected(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(v=P),                                           # keys and values in one place
    dict(k_head=64, k_token=64), dict(v_block=1024), dict(k_token=2048, k_head=64, k_block=4096),
])
def test_append_to_rows_on_one_another_is_rejected(kw):
    assert append(cache(**kw)) == -10


def test_scales_inside_what_is_written_are_rejected():
    assert append(cache(ks=9 * P)) == -10 and append(cache(vs=P)) == -10
    assert decode(cache(ks=6 * P)) == -10 and decode(cache(vs=7 * P)) == -10


def test_append_calls_that_pass_the_checks():
    assert append(T=0) == 0
    if not torch.cuda.is_available():
        row = 8 * 64
        for kw in (dict(), dict(k_out=0), dict(q_out=3 * P), dict(k_out=4 * P), dict(r=0, freq=0), dict(T=1, qs=0, qos=0),
                   # slices of one projection, turned in place
                   dict(q=3 * P, k=3 * P + 512, v=3 * P + 768, qs=row, ks=row, vs=row, q_out=3 * P, qos=row,
                        k_out=3 * P + 512, kos=row),
                   # outputs side by side in one buffer
                   dict(q_out=9 * P, qos=row, k_out=9 * P + 512, kos=row)):
            assert append(**kw) == -5, kw
        for kw in (dict(q=3 * P, k=3 * P, v=3 * P + 768, qs=row, ks=row, vs=row, q_out=3 * P, qos=row),     # k is q's first heads
                   dict(q=3 * P, k=3 * P + 512, v=3 * P + 512, qs=row, ks=row, vs=row, q_out=3 * P, qos=row,
                        k_out=3 * P + 512, kos=row),                                                        # v is k
                   dict(q=3 * P, k=3 * P + 384, v=3 * P + 768, qs=row, ks=row, vs=row, q_out=3 * P, qos=row),
                   dict(q=3 * P, k=3 * P + row * 2 * 3 + 768, v=5 * P, qs=row, ks=row, q_out=3 * P, qos=row, k_out=3 * P + 768,
                        kos=row)):                                                                          # k_out is k, three tokens on
            assert append(**kw) == -10, kw


def maps(ctx=P, fresh=2 * P, table=3 * P, unused=4 * P, slots=5 * P, pos=6 * P, cu=7 * P, lens=8 * P, counts=9 * P, B=4,
         width=8, stride=8, n=10, page=16, T=20):
    return fa.fa_page_maps(ctx, fresh, table, unused, slots, pos, cu, lens, counts, B, width, stride, n, page, T, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ctx=0), -1), (dict(fresh=0), -1), (dict(table=0), -1), (dict(unused=0), -1), (dict(slots=0), -1),
    (dict(pos=0), -1), (dict(cu=0), -1), (dict(lens=0), -1), (dict(counts=0), -1),
    (dict(B=0), -2), (dict(B=8193), -2), (dict(width=0), -2), (dict(stride=7), -2), (dict(n=-1), -2), (dict(T=-1), -2),
    (dict(page=10), -2), (dict(page=8), -2),
    (dict(ctx=P + 2), -4), (dict(counts=9 * P + 1), -4), (dict(unused=4 * P + 2), -4),
    (dict(slots=P), -10), (dict(cu=7 * P, lens=7 * P + 16), -10), (dict(table=4 * P + 16), -10), (dict(pos=5 * P + 40), -10),
])
def test_bad_page_map_calls_are_rejected(kw, code):
    assert maps(**kw) == code


def test_page_map_calls_that_pass_the_checks():
    if not torch.cuda.is_available():
        for kw in (dict(), dict(T=0, slots=0, pos=0), dict(n=0, unused=0), dict(B=1, stride=0), dict(B=8192)):
            assert maps(**kw) == -5, kw


# ---- Python ------------------------------------------------------------------

def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _decode_args(**kw):
    a = dict(q=_bf(2, 4, 64), k_cache=_bf(3, 16, 2, 64), v_cache=_bf(3, 16, 2, 64), block_table=_i(2, 5), seq_lens=_i(2))
    return a | kw


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(2, 4, 64)), TypeError), (dict(q=7), TypeError), (dict(block_table=torch.zeros(2, 5)), TypeError),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError), (dict(k_cache=torch.zeros(3, 16, 2, 64)), TypeError),
    (dict(v_cache=_bf(3, 16, 2, 64).half()), TypeError), (dict(k_cache=_bf(3, 16, 2, 128)), ValueError),
    (dict(q=_bf(2, 64)), ValueError), (dict(seq_lens=_i(3)), ValueError), (dict(block_table=_i(3, 5)), ValueError),
    (dict(block_table=_i(5, 2).t()), ValueError), (dict(q=_bf(2, 64, 4).transpose(1, 2)), ValueError),
    (dict(k_cache=_bf(3, 16, 64, 2).transpose(2, 3)), ValueError), (dict(v_cache=_bf(4, 16, 2, 64)), ValueError),
    (dict(k_scale=torch.ones(3)), ValueError), (dict(v_scale=torch.ones(2, dtype=torch.float64)), ValueError),
    (dict(out=_bf(2, 4, 128)), ValueError), (dict(lse=torch.zeros(2, 5)), ValueError), (dict(out=torch.zeros(2, 4, 64)), ValueError),
    (dict(workspace=_i(100)), ValueError), (dict(scale="x"), TypeError), (dict(), ValueError),   # the last: CPU tensors
])
def test_bad_python_decode_calls(kw, error):
    with pytest.raises(error):
        fa.attention_decode_paged(**_decode_args(**kw))


@pytest.mark.parametrize("kw,error", [
    (dict(x=torch.zeros(2, 3, 4, 64)), TypeError), (dict(positions=torch.zeros(4)), TypeError),
    (dict(positions=_i(5)), ValueError), (dict(positions=_i(3, 4)), ValueError), (dict(x=_bf(4, 64)), ValueError),
    (dict(x=_bf(2, 3, 64, 4).transpose(2, 3)), ValueError), (dict(inv_freq=torch.zeros(32)), ValueError),
    (dict(inv_freq=torch.zeros(2, 16, dtype=torch.float64)), ValueError), (dict(out=_bf(2, 3, 4, 128)), ValueError),
    (dict(factor=None), TypeError), (dict(), ValueError),
])
def test_bad_python_rotary_calls(kw, error):
    a = dict(x=_bf(2, 3, 4, 64), positions=_i(4), inv_freq=torch.zeros(32, dtype=torch.float64)) | kw
    with pytest.raises(error):
        fa.rotary(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(5, 4, 64)), TypeError), (dict(slots=torch.zeros(5, dtype=torch.int64)), TypeError),
    (dict(k=_bf(5, 3, 64)), ValueError), (dict(v=_bf(5, 2, 128)), ValueError), (dict(q=_bf(6, 4, 64)), ValueError),
    (dict(positions=_i(6)), ValueError), (dict(slots=_i(10)[::2]), ValueError), (dict(k_cache=_bf(3, 16, 3, 64)), ValueError),
    (dict(q=_bf(4, 5, 64).transpose(0, 1)), ValueError), (dict(q_out=_bf(5, 4, 128)), ValueError),
    (dict(k_out=_bf(5, 2, 64).float()), ValueError), (dict(k_scale=torch.ones(1)), ValueError), (dict(), ValueError),
])
def test_bad_python_append_calls(kw, error):
    a = dict(q=_bf(5, 4, 64), k=_bf(5, 2, 64), v=_bf(5, 2, 64), positions=_i(5), slots=_i(5), inv_freq=None,
             k_cache=_bf(3, 16, 2, 64), v_cache=_bf(3, 16, 2, 64)) | kw
    with pytest.raises(error):
        fa.cache_append(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(context_lens=torch.zeros(3)), TypeError), (dict(unused_blocks=torch.zeros(9, dtype=torch.int64)), TypeError),
    (dict(new_lens=_i(4)), ValueError), (dict(block_table=_i(15)), ValueError), (dict(unused_blocks=_i(3, 3)), ValueError),
    (dict(block_table=_i(5, 3).t()), ValueError), (dict(num_tokens=-1), ValueError), (dict(page_size=2.5), TypeError),
    (dict(out=fa.PageMaps(_i(7), _i(7), _i(4), _i(3), _i(3))), ValueError), (dict(out=[1]), TypeError), (dict(), ValueError),
])
def test_bad_python_page_map_calls(kw, error):
    a = dict(context_lens=_i(3), new_lens=_i(3), block_table=_i(3, 5), unused_blocks=_i(9), page_size=16, num_tokens=7) | kw
    with pytest.raises(error):
        fa.page_maps(**a)


def test_statuses_are_raised_as_errors():
    """A status of the C call becomes FaError with its code and text."""
    bind = fa.load_binding()
    assert fa.load_binding() is bind
    with pytest.raises(TypeError):
        bind.setup(1, 2)
    if torch.cuda.is_available():
        return
    e = fa.FaError(-2, "fa_rotary")
    assert e.status == -2 and "fa_rotary" in str(e) and fa.fa_strerror(-2) in str(e)


def test_fake_implementations_give_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode

    from exact_attention_91_gb300 import torch_op  # noqa: F401
    with FakeTensorMode():
        def t(*s, dtype=torch.bfloat16):
            return torch.empty(*s, dtype=dtype, device="meta")
        i = torch.int32
        o, lse = torch.ops.fa91.attention_decode_paged(t(3, 8, 64), t(9, 16, 2, 64), t(9, 16, 2, 64), t(3, 5, dtype=i),
                                                       t(3, dtype=i), None, None, None)
        q = torch.ops.fa91.cache_append(t(7, 8, 64), t(7, 2, 64), t(7, 2, 64), t(7, dtype=i), t(7, dtype=i), None,
                                        t(9, 16, 2, 64), t(9, 16, 2, 64))
        m = torch.ops.fa91.page_maps(t(3, dtype=i), t(3, dtype=i), t(3, 5, dtype=i), t(9, dtype=i), 16, 7)
    assert o.shape == (3, 8, 64) and lse.shape == (3, 8) and lse.dtype == torch.float32
    assert q.shape == (7, 8, 64) and [x.shape[0] for x in m] == [7, 7, 4, 3, 4]


def test_structure_is_laid_out_as_in_the_header():
    assert ctypes.sizeof(fa.FaPagedCache) == 4 * 8 + 6 * 8 + 5 * 4 + 4
