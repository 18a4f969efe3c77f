"""What the serving functions write counts as written in place: a backward pass that
saved the tensor before raises, and does not use the new values."""
import pytest

from .test_decode_paged import _fa, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_written_tensors_are_marked_and_others_are_not():
    fa = _fa()
    x = make([40, 7, 33], 4, 2, 64, 16, seed=3)
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    k, v = torch.randn(3, 2, 64, device="cuda").bfloat16(), torch.randn(3, 2, 64, device="cuda").bfloat16()
    out, lse, k_out = torch.empty_like(x["q"]), torch.empty(3, 4, device="cuda"), torch.empty_like(k)
    maps = fa.page_maps(x["lens"], pos, x["table"].clone(), pos, 16, 9)
    table = x["table"].clone()
    calls = [
        ((out, lse), (x["q"], x["k"], x["v"], x["table"], x["lens"]),
         lambda: fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"], out=out, lse=lse)),
        ((out,), (x["q"], pos, freq), lambda: fa.rotary(x["q"], pos, freq, out=out)),
        ((out, k_out, x["k"], x["v"]), (x["q"], k, v, pos, freq),
         lambda: fa.cache_append(x["q"], k, v, pos, pos, freq, x["k"], x["v"], q_out=out, k_out=k_out)),
        ((table, *maps), (x["lens"], pos), lambda: fa.page_maps(x["lens"], pos, table, pos, 16, 9, out=maps)),
    ]
    for written, read, call in calls:
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > n for t, n in zip(written, before[0]))
        assert [t._version for t in read] == before[1]


def test_a_gradient_does_not_use_what_was_turned_in_place():
    fa = _fa()
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    w = torch.randn(5, 2, 64, device="cuda").bfloat16().requires_grad_()
    y = w * 2
    loss = (y * y).sum()                            # keeps y
    fa.rotary(y.detach(), pos, freq, out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_written_all_the_same():
    fa = _fa()
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    with torch.inference_mode():
        x = torch.randn(5, 2, 64, device="cuda").bfloat16()
        want = fa.rotary(x, pos, freq)
        assert torch.equal(fa.rotary(x, pos, freq, out=x), want)
    y = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    with torch.inference_mode():
        fa.rotary(x, pos, freq, out=y)
    assert y._version > 0
    fa.rotary(y, pos, freq, out=x)                  # an inference tensor outside the mode
