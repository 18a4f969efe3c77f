"""Temporaries given to a call on another stream: their memory is not handed out
again on the current one while the call may still use it."""
import pytest

from .test_decode_paged import _fa, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["decode", "rotary", "append", "maps"])
def test_temporaries_outlive_a_call_on_another_stream(op):
    fa = _fa()
    x = make([400, 90, 333], 8, 2, 128, 16, seed=61)
    freq = fa.rotary_inv_freq(128, device="cuda")[0]
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    out = fa.page_maps(x["lens"], pos, x["table"].clone(), pos, 16, 9)

    def run(own, **kw):
        """own(t): the tensor to give for t."""
        if op == "decode":
            return fa.attention_decode_paged(own(x["q"]), x["k"], x["v"], own(x["table"]), own(x["lens"]), **kw)
        if op == "rotary":
            return (fa.rotary(own(x["q"]), own(pos), own(freq), **kw),)
        if op == "append":
            kc, vc = torch.zeros_like(x["k"]), torch.zeros_like(x["v"])    # (the clones below have the stream wait for them)
            q, k = own(x["q"]), own(x["q"][:, :2])
            q = fa.cache_append(q, k, own(x["q"][:, 2:4]), own(pos), own(pos), own(freq), kc, vc, **kw)
            return q, kc, vc
        given = fa.PageMaps(*(own(t) for t in out)) if kw else None        # the results, in buffers that are dropped but one
        m = fa.page_maps(own(x["lens"]), own(pos), own(x["table"]), own(pos), 16, 9, out=given, **kw)
        return (m.slots.clone(),) if not kw else (m,)

    want = run(lambda t: t.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        sizes = []

        def own(t):
            sizes.append(t.numel() * t.element_size())
            y = t.clone(memory_format=torch.contiguous_format)
            side.wait_stream(torch.cuda.current_stream())
            return y

        with torch.cuda.stream(side):
            torch.cuda._sleep(20000000)
        got = run(own, stream=side)
        grabbed = [torch.full((n,), 0x41, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        if op == "maps":
            got = (got[0].slots,)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del grabbed, got
