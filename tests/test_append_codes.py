"""The codes that an append writes into an e4m3 cache: those of the value over the
head's scale, a quotient rounded once to fp32, and once to e4m3."""
import pytest

from .test_cache_append import _fa

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_codes_are_those_of_the_quotient(d, interleaved):
    """Every bf16 value over scales of all sizes (ordinary ones, the borders of
    fp32, zero, infinity, below zero): the codes of a fp32 division on the CPU,
    bit for bit, zeros' signs and NaN included."""
    fa = _fa()
    g = torch.Generator().manual_seed(d)
    scales = torch.cat((0.003 + 0.1 * torch.rand(55, generator=g),
                        torch.tensor([1.0, 3.0, -0.7, 1e-39, 2.0 ** 127, 1e-30, 0.0, float("inf"), float("nan")])))
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).reshape(65536 // d, 1, d).expand(-1, len(scales), d)
    T = v.shape[0]
    slots = torch.randperm(T, generator=g).int()
    kc, vc = (torch.zeros(T // 16, 16, len(scales), d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              for _ in range(2))
    x, s = v.contiguous().cuda(), scales.cuda()
    fa.cache_append(x[:, :1].contiguous(), x, x, slots.cuda(), slots.cuda(), None, kc, vc, interleaved=interleaved,
                    k_scale=s, v_scale=s)
    want = (v.float() / scales[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    for cache in (kc, vc):
        got = cache.view(torch.uint8).cpu().reshape(T, len(scales), d)[slots.long()]
        nan = (want & 127) == 127
        assert torch.equal((got & 127) == 127, nan)
        wrong = ((got != want) & ~nan).sum((0, 2))
        assert not wrong.any(), {float(scales[i]): int(n) for i, n in enumerate(wrong) if n}
