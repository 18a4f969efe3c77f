"""The join of a cluster's blocks in the small form of the paged decode: every
cluster size, blocks without a key among them, launch on launch (the blocks of a
cluster end while others of it may still read their shared memory, unless the
last barrier holds them)."""
import pytest

from . import serve_oracle as so
from .test_decode_paged import _fa, call, make, small_form, want

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,e4m3,hq,hkv", [(128, False, 4, 1), (128, False, 16, 1), (64, True, 20, 1), (64, False, 1, 1),
                                           (128, True, 11, 1)])
@pytest.mark.parametrize("tiles", [9, 17, 40, 256])                   # clusters of 2, 4, 8 and 8 blocks
def test_joined_results_of_launches_in_a_row(d, e4m3, hq, hkv, tiles):
    fa = _fa()
    keys = 4096 // (d if e4m3 else 2 * d)
    n = tiles * keys
    # requests with fewer tiles than blocks, without a key, with one, and whole ones
    x = make([n, 1, 0, keys, 2 * keys + 1, n - 1, 3 * keys, n], hq, hkv, d, 16, e4m3, seed=tiles)
    assert small_form(fa, x)
    o, lse = call(fa, x)
    torch.cuda.synchronize()
    so.assert_decode(so.f64(o), so.f64(lse), want(x), e4m3 and hq > 8 * hkv)
    outs = [(torch.full_like(o, 9.0), torch.full_like(lse, 9.0)) for _ in range(200)]
    for a, b in outs:
        call(fa, x, out=a, lse=b)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)
    lone = call(fa, x, return_lse=False)                               # no log-sum-exp asked for
    assert torch.equal(lone, o)
