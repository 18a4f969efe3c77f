"""Sizes that do not fit an int are refused, not wrapped around."""
import pytest

from .test_decode_paged import _fa

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16 - 2 ** 32, 16 + 2 ** 32, -16, 2 ** 31, -2 ** 63])
def test_page_sizes_past_an_int_are_refused(page):
    fa = _fa()
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(fa.FaError) as e:
        fa.page_maps(one, one, table, one, page, 1)
    assert e.value.status == -2
    torch.cuda.synchronize()
    assert (table == -1).all()
