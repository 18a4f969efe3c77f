"""Block tables and slot maps from request lengths (fa_page_maps) against the
step taken one token after the other on the host; all results are equal."""
import random

import pytest

from . import serve_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


def _int(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def step(fa, context, fresh, width, page, unused, T=None, seed=0, table=None):
    rng = random.Random(seed)
    held = [-(-max(c, 0) // page) for c in context]
    if table is None:
        ids = iter(rng.sample(range(10 ** 6), sum(held) + 1))
        table = [[next(ids) if i < min(h, width) else -1 - i for i in range(width)] for h in held]
    T = sum(max(n, 0) for n in fresh) if T is None else T
    t = _int(table)
    m = fa.page_maps(_int(context), _int(fresh), t, _int(unused) if unused else torch.empty(0, dtype=torch.int32).cuda(),
                     page, T)
    torch.cuda.synchronize()
    want = so.page_maps(context, fresh, table, unused, page, T)
    got = (t.tolist(), m.slots.tolist(), m.positions.tolist(), m.cu_seqlens.tolist(), m.seq_lens.tolist(), m.counts.tolist())
    for name, a, b in zip(("table", "slots", "positions", "cu", "lens", "counts"), got, want):
        assert a == b, name
    return got


@pytest.mark.parametrize("page", [16, 64])
def test_ordinary_steps(page):
    fa = _fa()
    unused = list(range(5000, 7000))
    step(fa, [0], [1], 4, page, unused)
    step(fa, [15, 16, 17, 31, 32], [1, 1, 1, 1, 1], 4, page, unused)            # one token each, around page ends
    step(fa, [0, 5, 100, 0], [300, 1, 0, 33], 40, page, unused, T=400)          # prompts, an idle request, padding
    step(fa, [0, 0, 0], [0, 0, 0], 4, page, unused, T=5)                        # nothing to do
    step(fa, [0, 0, 0], [0, 0, 0], 4, page, unused, T=0)
    step(fa, [0, 0, 7, 0, 0], [0, 0, 9, 0, 0], 4, page, unused)                 # empty requests around one


def test_many_requests_and_long_prompts():
    fa = _fa()
    rng = random.Random(1)
    for B in (31, 32, 33, 511, 512, 513, 1500):
        ctx = [rng.choice([0, 1, 16, rng.randint(0, 3000)]) for _ in range(B)]
        new = [rng.choice([0, 1, 1, 1, rng.randint(0, 200)]) for _ in range(B)]
        step(fa, ctx, new, 220, 16, list(range(100000, 140000)), T=sum(new) + 3, seed=B)
    step(fa, [0, 3], [70000, 60001], 5000, 16, list(range(9000)))


def test_most_requests():
    fa = _fa()
    B = 8192
    step(fa, [i % 50 for i in range(B)], [1] * B, 4, 16, list(range(10 ** 6, 10 ** 6 + B)))


def test_pages_run_out_and_tables_too_narrow():
    fa = _fa()
    g = step(fa, [10, 0, 40], [100, 50, 30], 20, 16, [7, 8, 9])                 # three pages of twelve
    assert g[5][:2] == [3, 9]
    step(fa, [10, 0, 40], [100, 50, 30], 20, 16, [])                            # none at all
    g = step(fa, [0, 5], [100, 10], 3, 16, list(range(50)))                     # wider than the table
    assert g[5][3] == 1
    step(fa, [200, 5], [10, 10], 3, 16, list(range(50)), table=[[1, 2, 3], [4, -1, -1]])   # context past the table
    step(fa, [20], [20], 4, 16, [3], table=[[-1, 6, 0, 0]])                     # a page that was given back


def test_fewer_rows_than_tokens_and_bad_lengths():
    fa = _fa()
    step(fa, [0, 0], [20, 20], 4, 16, list(range(50)), T=25)
    step(fa, [-3, 5, -2 ** 31], [4, -7, 1], 4, 16, list(range(50)))


def test_huge_lengths_stay_in_bounds():
    """Sums past 2^31 - 1 stay there; nothing outside the arrays is touched."""
    fa = _fa()
    big = 2 ** 31 - 1
    t = torch.full((3, 6), -1, dtype=torch.int32).cuda()
    m = fa.page_maps(_int([0, big, 5]), _int([big, big, big]), t, _int(list(range(8))), 16, 100)
    assert m.cu_seqlens.tolist() == [0, big, big, big] and m.seq_lens.tolist() == [big] * 3
    assert t.tolist() == [[0, 1, 2, 3, 4, 5], [-1] * 6, [-1, 6, 7, -1, -1, -1]]
    assert m.counts.tolist() == [8, 3, big, 3]
    assert m.slots.tolist() == list(range(96)) + [-1] * 4 and m.positions.tolist() == list(range(100))


def test_slots_past_31_bits_are_refused():
    fa = _fa()
    t = _int([[2 ** 27 - 1, 2 ** 27]])
    m = fa.page_maps(_int([14]), _int([4]), t, _int([]), 16, 4)
    assert m.slots.tolist() == [2 ** 31 - 2, 2 ** 31 - 1, -1, -1]


def test_strided_table_and_given_outputs():
    fa = _fa()
    wide = torch.full((2, 9), 77, dtype=torch.int32).cuda()
    wide[:, :3] = -1
    whole = torch.full((40,), 55, dtype=torch.int32).cuda()
    out = fa.PageMaps(whole[1:11], whole[12:22], whole[23:26], whole[27:29], whole[30:34])
    m = fa.page_maps(_int([0, 0]), _int([3, 5]), wide[:, :3], _int([4, 2]), 16, 10, out=out)
    assert m is out
    assert whole.tolist() == ([55] + [64, 65, 66, 32, 33, 34, 35, 36, -1, -1] + [55] + [0, 1, 2, 0, 1, 2, 3, 4, 0, 0] +
                              [55] + [0, 3, 8] + [55] + [3, 5] + [55] + [2, 0, 8, 0] + [55] * 6)
    assert wide.tolist() == [[4, -1, -1] + [77] * 6, [2, -1, -1] + [77] * 6]
