"""fa_cache_append writes keys and values: caches of one buffer are taken when their
rows lie apart, in any order in memory, and refused when they meet. Without a GPU:
the checks come before CUDA is touched; every answer is held against the list of the
bytes themselves."""
import itertools
import random

import pytest

import exact_attention_91_gb300 as fa

from .test_serve_abi import P, append, cache, lib  # noqa: F401  (lib: builds the library)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run on made-up addresses")

KV = 64 * P                                        # away from the other fake addresses


def call(c):
    row = c.heads * c.d
    return append(c, q=P, k=2 * P, v=3 * P, pos=4 * P, slots=5 * P, freq=6 * P, q_out=7 * P, k_out=8 * P, ks=row, vs=row,
                  kos=row, r=0)


def rows(c, name):
    """First bytes of all rows of the keys or the values."""
    elt = 1 if c.type == fa.CACHE_E4M3 else 2
    at = getattr(c, name)
    st = [getattr(c, f"{name}_{x}") * elt for x in ("block", "token", "head")]
    return sorted(at + b * st[0] + t * st[1] + h * st[2] for b, t, h in
                  itertools.product(range(c.num_blocks), range(c.page_size), range(c.heads)))


def meet(c):
    size = c.d * (1 if c.type == fa.CACHE_E4M3 else 2)
    both = sorted([(x, 0) for x in rows(c, "k")] + [(x, 1) for x in rows(c, "v")])
    return any(y - x < size for (x, _), (y, _) in zip(both, both[1:]))


@pytest.mark.parametrize("kind", [fa.CACHE_BF16, fa.CACHE_E4M3])
@pytest.mark.parametrize("k,v", [
    ((0, 0, 0, 0), (0, 0, 2, 0)),    # [block, token, 2 * heads, d]: the heads side by side
    ((0, 0, 0, 0), (0, 1, 0, 0)),    # [block, 2, token, heads, d]
    ((0, 0, 0, 0), (2, 0, 0, 0)),    # one after the other
])
def test_usual_layouts_are_taken(kind, k, v):
    d, page, heads, blocks = 64, 16, 2, 4
    elt = 1 if kind == fa.CACHE_E4M3 else 2
    if v[2]:
        st, off = dict(block=page * 2 * heads * d, token=2 * heads * d, head=d), heads * d
    elif v[1]:
        st, off = dict(block=2 * page * heads * d, token=heads * d, head=d), page * heads * d
    else:
        st, off = dict(block=page * heads * d, token=heads * d, head=d), blocks * page * heads * d
    s = {f"{n}_{x}": st[x] for n in "kv" for x in st}
    for a, b in ((0, off), (off, 0)):
        c = cache(KV + a * elt, KV + b * elt, page=page, heads=heads, d=d, blocks=blocks, kind=kind, **s)
        assert not meet(c) and call(c) != -10


def test_rows_side_by_side_and_other_orders_within_a_block_are_taken():
    d, page, heads, blocks = 64, 16, 2, 3
    s = dict(k_block=2 * page * heads * d, k_token=2 * heads * d, k_head=2 * d)
    c = cache(KV, KV + 2 * d, page=page, heads=heads, d=d, blocks=blocks, **s,
              **{"v" + n[1:]: x for n, x in s.items()})                                   # [block, token, head, 2, d]
    assert not meet(c) and call(c) != -10
    half = page * heads * d
    c = cache(KV, KV + 2 * half, page=page, heads=heads, d=d, blocks=blocks, k_block=2 * half, k_token=heads * d, k_head=d,
              v_block=2 * half, v_token=d, v_head=page * d)                               # k token by token, v head by head
    assert not meet(c) and call(c) != -10


@pytest.mark.parametrize("off", ["head", "token", "block", "half a row", "row and a half"])
@pytest.mark.parametrize("back", [False, True])
def test_values_on_the_keys_are_refused(off, back):
    d, page, heads, blocks = 64, 16, 4, 5
    st = dict(block=page * heads * d, token=heads * d, head=d)
    at = {"half a row": d // 2, "row and a half": d + d // 2}.get(off) or st[off]
    a, b = KV, KV + 2 * at
    c = cache(*((b, a) if back else (a, b)), page=page, heads=heads, d=d, blocks=blocks,
              **{f"{n}_{x}": st[x] for n in "kv" for x in st})
    assert meet(c) and call(c) == -10


def test_slices_of_one_tensor_that_share_a_head_are_refused():
    d, page, heads, blocks = 64, 16, 4, 3
    st = dict(block=page * heads * d, token=heads * d, head=d)
    s = {f"{n}_{x}": st[x] for n in "kv" for x in st}
    assert call(cache(KV, KV + 2 * d, page=page, heads=2, d=d, blocks=blocks, **s)) == -10         # kv[:, :, 0:2], kv[:, :, 1:3]
    assert call(cache(KV, KV + 4 * d, page=page, heads=2, d=d, blocks=blocks, **s)) != -10         # kv[:, :, 0:2], kv[:, :, 2:4]


def test_answers_are_those_of_the_bytes():
    """Random layouts in one buffer: what meets is refused, and of what lies apart
    everything with equal strides is taken."""
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        d, page, heads, blocks = 64, 16, rng.choice([1, 2, 3]), rng.choice([1, 2, 3])
        order = rng.choice([("block", "token", "head"), ("block", "head", "token"), ("token", "block", "head"),
                            ("head", "block", "token")])
        sizes = dict(block=blocks, token=page, head=heads)
        st, span = {}, d
        for x in reversed(order):
            st[x] = span + 16 * rng.choice([0, 0, 1, 4, 8, 12]) + span * rng.choice([0, 0, 1, 2])
            span = st[x] * (sizes[x] - 1) + span
        off = rng.choice([rng.randrange(0, span + 2 * d, 8), rng.choice(list(st.values())) * rng.randint(0, 3) +
                          rng.choice([0, d, d + 8, d - 8])])
        s = {f"{n}_{x}": st[x] for n in "kv" for x in st}
        a, b = KV, KV + 2 * off
        if rng.random() < 0.5:
            a, b = b, a
        c = cache(a, b, page=page, heads=heads, d=d, blocks=blocks, **s)
        m = meet(c)
        seen[m] += 1
        assert (call(c) == -10) == m, (order, sizes, st, off)
    assert min(seen.values()) > 300


def test_nothing_that_meets_is_taken_whatever_the_orders():
    """Keys and values with strides of their own, also one stride in common and the
    rest in another order: a meeting is never missed."""
    rng = random.Random(8)
    seen = 0
    for _ in range(6000):
        d, page, heads, blocks = 64, 16, rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3, 7])
        sizes = dict(block=blocks, token=page, head=heads)

        def lay(order, keep=None):
            st, span = {}, d
            for x in reversed(order):
                st[x] = keep[1] if keep and x == keep[0] and keep[1] >= span else span + rng.choice([0, 0, 64, 512])
                span = st[x] * (sizes[x] - 1) + span
            return st, span

        orders = list(itertools.permutations(("block", "token", "head")))
        ks, span = lay(rng.choice(orders))
        same = rng.choice(["block", "token", "head"])
        vs, vspan = lay(rng.choice(orders), (same, ks[same]))
        off = rng.randrange(-vspan, span, 8)
        c = cache(KV, KV + 2 * off, page=page, heads=heads, d=d, blocks=blocks, **{f"k_{x}": ks[x] for x in ks},
                  **{f"v_{x}": vs[x] for x in vs})
        if meet(c):
            seen += 1
            assert call(c) == -10, (sizes, ks, vs, off)
    assert seen > 1000
