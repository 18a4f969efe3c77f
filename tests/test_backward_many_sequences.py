"""Packed backward passes over thousands of sequences, numbered through all of them: how a block finds its sequence,
restated in Python after fa_bwd_kernel.cuh (BwdFind), and the kernels on such batches."""
import random

import numpy as np
import pytest

from . import grad_oracle as G

torch = pytest.importorskip("torch")

BLOCK = 128


class Find:
    """The kernel's walk over chunks of 32 sequences; `steps` counts the chunks that it looked at."""

    def __init__(self, cu, total, bound):
        self.cu, self.total, self.steps = cu, total, 0
        self.B = len(cu) - 1
        self.last = (self.B - 1) // 32 * 32
        lanes = [0] * 32
        for b in range(self.last):
            lanes[b % 32] = min(lanes[b % 32] + self.blocks(b), bound)
        self.last_before = min(sum(lanes), bound)
        self.b0, self.before = self.last, self.last_before
        self.load()
        self.count = min(self.before + self.sum, bound)

    def blocks(self, b):
        assert 0 <= b < self.B
        t0 = min(max(self.cu[b], 0), self.total)
        return (min(max(self.cu[b + 1], t0), self.total) - t0 + BLOCK - 1) // BLOCK

    def load(self):
        self.steps += 1
        n = [self.blocks(b) if b < self.B else 0 for b in range(self.b0, self.b0 + 32)]
        self.n, self.incl = n, list(np.cumsum(n))
        self.sum = int(self.incl[-1])

    def find(self, t):
        while True:
            below = t < self.before
            if not below and t < self.before + self.sum:
                break
            if self.b0 == (0 if below else self.last):
                return None
            if below:
                self.b0 -= 32
            elif self.count - t < t - (self.before + self.sum):
                self.b0, self.before = self.last, self.last_before
            else:
                self.b0, self.before = self.b0 + 32, self.before + self.sum
            self.load()
            if below:
                self.before -= self.sum
        at = next(i for i in range(32) if t < self.before + self.incl[i])
        return self.b0 + at, t - self.before - int(self.incl[at] - self.n[at])


def offsets(lens):
    return [0] + np.cumsum(lens).tolist()


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 70, 1000])
def test_every_block_is_found(B):
    r = random.Random(B)
    for kind in range(3):
        lens = [(r.randint(0, 700), r.choice([0, 0, 0, 5000]), r.randint(0, 3))[kind] for _ in range(B)]
        cu = offsets(lens)
        want = [(b, i) for b, n in enumerate(lens) for i in range((n + BLOCK - 1) // BLOCK)]
        f = Find(cu, cu[-1], cu[-1] // BLOCK + B)
        assert f.count == len(want)
        some = [r.randrange(len(want)) for _ in range(50)] if want else []
        for order in (range(len(want)), range(len(want) - 1, -1, -1), some):
            for t in order:
                assert f.find(t) == want[t]


@pytest.mark.parametrize("blocks", [1, 152])
def test_the_walk_is_short(blocks):
    """One block's claims, heads in groups of 16, each from the last block down: a group costs at most the chunks."""
    B, heads = 4096, 40
    f = Find(offsets([128] * B), 128 * B, 2 * B)
    assert f.count == B  # (not one unit without rows)
    for u in range(0, B * heads, blocks):
        g = u // (16 * B)
        idx = u - g * 16 * B
        assert f.find(B - 1 - idx // min(16, heads - 16 * g)) is not None
    assert f.steps <= 3 * (B // 32 + 2)


def test_any_offsets_end_in_range():
    r = random.Random(5)
    for _ in range(300):
        B = r.choice([1, 5, 40, 130])
        total = r.choice([0, 50, 10000])
        cu = [r.choice([r.randint(-2 ** 31, 2 ** 31 - 1), r.randint(0, total)]) for _ in range(B + 1)]
        bound = total // BLOCK + B
        f = Find(cu, total, bound)
        assert 0 <= f.count <= bound
        for _ in range(30):
            got = f.find(r.randrange(max(f.count, 1)))
            assert got is None or (0 <= got[0] < B and 0 <= got[1] < max(f.blocks(got[0]), 1))


# ---- on the GPU -------------------------------------------------------------


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


def f64(t):
    return t.detach().cpu().double().numpy()


def make(fa, lens, H, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    q, k, v, do = (torch.randn(T, H, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    cu = torch.tensor(offsets(lens), dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward_varlen(q, k, v, cu, cu, max(lens), causal=True)
    return do, q, k, v, o, lse, cu


def check(x, got, lens, some):
    do, q, k, v, o, lse, cu = x
    at = cu.tolist()
    for b in some:
        i = slice(at[b], at[b + 1])
        for h in (0, q.shape[1] - 1):
            want, bound = G.backward(*(f64(t[i, h]) for t in (do, q, k, v, o)), f64(lse[h, i]), np.zeros(lens[b]), True,
                                     q.shape[2] ** -0.5)
            G.assert_gradients([f64(t[i, h]) for t in got], want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("d,H", [(64, 20), (128, 3)])
def test_thousands_of_sequences(fa, d, H):
    """Loose bounds (blocks numbered through the sequences) and tight ones (each sequence's own) give the same bits."""
    r = random.Random(d)
    lens = [r.randint(0, 200) for _ in range(4096)]
    x = make(fa, lens, H, d, 1)
    do, q, k, v, o, lse, cu = x
    T = q.shape[0]
    loose = fa.attention_backward_varlen(do, q, k, v, o, lse, cu, cu, T, T, causal=True)
    tight = fa.attention_backward_varlen(do, q, k, v, o, lse, cu, cu, 200, 200, causal=True)
    for a, b in zip(loose, tight):
        assert torch.equal(a, b)
    assert fa.fa_device_status() == (0, 0)
    check(x, loose, lens, [0, 1, 31, 32, 33, 2047, 2048, 4064, 4095] + r.sample(range(4096), 20))


@pytest.mark.gpu
def test_many_sequences_without_rows_hold_no_block_up(fa):
    """28000 sequences without rows among 30000: no wait for a block's next unit comes near a twentieth of the usual limit."""
    lens = [3 if b % 16 == 5 else 0 for b in range(30000)]
    x = make(fa, lens, 16, 64, 2)
    do, q, k, v, o, lse, cu = x
    T = q.shape[0]
    some = torch.tensor(offsets([3] * (T // 3)), dtype=torch.int32, device="cuda")
    want = fa.attention_backward_varlen(do, q, k, v, o, lse, some, some, 3, 3, causal=True)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    lib = fa.load_library()
    lib.fa_set_wait_limit_ns(100_000_000)
    try:
        got = fa.attention_backward_varlen(do, q, k, v, o, lse, cu, cu, T, T, causal=True)
        torch.cuda.synchronize()
    finally:
        lib.fa_set_wait_limit_ns(0)
    assert fa.fa_device_status() == (0, 0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    check(x, got, lens, [5, 21, 29989])
