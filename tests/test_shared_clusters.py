"""The cluster form of the shared-prefix decode (few requests: the shared part's kernel, then a cluster of blocks for each
unit of own keys, which starts before it) under graph replay, on two streams, with lengths, shared lengths and pages
that change between replays. Each size's workspace says that the shared path runs, not paged decode's."""
import pytest

from . import serve_oracle as so
from .test_decode_shared import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_91_gb300 as fa
    return fa


def rand(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


# requests, query heads, key heads, d: units of own keys that make clusters of 8, 4, 2 and 1 blocks on 152 SMs
SIZES = [(8, 8, 2, 64), (8, 32, 8, 128), (30, 20, 5, 64), (36, 8, 4, 128), (70, 40, 2, 64), (40, 7, 7, 128)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("requests,hq,hkv,d", SIZES)
def test_captured_with_changing_lengths(fa, requests, hq, hkv, d, e4m3):
    page, pages = 16, 512
    kind = fa.CACHE_E4M3 if e4m3 else fa.CACHE_BF16
    # (a table with room for 128 MB of keys and values or less would be read as paged decode reads it)
    width = (1 << 27) // (requests * hkv * d * (2 if e4m3 else 4) * page) + 1
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shared_ws = fa.fa_decode_shared_workspace(requests, hq, hkv, d, kind, page, width, 2, sms)
    assert shared_ws != fa.fa_decode_paged_workspace(requests, hq, hkv, d, kind, page, width, sms)
    assert requests * hkv * ((hq // hkv + 15) // 16) <= 2 * sms  # (one wave of clusters: not the equal runs)
    kc, vc = (rand(pages, page, hkv, d, seed=s) for s in (1, 2))
    if e4m3:
        kc, vc = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    ks = torch.linspace(0.4, 1.2, hkv, device="cuda") if e4m3 else None
    vs = torch.linspace(1.1, 0.3, hkv, device="cuda") if e4m3 else None
    q = rand(requests, hq, d, seed=3)
    lens, prefix = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (requests, 2))
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    longest = min(1100, width * page)

    def fill(seed, shared):
        g = torch.Generator().manual_seed(seed)
        p = [min(n, longest) for n in shared]
        used = (longest + page - 1) // page
        t = torch.randint(0, pages, (requests, used), generator=g)
        for i in range(2):
            rows = slice(i * requests // 2, (i + 1) * requests // 2)
            t[rows, :p[i] // page] = t[rows.start, :p[i] // page]
        table[:, :used] = t.int().cuda()
        prefix.copy_(torch.tensor(p, dtype=torch.int32))
        n = torch.randint(0, longest + 1, (requests,), generator=g)
        n[0], n[-1] = 0, longest
        lens.copy_(n.int())

    def decode():
        return fa.attention_decode_shared(q, kc, vc, table, lens, prefix, k_scale=ks, v_scale=vs)

    fill(0, (300, 640))
    decode()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(decode())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for seed, shared in ((1, (700, 33)), (2, (0, 0)), (3, (1024, 15)), (4, (129, 512))):
        fill(seed, shared)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        ref = so.decode(so.f64(q), so.f64(kc), so.f64(vc), table.cpu().numpy(), lens.cpu().numpy(), d ** -0.5,
                        None if ks is None else so.f64(ks), None if vs is None else so.f64(vs))
        eager = decode()
        check(eager, ref)
        for got in outs:
            assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
    assert fa.fa_device_status() == (0, 0)
