"""Attention over a 4-bit cache where several CTAs share a row tile's keys, at the shapes
whose kernels differ (needs a B200): selections and pages that are copied row by row, blocks of 32
keys, the joins' places.  Each call is checked to take that path, by its workspace."""
import pytest
import torch

import test_gpu_cache as T
from test_gpu_cache import lib, no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


def shared(L, monkeypatch):
    """From here on every attention call without a workspace fails."""
    lib = L.load_library()
    size = lib.csa_cache_attention_workspace_size

    class Checked:
        def __getattr__(self, name):
            return getattr(lib, name)

        @staticmethod
        def csa_cache_attention_workspace_size(a):
            n = size(a)
            assert n > 0, "one CTA has the whole tile"
            return n

    monkeypatch.setattr(L, "load_library", lambda *_: Checked())


@pytest.mark.parametrize("HA", [8, 16])
@pytest.mark.parametrize("topk", [1500, 2048])
def test_selected(lib, monkeypatch, HA, topk):
    """Lists of more than four chunks, two queries of their own each, entries out of the sequence, a length of zero."""
    shared(lib, monkeypatch)
    T.check_attention(lib, B=4, S=2, HA=HA, H=1, Dk=128, Dv=128, page=24, lens=[4000, 0, 17, 2500], topk=topk, seed=topk + HA)


@pytest.mark.parametrize("HA,H", [(16, 2), (24, 2)])
def test_selected_grouped_heads(lib, monkeypatch, HA, H):
    shared(lib, monkeypatch)
    T.check_attention(lib, B=2, S=3, HA=HA, H=H, Dk=64, Dv=128, page=16, lens=[3000, 1200], topk=2048, seed=HA)


@pytest.mark.parametrize("HA,H,S", [(8, 1, 1), (16, 1, 1), (6, 2, 4), (4, 4, 9)])
@pytest.mark.parametrize("page", [24, 1])
def test_dense_row_by_row(lib, monkeypatch, HA, H, S, page):
    """Pages that hold no whole tiles of 16 keys."""
    shared(lib, monkeypatch)
    T.check_attention(lib, B=4, S=S, HA=HA, H=H, Dk=128, Dv=128, page=page, lens=[3000, 0, 17, 1100], seed=page + HA)


@pytest.mark.parametrize("HA", [8, 16])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("Dk,Dv", [(192, 128), (192, 192), (256, 256), (64, 256), (256, 64), (128, 256)])
def test_wide_rows(lib, monkeypatch, Dk, Dv, HA, page):
    """Blocks of 32 keys, three stages."""
    shared(lib, monkeypatch)
    T.check_attention(lib, B=3, S=1, HA=HA, H=1, Dk=Dk, Dv=Dv, page=page, lens=[3000, 0, 1111], seed=Dk + Dv + HA)


@pytest.mark.parametrize("HA", [8, 16])
def test_holes(lib, monkeypatch, HA):
    shared(lib, monkeypatch)
    T.check_attention(lib, B=4, S=2, HA=HA, H=1, Dk=128, Dv=128, page=16, lens=[2000, 1500, 64, 3], holes=True, seed=4)


@pytest.mark.parametrize("D,H", [(64, 1), (192, 1), (128, 3)])
def test_scale_strides_off_16(lib, monkeypatch, D, H):
    """Scale pages at distances that the bulk copies do not take: equal to the dense ones."""
    L, g, page, pages, n = lib, T.gen(D), 16, 200, 3000
    shared(L, monkeypatch)
    dense = [T.random_cache(L, "e2m1", pages, page, H, D, g) for _ in (0, 1)]
    loose = []
    for c in dense:
        row = H * page * (D // 16)
        buf = torch.full((pages, row + D // 16), 255, dtype=torch.uint8, device="cuda")
        buf[:, :row] = c.scale.reshape(pages, row)
        assert buf.stride(0) % 16 != 0
        scale = buf.as_strided(c.scale.shape, (buf.stride(0),) + c.scale.stride()[1:])
        loose.append(L.Cache("e2m1", c.data, scale))
    table = T.pages_of(2, 100, pages, g)
    lens = torch.tensor([1600, 1111], dtype=torch.int32, device="cuda")
    for HA in (8 * H, 16 * H):
        q = torch.randn((2, 1, HA, D), generator=g, device="cuda").to(torch.bfloat16)
        a, b = (L.cache_attention(q, k, v, table, lens, scale=D ** -0.5, return_lse=True) for k, v in (dense, loose))
        # the same keys in the same shares and blocks: only the copies differ
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    no_device_error(L)


@pytest.mark.parametrize("HA,topk", [(8, 0), (16, 0), (8, 2048), (16, 2048)])
def test_replay_with_other_lengths(lib, monkeypatch, HA, topk):
    """A captured call shares out the chunks of the lengths that it finds when it is replayed."""
    L, g, n = lib, T.gen(7), 5000
    shared(L, monkeypatch)
    page = 64 if not topk else 24
    per = -(-n // page)
    c = T.random_cache(L, "e2m1", 3 * per, page, 1, 128, g)
    table = T.pages_of(3, per, 3 * per, g)
    lens = torch.tensor([n, 4000, 1], dtype=torch.int32, device="cuda")
    q = torch.randn((3, 1, HA, 128), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randint(-5, n, (3, 1, topk), generator=g, device="cuda", dtype=torch.int32) if topk else None
    call = lambda: L.cache_attention(q, c, c, table, lens, scale=0.09, idx=idx, return_lse=True)  # noqa: E731
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = call()
    for new in ([n, 4000, 1], [1, 0, 0], [0, 0, 0], [300, n, 2999], [0, 257, 0], [n, n, n]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(kept, want):
            assert torch.equal(x, y), new
    no_device_error(L)


@pytest.mark.parametrize("HA", [8, 16])
def test_more_sequences_than_ctas(lib, monkeypatch, HA):
    """Shares that take whole tiles of several sequences, begin in one and end in another."""
    shared(lib, monkeypatch)
    lens = [(37 * i * i) % 1400 for i in range(300)]
    T.check_attention(lib, B=len(lens), S=1, HA=HA, H=1, Dk=64, Dv=64, page=24, lens=lens, seed=HA)


@pytest.mark.parametrize("HA,H", [(8, 1), (16, 2), (64, 1), (128, 1)])
@pytest.mark.parametrize("topk", [40, 1500])
def test_selected_without_causality(lib, HA, H, topk):
    """causal=False: every listed key of the sequence, whatever the query's place."""
    T.check_attention(lib, B=3, S=3, HA=HA, H=H, Dk=128, Dv=64, page=16, lens=[2000, 2, 0], topk=topk, causal=False, seed=HA + topk)


@pytest.mark.parametrize("HA", [8, 16, 64, 128])
@pytest.mark.parametrize("page,pages", [(16, 20), (64, 40), (24, 100)])
def test_sequences_longer_than_their_table(lib, HA, page, pages):
    """kv_len past the pages that the table lists: as many positions as it reaches."""
    L, g, n = lib, T.gen(page), page * pages
    c = T.random_cache(L, "e2m1", 2 * pages, page, 1, 128, g)
    table = T.pages_of(2, pages, 2 * pages, g)
    q = torch.randn((2, 1, HA, 128), generator=g, device="cuda").to(torch.bfloat16)
    call = lambda lens: L.cache_attention(q, c, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.09,  # noqa: E731
                                          return_lse=True)
    for long in (n + 1, 10 ** 6, 2 ** 31 - 1):
        for x, y in zip(call([long, 77]), call([n, 77])):
            assert torch.equal(x, y)
    no_device_error(L)
