"""Refusals of the cache operators that depend on several arguments together, without a
GPU: a call that passes every check ends at the missing device, before any launch."""
import random

import pytest
import torch

import lightning_indexer_top_02_b200 as L
from lightning_indexer_top_02_b200 import cache as C
from lightning_indexer_top_02_b200.build import build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its addresses are made up")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return L.load_library()


def cache(dtype, at, *, H=2, D=64, pages=8, page=16, page_stride=0, scale_stride=0):
    c = C.CsaCache()
    c.dtype, c.H, c.D, c.num_pages, c.page_size, c.tensor_scale = dtype, H, D, pages, page, 1.0
    c.data, c.scale = at if isinstance(at, tuple) else (at, at + (1 << 24))
    if dtype == C.CSA_CACHE_BF16:
        c.scale = None
    c.page_stride, c.scale_page_stride = page_stride, scale_stride
    return c


def append(cache_k, cache_v=None):
    a = C.CsaAppendArgs()
    a.k = a.kv_len = a.page_table = 1 << 30
    a.k_token_stride, a.k_head_stride = cache_k.H * cache_k.D, cache_k.D
    a.B, a.S, a.N = 2, 1, 2
    a.max_pages = a.table_stride = 4
    a.cache_k = cache_k
    if cache_v is not None:
        a.v, a.cache_v = 1 << 30, cache_v
        a.v_token_stride, a.v_head_stride = cache_v.H * cache_v.D, cache_v.D
    return L.csa_cache_append(a, None)


def row_bytes(c):
    return {C.CSA_CACHE_BF16: (2 * c.D, 0), C.CSA_CACHE_E4M3: (c.D, 4), C.CSA_CACHE_E2M1: (c.D // 2, c.D // 16)}[c.dtype]


def memory(c):
    """The bytes of a cache's data and of its scales, as sets."""
    out = []
    for at, stride, row in ((c.data, c.page_stride, row_bytes(c)[0]), (c.scale, c.scale_page_stride, row_bytes(c)[1])):
        n = c.H * c.page_size * row
        out.append({at + p * (stride or n) + i for p in range(c.num_pages) for i in range(n)} if row else set())
    return out


def test_append_refuses_shared_memory():
    big = 1 << 26
    k, E = cache(2, big), 64 * 16 * 2 // 2 * 8                       # E: bytes of a cache's codes
    assert append(k) == append(k, cache(2, 2 * big)) == L.CSA_ERR_CUDA
    for at in ((big, 2 * big), (big + 16, 2 * big), (big + E - 16, 2 * big), (big - E + 16, 2 * big), (2 * big, big),
               (2 * big, big + (1 << 24)), (2 * big, big + (1 << 24) + 16), (big + (1 << 24), 2 * big)):
        assert append(k, cache(2, at)) == L.CSA_ERR_INVALID_ARG, at
    for at in ((big + E, 2 * big), (big - E, 2 * big), (2 * big, big + E)):
        assert append(k, cache(2, at)) == L.CSA_ERR_CUDA, at
    assert append(cache(2, (big, big))) == append(cache(1, (big, big + 64))) == L.CSA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [C.CSA_CACHE_BF16, C.CSA_CACHE_E4M3, C.CSA_CACHE_E2M1])
def test_append_takes_interleaved_pages(dtype):
    """Codes and scales of keys and values page by page in one allocation, in any order; one byte less is refused."""
    one = cache(dtype, 1 << 26)
    data, scale = (one.H * one.page_size * b for b in row_bytes(one))
    step = 2 * (data + scale)
    at = [(1 << 26) + o for o in (0, data, data + scale, 2 * data + scale)]
    how = dict(page_stride=step, scale_stride=step)
    assert append(cache(dtype, (at[0], at[1]), **how), cache(dtype, (at[2], at[3]), **how)) == L.CSA_ERR_CUDA
    if scale:
        assert append(cache(dtype, (at[0], at[1]), **how), cache(dtype, (at[2], at[3] - 16), **how)) == L.CSA_ERR_INVALID_ARG
    assert append(cache(dtype, (at[0], at[1]), **how), cache(dtype, (at[2] - 16, at[3]), **how)) == L.CSA_ERR_INVALID_ARG


def test_append_shared_memory_byte_by_byte():
    """Small caches at random places and distances, against their bytes as sets."""
    rng, seen = random.Random(1), {L.CSA_ERR_CUDA: 0, L.CSA_ERR_INVALID_ARG: 0}
    for _ in range(1500):
        dtype, pages, page = rng.choice([0, 1, 2]), rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 2])

        def one():
            H, D = 1, 32 * rng.choice([1, 1, 2])
            c = cache(dtype, (16 * rng.randint(64, 200), 16 * rng.randint(64, 200)), H=H, D=D, pages=pages, page=page)
            n, s = (H * page * b for b in row_bytes(c))
            if pages > 1 and rng.random() < 0.8:
                c.page_stride = (n + 15) // 16 * 16 + 16 * rng.choice([0, 1, 4, 9])
                if s:
                    c.scale_page_stride = s + row_bytes(c)[1] * rng.choice([0, 1, 8, 30])
            return c

        k, v = one(), one()
        sets = memory(k) + memory(v)
        clash = any(sets[i] & sets[j] for i in range(4) for j in range(i))
        want = L.CSA_ERR_INVALID_ARG if clash else L.CSA_ERR_CUDA
        assert append(k, v) == want, [(c.data, c.scale, c.page_stride, c.scale_page_stride, c.D, pages, page) for c in (k, v)]
        seen[want] += 1
    assert min(seen.values()) > 200, seen


def attention(workspace=None, **fields):
    """B = 2, S = 3, 8 heads of 64: q and out of 6,144 bytes, lse of 192, idx of 6 * 40 entries."""
    a = C.CsaCacheAttnArgs()
    a.cache_k, a.cache_v = cache(2, 1 << 26), cache(2, 1 << 27)
    a.kv_len = a.page_table = 1 << 28
    a.max_pages = a.table_stride = 4
    a.B, a.S, a.HA, a.topk, a.causal, a.scale = 2, 3, 8, 40, 1, 0.1
    a.q, a.out, a.lse, a.idx = 1 << 20, 1 << 21, 1 << 22, 1 << 23
    for f, v in fields.items():
        setattr(a, f, v)
    return L.csa_cache_attention(a, workspace, 1 << 20, None)


@pytest.mark.parametrize("size,other,other_size,field", [(6144, "q", 6144, "out"), (6144, "idx", 960, "out"), (192, "q", 6144, "lse"),
                                                         (192, "out", 6144, "lse"), (192, "idx", 960, "lse")])
def test_attention_refuses_overlapping_outputs(size, other, other_size, field):
    at = dict(q=1 << 20, out=1 << 21, lse=1 << 22, idx=1 << 23)[other]
    assert attention() == L.CSA_ERR_CUDA
    for d in (0, 16, other_size - 16, 16 - size):
        assert attention(**{field: at + d}) == L.CSA_ERR_INVALID_ARG, d
    for d in (other_size, -size):
        assert attention(**{field: at + d}) == L.CSA_ERR_CUDA, d
    assert attention(lse=None, idx=None) == L.CSA_ERR_CUDA


@pytest.mark.parametrize("dtype", [C.CSA_CACHE_BF16, C.CSA_CACHE_E4M3, C.CSA_CACHE_E2M1])
def test_append_refuses_heads_past_an_int(dtype):
    """2^30 heads of 4 lanes each: their product is 0 in 32 bits, which the host divided by."""
    far = (1 << 40, 1 << 50)
    assert append(cache(dtype, far, H=1 << 30, pages=1, page=1)) == L.CSA_ERR_UNSUPPORTED
    k, v = (cache(dtype, at, H=1 << 28, D=D, pages=1, page=1) for at, D in ((far, 32), ((1 << 41, 1 << 51), 128)))
    assert append(k, v) == L.CSA_ERR_UNSUPPORTED
    assert append(k) == L.CSA_ERR_CUDA


def test_scales_whose_product_is_not_finite():
    """Each is finite; their products, which the kernels compute with, are not."""
    k = cache(2, 1 << 26)
    k.tensor_scale = 4.0
    assert attention(cache_k=k, scale=1e38) == L.CSA_ERR_INVALID_ARG
    assert attention(cache_k=k, scale=-1e38) == L.CSA_ERR_INVALID_ARG
    assert attention(cache_k=k, scale=1e37) == L.CSA_ERR_CUDA
    v = cache(2, 1 << 27)
    v.tensor_scale = 1e38
    assert append(v) == append(k, v) == L.CSA_ERR_INVALID_ARG
    assert attention(cache_v=v) == append(k) == L.CSA_ERR_CUDA
