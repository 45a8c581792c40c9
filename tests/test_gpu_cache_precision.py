"""How far the cache operators' arithmetic reaches: keys far below a row's
largest, query elements far below theirs (needs a B200).

Bounds:
* attention: P is f16 relative to 2^7 at least, so an absolute error of 2^-25 is 2^-32 of the
  largest weight; the rest as in test_gpu_cache.py (2^-11 of P, 2^-8 of out, a logit's
  e = Dk * 2^-22 * scale * sum |q| |k|).
"""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lightning_indexer_top_02_b200 as L
    from lightning_indexer_top_02_b200.build import build
    build()
    L.load_library()
    return L


def no_device_error(L):
    torch.cuda.synchronize()
    assert L.csa_last_device_error(None) == L.CSA_OK


def dense(L, data, scale):
    """A cache of one page with the rows [n, 1, D] given as codes and scale bytes."""
    n = data.shape[0]
    return L.Cache("e2m1", data.view(1, 1, n, -1).contiguous(), scale.view(1, 1, n, -1).contiguous())


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("HA", [8, 16, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("log2", [25.5, 26.0, 28.0])
def test_attention_weights_far_below_the_largest(lib, HA, D, log2):
    """Every 64th key is 2^log2 times as heavy as the others, and has a value of zero: the
    output is what all the light keys together leave."""
    L, n = lib, 1 << 14
    heavy = torch.arange(n, device="cuda") % 64 == 0
    codes = torch.zeros((n, D // 2), dtype=torch.uint8, device="cuda")
    codes[heavy, 0] = 7                                  # element 0: 6
    ones = torch.full((n, D // 16), 0x38, dtype=torch.uint8, device="cuda")
    k = dense(L, codes, ones)
    codes = torch.full((n, D // 2), 0x22, dtype=torch.uint8, device="cuda")              # 1 everywhere
    codes[heavy] = 0
    v = dense(L, codes, ones)
    q = torch.zeros((1, 1, HA, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = log2 * math.log(2.0) / 6
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = L.cache_attention(q, k, v, table, lens, scale=scale, return_lse=True)
    no_device_error(L)
    nh = int(heavy.sum())
    mass = nh + (n - nh) * 2.0 ** -log2                  # in units of the largest weight
    ref = (n - nh) * 2.0 ** -log2 / mass
    e = D * 2.0 ** -22 * 6 * scale
    tol = ref * (2.0 ** -8 + 2.0 ** -11 + 2 * e) + (n - nh) * 2.0 ** -32 / mass
    assert tol < ref                                     # (an output of zeros is not within it)
    assert (out.double() - ref).abs().max() <= tol
    want = log2 * math.log(2.0) + math.log(mass)
    assert (lse.double() - want).abs().max() <= e + 2.0 ** -20 * (1 + want)


@pytest.mark.parametrize("HA", [8, 16, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("low", [2.0 ** -18, 2.0 ** -24])
def test_attention_small_query_elements(lib, HA, D, low):
    """One query element is far larger than the others and meets zeros only: the others
    decide the softmax, and none of their bits is lost."""
    L, n = lib, 700
    g = torch.Generator(device="cuda").manual_seed(D + HA)
    rows = lambda: R.stored(torch.randn((n, D), generator=g, device="cuda"), "e2m1")  # noqa: E731
    kd, ks = rows()
    kd[:, 0] &= 0xF0                                     # element 0 of every key: zero
    vd, vs = rows()
    q = torch.randn((1, 1, HA, D), generator=g, device="cuda")
    q = (q.sign() * (0.5 + q.abs().clamp(max=3.0)) * low).to(torch.bfloat16)             # low / 2 .. 3.5 low
    q[..., 0] = 1.0
    scale = D ** -0.5 / low
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = L.cache_attention(q, dense(L, kd, ks), dense(L, vd, vs), table, lens, scale=scale, return_lse=True)
    no_device_error(L)
    k, v = R.held("e2m1", kd, ks)[:, None], R.held("e2m1", vd, vs)[:, None]
    ref, rl, mean, size = R.attention(q[0, 0], k, v, torch.ones(n, dtype=torch.bool, device="cuda"), scale)
    e = D * 2.0 ** -22 * size[:, None]
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e) * mean * 1.01 + n * 2.0 ** -32 * v.abs().max()
    assert ((out[0, 0].double() - ref).abs() <= tol).all()
    assert ((lse[0, 0].double() - rl).abs() <= e[:, 0] + 2.0 ** -20 * (1 + rl.abs())).all()
