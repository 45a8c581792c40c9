"""How far the cache operators' arithmetic reaches: keys far below a row's
largest, query elements far below theirs, angles of far positions (needs a B200).

Bounds:
* attention: P is f16 relative to 2^7 at least, so an absolute error of 2^-25 is 2^-32 of the
  largest weight; the rest as in test_gpu_cache.py (2^-11 of P, 2^-8 of out, a logit's
  e = Dk * 2^-22 * scale * sum |q| |k|);
* rotary: half turns are rounded to fp32 (at most 2^-25 of a half turn: 9.36e-8 rad) and
  sincospi is good to one step of a value below one (5.97e-8); with pairs (1, 0) and a
  factor of one nothing else rounds: 1.54e-7;
* append: the stored value is the exactly rotated one, rounded to fp32 and to bf16.
"""
import math
from fractions import Fraction

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


# ---------------------------------------------------------------- angles

def pi_fraction(bits=256):
    """pi from Machin's formula, in integers."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(x):
        term = total = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    return Fraction(4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), one)


def exact_cos_sin(pos, freq):
    """cos and sin [N, half] of pos * freq, the angle reduced in rational arithmetic."""
    inv = 1 / (2 * pi_fraction())
    c, s = [], []
    for f in [Fraction(x) * inv for x in freq.double().tolist()]:
        col = []
        for p in pos.tolist():
            t = p * f
            col.append(2 * math.pi * float(t - round(t)))
        c.append([math.cos(a) for a in col])
        s.append([math.sin(a) for a in col])
    return torch.tensor(c, dtype=torch.float64).T.cuda(), torch.tensor(s, dtype=torch.float64).T.cuda()


def far_positions(n, seed):
    """Near both ends of int32, and between."""
    g = torch.Generator().manual_seed(seed)
    p = 2 ** 31 - 1 - torch.randint(0, 1 << 20, (n,), generator=g)
    p[::4] = -p[::4]
    p[1::8] = torch.randint(1 << 29, 1 << 31, (len(p[1::8]),), generator=g)
    return p.to(torch.int32).cuda()


def test_rotary_far_positions(lib):
    L = lib
    freq, _ = L.rope_frequencies(64, device="cuda")
    pos = far_positions(256, 1)
    x = torch.zeros((256, 1, 64), device="cuda")
    x[..., :32] = 1.0
    got = L.rotary(x, pos, freq)[:, 0].double()
    c, s = exact_cos_sin(pos, freq.cpu())
    no_device_error(L)
    assert (got[:, :32] - c).abs().max() <= 1.54e-7
    assert (got[:, 32:] - s).abs().max() <= 1.54e-7


@pytest.mark.parametrize("inter", [False, True])
def test_append_far_positions(lib, inter):
    """What a bf16 cache holds of keys rotated by far positions, bit by bit."""
    L, N, H = lib, 512, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    freq, _ = L.rope_frequencies(64, device="cuda")
    pos = far_positions(N, 3)
    k = torch.randn((1, N, H, 64), generator=g, device="cuda").to(torch.bfloat16)
    cache = L.make_cache("bf16", 1, N, H, 64, device="cuda")
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([N], dtype=torch.int32, device="cuda")
    L.cache_append(k, cache, table, lens, positions=pos.view(1, N), inv_freq=freq, interleaved=inter)
    no_device_error(L)
    c, s = (t[:, None] for t in exact_cos_sin(pos, freq.cpu()))
    x = k[0].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    u, w = a * c - b * s, b * c + a * s
    want = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    assert torch.equal(cache.data[0].transpose(0, 1), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("far", [100, 1_000_000, 2 ** 31 - 1])
def test_rotary_angles_to_the_last_bit(lib, far):
    """cos and sin to one step of sincospi (5.97e-8) and of the sum that corrects it (half a step: 2.98e-8); the
    angle's own rounding to fp32, 9.4e-8 by itself, is put back."""
    L = lib
    g = torch.Generator().manual_seed(far % 1000)
    freq, _ = L.rope_frequencies(64, device="cuda")
    pos = torch.randint(0, far, (400,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    x = torch.zeros((400, 1, 64), device="cuda")
    x[..., :32] = 1.0
    got = L.rotary(x, pos, freq)[:, 0].double()
    c, s = exact_cos_sin(pos, freq.cpu())
    no_device_error(L)
    assert max((got[:, :32] - c).abs().max(), (got[:, 32:] - s).abs().max()) <= 8.95e-8
