"""The cache operators on the GPU against plain implementations in 64 bits
(needs a B200).

Bounds, from the arithmetic that include/csa_cache.h states:
* rotary: the angle's reduced half turns are rounded to fp32 (2^-25 of a half
  turn: 9.4e-8 rad), sincospi is good to one step (2^-24 of a value up to one,
  6e-8), and the factor, two products and their sum round by 2^-24 each: at
  most 3.6e-7 * scale * (|a| + |b|), and half a step of the element type;
* append, read: what is stored is a function of the exactly rounded rotated
  element, so codes, scales and values are equal (the kernel carries the
  products in 40 bits: a differing code has a chance of about 1e-9 an element);
* attention: P is rounded to 16 bits (half a step of f16: 2^-11 relative,
  below 2^-14 2^-25 absolute) and out to bf16 (2^-8); q.k accumulates Dk
  products in fp32 (each sum off by at most 2^-22 of the largest partial sum,
  which the tensor cores' truncation allows), so a logit is off by at most
  e = Dk * 2^-22 * max_j scale * sum |q||k_j|, and a softmax weight by 2 e
  relatively.  The running maximum may lag by 2^8, so that the denominator is at least
  one and n absolute errors of 2^-25 add.
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def no_device_error(L):
    torch.cuda.synchronize()
    assert L.csa_last_device_error(None) == L.CSA_OK


# ---------------------------------------------------------------- rotary

def check_rotary(got, x, pos, freq, **how):
    ref = R.turn(x, pos, freq, **how)
    half, off, inter = freq.numel(), how.get("off", 0), how.get("inter", False)
    i = torch.arange(half, device=x.device)
    u, w = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + half + i)
    size = torch.zeros_like(ref)
    size[..., u] = size[..., w] = x.double()[..., u].abs() + x.double()[..., w].abs()
    fi = torch.finfo(x.dtype)
    tol = ref.abs() * fi.eps / 2 + fi.smallest_normal * fi.eps + 3.6e-7 * abs(how.get("scale", 1.0)) * size * (1 + fi.eps)
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (err - tol).max().item()
    rest = torch.ones(x.shape[-1], dtype=torch.bool)
    rest[u.cpu()] = rest[w.cpu()] = False
    assert torch.equal(got[..., rest.cuda()], x[..., rest.cuda()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N,H,D,rot,off", [(1, 1, 2, 2, 0), (5, 3, 10, 6, 2), (3, 2, 64, 64, 0), (37, 8, 128, 64, 0),
                                           (37, 5, 192, 64, 128), (2, 128, 128, 32, 64), (300, 1, 96, 48, 24),
                                           (4099, 2, 80, 16, 8), (1, 7, 1024, 1024, 0)])
def test_rotary(lib, dtype, inter, N, H, D, rot, off):
    g = gen(N * D + rot)
    x = torch.randn((N, H, D), generator=g, device="cuda").to(dtype)
    pos = torch.randint(-1000, 1_000_000, (N,), generator=g, device="cuda", dtype=torch.int32)
    freq, m = lib.rope_frequencies(rot, scaling="yarn", factor=4.0, original_len=4096, device="cuda")
    for inverse in (False, True):
        got = lib.rotary(x, pos, freq, rot_offset=off, interleaved=inter, scale=m, inverse=inverse)
        check_rotary(got, x, pos, freq, off=off, inter=inter, scale=m, inverse=inverse)
        same = x.clone()
        assert lib.rotary(same, pos, freq, rot_offset=off, interleaved=inter, scale=m, inverse=inverse, out=same) is same
        assert torch.equal(same, got)
    no_device_error(lib)


def test_rotary_strides(lib):
    """Heads inside a wider projection, at offsets that no 16-byte load takes, [B, S] tokens, heads outermost."""
    g = gen(3)
    freq, _ = lib.rope_frequencies(32, device="cuda")
    pos = torch.randint(0, 9000, (4, 6), generator=g, device="cuda", dtype=torch.int32)
    wide = torch.randn((4, 6, 3, 200), generator=g, device="cuda").to(torch.bfloat16)
    for lo in (0, 8, 3):
        x = wide[..., lo:lo + 64]
        out = torch.full((4, 6, 5, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        got = lib.rotary(x, pos, freq, out=out[:, :, 1:4, 4:68])
        check_rotary(got.reshape(24, 3, 64), x.reshape(24, 3, 64), pos.flatten(), freq)
        keep = torch.ones(5, 72, dtype=torch.bool)
        keep[1:4, 4:68] = False
        assert (out[:, :, keep] == 7.0).all()
    outer = wide[0, :, :, :64].transpose(0, 1).contiguous().transpose(0, 1)     # [6, 3, 64], heads outermost
    check_rotary(lib.rotary(outer, pos[0], freq), outer.contiguous(), pos[0], freq)
    with pytest.raises(ValueError):
        lib.rotary(wide[:, ::2, :, :64][:, :2], pos[:, :2].contiguous(), freq)  # unevenly spaced tokens


def test_rotary_positions(lib):
    """The ends of int32, and no tokens at all."""
    freq, _ = lib.rope_frequencies(64, device="cuda")
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123_456_789], dtype=torch.int32, device="cuda")
    x = torch.randn((6, 2, 64), generator=gen(1), device="cuda")
    check_rotary(lib.rotary(x, pos, freq), x, pos, freq)
    assert lib.rotary(x[:0], pos[:0], freq).shape == (0, 2, 64)
    no_device_error(lib)


def test_rotary_gradient(lib):
    """inverse=True is the gradient: against the transposed matrix, and against differences."""
    g = gen(5)
    freq, _ = lib.rope_frequencies(16, device="cuda")
    pos = torch.randint(0, 5000, (11,), generator=g, device="cuda", dtype=torch.int32)
    how = dict(rot_offset=4, interleaved=True, scale=1.25)
    x = torch.randn((11, 2, 24), generator=g, device="cuda")
    up = torch.randn((11, 2, 24), generator=g, device="cuda")
    grad = lib.rotary(up, pos, freq, inverse=True, **how)
    eye = torch.eye(24, device="cuda").expand(11, 24, 24).contiguous()            # rows of R^T as heads
    rows = R.turn(eye, pos, freq, off=4, inter=True, scale=1.25)
    want = torch.einsum("nij,nhj->nhi", rows, up.double())
    assert (grad.double() - want).abs().max() <= 3.6e-7 * 1.25 * 2 * up.abs().max() + 2 ** -23 * 2 * up.abs().max()
    # the map is linear: a difference of step one is exact but for fp32 (two outputs' bounds)
    d = torch.randn((11, 2, 24), generator=g, device="cuda")
    y = [lib.rotary(v, pos, freq, **how).double() for v in (x, x + d)]
    dx = (x + d).double() - x.double()
    lhs, rhs = ((y[1] - y[0]) * up.double()).sum(), (grad.double() * dx).sum()
    size = (up.double().abs() * (2 * 1.25 * (x.double().abs().max() * 2 + d.double().abs().max()))).sum()
    assert abs(lhs - rhs) <= 2 * 4.3e-7 * size
    with pytest.raises(ValueError):
        lib.rotary(x.requires_grad_(), pos, freq)


# ---------------------------------------------------------------- append and read

def pages_of(B, per, num_pages, g):
    """Distinct random pages for [B, per] places."""
    return torch.randperm(num_pages, generator=g, device="cuda")[:B * per].to(torch.int32).view(B, per)


def random_cache(L, kind, pages, page, H, D, g, tensor_scale=1.0):
    c = L.make_cache(kind, pages, page, H, D, device="cuda", tensor_scale=tensor_scale)
    if kind == "bf16":
        c.data.copy_(torch.randn(c.data.shape, generator=g, device="cuda"))
    else:
        r = torch.randn((pages, H, page, D), generator=g, device="cuda")
        data, scale = R.stored(r, kind, tensor_scale)
        c.data.copy_(data)
        c.scale.copy_(scale)
    return c


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("H,D,Dv,page,rot,off,inter", [(1, 128, 0, 40, 64, 64, True), (3, 64, 128, 16, 64, 0, False),
                                                       (2, 192, 64, 7, 48, 8, False), (8, 128, 128, 64, 0, 0, False),
                                                       (1, 512, 32, 1, 512, 0, True), (5, 96, 96, 24, 6, 2, False),
                                                       (1, 256, 256, 33, 30, 100, True)])
@pytest.mark.parametrize("ragged", [False, True])
def test_append(lib, kind, H, D, Dv, page, rot, off, inter, ragged):
    """Every row of the caches afterwards: new tokens rotated and rounded, all others as they were.  Unused
    places, positions below zero, missing pages, a table that is too short, packed rows past the last sequence."""
    L, g = lib, gen(H * D + page)
    B, S, per = 6, 9, max(1, -(-40 // page))
    new = [9, 1, 4, 9, 0, 7] if ragged else [S] * B
    lens = [40, 25, 3, 0, 12, 900]                       # 3: part of a step of 9 lies below zero; 900: past the table
    if not ragged:
        lens[4] = 11
    num_pages = B * per + 3
    table = pages_of(B, per, num_pages, g)
    if per > 1:
        table[0, per - 1] = -1                           # the last rows have no page
        table[1, 0] = num_pages                          # nor do these (out of range)
    N = sum(new)
    lead = (N + 5,) if ragged else (B, S)
    k = torch.randn(lead + (H, D), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(lead + (H, Dv), generator=g, device="cuda").to(torch.bfloat16) if Dv else None
    k[0] *= 0.0                                          # rows of zeros
    caches = [random_cache(L, kind, num_pages, page, H, d, g, 0.37 if kind == "e2m1" else 1.0) for d in (D, Dv) if d]
    want = [(c.data.clone(), None if c.scale is None else c.scale.clone()) for c in caches]
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda") if ragged else None
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    freq, m = (L.rope_frequencies(rot, scaling="yarn", factor=2.0, original_len=64, device="cuda")) if rot else (None, 1.0)
    override = torch.randint(0, 70000, lead, generator=g, device="cuda", dtype=torch.int32) if page == 24 else None
    L.cache_append(k, caches[0], table, kv_len, v=v, cache_v=caches[1] if Dv else None, cu_tokens=cu, positions=override,
                   inv_freq=freq, rot_offset=off, interleaved=inter, rope_scale=m)
    no_device_error(L)
    cpu_table, n = table.cpu(), 0
    for b in range(B):
        for j in range(new[b]):
            pos = lens[b] - new[b] + j
            at = R.place(cpu_table, b, pos, page, num_pages) if lens[b] > 0 else None
            if at is not None:
                for x, c, w in zip((k, v), caches, want):
                    r = x.reshape(-1, H, x.shape[-1])[n:n + 1]
                    if rot and x is k:
                        p = override.flatten()[n:n + 1] if override is not None else torch.tensor([pos], device="cuda")
                        r = R.turn(r, p, freq, off=off, inter=inter, scale=m)
                    data, scale = R.stored(r[0].float(), kind, c.tensor_scale)
                    w[0][at[0], :, at[1]] = data
                    if scale is not None:
                        w[1][at[0], :, at[1]] = scale
            n += 1
    for c, w in zip(caches, want):
        # as values: a code of -0 is a zero too
        assert torch.equal(R.held(kind, c.data, c.scale), R.held(kind, *w))
        assert c.scale is None or torch.equal(c.scale, w[1])


def test_append_extremes(lib):
    """4-bit rounding at its borders: ties, saturation, scales that vanish or reach the largest."""
    L = lib
    x = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.5])
    rows = torch.stack([x, x * 448, x * 2.0 ** 20, x * 2.0 ** -9, x * 2.0 ** -12, x * 2.0 ** -30, x * 0, -x])
    rows = rows.repeat(1, 2).view(8, 1, 1, 32).to(torch.bfloat16).cuda()
    for ts in (1.0, 2.0 ** -6, 0.01):
        c = L.make_cache("e2m1", 8, 1, 1, 32, device="cuda", tensor_scale=ts)
        table = torch.arange(8, dtype=torch.int32, device="cuda").view(8, 1)
        L.cache_append(rows, c, table, torch.ones(8, dtype=torch.int32, device="cuda"))
        data, scale = R.stored(rows.float()[:, 0], "e2m1", ts)
        assert torch.equal(c.scale[:, :, 0], scale)
        assert torch.equal(R.held("e2m1", c.data, c.scale)[:, :, 0], R.held("e2m1", data, scale))
    no_device_error(L)


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
def test_append_vanishing_rows(lib, kind):
    """Rows whose scale is too small for its type are rows of zeros, not of 0 / 0."""
    L = lib
    c = L.make_cache(kind, 2, 4, 1, 64, device="cuda")
    table = torch.arange(2, dtype=torch.int32, device="cuda").view(2, 1)
    k = torch.full((2, 4, 1, 64), 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    k[:, :, :, 1::2] = 0
    pos = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    # rotated: 2^-145, and 2^-145 / 448 is 0 in fp32
    L.cache_append(k, c, table, torch.full((2,), 4, dtype=torch.int32, device="cuda"), inv_freq=torch.ones(32, device="cuda"),
                   positions=pos, rope_scale=2.0 ** -45)
    no_device_error(L)
    assert (R.held(kind, c.data, c.scale) == 0).all()
    assert (c.scale == (1.0 if kind == "e4m3" else 0)).all()
    assert (L.cache_read(c, table, torch.full((2,), 4, dtype=torch.int32, device="cuda"), 4) == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("B,T,H,D,page", [(1, 1, 1, 64, 1), (3, 100, 2, 128, 16), (4, 77, 3, 192, 24), (2, 50, 1, 512, 7), (3, 65, 8, 32, 64)])
def test_read(lib, kind, B, T, H, D, page):
    L, g = lib, gen(T * D)
    per = -(-T // page)
    num_pages = B * per + 2
    table = pages_of(B, per, num_pages, g)
    if per > 2:
        table[0, 1] = -1
        table[B - 1, 0] = num_pages + 7
    lens = torch.tensor([T, T // 2, 0, 5000][:B], dtype=torch.int32, device="cuda")
    c = random_cache(L, kind, num_pages, page, H, D, g, 2.0 ** -3)
    got = L.cache_read(c, table, lens, T)
    no_device_error(L)
    values = R.held(kind, c.data, c.scale, c.tensor_scale if kind == "e2m1" else 1.0)
    want = torch.zeros((B, T, H, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        for t in range(min(T, int(lens[b]))):
            at = R.place(table.cpu(), b, t, page, num_pages)
            if at is not None:
                want[b, t] = values[at[0], :, at[1]]
    # E4M3: the product with the fp32 scale is rounded to fp32 first
    assert torch.equal(got, (want.float() if kind == "e4m3" else want).to(torch.bfloat16))
    assert L.cache_read(c, table, lens, 0).shape == (B, 0, H, D)


# ---------------------------------------------------------------- attention

def check_attention(L, *, B, S, HA, H, Dk, Dv, page, lens, topk=0, causal=True, seed=0, scale=None, holes=False, ts=(1.0, 1.0),
                    q_size=1.0, idx=None, rows=None):
    g = gen(seed)
    per = -(-max(max(lens), 1) // page)
    num_pages = B * per + 2
    table = pages_of(B, per, num_pages, g)
    kc = random_cache(L, "e2m1", num_pages, page, H, Dk, g, ts[0])
    vc = random_cache(L, "e2m1", num_pages, page, H, Dv, g, ts[1])
    # whatever lies outside the sequences' rows is not used: bytes of all ones (scales: NaN)
    used = torch.zeros((num_pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(per):
            used[int(table[b, p]), :max(0, min(page, n - p * page))] = True
    if holes and per > 1:
        for b in range(B):
            hole = int(table[b, b % (per - 1)])
            used[hole] = False
            table[b, b % (per - 1)] = [-1, num_pages, -2 ** 31][b % 3]
    bad = ~used[:, None, :, None].cuda()
    for c in (kc, vc):
        c.data.masked_fill_(bad, 255)
        c.scale.masked_fill_(bad, 255)
    q = (torch.randn((B, S, HA, Dk), generator=g, device="cuda") * q_size).to(torch.bfloat16)
    if topk and idx is None:
        idx = torch.randint(-3, max(lens) + 5, (B, S, topk), generator=g, device="cuda", dtype=torch.int32)
    scale = Dk ** -0.5 if scale is None else scale
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = L.cache_attention(q, kc, vc, table, kv_len, scale=scale, idx=idx, causal=causal, return_lse=True)
    no_device_error(L)
    assert torch.equal(L.cache_attention(q, kc, vc, table, kv_len, scale=scale, idx=idx, causal=causal), out)
    kh, vh = R.held("e2m1", kc.data, kc.scale, ts[0]), R.held("e2m1", vc.data, vc.scale, ts[1])
    cpu = table.cpu()
    for b in range(B):
        at = [R.place(cpu, b, t, page, num_pages) for t in range(max(lens[b], 0))]
        have = torch.tensor([a is not None for a in at], dtype=torch.bool, device="cuda")
        pg = torch.tensor([a[0] if a else 0 for a in at], dtype=torch.long, device="cuda")
        of = torch.tensor([a[1] if a else 0 for a in at], dtype=torch.long, device="cuda")
        k = kh[pg, :, of].nan_to_num(0.0) if at else kh[:0, :, 0]
        v = vh[pg, :, of].nan_to_num(0.0) if at else vh[:0, :, 0]
        for i in range(S) if rows is None else rows:
            see = lens[b] - S + i + 1 if causal else lens[b]
            vis = have & (torch.arange(len(at), device="cuda") < see)
            ki, vi = k, v
            if idx is not None and at:
                pick = idx[b, i][(idx[b, i] >= 0) & (idx[b, i] < len(at))].long()   # a key twice counts twice
                ki, vi, vis = k[pick], v[pick], vis[pick]
            ref, rl, mean, size = R.attention(q[b, i], ki, vi, vis, scale)
            e = Dk * 2.0 ** -22 * size[:, None]
            n = int(vis.sum())
            vmax = vi[vis].abs().max() if n else 0.0
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e) * mean * 1.01 + n * 2.0 ** -25 * vmax
            err = (out[b, i].double() - ref).abs()
            assert (err <= tol).all(), (b, i, (err / tol).max().item())
            if n:
                assert ((lse[b, i].double() - rl).abs() <= e[:, 0] + 2.0 ** -20 * (1 + rl.abs())).all()
            else:
                assert (out[b, i] == 0).all() and (lse[b, i] == -math.inf).all()
    return out


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128), (128, 64), (256, 256), (64, 192), (192, 192), (128, 256), (256, 64)])
@pytest.mark.parametrize("HA,H,S", [(8, 1, 1), (3, 3, 1), (10, 2, 2), (20, 1, 1)])
def test_attention(lib, Dk, Dv, HA, H, S):
    check_attention(lib, B=3, S=S, HA=HA, H=H, Dk=Dk, Dv=Dv, page=16, lens=[150, 33, 1], seed=Dk + Dv + HA)


@pytest.mark.parametrize("lens", [[0], [1], [31], [32], [33], [127], [128], [129], [1000], [0, 5, 0, 257]])
@pytest.mark.parametrize("page", [1, 16, 24, 64, 1024])
def test_attention_lengths(lib, lens, page):
    """Lengths around the tiles, pages that end inside one, unused places."""
    check_attention(lib, B=len(lens), S=1, HA=16, H=2, Dk=128, Dv=128, page=page, lens=lens, seed=page + lens[0])


@pytest.mark.parametrize("HA,H", [(1, 1), (7, 1), (9, 1), (16, 1), (17, 1), (40, 1), (64, 1), (65, 1), (128, 1), (96, 2), (256, 2)])
@pytest.mark.parametrize("S", [1, 3])
def test_attention_heads(lib, HA, H, S):
    check_attention(lib, B=2, S=S, HA=HA, H=H, Dk=128, Dv=128, page=16, lens=[300, 70], seed=HA)


@pytest.mark.parametrize("S", [2, 5, 40, 130])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_several_queries(lib, S, causal):
    """Causal rows within a tile, queries before the sequence's first position (they see nothing)."""
    check_attention(lib, B=3, S=S, HA=12, H=2, Dk=64, Dv=64, page=24, lens=[200, S // 2, 0], causal=causal, seed=S)


@pytest.mark.parametrize("HA,H", [(8, 1), (16, 1), (64, 1), (128, 1), (40, 2)])
@pytest.mark.parametrize("topk", [1, 33, 300])
def test_attention_selected(lib, HA, H, topk):
    """Lists with padding anywhere, entries past the sequence or after the query, keys listed twice."""
    check_attention(lib, B=3, S=2, HA=HA, H=H, Dk=128, Dv=128, page=24, lens=[400, 60, 0], topk=topk, seed=topk + HA)


def test_attention_selected_rows_without_keys(lib):
    idx = torch.full((1, 4, 200), -1, dtype=torch.int32, device="cuda")
    idx[0, 1, 199] = 7
    idx[0, 2, 100:130] = torch.arange(30, dtype=torch.int32, device="cuda")
    idx[0, 3, ::7] = 2 ** 31 - 1
    out = check_attention(lib, B=1, S=4, HA=64, H=1, Dk=128, Dv=128, page=16, lens=[64], topk=200, idx=idx)
    assert (out[0, 0] == 0).all() and (out[0, 3] == 0).all() and (out[0, 1] != 0).any()


@pytest.mark.parametrize("HA", [8, 16, 64])
def test_attention_missing_pages(lib, HA):
    check_attention(lib, B=4, S=2, HA=HA, H=1, Dk=128, Dv=128, page=16, lens=[100, 17, 64, 33], holes=True, seed=4)


@pytest.mark.parametrize("HA", [8, 16, 96])
@pytest.mark.parametrize("scale,q_size", [(2.0, 1.0), (-0.09, 1.0), (0.0, 1.0), (1e-4, 2.0 ** 90), (0.09, 2.0 ** -100), (0.09, 0.0)])
def test_attention_scales(lib, HA, scale, q_size):
    """Sharp, flipped and flat softmaxes; queries at the ends of bf16's range; scales of the whole tensors."""
    if q_size > 1.0:
        scale = scale * 2.0 ** -90 * 100
    check_attention(lib, B=2, S=1, HA=HA, H=1, Dk=128, Dv=128, page=64, lens=[700, 90], scale=scale, q_size=q_size,
                    ts=(0.5, 3.0), seed=6)


def test_attention_long(lib):
    """A long sequence beside short ones: many shares of the keys."""
    check_attention(lib, B=3, S=1, HA=8, H=1, Dk=128, Dv=128, page=64, lens=[70000, 3, 1000], seed=8)
    check_attention(lib, B=2, S=1, HA=128, H=1, Dk=128, Dv=128, page=64, lens=[20000, 130], seed=9)


def test_attention_far_offsets(lib):
    """Rows that lie more than 2^32 bytes into the allocation."""
    L, g = lib, gen(1)
    page, H, D, pages = 1024, 8, 256, 4400               # 1 MB of codes a page
    data = torch.empty((pages, H, page, D // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, H, page, D // 16), dtype=torch.uint8, device="cuda")
    assert data.numel() > 2 ** 32
    small = random_cache(L, "e2m1", 2, page, H, D, g)
    data[[0, pages - 1]], scale[[0, pages - 1]] = small.data, small.scale
    far = L.Cache("e2m1", data, scale)
    lens = torch.tensor([1500], dtype=torch.int32, device="cuda")
    near_t = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    far_t = torch.tensor([[0, pages - 1]], dtype=torch.int32, device="cuda")
    for HA in (H, 16 * H):
        q = torch.randn((1, 1, HA, D), generator=g, device="cuda").to(torch.bfloat16)
        assert torch.equal(L.cache_attention(q, far, far, far_t, lens, scale=0.06),
                           L.cache_attention(q, small, small, near_t, lens, scale=0.06))
    assert torch.equal(L.cache_read(far, far_t, lens, 1500), L.cache_read(small, near_t, lens, 1500))
    k = torch.randn((1, 3, H, D), generator=g, device="cuda").to(torch.bfloat16)
    L.cache_append(k, far, far_t, lens)
    L.cache_append(k, small, near_t, lens)
    assert torch.equal(data[pages - 1], small.data[1]) and torch.equal(scale[pages - 1], small.scale[1])
    no_device_error(L)


def test_strided_pages(lib):
    """Keys and values of one layer inside an allocation that interleaves them page by page."""
    L, g = lib, gen(2)
    pages, H, page, D = 9, 2, 16, 128
    both = torch.full((pages, 2, H, page, D // 2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, 2, H, page, D // 16), 255, dtype=torch.uint8, device="cuda")
    kc, vc = (L.Cache("e2m1", both[:, i], scales[:, i]) for i in (0, 1))
    dense = [L.make_cache("e2m1", pages, page, H, D, device="cuda") for _ in (0, 1)]
    table = pages_of(2, 4, pages, g)
    lens = torch.tensor([60, 20], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 60, 80], dtype=torch.int32, device="cuda")
    kv = torch.randn((80, 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)   # k and v of one projection
    k, v = kv[:, :H], kv[:, H:]
    freq, _ = L.rope_frequencies(64, device="cuda")
    q = torch.randn((2, 1, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    outs = []
    for a, b in ((kc, vc), dense):
        L.cache_append(k, a, table, lens, v=v, cache_v=b, cu_tokens=cu, inv_freq=freq)
        outs.append((L.cache_attention(q, a, b, table, lens, scale=0.09), L.cache_read(a, table, lens, 60),
                     L.cache_read(b, table, lens, 60)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    no_device_error(L)


def test_workspace(lib):
    L, g = lib, gen(3)
    c = random_cache(L, "e2m1", 64, 64, 1, 128, g)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 1, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    want = L.cache_attention(q, c, c, table, lens, scale=0.09)
    with pytest.raises(L.CsaError) as e:
        L.cache_attention(q, c, c, table, lens, scale=0.09, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == L.CSA_ERR_WORKSPACE
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")          # its contents do not matter
    for _ in range(2):
        assert torch.equal(L.cache_attention(q, c, c, table, lens, scale=0.09, workspace=ws), want)
    a = L.cache.CsaCacheAttnArgs()                                              # and without one: stream-ordered
    a.cache_k = a.cache_v = L.cache._cache_struct("c", c)
    out = torch.empty((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    a.q, a.out, a.kv_len, a.page_table = q.data_ptr(), out.data_ptr(), lens.data_ptr(), table.data_ptr()
    a.max_pages = a.table_stride = 64
    a.B, a.S, a.HA, a.causal, a.scale = 1, 1, 8, 1, 0.09
    assert L.csa_cache_attention(a, None, 0, None) == L.CSA_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_attention_empty_selection(lib):
    """An empty list is not "every position"."""
    L, g = lib, gen(4)
    c = random_cache(L, "e2m1", 4, 16, 1, 128, g)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    q = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        L.cache_attention(q, c, c, table, lens, scale=1.0, idx=torch.zeros((1, 1, 0), dtype=torch.int32, device="cuda"))
    with pytest.raises(L.CsaError):                        # in place: q is read while out is written
        L.cache_attention(q, c, c, table, lens, scale=1.0, out=q)
    none = L.cache_attention(q[:0], c, c, table[:0], lens[:0], scale=1.0, return_lse=True)
    assert none[0].shape == (0, 1, 8, 128) and none[1].shape == (0, 1, 8)


@pytest.mark.parametrize("HA,page", [(64, 64), (128, 24)])
def test_attention_wait_limit(lib, HA, page):
    """A wait that runs out ends the call with an error status, and the next call is right.  (Up to 16 rows a
    copy from L2 has often landed before it is first waited for.)"""
    L, g = lib, gen(HA)
    c = random_cache(L, "e2m1", 200, page, 1, 128, g)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(1, 200)
    q = torch.randn((1, 1, HA, 128), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
    want = L.cache_attention(q, c, c, table, lens, scale=0.09)
    no_device_error(L)
    L.csa_set_wait_limit(1)
    try:
        L.cache_attention(q, c, c, table, lens, scale=0.09)
        assert L.csa_last_device_error(None) == L.CSA_ERR_TIMEOUT
    finally:
        L.csa_set_wait_limit(0)
    assert torch.equal(L.cache_attention(q, c, c, table, lens, scale=0.09), want)
    no_device_error(L)


def test_attention_ragged_batches(lib):
    """Many sequences of very different lengths: shares that begin and end anywhere, whole tiles, unused places."""
    lens = [0, 1, 3000, 17, 0, 255, 256, 257, 1024, 5, 0, 0, 700] * 12        # more sequences than threads in a block
    for HA, H, S in ((8, 2, 1), (16, 1, 1), (4, 4, 3)):
        check_attention(lib, B=len(lens), S=S, HA=HA, H=H, Dk=64, Dv=64, page=32, lens=lens, seed=HA + S)


def test_calls_at_once(lib):
    """Two streams at a time, each with what it allocates itself."""
    L = lib
    states = [step_state(L, T=200), step_state(L, T=200)]
    want = [L.cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=0.09) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [[], []]
    for _ in range(20):
        for i, (s, st) in enumerate(zip(states, streams)):
            got[i].append(L.cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=0.09, stream=st))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x in g:
            assert torch.equal(x, w)
    no_device_error(L)


# ---------------------------------------------------------------- together

def decode_step(L, s, stream=None):
    """One decode step as a model runs it: rotate, append to the indexer's and the attention's caches, select, attend."""
    q = L.rotary(s["q"], s["pos"], s["freq"], rot_offset=64, stream=stream)
    iq = L.rotary(s["iq"], s["pos"], s["freq"], interleaved=True, stream=stream)
    L.cache_append(s["ik"], s["index"], s["index_table"], s["lens"], inv_freq=s["freq"], interleaved=True, stream=stream)
    L.cache_append(s["k"], s["kc"], s["table"], s["lens"], v=s["v"], cache_v=s["vc"], inv_freq=s["freq"], rot_offset=64,
                   stream=stream)
    B, _, T, d = s["index"].data.shape
    idx, _ = L.indexer_topk(iq, s["w"], s["index"].data.view(B, T, d), k_scale=s["index"].scale.view(B, T), m=1, topk=64,
                            q_offset=s["T"] - 1, stream=stream)
    return L.cache_attention(q, s["kc"], s["vc"], s["table"], s["lens"], scale=0.09, idx=idx, stream=stream), idx, q


def step_state(L, T=200, B=2):
    g = gen(12)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    s = dict(T=T, q=rnd(B, 1, 64, 128), iq=rnd(B, 1, 16, 128), ik=rnd(B, 1, 1, 128), k=rnd(B, 1, 1, 128), v=rnd(B, 1, 1, 128),
             w=torch.randn((B, 1, 16), generator=g, device="cuda"), pos=torch.full((B, 1), T - 1, dtype=torch.int32, device="cuda"),
             lens=torch.full((B,), T, dtype=torch.int32, device="cuda"), freq=L.rope_frequencies(64, device="cuda")[0])
    s["index"] = random_cache(L, "e4m3", B, T, 1, 128, g)          # one page a sequence: the indexer's [B, T, d]
    s["index_table"] = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    per = -(-T // 16)
    s["table"] = pages_of(B, per, B * per, g)
    s["kc"], s["vc"] = (random_cache(L, "e2m1", B * per, 16, 1, 128, g) for _ in (0, 1))
    return s


def test_decode_step(lib):
    """The operators in a row, against the library's own bf16 path over the rows read back."""
    L = lib
    s = step_state(L)
    out, idx, q = decode_step(L, s)
    no_device_error(L)
    assert (idx >= 0).all()                                        # 200 visible keys, 64 taken
    k, v = (L.cache_read(s[c], s["table"], s["lens"], s["T"])[:, :, 0] for c in ("kc", "vc"))
    # exact in bf16 (six significant bits), so only P's rounding differs: bf16 there, 2^-8 of the mean |v|
    ref = L.sparse_attention(q, k.contiguous(), idx, scale=0.09, v=v.contiguous())
    bound = 2 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * v.float().abs().max()
    assert ((out.float() - ref).abs() <= bound).all()
    # the appended key reads back as the rotated one, rounded to 4 bits
    want = R.turn(s["k"][:, 0], s["pos"][:, 0], s["freq"], off=64).float()
    assert torch.equal(k[:, -1].double(), R.held("e2m1", *R.stored(want[:, 0], "e2m1")))


def test_streams_and_graph(lib):
    """On a side stream, and captured into a graph that is replayed on new inputs and lengths."""
    L = lib
    s = step_state(L)
    want = decode_step(L, s)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = decode_step(L, s, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        decode_step(L, s)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = L.cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=0.09)
        L.cache_append(s["k"], s["kc"], s["table"], s["lens"], inv_freq=s["freq"])
        back = L.cache_read(s["kc"], s["table"], s["lens"], s["T"])
    for n in (200, 1, 77, 0):
        s["lens"].fill_(n)
        s["q"].normal_(generator=gen(n))
        want = L.cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=0.09)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
        assert torch.equal(back, L.cache_read(s["kc"], s["table"], s["lens"], s["T"]))
    no_device_error(L)


def test_launch_events(lib):
    """The measurement hook counts this module's launches too."""
    L = lib
    s = step_state(L)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    assert L.csa_set_launch_events(ev) == L.CSA_OK
    try:
        L.cache_read(s["kc"], s["table"], s["lens"], s["T"])
    finally:
        L.csa_set_launch_events(None)
    torch.cuda.synchronize()
    assert ev[0].elapsed_time(ev[1]) > 0
