"""The cache operators where inputs and outputs pass 2^31 elements or 2^32 bytes
(needs a B200): rows at the far end are those of a small call, or of 64 bits."""
import pytest
import torch

import cache_ref as R
import test_gpu_cache as T
from test_gpu_cache import lib, no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
def test_rotary(lib, inter):
    L, N, H, D = lib, 270_000, 64, 128                   # 2.2e9 elements
    g = T.gen(1)
    x = torch.zeros((N, H, D), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((50, H, D), generator=g, device="cuda").to(torch.bfloat16)
    x[-50:] = tail
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freq, _ = L.rope_frequencies(64, device="cuda")
    got = L.rotary(x, pos, freq, rot_offset=32, interleaved=inter)
    assert torch.equal(got[-50:], L.rotary(tail, pos[-50:].clone(), freq, rot_offset=32, interleaved=inter))
    assert not got[:100].any() and not got[N // 2:N // 2 + 100].any()
    assert L.rotary(x, pos, freq, rot_offset=32, interleaved=inter, out=x) is x
    assert torch.equal(x, got)
    no_device_error(L)


def test_append_from_far_rows(lib):
    """Tokens four million elements apart."""
    L, N, step = lib, 1100, 1 << 22
    g = T.gen(2)
    buf = torch.empty(N * step, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((1, N, 2, 64), (N * step, step, 1 << 20, 1))
    rows = torch.randn((1, N, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    k.copy_(rows)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([N], dtype=torch.int32, device="cuda")
    freq, _ = L.rope_frequencies(32, device="cuda")
    for kind in ("bf16", "e2m1"):
        a, b = (L.make_cache(kind, 1, N, 2, 64, device="cuda") for _ in (0, 1))
        L.cache_append(k, a, table, lens, inv_freq=freq)
        L.cache_append(rows, b, table, lens, inv_freq=freq)
        assert torch.equal(a.data, b.data) and (a.scale is None or torch.equal(a.scale, b.scale))
    no_device_error(L)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_read(lib, kind):
    L, B, n, H, D, page = lib, 5, 120_000, 8, 512, 64     # 2.5e9 elements out
    g = T.gen(3)
    c = T.random_cache(L, kind, 3, page, H, D, g)
    table = torch.full((B, n // page), -1, dtype=torch.int32, device="cuda")
    table[-1, -1], table[-1, 0], table[0, 0] = 2, 1, 0
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out = L.cache_read(c, table, lens, n)
    near = L.cache_read(c, torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3), torch.full((1,), 3 * page, dtype=torch.int32, device="cuda"),
                        3 * page)[0]
    assert out.numel() > 2 ** 31
    assert torch.equal(out[0, :page], near[:page]) and torch.equal(out[-1, :page], near[page:2 * page])
    assert torch.equal(out[-1, -page:], near[2 * page:])
    assert not out[0, page:].any() and not out[1].any() and not out[-1, page:-page].any()
    no_device_error(L)


@pytest.mark.parametrize("HA", [8, 128])
@pytest.mark.parametrize("topk", [0, 40])
def test_attention(lib, HA, topk):
    """Queries and outputs of more than 2^31 elements; most of a dense call's queries stand before its first key."""
    L, D = lib, 256
    S = 2 ** 31 // (HA * D) + 1000
    g = T.gen(4)
    c = T.random_cache(L, "e2m1", 8, 16, 1, D, g)
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), torch.tensor([100], dtype=torch.int32, device="cuda")
    q = torch.zeros((1, S, HA, D), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((1, 100, HA, D), generator=g, device="cuda").to(torch.bfloat16)
    q[:, -100:] = tail
    idx = torch.full((1, S, topk), -1, dtype=torch.int32, device="cuda") if topk else None
    if topk:
        idx[:, -100:] = torch.randint(-5, 100, (1, 100, topk), generator=g, device="cuda", dtype=torch.int32)
    out, lse = L.cache_attention(q, c, c, table, lens, scale=0.06, idx=idx, return_lse=True)
    k = R.held("e2m1", c.data, c.scale)[:, 0].reshape(1, 128, D).transpose(0, 1)      # positions in order
    for i in range(100):
        see = torch.arange(128, device="cuda") <= i
        keys, vis = k, see
        if topk:
            pick = idx[0, S - 100 + i]
            pick = pick[pick >= 0].long()
            keys, vis = k[pick], see[pick]
        ref, rl, mean, size = R.attention(tail[0, i], keys, keys, vis, 0.06)
        e = D * 2.0 ** -22 * size[:, None]              # (the bounds of test_gpu_cache.py)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e) * mean * 1.01 + 128 * 2.0 ** -32 * k.abs().max()
        assert ((out[0, S - 100 + i].double() - ref).abs() <= tol).all(), i
        if vis.any():
            assert ((lse[0, S - 100 + i].double() - rl).abs() <= e[:, 0] + 2.0 ** -20 * (1 + rl.abs())).all(), i
        else:
            assert (lse[0, S - 100 + i] == -torch.inf).all()
    assert not out[:, :-100].any() and (lse[:, :-100] == -torch.inf).all()
    no_device_error(L)
