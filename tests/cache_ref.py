"""Plain implementations, in 64 bits, of the cache operators
(include/csa_cache.h), for the tests.  Torch on any device; no library code."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def turn(x, pos, freq, *, off=0, inter=False, scale=1.0, inverse=False):
    """x [N, H, D] rotated by pos [N], in 64 bits."""
    x = x.double().clone()
    a = pos.double()[:, None, None] * freq.double()
    c, s = torch.cos(a) * scale, torch.sin(a) * (-scale if inverse else scale)
    half = freq.numel()
    i = torch.arange(half, device=x.device)
    u, w = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + half + i)
    p, q = x[..., u], x[..., w]
    x[..., u], x[..., w] = p * c - q * s, q * c + p * s
    return x


def stored(r, kind, tensor_scale=1.0):
    """fp32 rows [..., D] as a cache stores them: (data, scale)."""
    if kind == "bf16":
        return r.to(torch.bfloat16), None
    if kind == "e4m3":
        peak = r.abs().amax(-1).double()
        s = torch.where(peak > 0, (peak / 448).float(), 1.0)
        return (r.double() / s.double()[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8), s
    y = r.unflatten(-1, (-1, 16)).double()
    ts = torch.tensor(tensor_scale, dtype=torch.float32)
    six = (6 * ts).double().item()
    s8 = (y.abs().amax(-1) / six).float().clamp(max=448).to(torch.float8_e4m3fn)
    s = (s8.float() * ts.to(r.device)).double()[..., None]
    z = torch.where(s > 0, y / torch.where(s > 0, s, 1.0), 0.0).float().double()
    # nearest magnitude, a tie to the even code
    d = (z.abs()[..., None] - E2M1.to(r.device)).abs()
    tie = torch.arange(8, device=r.device) % 2 * 1e-12
    code = (d + tie).argmin(-1) + 8 * (z < 0)
    code = code.flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), s8.view(torch.uint8)


def held(kind, data, scale, tensor_scale=1.0):
    """The values that stored rows stand for, in 64 bits."""
    if kind == "bf16":
        return data.double()
    if kind == "e4m3":
        return data.view(torch.float8_e4m3fn).double() * scale.double()[..., None]
    codes = torch.stack((data & 15, data >> 4), -1).flatten(-2).long()
    v = torch.cat((E2M1, -E2M1)).to(data.device)[codes]
    ts = torch.tensor(tensor_scale, dtype=torch.float32).double().item()
    return v * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * ts


def place(table, b, pos, page_size, num_pages):
    """(page, row) of one position, or None."""
    n = pos // page_size
    if pos < 0 or n >= table.shape[1]:
        return None
    p = int(table[b, n])
    return (p, pos % page_size) if 0 <= p < num_pages else None


def attention(q, k, v, visible, scale):
    """One query row's heads: q [HA, Dk], k [n, H, Dk], v [n, H, Dv] (64 bits),
    visible [n] bool.  Returns out [HA, Dv], lse [HA], the mean of |v| under the
    softmax, and the largest scale * sum |q| |k|."""
    HA, H = q.shape[0], k.shape[1]
    k, v = k[visible], v[visible]
    if k.shape[0] == 0:
        z = torch.zeros((HA, v.shape[-1]), dtype=torch.float64, device=q.device)
        return z, torch.full((HA,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[:, 0])
    kk = k.repeat_interleave(HA // H, 1)
    vv = v.repeat_interleave(HA // H, 1)
    t = torch.einsum("hd,nhd->hn", q.double(), kk) * scale
    p = torch.softmax(t, -1)
    size = abs(scale) * torch.einsum("hd,nhd->hn", q.double().abs(), kk.abs()).amax(-1)
    return torch.einsum("hn,nhd->hd", p, vv), torch.logsumexp(t, -1), torch.einsum("hn,nhd->hd", p, vv.abs()), size
