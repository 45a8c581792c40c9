"""The cache operators on torch tensors: rotary positions, appending to a paged
cache, reading it back as bf16 rows, and attention over a cache held in 4 bits.

The same calls as ``include/csa_cache.h`` (operation, layouts and limits are
stated there), marshalled with ctypes; outputs and workspaces are allocated on
the tensors' device if not given.  Nothing here records a gradient: a tensor
that would need one, or that carries a forward-mode tangent, is refused
(``rotary(..., inverse=True)`` is the gradient of ``rotary``).
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import lightning_indexer_top_02_b200 as L

CSA_CACHE_BF16, CSA_CACHE_E4M3, CSA_CACHE_E2M1 = 0, 1, 2
CACHE_DTYPES = {"bf16": CSA_CACHE_BF16, "e4m3": CSA_CACHE_E4M3, "e2m1": CSA_CACHE_E2M1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}

_P, _I, _LL, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class CsaCache(ctypes.Structure):
    _fields_ = [("data", _P), ("scale", _P), ("dtype", _I), ("H", _I), ("D", _I), ("num_pages", _I),
                ("page_size", _I), ("page_stride", _LL), ("scale_page_stride", _LL), ("tensor_scale", _F)]


class CsaRotaryArgs(ctypes.Structure):
    _fields_ = [("x", _P), ("out", _P), ("dtype", _I), ("N", _I), ("H", _I), ("D", _I),
                ("x_token_stride", _LL), ("x_head_stride", _LL), ("out_token_stride", _LL),
                ("out_head_stride", _LL), ("positions", _P), ("inv_freq", _P), ("rot_dim", _I),
                ("rot_offset", _I), ("interleaved", _I), ("inverse", _I), ("scale", _F)]


class CsaAppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_token_stride", _LL), ("k_head_stride", _LL),
                ("v_token_stride", _LL), ("v_head_stride", _LL), ("N", _I), ("B", _I), ("S", _I),
                ("cu_tokens", _P), ("kv_len", _P), ("page_table", _P), ("max_pages", _I),
                ("table_stride", _LL), ("cache_k", CsaCache), ("cache_v", CsaCache), ("inv_freq", _P),
                ("positions", _P), ("rot_dim", _I), ("rot_offset", _I), ("interleaved", _I),
                ("rope_scale", _F)]


class CsaCacheReadArgs(ctypes.Structure):
    _fields_ = [("cache", CsaCache), ("kv_len", _P), ("page_table", _P), ("max_pages", _I),
                ("table_stride", _LL), ("B", _I), ("T", _I), ("out", _P)]


class CsaCacheAttnArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("cache_k", CsaCache), ("cache_v", CsaCache), ("kv_len", _P),
                ("page_table", _P), ("max_pages", _I), ("table_stride", _LL), ("idx", _P), ("topk", _I),
                ("B", _I), ("S", _I), ("HA", _I), ("causal", _I), ("scale", _F), ("out", _P), ("lse", _P)]


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    lib.csa_rope_frequencies.argtypes = [_I, ctypes.c_double, _I, ctypes.c_double, _I, ctypes.c_double,
                                         ctypes.c_double, _P, _P]
    lib.csa_rotary.argtypes = [ctypes.POINTER(CsaRotaryArgs), _P]
    lib.csa_cache_append.argtypes = [ctypes.POINTER(CsaAppendArgs), _P]
    lib.csa_cache_read.argtypes = [ctypes.POINTER(CsaCacheReadArgs), _P]
    lib.csa_cache_attention.argtypes = [ctypes.POINTER(CsaCacheAttnArgs), _P, ctypes.c_size_t, _P]
    lib.csa_cache_attention_workspace_size.argtypes = [ctypes.POINTER(CsaCacheAttnArgs)]
    for fn in (lib.csa_rope_frequencies, lib.csa_rotary, lib.csa_cache_append, lib.csa_cache_read,
               lib.csa_cache_attention):
        fn.restype = _I
    lib.csa_cache_attention_workspace_size.restype = ctypes.c_size_t


# ----------------------------------------------------------------- raw C-ABI mirrors

def csa_rope_frequencies(rot_dim, base, scaling, factor, original_len, beta_fast, beta_slow, inv_freq_ptr,
                         scale_ptr) -> int:
    return L.load_library().csa_rope_frequencies(rot_dim, base, scaling, factor, original_len, beta_fast,
                                                 beta_slow, inv_freq_ptr, scale_ptr)


def csa_rotary(args: CsaRotaryArgs, stream_ptr) -> int:
    return L.load_library().csa_rotary(ctypes.byref(args), stream_ptr)


def csa_cache_append(args: CsaAppendArgs, stream_ptr) -> int:
    return L.load_library().csa_cache_append(ctypes.byref(args), stream_ptr)


def csa_cache_read(args: CsaCacheReadArgs, stream_ptr) -> int:
    return L.load_library().csa_cache_read(ctypes.byref(args), stream_ptr)


def csa_cache_attention(args: CsaCacheAttnArgs, workspace_ptr, workspace_bytes: int, stream_ptr) -> int:
    return L.load_library().csa_cache_attention(ctypes.byref(args), workspace_ptr, workspace_bytes, stream_ptr)


def csa_cache_attention_workspace_size(args: CsaCacheAttnArgs) -> int:
    return L.load_library().csa_cache_attention_workspace_size(ctypes.byref(args))


# ----------------------------------------------------------------- torch convenience

@dataclass
class Cache:
    """One paged cache: ``dtype`` "bf16", "e4m3" or "e2m1"; ``data`` [pages, H,
    page_size, row bytes or bf16 values] and ``scale`` (None; fp32 [pages, H,
    page_size]; E4M3 bytes [pages, H, page_size, D / 16]).  Pages may be
    strided (a slice of a wider allocation); what lies within a page is dense.
    ``make_cache`` allocates one."""
    dtype: str
    data: object
    scale: object = None
    tensor_scale: float = 1.0

    @property
    def D(self) -> int:
        return self.data.shape[3] * (2 if self.dtype == "e2m1" else 1)


def make_cache(dtype: str, num_pages: int, page_size: int, H: int, D: int, *, device, tensor_scale: float = 1.0):
    """A cache of zeros (scales of one for "e4m3", so that a row never written reads as zeros)."""
    import torch

    shape = (num_pages, H, page_size)
    if dtype == "bf16":
        return Cache(dtype, torch.zeros(shape + (D,), dtype=torch.bfloat16, device=device))
    if dtype == "e4m3":
        return Cache(dtype, torch.zeros(shape + (D,), dtype=torch.uint8, device=device),
                     torch.ones(shape, dtype=torch.float32, device=device))
    if dtype != "e2m1":
        raise ValueError(f"unknown cache type {dtype!r}")
    return Cache(dtype, torch.zeros(shape + (D // 2,), dtype=torch.uint8, device=device),
                 torch.zeros(shape + (D // 16,), dtype=torch.uint8, device=device), tensor_scale)


def _page_stride(t):
    """Bytes from page to page of a tensor that is dense within a page (0: dense altogether)."""
    if t.is_contiguous():
        return 0
    n = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != n:
            raise ValueError("a cache must be dense within a page")
        n *= size
    if t.shape[0] == 1:
        return n * t.element_size()
    if t.stride(0) < n:                     # (0 would be taken for dense)
        raise ValueError("the pages of a cache must not overlap")
    return t.stride(0) * t.element_size()


def _cache_struct(name: str, c: Cache) -> CsaCache:
    import torch

    kind = CACHE_DTYPES.get(c.dtype)
    if kind is None:
        raise ValueError(f"unknown cache type {c.dtype!r}")
    data, scale = c.data, c.scale
    dtype = data.dtype
    if dtype != (torch.bfloat16 if kind == CSA_CACHE_BF16 else torch.uint8) and \
            not (kind == CSA_CACHE_E4M3 and dtype == torch.float8_e4m3fn) or data.dim() != 4:
        raise TypeError(f"{name}.data must be a 4-dimensional {'bfloat16' if kind == 0 else 'uint8'} tensor")
    pages, H, page, D = data.shape
    if data.numel() > _INT_MAX // 2:
        _ints(**{f"{name}'s pages": pages, "H": H, "page_size": page, "D": 2 * D})
    if kind == CSA_CACHE_BF16:
        return CsaCache(data.data_ptr(), None, kind, H, D, pages, page, _page_stride(data), 0, c.tensor_scale)
    want = (pages, H, page)
    if kind == CSA_CACHE_E2M1:
        D *= 2
        want = (pages, H, page, D // 16)
    if scale is None or scale.shape != want or \
            scale.dtype != (torch.float32 if kind == CSA_CACHE_E4M3 else torch.uint8) and \
            not (kind == CSA_CACHE_E2M1 and scale.dtype == torch.float8_e4m3fn):
        raise TypeError(f"{name}.scale must be {'float32' if kind == CSA_CACHE_E4M3 else 'uint8'} {want}")
    return CsaCache(data.data_ptr(), scale.data_ptr(), kind, H, D, pages, page, _page_stride(data), _page_stride(scale),
                    c.tensor_scale)


_autograd = _increment_version = None       # torch.autograd's, from the first call on


def _load_autograd():
    global _autograd, _increment_version
    from torch.autograd import forward_ad, graph

    _increment_version = graph.increment_version    # before _autograd, which other threads look at
    _autograd = forward_ad
    return forward_ad


def _on(dev, names, *tensors):
    """Every tensor on one CUDA device, and none that would need a gradient or carries a
    tangent.  (Checked in one go, names looked up only for an error: this is on every
    call's path.)"""
    forward_ad = _autograd or _load_autograd()
    for t in tensors:
        if t is not None and (t.get_device() != dev or t.requires_grad):
            break
    else:
        if dev >= 0 and forward_ad._current_level < 0:
            return
    import torch

    for name, t in zip(names.split(), tensors):
        if t is None:
            continue
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be on " + (f"CUDA device {dev}" if dev >= 0 else "a CUDA device"))
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} needs a gradient, which this call does not record")
        if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{name} carries a tangent, which this call does not pass on")


_INT_MAX = 2 ** 31 - 1


def _ints(**sizes):
    """An argument struct's 32-bit fields would take larger numbers modulo 2^32."""
    for name, n in sizes.items():
        if not -_INT_MAX <= n <= _INT_MAX:
            raise ValueError(f"{name} = {n} does not fit in 32 bits")


def _wrote(*tensors):
    """Counts a change of the caller's tensors that a call (past _on) writes through their
    addresses, so that autograd refuses to use a value it had kept of them."""
    _increment_version(tensors)


def _int32(name, t, shape):
    import torch

    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _freq(inv_freq):
    import torch

    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float32 vector")
    return inv_freq.data_ptr()


def _table(page_table, kv_len):
    """(kv_len, page_table, max_pages, table_stride) for the argument structs, after B."""
    import torch

    if page_table.dtype != torch.int32 or page_table.dim() != 2:
        raise TypeError("page_table must be int32 [B, max_pages]")
    B, n = page_table.shape
    if page_table.numel() > _INT_MAX:
        _ints(B=B, max_pages=n)
    stride = n
    if not page_table.is_contiguous():
        if n > 1 and page_table.stride(1) != 1:
            raise TypeError("page_table must have dense rows")
        stride = page_table.stride(0) if B > 1 else n
    if kv_len.dtype != torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
        raise TypeError(f"kv_len must be a contiguous int32 tensor of shape ({B},)")
    return B, (kv_len.data_ptr(), page_table.data_ptr(), n, stride)


@contextlib.contextmanager
def _elsewhere(device, stream):
    import torch

    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _launch(t, stream):
    """The call's stream handle, and a context in which the tensor's device is
    current and allocations belong to that stream (memory handed out on another one
    could still be in use there)."""
    import torch

    dev = t.get_device()
    if stream is None:
        if dev == torch.cuda.current_device():
            return torch._C._cuda_getCurrentRawStream(dev), _HERE
        stream = torch.cuda.current_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream must be on the tensors' device, {dev}")
    return stream.cuda_stream, _elsewhere(dev, stream)


def _check(status, what):
    if status != L.CSA_OK:
        raise L.CsaError(status, what)


def rope_frequencies(rot_dim: int, *, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotation frequencies (fp32 [rot_dim / 2] on ``device``) and the factor on
    cos and sin, for the ``scale`` of ``rotary`` and ``rope_scale`` of
    ``cache_append``."""
    import torch

    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}")
    _ints(rot_dim=rot_dim, original_len=original_len)
    f = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float32)
    m = ctypes.c_float()
    _check(csa_rope_frequencies(rot_dim, base, ROPE_SCALINGS[scaling], factor, original_len, beta_fast,
                                beta_slow, f.data_ptr() or None, ctypes.addressof(m)), "csa_rope_frequencies")
    return (f if device is None else f.to(device)), m.value


def rotary(x, positions, inv_freq, *, rot_offset: int = 0, interleaved: bool = False, scale: float = 1.0,
           inverse: bool = False, out=None, stream=None):
    """Rotates part of every head of ``x`` [..., H, D] (bf16, fp16 or fp32; any
    strides that leave a head's elements adjacent and the tokens evenly
    spaced) by ``positions`` int32 [...]; returns ``out`` (``out=x``: in
    place).  ``inverse`` rotates back: the gradient."""
    import torch

    kind = 0 if x.dtype == torch.bfloat16 else 1 if x.dtype == torch.float16 else 2 if x.dtype == torch.float32 else None
    shape = x.shape
    if kind is None or len(shape) < 2:
        raise TypeError("x must be a bfloat16, float16 or float32 tensor [..., H, D]")
    dev = x.get_device()
    pos = _int32("positions", positions, shape[:-2])
    freq = _freq(inv_freq)
    N, rot = positions.numel(), 2 * inv_freq.numel()
    if x.numel() > _INT_MAX or rot > _INT_MAX or not -_INT_MAX < rot_offset < _INT_MAX:
        _ints(tokens=N, H=shape[-2], D=shape[-1], rot_dim=rot, rot_offset=rot_offset)
    xs = _token_strides("x", x)
    if out is not None and (out.shape != shape or out.dtype != x.dtype):
        raise TypeError("out must have the shape and type of x")
    _on(dev, "x positions inv_freq out", x, positions, inv_freq, out)
    s, ctx = _launch(x, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)
        else:
            _wrote(out)
        if x.numel():
            os = xs if out is x else _token_strides("out", out)
            st = L.load_library().csa_rotary(
                ctypes.byref(CsaRotaryArgs(x.data_ptr(), out.data_ptr(), kind, N, shape[-2], shape[-1],
                                           *xs, *os, pos, freq, rot, rot_offset, bool(interleaved),
                                           bool(inverse), scale)), s)
            if st:
                raise L.CsaError(st, "csa_rotary")
    return out


def _token_strides(name, x):
    """(token, head) strides of [..., H, D] whose leading dimensions step evenly."""
    if x.is_contiguous():
        D = x.shape[-1]
        return x.shape[-2] * D, D
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}: a head's elements must be adjacent")
    step = None
    for size, stride in zip(reversed(x.shape[:-2]), reversed(x.stride()[:-2])):
        if size == 1:
            continue
        if step is None:
            step, n = stride, size
        elif stride != step * n:
            raise ValueError(f"{name}: the tokens must be evenly spaced")
        else:
            n *= size
    heads = x.stride(-2) if x.shape[-2] > 1 else x.shape[-1]
    return (heads * x.shape[-2] if step is None else step), heads


def cache_append(k, cache_k: Cache, page_table, kv_len, *, v=None, cache_v: Optional[Cache] = None,
                 cu_tokens=None, positions=None, inv_freq=None, rot_offset: int = 0, interleaved: bool = False,
                 rope_scale: float = 1.0, stream=None) -> None:
    """Appends new keys ``k`` bf16 [B,S,H,Dk] (packed: [N,H,Dk] with
    ``cu_tokens`` int32 [B+1]) and values ``v`` to their caches, the keys
    rotated if ``inv_freq`` is given.  ``kv_len`` int32 [B] counts the new tokens
    already (0: an unused place); ``page_table`` int32 [B, max_pages]."""
    import torch

    dev = k.get_device()
    B, pages = _table(page_table, kv_len)
    if (v is None) != (cache_v is None):
        raise ValueError("v and cache_v go together")
    shape = k.shape
    lead = shape[:-2]
    if len(shape) != (4 if cu_tokens is None else 3) or (cu_tokens is None and shape[0] != B):
        raise ValueError("k must be [B, S, H, Dk], or [N, H, Dk] with cu_tokens")

    def rows(name, x, c):
        st = _cache_struct("cache_" + name, c)
        if x.dtype != torch.bfloat16 or x.shape[:-2] != lead or x.shape[-2] != st.H or x.shape[-1] != st.D:
            raise TypeError(f"{name} must be bfloat16 with the tokens of k and the heads and D of cache_{name}")
        return x.data_ptr(), _token_strides(name, x), st

    kp, ks, kc = rows("k", k, cache_k)
    vp, vs, vc = rows("v", v, cache_v) if v is not None else (None, (0, 0), kc)
    N, S = (shape[0], 0) if cu_tokens is not None else (shape[0] * shape[1], shape[1])
    cu = _int32("cu_tokens", cu_tokens, (B + 1,)) if cu_tokens is not None else None
    pos = _int32("positions", positions, lead) if positions is not None else None
    freq, rot = (_freq(inv_freq), 2 * inv_freq.numel()) if inv_freq is not None else (None, 0)
    if N > _INT_MAX or rot > _INT_MAX or not -_INT_MAX < rot_offset < _INT_MAX:
        _ints(tokens=N, rot_dim=rot, rot_offset=rot_offset)
    _on(dev, "k cache_k.data cache_k.scale v cache_v.data cache_v.scale page_table kv_len cu_tokens positions inv_freq",
        k, cache_k.data, cache_k.scale, v, cache_v and cache_v.data, cache_v and cache_v.scale, page_table, kv_len,
        cu_tokens, positions, inv_freq)
    a = CsaAppendArgs(kp, vp, *ks, *vs, N, B, S, cu, *pages, kc, vc, freq, pos, rot, rot_offset, bool(interleaved),
                      rope_scale)
    s, ctx = _launch(k, stream)
    with ctx:
        st = L.load_library().csa_cache_append(ctypes.byref(a), s)
    if st:
        raise L.CsaError(st, "csa_cache_append")
    _wrote(cache_k.data) if cache_k.scale is None else _wrote(cache_k.data, cache_k.scale)
    if cache_v is not None:
        _wrote(cache_v.data) if cache_v.scale is None else _wrote(cache_v.data, cache_v.scale)


def cache_read(cache: Cache, page_table, kv_len, T: int, *, out=None, stream=None):
    """Positions 0 .. T-1 of every sequence as bf16 [B, T, H, D], zeros past ``kv_len``."""
    import torch

    dev = cache.data.get_device()
    B, pages = _table(page_table, kv_len)
    c = _cache_struct("cache", cache)
    T = int(T)
    if not -_INT_MAX <= T <= _INT_MAX:
        _ints(T=T)
    shape = (B, T, c.H, c.D)
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != shape or not out.is_contiguous()):
        raise TypeError(f"out must be a contiguous bfloat16 tensor of shape {shape}")
    _on(dev, "cache.data cache.scale page_table kv_len out", cache.data, cache.scale, page_table, kv_len, out)
    s, ctx = _launch(cache.data, stream)
    with ctx:
        if out is None:
            out = cache.data.new_empty(shape, dtype=torch.bfloat16)
        else:
            _wrote(out)
        st = L.load_library().csa_cache_read(ctypes.byref(CsaCacheReadArgs(c, *pages, B, T, out.data_ptr())), s)
    if st:
        raise L.CsaError(st, "csa_cache_read")
    return out


def cache_attention(q, cache_k: Cache, cache_v: Cache, page_table, kv_len, *, scale: float, idx=None,
                    causal: bool = True, return_lse: bool = False, out=None, lse=None, workspace=None, stream=None):
    """Attention of ``q`` bf16 [B,S,HA,Dk] over 4-bit caches: every visible
    position, or those of ``idx`` int32 [B,S,topk].  Returns ``out`` bf16
    [B,S,HA,Dv], with ``return_lse`` (out, lse fp32 [B,S,HA]).
    ``workspace`` (dense uint8 CUDA tensor) is allocated if not given."""
    import torch

    dev = q.get_device()
    B, pages = _table(page_table, kv_len)
    kc, vc = _cache_struct("cache_k", cache_k), _cache_struct("cache_v", cache_v)
    if q.dtype != torch.bfloat16 or q.dim() != 4 or q.shape[0] != B or not q.is_contiguous() or q.shape[-1] != kc.D:
        raise TypeError("q must be a contiguous bfloat16 tensor [B, S, HA, Dk]")
    _, S, HA, _ = q.shape
    if q.numel() > _INT_MAX or idx is not None and idx.numel() > _INT_MAX:
        _ints(S=S, HA=HA, topk=0 if idx is None else idx.shape[-1])
    if idx is not None and idx.numel() == 0 and B * S:
        raise ValueError("idx has no entries (leave it out for every visible position)")
    ip, topk = (None, 0) if idx is None else (_int32("idx", idx, (B, S, idx.shape[-1])), idx.shape[-1])
    for name, t, dtype, shape in (("out", out, torch.bfloat16, (B, S, HA, vc.D)),
                                  ("lse", lse, torch.float32, (B, S, HA))):
        if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    if workspace is not None and not workspace.is_contiguous():
        raise TypeError("workspace must be contiguous")
    _on(dev, "q cache_k.data cache_k.scale cache_v.data cache_v.scale page_table kv_len idx out lse workspace", q,
        cache_k.data, cache_k.scale, cache_v.data, cache_v.scale, page_table, kv_len, idx, out, lse, workspace)
    s, ctx = _launch(q, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(q) if vc.D == kc.D else q.new_empty((B, S, HA, vc.D))
        else:
            _wrote(out)
        if lse is not None:
            _wrote(lse)
        elif return_lse:
            lse = q.new_empty((B, S, HA), dtype=torch.float32)
        a = CsaCacheAttnArgs(q.data_ptr(), kc, vc, *pages, ip, topk, B, S, HA, bool(causal), scale, out.data_ptr(),
                             None if lse is None else lse.data_ptr())
        lib, a = L.load_library(), ctypes.byref(a)
        if workspace is None:
            size = lib.csa_cache_attention_workspace_size(a)
            ws = q.new_empty(size, dtype=torch.uint8) if size else None
        else:
            ws, size = workspace, workspace.numel() * workspace.element_size()
        st = lib.csa_cache_attention(a, None if ws is None else ws.data_ptr(), size, s)
    if st:
        raise L.CsaError(st, "csa_cache_attention")
    return (out, lse) if return_lse else out
