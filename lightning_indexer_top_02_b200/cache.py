"""The cache operators on torch tensors: rotary positions, appending to a paged
cache, reading it back as bf16 rows, and attention over a cache held in 4 bits.

The same calls as ``include/csa_cache.h`` (operation, layouts and limits are
stated there), marshalled with ctypes; outputs and workspaces are allocated on
the tensors' device if not given.  Nothing here records a gradient: a tensor
that would need one is refused (``rotary(..., inverse=True)`` is the gradient
of ``rotary``).
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


def _dense_but_pages(name, t):
    """The stride in bytes from page to page of a tensor that is dense within a page."""
    n = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != n:
            raise ValueError(f"{name} must be dense within a page")
        n *= size
    return (t.stride(0) if t.shape[0] > 1 else n) * t.element_size()


def _cache_struct(name: str, c: Cache, device) -> CsaCache:
    import torch

    if c.dtype not in CACHE_DTYPES:
        raise ValueError(f"unknown cache type {c.dtype!r}")
    data, scale = c.data, c.scale
    want = (torch.bfloat16,) if c.dtype == "bf16" else (torch.uint8, torch.float8_e4m3fn) if c.dtype == "e4m3" \
        else (torch.uint8,)
    if data.dtype not in want or data.dim() != 4:
        raise TypeError(f"{name}.data must be a 4-dimensional {want[0]} tensor")
    s = CsaCache()
    s.dtype = CACHE_DTYPES[c.dtype]
    s.num_pages, s.H, s.page_size = data.shape[:3]
    s.D = c.D
    _on(device, **{name + ".data": data})
    s.data, s.page_stride = data.data_ptr(), _dense_but_pages(name + ".data", data)
    if c.dtype != "bf16":
        kinds = (torch.float32,) if c.dtype == "e4m3" else (torch.uint8, torch.float8_e4m3fn)
        tail = () if c.dtype == "e4m3" else (s.D // 16,)
        if scale is None or scale.dtype not in kinds or tuple(scale.shape) != tuple(data.shape[:3]) + tail:
            raise TypeError(f"{name}.scale must be {kinds[0]} {tuple(data.shape[:3]) + tail}")
        _on(device, **{name + ".scale": scale})
        s.scale, s.scale_page_stride = scale.data_ptr(), _dense_but_pages(name + ".scale", scale)
    s.tensor_scale = float(c.tensor_scale)
    return s


def _on(device, **tensors):
    import torch

    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{name} must be on {device}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} needs a gradient, which this call does not record")


def _int32(name, t, shape):
    import torch

    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")


def _freq(inv_freq):
    import torch

    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float32 vector")


def _table(page_table, kv_len):
    import torch

    if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise TypeError("page_table must be int32 [B, max_pages] with dense rows")
    _int32("kv_len", kv_len, (page_table.shape[0],))
    B, n = page_table.shape
    return B, n, page_table.stride(0) if B > 1 else n


@contextlib.contextmanager
def _elsewhere(device, stream):
    import torch

    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _launch(t, stream):
    """The call's stream, and a context in which the tensor's device is current
    and allocations belong to that stream (memory handed out on another one
    could still be in use there)."""
    import torch

    here = torch.cuda.current_stream(t.device)
    if stream is None:
        stream = here
    same = stream == here and torch.cuda.current_device() == t.device.index
    return stream, contextlib.nullcontext() if same else _elsewhere(t.device, stream)


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

    kinds = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    if x.dtype not in kinds or x.dim() < 2:
        raise TypeError("x must be a bfloat16, float16 or float32 tensor [..., H, D]")
    _int32("positions", positions, x.shape[:-2])
    _freq(inv_freq)
    s, ctx = _launch(x, stream)
    if out is None:
        with ctx:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise TypeError("out must have the shape and type of x")
    _on(x.device, x=x, positions=positions, inv_freq=inv_freq, out=out)
    a = CsaRotaryArgs()
    a.x, a.out, a.dtype = x.data_ptr(), out.data_ptr(), kinds[x.dtype]
    a.H, a.D = x.shape[-2:]
    a.N = positions.numel()
    a.x_token_stride, a.x_head_stride = _token_strides("x", x)
    a.out_token_stride, a.out_head_stride = _token_strides("out", out)
    a.positions, a.inv_freq = positions.data_ptr(), inv_freq.data_ptr()
    a.rot_dim, a.rot_offset = 2 * inv_freq.numel(), int(rot_offset)
    a.interleaved, a.inverse, a.scale = int(bool(interleaved)), int(bool(inverse)), float(scale)
    if x.numel() == 0:
        return out
    with _launch(x, stream)[1]:
        _check(csa_rotary(a, ctypes.c_void_p(s.cuda_stream)), "csa_rotary")
    return out


def _token_strides(name, x):
    """(token, head) strides of [..., H, D] whose leading dimensions step evenly."""
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

    B, n, stride = _table(page_table, kv_len)
    if (v is None) != (cache_v is None):
        raise ValueError("v and cache_v go together")
    lead = k.shape[:-2]
    if k.dim() != (4 if cu_tokens is None else 3) or (cu_tokens is None and k.shape[0] != B):
        raise ValueError("k must be [B, S, H, Dk], or [N, H, Dk] with cu_tokens")
    a = CsaAppendArgs()
    for name, x, c in (("k", k, cache_k), ("v", v, cache_v)):
        if x is None:
            continue
        if x.dtype != torch.bfloat16 or x.shape[:-2] != lead or x.shape[-2] != c.data.shape[1] or x.shape[-1] != c.D:
            raise TypeError(f"{name} must be bfloat16 with the tokens of k and the heads and D of cache_{name}")
        token, head = _token_strides(name, x)
        setattr(a, name, x.data_ptr())
        setattr(a, name + "_token_stride", token)
        setattr(a, name + "_head_stride", head)
        setattr(a, "cache_" + name, _cache_struct("cache_" + name, c, k.device))
    a.N = k.shape[0] if cu_tokens is not None else k.shape[0] * k.shape[1]
    a.B, a.S = B, 0 if cu_tokens is not None else k.shape[1]
    if cu_tokens is not None:
        _int32("cu_tokens", cu_tokens, (B + 1,))
        a.cu_tokens = cu_tokens.data_ptr()
    if positions is not None:
        _int32("positions", positions, lead)
        a.positions = positions.data_ptr()
    if inv_freq is not None:
        _freq(inv_freq)
        a.inv_freq, a.rot_dim, a.rot_offset = inv_freq.data_ptr(), 2 * inv_freq.numel(), int(rot_offset)
        a.interleaved, a.rope_scale = int(bool(interleaved)), float(rope_scale)
    _on(k.device, k=k, v=v, page_table=page_table, kv_len=kv_len, cu_tokens=cu_tokens, positions=positions,
        inv_freq=inv_freq)
    a.kv_len, a.page_table, a.max_pages, a.table_stride = kv_len.data_ptr(), page_table.data_ptr(), n, stride
    s, ctx = _launch(k, stream)
    with ctx:
        _check(csa_cache_append(a, ctypes.c_void_p(s.cuda_stream)), "csa_cache_append")


def cache_read(cache: Cache, page_table, kv_len, T: int, *, out=None, stream=None):
    """Positions 0 .. T-1 of every sequence as bf16 [B, T, H, D], zeros past ``kv_len``."""
    import torch

    B, n, stride = _table(page_table, kv_len)
    dev = cache.data.device
    a = CsaCacheReadArgs()
    a.cache = _cache_struct("cache", cache, dev)
    shape = (B, int(T), a.cache.H, a.cache.D)
    s, ctx = _launch(cache.data, stream)
    if out is None:
        with ctx:
            out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != shape or not out.is_contiguous():
        raise TypeError(f"out must be a contiguous bfloat16 tensor of shape {shape}")
    _on(dev, page_table=page_table, kv_len=kv_len, out=out)
    a.kv_len, a.page_table, a.max_pages, a.table_stride = kv_len.data_ptr(), page_table.data_ptr(), n, stride
    a.B, a.T, a.out = B, int(T), out.data_ptr()
    with _launch(cache.data, stream)[1]:
        _check(csa_cache_read(a, ctypes.c_void_p(s.cuda_stream)), "csa_cache_read")
    return out


def cache_attention(q, cache_k: Cache, cache_v: Cache, page_table, kv_len, *, scale: float, idx=None,
                    causal: bool = True, return_lse: bool = False, out=None, lse=None, workspace=None, stream=None):
    """Attention of ``q`` bf16 [B,S,HA,Dk] over 4-bit caches: every visible
    position, or those of ``idx`` int32 [B,S,topk].  Returns ``out`` bf16
    [B,S,HA,Dv], with ``return_lse`` (out, lse fp32 [B,S,HA]).
    ``workspace`` (uint8 CUDA tensor) is allocated if not given."""
    import torch

    B, n, stride = _table(page_table, kv_len)
    if q.dtype != torch.bfloat16 or q.dim() != 4 or q.shape[0] != B or not q.is_contiguous() \
            or q.shape[-1] != cache_k.D:
        raise TypeError("q must be a contiguous bfloat16 tensor [B, S, HA, Dk]")
    S, HA = q.shape[1:3]
    a = CsaCacheAttnArgs()
    a.cache_k = _cache_struct("cache_k", cache_k, q.device)
    a.cache_v = _cache_struct("cache_v", cache_v, q.device)
    if idx is not None:
        _int32("idx", idx, (B, S, idx.shape[-1]))
        a.idx, a.topk = idx.data_ptr(), idx.shape[-1]
    for name, t, dtype, shape in (("out", out, torch.bfloat16, (B, S, HA, a.cache_v.D)),
                                  ("lse", lse, torch.float32, (B, S, HA))):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    s, ctx = _launch(q, stream)
    with ctx:
        if out is None:
            out = torch.empty((B, S, HA, a.cache_v.D), dtype=torch.bfloat16, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((B, S, HA), dtype=torch.float32, device=q.device)
        _on(q.device, q=q, page_table=page_table, kv_len=kv_len, idx=idx, out=out, lse=lse, workspace=workspace)
        a.q, a.out = q.data_ptr(), out.data_ptr()
        a.lse = lse.data_ptr() if lse is not None else None
        a.kv_len, a.page_table, a.max_pages, a.table_stride = kv_len.data_ptr(), page_table.data_ptr(), n, stride
        a.B, a.S, a.HA, a.causal, a.scale = B, S, HA, int(bool(causal)), float(scale)
        if workspace is None:
            need = csa_cache_attention_workspace_size(a)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws, size = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
            if workspace is not None else (None, 0)
        _check(csa_cache_attention(a, ws, size, ctypes.c_void_p(s.cuda_stream)), "csa_cache_attention")
    return (out, lse) if return_lse else out
