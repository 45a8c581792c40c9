"""The cache operators' entry points without a GPU: refusals before any launch,
rotation frequencies against their formulas, the binding's own checks."""
import math

import pytest
import torch

import lightning_indexer_top_02_b200 as L
from lightning_indexer_top_02_b200 import cache as C
from lightning_indexer_top_02_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return L.load_library()


def good_cache(dtype=C.CSA_CACHE_E2M1, D=128, H=2):
    c = C.CsaCache()
    c.data, c.scale, c.dtype, c.H, c.D = 4096, 4096, dtype, H, D
    c.num_pages, c.page_size, c.tensor_scale = 8, 16, 1.0
    return c


def good_attn():
    a = C.CsaCacheAttnArgs()
    a.q = a.kv_len = a.page_table = 4096
    a.out = 8192
    a.cache_k, a.cache_v = good_cache(), good_cache()
    a.max_pages = a.table_stride = 4
    a.B, a.S, a.HA, a.causal, a.scale = 0, 1, 8, 1, 0.1       # B = 0: valid, and launches nothing
    return a


def good_append():
    a = C.CsaAppendArgs()
    a.k = a.kv_len = a.page_table = a.inv_freq = 4096
    a.k_token_stride, a.k_head_stride = 256, 128
    a.B, a.S, a.N = 2, 0, 0                                   # no tokens: launches nothing
    a.max_pages = a.table_stride = 4
    a.cache_k = good_cache()
    a.rot_dim, a.rope_scale = 64, 1.0
    return a


def good_rotary():
    a = C.CsaRotaryArgs()
    a.x = a.out = a.positions = a.inv_freq = 4096
    a.N, a.H, a.D, a.rot_dim, a.scale = 0, 4, 128, 64, 1.0
    a.x_token_stride = a.out_token_stride = 512
    a.x_head_stride = a.out_head_stride = 128
    return a


def set_path(a, path, value):
    *head, last = path.split(".")
    for h in head:
        a = getattr(a, h)
    setattr(a, last, value)


CACHE_FAULTS = [("dtype", 3, 1), ("dtype", -1, 1), ("H", 0, 1), ("D", 0, 1), ("D", 24, 2), ("D", 48, 2), ("D", 544, 2),
                ("num_pages", 0, 1), ("page_size", 0, 1), ("data", 0, 1), ("data", 4104, 1), ("scale", 0, 1),
                ("page_stride", 8, 1), ("page_stride", 16, 1), ("page_stride", -16, 1), ("scale_page_stride", 8, 1),
                ("tensor_scale", 0.0, 1), ("tensor_scale", math.nan, 1), ("tensor_scale", math.inf, 1)]


@pytest.mark.parametrize("field,value,status", [("cache_k." + f, v, s) for f, v, s in CACHE_FAULTS]
                         + [("cache_v." + f, v, s) for f, v, s in CACHE_FAULTS]
                         + [("B", -1, 1), ("S", -1, 1), ("HA", 0, 1), ("HA", 7, 1), ("HA", 258, 2), ("scale", math.nan, 1),
                            ("scale", math.inf, 1), ("cache_v.page_size", 8, 1), ("cache_v.H", 1, 1),
                            ("cache_v.num_pages", 9, 1), ("cache_k.dtype", 1, 1), ("cache_k.D", 96, 2),
                            ("cache_v.D", 320, 2)])
def test_attention_refuses(field, value, status):
    a = good_attn()
    assert L.csa_cache_attention(a, None, 0, None) == L.CSA_OK
    set_path(a, field, value)
    assert L.csa_cache_attention(a, None, 0, None) == status
    assert L.csa_cache_attention_workspace_size(a) == 0


@pytest.mark.parametrize("field,value,status", [("q", 0, 1), ("q", 4104, 1), ("q", 8192, 1), ("out", 0, 1), ("out", 4104, 1), ("kv_len", 0, 1),
                                                ("page_table", 0, 1), ("page_table", 4098, 1), ("max_pages", 0, 1),
                                                ("table_stride", 3, 1), ("max_pages", 1 << 28, 1), ("idx", 4098, 1),
                                                ("lse", 4098, 1)])
def test_attention_refuses_pointers(field, value, status):
    """With work to do, before any launch."""
    a = good_attn()
    a.B = 1
    a.topk = 4
    setattr(a, field, value)
    assert L.csa_cache_attention(a, None, 0, None) == status


def test_attention_refuses_large():
    a = good_attn()
    a.B, a.max_pages, a.table_stride = 1, 1 << 27, 1 << 27    # 2^31 positions
    assert L.csa_cache_attention(a, None, 0, None) == L.CSA_ERR_UNSUPPORTED
    a = good_attn()
    a.B, a.S = 1 << 16, 1 << 16
    assert L.csa_cache_attention(a, None, 0, None) == L.CSA_ERR_UNSUPPORTED
    a = good_attn()
    a.B, a.idx, a.topk = 1, 4096, 0
    assert L.csa_cache_attention(a, None, 0, None) == L.CSA_ERR_INVALID_ARG
    assert L.load_library().csa_cache_attention(None, None, 0, None) == L.CSA_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [("cache_k." + f, v, s) for f, v, s in CACHE_FAULTS]
                         + [("N", -1, 1), ("N", 1, 1), ("B", -1, 1), ("S", -1, 1), ("rot_dim", 3, 1), ("rot_dim", 0, 1), ("rot_dim", 130, 1),
                            ("rot_offset", 1, 1), ("rot_offset", 66, 1), ("rot_offset", -2, 1), ("rope_scale", math.nan, 1),
                            ("inv_freq", 4098, 1), ("v", 4096, 1)])
def test_append_refuses(field, value, status):
    a = good_append()
    assert L.csa_cache_append(a, None) == L.CSA_OK
    set_path(a, field, value)
    assert L.csa_cache_append(a, None) == status


@pytest.mark.parametrize("field,value", [("k", 0), ("k", 4104), ("v", 4104), ("kv_len", 0), ("page_table", 0), ("k_token_stride", 4),
                                         ("k_head_stride", -8), ("v_token_stride", 4), ("cu_tokens", 4098), ("positions", 4098),
                                         ("table_stride", 0), ("max_pages", 0), ("cache_v.data", 4096)])
def test_append_refuses_pointers(field, value):
    a = good_append()
    a.S, a.N = 1, 2
    a.v, a.cache_v, a.v_token_stride, a.v_head_stride = 4096, good_cache(), 256, 128
    a.cache_v.data = 8192
    set_path(a, field, value)
    assert L.csa_cache_append(a, None) == L.CSA_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [("dtype", 3, 1), ("N", -1, 1), ("H", 0, 1), ("D", 0, 1), ("rot_dim", 1, 1),
                                                ("rot_dim", 7, 1), ("rot_offset", 3, 1), ("rot_offset", 66, 1), ("scale", math.inf, 1),
                                                ("D", 1026, 2), ("H", 1 << 25, 2)])
def test_rotary_refuses(field, value, status):
    a = good_rotary()
    assert L.csa_rotary(a, None) == L.CSA_OK
    setattr(a, field, value)
    assert L.csa_rotary(a, None) == status


@pytest.mark.parametrize("fields", [dict(x=0), dict(out=0), dict(x=4097), dict(positions=0), dict(inv_freq=0), dict(positions=4098),
                                    dict(out_head_stride=64), dict(out_token_stride=64), dict(x_token_stride=-512),
                                    dict(out_token_stride=256),            # a token's heads within another's
                                    dict(x_token_stride=1024),             # in place with other strides
                                    dict(out_head_stride=0)])
def test_rotary_refuses_pointers(fields):
    a = good_rotary()
    a.N = 2
    for f, v in fields.items():
        setattr(a, f, v)
    assert L.csa_rotary(a, None) == L.CSA_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [("cache." + f, v, s) for f, v, s in CACHE_FAULTS] + [("B", -1, 1), ("T", -1, 1)])
def test_read_refuses(field, value, status):
    a = C.CsaCacheReadArgs()
    a.cache, a.kv_len, a.page_table, a.out = good_cache(), 4096, 4096, 4096
    a.max_pages = a.table_stride = 4
    assert L.csa_cache_read(a, None) == L.CSA_OK              # T = 0
    set_path(a, field, value)
    assert L.csa_cache_read(a, None) == status


def test_frequencies():
    """Each scaling against its formula, written with torch in 64 bits; fp32 values, half a step off at most."""
    rot, base, factor, n = 64, 10000.0, 8.0, 4096
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    plain = base ** (-i / rot)
    low = math.floor(rot * math.log(n / (32 * 2 * math.pi)) / (2 * math.log(base)))
    high = math.ceil(rot * math.log(n / (1 * 2 * math.pi)) / (2 * math.log(base)))
    ramp = ((i / 2 - low) / (high - low)).clamp(0, 1)
    want = {"plain": plain, "linear": plain / factor, "ntk": (base * factor ** (rot / (rot - 2))) ** (-i / rot),
            "yarn": plain * (1 - ramp) + plain / factor * ramp}
    assert 0 < low < high < rot // 2
    for how, f in want.items():
        got, m = L.rope_frequencies(rot, base=base, scaling=how, factor=factor, original_len=n)
        assert got.dtype == torch.float32
        assert ((got.double() - f).abs() <= f * (2.0 ** -24 + 1e-14)).all(), how
        assert m == pytest.approx(0.1 * math.log(factor) + 1 if how == "yarn" else 1.0, rel=2 ** -24)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=math.nan), dict(scaling="linear", factor=0.5),
                                dict(scaling="ntk", rot_dim=2, factor=2.0), dict(scaling="yarn", factor=2.0, original_len=0),
                                dict(scaling="yarn", factor=2.0, original_len=8, beta_fast=1.0, beta_slow=2.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(L.CsaError):
        L.rope_frequencies(**{"rot_dim": 64, **kw})


def test_binding_refuses():
    """Types, shapes and devices that the binding can see."""
    f = torch.ones(32)
    x = torch.zeros(2, 4, 128)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        L.rotary(x, pos.long(), f)
    with pytest.raises(TypeError):
        L.rotary(x.double(), pos, f)
    with pytest.raises(TypeError):
        L.rotary(x, pos, f.double())
    with pytest.raises(ValueError):
        L.rope_frequencies(64, scaling="other")
    with pytest.raises(ValueError):
        L.make_cache("int4", 1, 1, 1, 64, device="cpu")
    c = L.make_cache("e2m1", 4, 16, 2, 128, device="cpu")
    assert c.D == 128 and c.data.shape == (4, 2, 16, 64) and c.scale.shape == (4, 2, 16, 8)
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        L.cache_attention(q.float(), c, c, table, lens, scale=1.0)
    with pytest.raises(TypeError):
        L.cache_attention(q, c, c, table.long(), lens, scale=1.0)
    with pytest.raises(TypeError):
        L.cache_attention(q, c, c, table, lens.long(), scale=1.0)
    with pytest.raises(ValueError):                            # not on a GPU: there is no CPU fallback
        L.cache_attention(q, c, c, table, lens, scale=1.0)
    with pytest.raises(ValueError):
        L.cache_append(q, c, table, lens, v=q)
    with pytest.raises(ValueError):
        L.cache_append(q[0], c, table, lens)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
def test_binding_refuses_overlapping_pages(dtype):
    """Pages laid over one another (an expanded tensor's): neither dense nor strided."""
    one, many = L.make_cache(dtype, 1, 16, 2, 64, device="cpu"), L.make_cache(dtype, 4, 16, 2, 64, device="cpu")
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    n = one.data[0].numel()
    for data in (one.data.expand(4, -1, -1, -1), many.data.as_strided(many.data.shape, (n // 2,) + many.data.stride()[1:])):
        with pytest.raises(ValueError, match="overlap"):
            L.cache_read(L.Cache(dtype, data, many.scale), table, lens, 4)
    if dtype != "bf16":
        scale = one.scale.expand(4, *one.scale.shape[1:])
        with pytest.raises(ValueError, match="overlap"):
            L.cache_read(L.Cache(dtype, many.data, scale), table, lens, 4)


def test_binding_refuses_spread_workspace():
    """An expanded tensor counts more bytes than it has."""
    c = L.make_cache("e2m1", 4, 16, 2, 128, device="cpu")
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(TypeError, match="workspace"):
            L.cache_attention(q, c, c, table, lens, scale=1.0, workspace=ws)


def test_binding_refuses_sizes_past_32_bits():
    """The argument structs' fields are 32 bits wide: larger numbers would arrive modulo 2^32."""
    x, pos, f = torch.zeros(2, 4, 128), torch.zeros(2, dtype=torch.int32), torch.ones(32)
    c = L.make_cache("e2m1", 4, 16, 2, 128, device="cpu")
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: L.rotary(x, pos, f, rot_offset=2 ** 32), lambda: L.rotary(x, pos, f, rot_offset=-2 ** 32),
                 lambda: L.cache_append(k, c, table, lens, inv_freq=f, rot_offset=2 ** 32),
                 lambda: L.cache_append(k[0, 0].expand(2 ** 32 + 1, 2, 128), c, table, lens, cu_tokens=cu),
                 lambda: L.cache_read(c, table, lens, 2 ** 32 + 4), lambda: L.rope_frequencies(2 ** 32 + 64),
                 lambda: L.rope_frequencies(64, scaling="yarn", factor=2.0, original_len=2 ** 32 + 4096)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_refuses_a_stream_of_another_device():
    """Its device would become the current one, where the tensors' addresses mean nothing."""
    from types import SimpleNamespace as Fake

    t = Fake(get_device=lambda: 0)
    handle, _ = C._launch(t, Fake(device_index=0, cuda_stream=5))
    assert handle == 5
    with pytest.raises(ValueError, match="stream"):
        C._launch(t, Fake(device_index=1, cuda_stream=5))
