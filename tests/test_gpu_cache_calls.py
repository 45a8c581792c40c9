"""What calls of the cache operators touch beside their outputs (needs a B200)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lightning_indexer_top_02_b200 as L
    from lightning_indexer_top_02_b200.build import build
    build()
    L.load_library()
    return L


def run_script(text, **env):
    r = subprocess.run([sys.executable, "-c", text.format(root=ROOT, here=HERE)], capture_output=True, text=True,
                       env=dict(os.environ, **env), timeout=600)
    assert r.returncode == 0 and "script ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


_APPEND_SCRIPT = r"""
import sys
sys.path.insert(0, {root!r})
import torch, lightning_indexer_top_02_b200 as L
assert L.LIB_PATH.endswith("libcsa_indexer_debug.so"), L.LIB_PATH
for kind in ("bf16", "e4m3", "e2m1"):
    for N, ends in ((40, [0, 7, 7, 20]), (3000, [0, 1, 2, 900]), (64, [0, 0, 0, 0]), (50, [0, 10, 30, 50])):
        for rot in (0, 64):
            k = torch.randn((N, 2, 128), device="cuda").to(torch.bfloat16)
            v = torch.randn((N, 2, 64), device="cuda").to(torch.bfloat16)
            ck, cv = (L.make_cache(kind, 200, 16, 2, D, device="cuda") for D in (128, 64))
            table = torch.arange(180, dtype=torch.int32, device="cuda").view(3, 60)
            lens = torch.full((3,), 900, dtype=torch.int32, device="cuda")
            freq = L.rope_frequencies(rot, device="cuda")[0] if rot else None
            L.cache_append(k, ck, table, lens, v=v, cache_v=cv, cu_tokens=torch.tensor(ends, dtype=torch.int32, device="cuda"),
                           inv_freq=freq, positions=torch.zeros(N, dtype=torch.int32, device="cuda"))
            assert L.csa_last_device_error(None) == L.CSA_OK, (kind, N, ends, rot)
print("script ok")
"""


def test_append_reads_no_row_past_the_last_sequence(lib):
    """The debug build checks every row that a packed append reads against cu_tokens[B].  (The rows are all there.)"""
    from lightning_indexer_top_02_b200.build import build
    run_script(_APPEND_SCRIPT, CSA_INDEXER_LIB=build(debug=True))


def test_workspace_over_outputs_is_refused(lib):
    L = lib
    c = L.make_cache("e2m1", 64, 64, 1, 128, device="cuda")
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
    buf = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    inside = lambda at: buf[at:at + 2048].view(torch.bfloat16).view(1, 1, 8, 128)  # noqa: E731
    q = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    for query, out in ((q, inside(0)), (q, inside(4096)), (inside(512), None)):
        with pytest.raises(L.CsaError) as e:
            L.cache_attention(query, c, c, table, lens, scale=0.1, out=out, workspace=buf)
        assert e.value.status == L.CSA_ERR_INVALID_ARG
    L.cache_attention(inside(0), c, c, table, lens, scale=0.1, out=inside(2048), workspace=buf[4096:])
    torch.cuda.synchronize()
    assert L.csa_last_device_error(None) == L.CSA_OK


# ---------------------------------------------------------------- autograd

def step(L):
    c = L.make_cache("e4m3", 2, 16, 1, 64, device="cuda")
    x = torch.randn((1, 3, 1, 64), device="cuda").to(torch.bfloat16)
    table = torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2)
    return c, x, table, torch.full((1,), 3, dtype=torch.int32, device="cuda"), torch.zeros((1, 3), dtype=torch.int32, device="cuda")


def test_tangents_are_refused(lib):
    """A tensor that carries a forward-mode tangent, which no call here would pass on."""
    import torch.autograd.forward_ad as fw
    L = lib
    c, x, table, lens, pos = step(L)
    freq = torch.ones(8, device="cuda")
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            L.rotary(d, pos, freq)
        with pytest.raises(ValueError, match="tangent"):
            L.cache_append(d, c, table, lens)
        with pytest.raises(ValueError, match="tangent"):
            L.cache_read(L.Cache("bf16", fw.make_dual(x, x)), table, lens, 1)
        e = L.make_cache("e2m1", 2, 16, 1, 64, device="cuda")
        with pytest.raises(ValueError, match="tangent"):
            L.cache_attention(d, e, e, table, lens, scale=0.1)
        assert torch.equal(L.rotary(x, pos, freq), x)    # (others pass; position 0)
    assert torch.equal(L.rotary(d, pos, freq), x)        # the level has ended: an ordinary tensor


def test_writes_are_seen_by_autograd(lib):
    """What a call writes counts as changed, so that a product's gradient is not computed from it."""
    L = lib
    c, x, table, lens, pos = step(L)
    freq = torch.ones(8, device="cuda")
    y = torch.randn_like(x).requires_grad_()
    z = (x * y).sum()                                    # keeps x for y's gradient
    L.rotary(x, pos + 1, freq, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()

    def changes(call, *tensors):
        was = [t._version for t in tensors]
        call()
        return [t._version > w for t, w in zip(tensors, was)]

    out = torch.empty_like(x)
    assert changes(lambda: L.rotary(x, pos, freq, out=out), out, x) == [True, False]
    assert changes(lambda: L.cache_append(x, c, table, lens), c.data, c.scale, x) == [True, True, False]
    b = L.make_cache("bf16", 2, 16, 1, 64, device="cuda")
    assert changes(lambda: L.cache_append(x, c, table, lens, v=x, cache_v=L.make_cache("e4m3", 2, 16, 1, 64, device="cuda")),
                   c.data, c.scale) == [True, True]
    assert changes(lambda: L.cache_append(x, b, table, lens), b.data) == [True]
    out = torch.empty((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    assert changes(lambda: L.cache_read(c, table, lens, 4, out=out), out, c.data) == [True, False]
    e = L.make_cache("e2m1", 2, 16, 1, 64, device="cuda")
    out, lse = torch.empty_like(x), torch.empty((1, 3, 1), device="cuda")
    assert changes(lambda: L.cache_attention(x, e, e, table, lens, scale=0.1, out=out, lse=lse), out, lse, x, e.data) == \
        [True, True, False, False]
    with torch.inference_mode():
        t = torch.zeros((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
        L.rotary(t, pos, freq, out=t)                    # (no version to count)


# ---------------------------------------------------------------- costs

_ERROR_WORD_SCRIPT = r"""
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {here!r})
import torch, lightning_indexer_top_02_b200 as L
from torch.profiler import profile, ProfilerActivity

def copies():
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
        assert L.csa_last_device_error(None) == L.CSA_OK
        torch.cuda.synchronize()
    return sum(e.count for e in p.key_averages() if "DtoH" in e.key)

q = torch.randn((1, 4, 16, 128), device="cuda").to(torch.bfloat16)
k = torch.randn((1, 300, 128), device="cuda").to(torch.bfloat16)
L.indexer_topk(q, torch.randn((1, 4, 16), device="cuda"), k, m=1, topk=16)
assert L.csa_last_device_error(None) == L.CSA_OK
print("indexer alone:", copies())
assert copies() == 1
c = L.make_cache("e2m1", 4, 16, 1, 128, device="cuda")
table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
L.cache_attention(q[:, :1], c, c, table, torch.tensor([60], dtype=torch.int32, device="cuda"), scale=0.1)
print("with attention:", copies())
assert copies() == 2
print("script ok")
"""


def test_error_word_costs_what_has_run(lib):
    """csa_last_device_error copies the words of the units that a call has used, the indexer's alone to begin with."""
    run_script(_ERROR_WORD_SCRIPT)


@pytest.mark.parametrize("HA", [8, 16])
@pytest.mark.parametrize("Dv", [64, 128, 192, 256])
@pytest.mark.parametrize("Dk", [64, 128, 192, 256])
def test_attention_shares_fit_the_sms(lib, Dk, Dv, HA):
    """The chunks are shared among CTAs that the GPU holds at a time: their staging (blocks of 64 keys twice, of
    32 keys three times where rows are wide, four warps) fits in the SMs' shared memory."""
    L = lib
    a = L.cache.CsaCacheAttnArgs()
    for c, D in ((a.cache_k, Dk), (a.cache_v, Dv)):
        c.data, c.scale, c.dtype, c.H, c.D = 4096, 4096, L.cache.CSA_CACHE_E2M1, 1, D
        c.num_pages, c.page_size, c.tensor_scale = 1, 1 << 24, 1.0
    a.q, a.out, a.kv_len, a.page_table = 4096, 1 << 20, 4096, 4096
    a.max_pages = a.table_stride = 1
    a.B, a.S, a.HA, a.causal, a.scale = 1, 1, HA, 1, 0.1
    size = L.csa_cache_attention_workspace_size(a)
    props = torch.cuda.get_device_properties(0)
    per_sm, rest = divmod(size, 2 * props.multi_processor_count * HA * (Dv + 2) * 4)
    assert rest == 0 and per_sm >= 1
    block = 64 if Dk + Dv <= 256 else 32
    staging = 4 * (2 if block == 64 else 3) * block * (Dk + Dv) * 9 // 16
    assert per_sm * (staging + 1024) <= props.shared_memory_per_multiprocessor


# ---------------------------------------------------------------- errors

_FAILED_CALL_SCRIPT = r"""
import sys
sys.path.insert(0, {root!r})
import torch, lightning_indexer_top_02_b200 as L
C = L.cache
c = L.make_cache("e2m1", 64, 64, 1, 128, device="cuda")
table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
q, out = (torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
back = torch.empty((1, 100, 1, 128), dtype=torch.bfloat16, device="cuda")
s = C._cache_struct("c", c)
pages = (lens.data_ptr(), table.data_ptr(), 64, 64)
attend = C.CsaCacheAttnArgs(q.data_ptr(), s, s, *pages, None, 0, 1, 1, 8, 1, 0.1, out.data_ptr(), None)
read = C.CsaCacheReadArgs(s, *pages, 1, 100, back.data_ptr())
assert L.csa_cache_attention(attend, None, 0, None) == L.CSA_OK
torch.cuda.synchronize()
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(side):
    graph.capture_begin(capture_error_mode="thread_local")
    try:
        side.synchronize()                  # not allowed while capturing: the capture is void from here on
    except RuntimeError as e:
        print("void:", str(e).splitlines()[0])
    status = L.csa_cache_attention(attend, None, 0, side.cuda_stream)
    try:
        graph.capture_end()
    except RuntimeError:
        pass
print("in the void capture:", status)
assert status == L.CSA_ERR_CUDA
assert L.csa_cache_read(read, None) == L.CSA_OK
torch.cuda.synchronize()
assert (back == 0).all()
print("script ok")
"""


def test_a_failed_call_leaves_no_error_behind(lib):
    """A workspace that cannot be allocated is that call's error, not the next one's."""
    run_script(_FAILED_CALL_SCRIPT)


# ---------------------------------------------------------------- forms of the arguments

def test_views_as_arguments(lib):
    """Tables inside wider ones, caches as E4M3 tensors, heads and tokens broadcast: as their plain copies."""
    import test_gpu_cache as T
    L, g = lib, T.gen(21)
    wide = torch.randperm(2 * 40, generator=g, device="cuda")[:80].to(torch.int32).view(2, 40)
    table = wide[:, 8:32]
    lens = torch.tensor([380, 100], dtype=torch.int32, device="cuda")
    kc, vc = (T.random_cache(L, "e2m1", 80, 16, 2, 128, g) for _ in (0, 1))
    as8 = lambda c: L.Cache(c.dtype, c.data if c.dtype == "e2m1" else c.data.view(torch.float8_e4m3fn),  # noqa: E731
                            c.scale.view(torch.float8_e4m3fn) if c.dtype == "e2m1" else c.scale, c.tensor_scale)
    for HA in (16, 64):
        q = torch.randn((2, 1, HA, 128), generator=g, device="cuda").to(torch.bfloat16)
        assert torch.equal(L.cache_attention(q, as8(kc), as8(vc), table, lens, scale=0.09),
                           L.cache_attention(q, kc, vc, table.contiguous(), lens, scale=0.09))
    row = torch.randn((1, 1, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    freq, _ = L.rope_frequencies(64, device="cuda")
    for kind in ("bf16", "e4m3", "e2m1"):
        a = T.random_cache(L, kind, 80, 16, 2, 128, g)
        b = L.Cache(kind, a.data.clone(), None if a.scale is None else a.scale.clone())
        c8 = as8(a) if kind != "bf16" else a
        L.cache_append(row.expand(2, 7, 2, 128), c8, table, lens, inv_freq=freq)
        L.cache_append(row.expand(2, 7, 2, 128).contiguous(), b, table.contiguous(), lens, inv_freq=freq)
        assert torch.equal(a.data, b.data) and (a.scale is None or torch.equal(a.scale, b.scale))
        assert torch.equal(L.cache_read(c8, table, lens, 390), L.cache_read(b, table.contiguous(), lens, 390))
    pos = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7)
    assert torch.equal(L.rotary(row.expand(2, 7, 2, 128), pos, freq), L.rotary(row.expand(2, 7, 2, 128).contiguous(), pos, freq))
    T.no_device_error(L)


def test_calls_from_two_threads(lib):
    """Two host threads, a stream each, at the same time."""
    import threading

    import test_gpu_cache as T
    L = lib
    states = [T.step_state(L, T=200), T.step_state(L, T=777)]
    want = [T.decode_step(L, s)[0] for s in states]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                got[i].append(T.decode_step(L, states[i], stream=stream)[0])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for g, w in zip(got, want):
        assert len(g) == 30 and all(torch.equal(x, w) for x in g)
    T.no_device_error(L)
