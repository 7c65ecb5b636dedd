"""libropekv_serving.so loads, exports what include/ropekv_serving.h declares
and refuses bad arguments on the host (no GPU: only calls that must be rejected
before any CUDA call, or that have nothing to do), and the binding refuses
tensors that do not fit."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import rope_kv_cache_gb300 as rk
from rope_kv_cache_gb300 import _serving, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0)
OK, NULL, MISALIGNED, HEAD_DIM, ROTARY_DIM, HEADS, SHAPE, CAPACITY, STYLE = 0, -1, -2, -3, -4, -5, -6, -8, -9


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return rk.load_serving_library()


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "ropekv_serving.h")).read()
    names = re.findall(r"ROPEKV_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == {"rope_write_kv_mrope", "rope_write_kv_slot_mapping_quant",
                          "paged_kv_read", "paged_attention_workspace_size",
                          "paged_attention_shared_prefix"}
    for n in names:
        assert hasattr(lib, n), n


def _axis(values):
    return (ctypes.c_int32 * len(values))(*values)


def _mrope(lib, ptrs=None, axis=None, axes=3, qs=48 * 128, ks=48 * 128, vs=48 * 128, T=4, Hq=32,
           Hkv=8, D=128, r=128, rows=16, blocks=4, bs=16, style=0):
    p = ptrs or [A] * 10
    return lib.rope_write_kv_mrope(p[0], p[1], axis if axis is not None else _axis([0] * 128), axes,
                                   p[2], qs, p[3], ks, p[4], vs, p[5], p[6], p[7], p[8], p[9], T, Hq,
                                   Hkv, D, r, rows, blocks, bs, style, NUL)


def _quant(lib, ptrs=None, qs=48 * 128, ks=48 * 128, vs=48 * 128, T=4, Hq=32, Hkv=8, D=128, r=128,
           rows=16, blocks=4, bs=16, fmt=1, style=0):
    p = ptrs or [A] * 11
    return lib.rope_write_kv_slot_mapping_quant(p[0], p[1], p[2], qs, p[3], ks, p[4], vs, p[5], p[6],
                                                p[7], p[8], p[9], p[10], T, Hq, Hkv, D, r, rows,
                                                blocks, bs, fmt, style, NUL)


@pytest.mark.parametrize("call", [_mrope, _quant])
def test_writes_refuse_bad_sizes(lib, call):
    assert call(lib, style=2) == STYLE
    assert call(lib, D=96, r=96) == HEAD_DIM
    assert call(lib, r=24) == ROTARY_DIM and call(lib, D=64, r=80) == ROTARY_DIM
    assert call(lib, Hq=12) == HEADS and call(lib, Hkv=0) == HEADS
    assert call(lib, T=-1) == SHAPE and call(lib, blocks=-1) == SHAPE and call(lib, bs=0) == SHAPE
    assert call(lib, qs=100) == SHAPE and call(lib, ks=8 * 128 + 4) == SHAPE and call(lib, vs=0) == SHAPE
    assert call(lib, blocks=1 << 40, bs=(1 << 31) - 1) == SHAPE
    n = 10 if call is _mrope else 11
    for i in range(n):
        ptrs = [A] * n
        ptrs[i] = MIS
        assert call(lib, ptrs=ptrs) == MISALIGNED, i
        ptrs[i] = NUL
        if call is _quant or i < 9:     # k_out of the multi-axis call may be NULL
            assert call(lib, ptrs=ptrs) == NULL, i
    assert call(lib, T=0, ptrs=[NUL] * n) == OK


def test_mrope_refuses_bad_axes(lib):
    assert _mrope(lib, axes=0) == SHAPE and _mrope(lib, axes=5) == SHAPE
    bad = [0] * 64
    bad[63] = 3
    assert _mrope(lib, axis=_axis(bad)) == SHAPE
    bad[63] = -1
    assert _mrope(lib, axis=_axis(bad)) == SHAPE
    assert _mrope(lib, axis=NUL) == NULL


def test_quant_refuses_bad_formats(lib):
    for fmt in (-1, 0, 3):
        assert _quant(lib, fmt=fmt) == STYLE


def _read(lib, ptrs=None, N=16, B=4, Hkv=8, D=128, P=16, M=8, tpp=64, fmt=1):
    p = ptrs or [A] * 7
    return lib.paged_kv_read(*p, N, B, Hkv, D, P, M, tpp, fmt, NUL)


def test_read_refuses_bad_arguments(lib):
    assert _read(lib, fmt=3) == STYLE and _read(lib, fmt=-1) == STYLE
    assert _read(lib, D=80) == HEAD_DIM and _read(lib, Hkv=0) == HEADS
    for kw in (dict(N=-1), dict(B=-1), dict(P=-1), dict(M=-1), dict(tpp=0), dict(P=1 << 24, tpp=64)):
        assert _read(lib, **kw) == SHAPE, kw
    for i in range(7):
        ptrs = [A] * 7
        ptrs[i] = MIS
        assert _read(lib, ptrs=ptrs) == MISALIGNED
        ptrs[i] = NUL
        assert _read(lib, ptrs=ptrs) == NULL
    assert _read(lib, N=0, ptrs=[NUL] * 7) == OK and _read(lib, B=0) == OK


def _dims(**kw):
    d = dict(batch=4, seqLen=1, numQHeads=32, numKVHeads=8, headDim=128, numPages=64,
             tokensPerPage=64, maxPagesPerSeq=8, prefixLen=200, maxPrefixPages=4, cacheFormat=0)
    d.update(kw)
    return _serving.ropekv_attention_dims(**d)


def _attn(lib, ptrs=None, size=1 << 40, scale=0.1, **kw):
    p = ptrs or [A] * 9
    return lib.paged_attention_shared_prefix(*p, size, ctypes.byref(_dims(**kw)), scale, NUL)


def test_attention_refuses_bad_arguments(lib):
    assert _attn(lib, cacheFormat=3) == STYLE
    assert _attn(lib, headDim=96) == HEAD_DIM
    assert _attn(lib, numQHeads=30) == HEADS and _attn(lib, numKVHeads=0) == HEADS
    for kw in (dict(batch=-1), dict(seqLen=-1), dict(seqLen=40000), dict(numPages=-1),
               dict(tokensPerPage=0), dict(maxPagesPerSeq=-1), dict(prefixLen=-1),
               dict(prefixLen=257), dict(maxPrefixPages=-1), dict(numPages=1 << 24),
               dict(maxPagesPerSeq=1 << 25), dict(batch=1 << 20, seqLen=1 << 10)):
        assert _attn(lib, **kw) == SHAPE, kw
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert _attn(lib, scale=bad) == SHAPE
    for i in range(9):
        ptrs = [A] * 9
        ptrs[i] = MIS
        assert _attn(lib, ptrs=ptrs, cacheFormat=1) == MISALIGNED, i
        ptrs[i] = NUL
        if i != 7:                      # lse may be NULL
            assert _attn(lib, ptrs=ptrs, cacheFormat=1) == NULL, i
    assert _attn(lib, size=lib.paged_attention_workspace_size(ctypes.byref(_dims())) - 1) == CAPACITY
    assert _attn(lib, batch=0, ptrs=[NUL] * 9, size=0) == OK
    assert lib.paged_attention_shared_prefix(*[A] * 9, 0, None, 0.1, NUL) == NULL


def test_workspace_size(lib):
    size = lib.paged_attention_workspace_size
    assert size(ctypes.byref(_dims(batch=0))) == 0 and size(ctypes.byref(_dims(seqLen=0))) == 0
    assert size(ctypes.byref(_dims())) >= 4 * 32 * 128 * 4
    assert size(ctypes.byref(_dims(headDim=32))) == HEAD_DIM
    assert size(None) == NULL


def test_freq_axis():
    f = rk.mrope_freq_axis
    assert f([2, 1, 1]).tolist() == [0, 0, 1, 2]
    assert f([4, 2, 2], interleaved=True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert f([16], interleaved=True).tolist() == [0] * 16
    for bad in ([], [1] * 5, [3, -1]):
        with pytest.raises(ValueError):
            f(bad)
    with pytest.raises(ValueError):
        f([0, 4, 4], interleaved=True)


def test_binding_refuses_cpu_tensors_types_and_shapes():
    build.build_library()
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)
    cs, q, k, cache = torch.zeros(16, 64), h(3, 4, 64), h(3, 2, 64), h(2, 16, 2, 64)
    axis = rk.mrope_freq_axis([16, 8, 8])
    with pytest.raises(ValueError, match="CUDA"):
        rk.rope_write_kv_mrope(cs, i64(3, 3), axis, q, k, k, i64(3), cache, cache.clone(), h(3, 4, 64))
    with pytest.raises(ValueError, match="freq_axis"):
        rk.rope_write_kv_mrope(cs, i64(3, 3), axis[:-1], q, k, k, i64(3), cache, cache.clone(), h(3, 4, 64))
    with pytest.raises(ValueError, match="inconsistent"):
        rk.rope_write_kv_mrope(cs, i64(3, 4), axis, q, k, k, i64(3), cache, cache.clone(), h(3, 4, 64))
    c8, s8 = torch.zeros(2, 16, 2, 64, dtype=torch.int8), torch.zeros(2, 2, 16)
    with pytest.raises(TypeError, match="key_cache"):
        rk.rope_write_kv_slot_mapping_quant(cs, i64(3), q, k, k, i64(3), cache, cache, s8, s8, h(3, 4, 64))
    with pytest.raises(ValueError, match="key_scales"):
        rk.rope_write_kv_slot_mapping_quant(cs, i64(3), q, k, k, i64(3), c8, c8, s8[:1], s8, h(3, 4, 64))
    pool, tab = h(2, 4, 16, 2, 64), i32(3, 2, 2)
    with pytest.raises(ValueError, match="kv_scales"):
        rk.paged_kv_read(pool.to(torch.int8), tab, i32(5), i32(5), h(5, 2, 64), h(5, 2, 64))
    with pytest.raises(ValueError, match="no kv_scales"):
        rk.paged_kv_read(pool, tab, i32(5), i32(5), h(5, 2, 64), h(5, 2, 64), kv_scales=torch.zeros(2, 4, 2, 16))
    with pytest.raises(ValueError, match="row_positions"):
        rk.paged_kv_read(pool, tab, i32(5), i32(4), h(5, 2, 64), h(5, 2, 64))
    att = lambda **kw: rk.paged_attention_shared_prefix(
        kw.get("q", h(3, 1, 4, 64)), kw.get("pool", pool), i32(2, 1), kw.get("P", 16), kw.get("tab", tab),
        kw.get("lens", i32(3)), kw.get("out", h(3, 1, 4, 64)), lse=kw.get("lse"))
    for kw in (dict(), dict(lens=i32(2)), dict(out=h(3, 1, 2, 64)), dict(lse=torch.zeros(3, 4)),
               dict(q=h(2, 1, 4, 64)), dict(tab=i32(3, 1, 2))):
        with pytest.raises(ValueError):
            att(**kw)
    with pytest.raises(TypeError):
        att(pool=pool.float())
