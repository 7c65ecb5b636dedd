"""GPU results of the multi-axis write, the 8-bit write and the paged read
against plain 64-bit implementations, with bounds derived from the roundings
each kernel makes."""
import numpy as np
import pytest

import serving_plain as sp
from serving_plain import E4M3, F16, GPTJ, INT8, NEOX

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
SENT = 0x7E5A      # an FP16 NaN that no result has


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def sentinel(shape):
    return torch.full(shape, SENT, dtype=torch.int16, device=DEV).view(torch.float16)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def make(seed, T, Hq, Hkv, D, bs, strided):
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float16)
    t = dev(x)
    q, k, v = t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    blocks = -(-T // bs) + 3
    slots = rng.permutation(blocks * bs)[:T].astype(np.int64)
    return rng, x, (q, k, v), blocks, slots


WRITES = [
    # T, Hq, Hkv, D, r, style, block size, strided
    (1, 1, 1, 64, 64, NEOX, 16, False),
    (7, 4, 2, 64, 32, GPTJ, 1, True),
    (37, 8, 2, 128, 128, NEOX, 64, True),
    (130, 6, 3, 128, 64, GPTJ, 5, False),
    (23, 8, 8, 256, 256, NEOX, 32, True),
    (11, 5, 1, 256, 48, GPTJ, 7, False),
    (1025, 32, 8, 128, 128, NEOX, 64, True),
    (1100, 10, 2, 64, 16, NEOX, 16, True),
]


# ------------------------------------------------------------- multi-axis --

def axis_maps(r):
    import rope_kv_cache_gb300 as rk
    n = r // 2
    rest = n * 3 // 8
    sec = [n - 2 * rest, rest, rest]
    inter = [n - 2 * (n // 3), n // 3, n // 3]
    rng = np.random.Generator(np.random.PCG64(r))
    return {"one": (1, torch.zeros(n, dtype=torch.int32)),
            "chunked": (3, rk.mrope_freq_axis(sec)),
            "interleaved": (3, rk.mrope_freq_axis(inter, interleaved=True)),
            "four": (4, torch.from_numpy(rng.integers(0, 4, n).astype(np.int32)))}


@pytest.mark.parametrize("kind", ["one", "chunked", "interleaved", "four"])
@pytest.mark.parametrize("idx", range(len(WRITES)))
def test_mrope(idx, kind):
    import rope_kv_cache_gb300 as rk
    T, Hq, Hkv, D, r, style, bs, strided = WRITES[idx]
    rng, x, (q, k, v), blocks, slots = make(100 + idx, T, Hq, Hkv, D, bs, strided)
    axes, freq = axis_maps(r)[kind]
    rows = 97
    tab = sp.table(rows, r)
    pos = rng.integers(0, rows, (axes, T))
    pos[:, ::3] = pos[:1, ::3]                  # every third token agrees on all axes (text)
    skip = np.zeros(T, bool)
    if T > 5:
        pos[0, 2], pos[axes - 1, 4] = rows, -1   # past the table, negative: skipped whole
        skip[[2, 4]] = True
        slots[3], slots[5] = -1, blocks * bs     # no cache write, Q still rotated
    kc, vc, qo, ko = sentinel((blocks, bs, Hkv, D)), sentinel((blocks, bs, Hkv, D)), \
        sentinel((T, Hq, D)), sentinel((T, Hkv, D))
    rk.rope_write_kv_mrope(dev(tab), dev(pos), freq, q, k, v, dev(slots), kc, vc, qo,
                           k_out=ko if idx % 2 else None, style=style)
    torch.cuda.synchronize()
    f, h = freq.numpy(), np.arange(r // 2)
    p = np.clip(pos, 0, rows - 1)[f].T           # [T, r/2]
    cos, sin = tab[p, h].astype(np.float64), tab[p, h + r // 2].astype(np.float64)
    xd = x.astype(np.float64)
    yq, mq = sp.rotate(xd[:, :Hq], cos, sin, r, style)
    yk, mk = sp.rotate(xd[:, Hq:Hq + Hkv], cos, sin, r, style)
    live = ~skip
    stored = live & (slots >= 0) & (slots < blocks * bs)
    qb = bits(qo)
    assert (qb[skip] == SENT).all()
    sp.check_f16(qb.view(np.float16)[live], yq[live], mq[live], "q_out")
    want_v = np.full((blocks * bs, Hkv, D), SENT, np.uint16)
    want_v[slots[stored]] = x[stored, Hq + Hkv:].view(np.uint16)
    assert np.array_equal(bits(vc).reshape(want_v.shape), want_v)
    kb = bits(kc).reshape(blocks * bs, Hkv, D)
    untouched = np.ones(blocks * bs, bool)
    untouched[slots[stored]] = False
    assert (kb[untouched] == SENT).all()
    sp.check_f16(kb[slots[stored]].view(np.float16), yk[stored], mk[stored], "key cache")
    assert np.array_equal(kb[slots[stored]][..., r:],
                          x[stored, Hq:Hq + Hkv, r:].view(np.uint16))     # past r: bits
    kob = bits(ko)
    if idx % 2:
        assert np.array_equal(kob[stored], kb[slots[stored]]) and (kob[~stored] == SENT).all()
    else:
        assert (kob == SENT).all()


def test_mrope_equal_axes_is_the_slot_mapping_call():
    """A token whose positions agree on all axes gets exactly what the one-axis call writes,
    whatever the frequencies' axes."""
    import rope_kv_cache_gb300 as rk
    for T, D, r, style in ((300, 128, 128, NEOX), (1500, 64, 48, GPTJ)):
        rng, x, (q, k, v), blocks, slots = make(7, T, 8, 2, D, 16, True)
        tab, pos = dev(sp.table(200, r)), rng.integers(0, 200, T)
        out = []
        for kind in ("plain", "four"):
            kc, vc, qo = sentinel((blocks, 16, 2, D)), sentinel((blocks, 16, 2, D)), sentinel((T, 8, D))
            if kind == "plain":
                rk.rope_write_kv_slot_mapping(tab, dev(pos), q, k, v, dev(slots), kc, vc, qo, style=style)
            else:
                rk.rope_write_kv_mrope(tab, dev(np.stack([pos] * 4)), axis_maps(r)[kind][1], q, k, v,
                                       dev(slots), kc, vc, qo, style=style)
            out.append((bits(kc), bits(vc), bits(qo)))
        for a, b in zip(*out):
            assert np.array_equal(a, b)


# ------------------------------------------------------------ 8-bit write --

def empty8(fmt, shape):
    t = torch.full(shape, 0x55, dtype=torch.uint8, device=DEV)
    return t.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8)


def quantise(fmt, shape, x=None, seed=0, tab=None, bad=True):
    import rope_kv_cache_gb300 as rk
    T, Hq, Hkv, D, r, style, bs, strided = shape
    rng, x0, (q, k, v), blocks, slots = make(seed, T, Hq, Hkv, D, bs, strided)
    if x is not None:
        x0, t = x, dev(x)
        q, k, v = t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]
    tab = sp.table(61, r) if tab is None else tab
    pos = rng.integers(0, len(tab), T)
    skip = np.zeros(T, bool)
    if T > 5 and bad:
        pos[2], pos[4] = len(tab), -5
        skip[[2, 4]] = True
        slots[3], slots[5] = -1, blocks * bs
    kc, vc = empty8(fmt, (blocks, bs, Hkv, D)), empty8(fmt, (blocks, bs, Hkv, D))
    ks = torch.full((blocks, Hkv, bs), -3.0, device=DEV)
    vs = torch.full((blocks, Hkv, bs), -3.0, device=DEV)
    qo = sentinel((T, Hq, D))
    rk.rope_write_kv_slot_mapping_quant(dev(tab), dev(pos), q, k, v, dev(slots), kc, vc, ks, vs, qo,
                                        style=style)
    torch.cuda.synchronize()
    p = np.clip(pos, 0, len(tab) - 1)
    cos, sin = tab[p, :r // 2].astype(np.float64), tab[p, r // 2:].astype(np.float64)
    stored = ~skip & (slots >= 0) & (slots < blocks * bs)
    flat = lambda c: c.view(torch.uint8).cpu().numpy().reshape(blocks * bs, Hkv, D)
    scal = lambda s: s.cpu().numpy().transpose(0, 2, 1).reshape(blocks * bs, Hkv)
    return dict(x=x0, cos=cos, sin=sin, slots=slots, stored=stored, skip=skip, codes=(flat(kc), flat(vc)),
                scales=(scal(ks), scal(vs)), q=bits(qo))


def check_quant(fmt, res, Hq, Hkv, r, style):
    xd = res["x"].astype(np.float64)
    yk, mk = sp.rotate(xd[:, Hq:Hq + Hkv], res["cos"], res["sin"], r, style)
    yv = xd[:, Hq + Hkv:]
    st, sl = res["stored"], res["slots"]
    rest = np.ones(len(res["codes"][0]), bool)
    rest[sl[st]] = False
    for codes, scales, y, mag in zip(res["codes"], res["scales"], (yk, yv), (mk, np.zeros_like(yv))):
        assert (codes[rest] == 0x55).all() and (scales[rest] == -3.0).all()
        y, mag, s = y[st], mag[st], scales[sl[st]].astype(np.float64)
        fp32 = 3 * 2.0 ** -24 * mag                        # the rotated value in FP32
        amax = np.abs(y).max(-1)
        # the scale: an FP32 maximum, one FP32 division
        assert (np.abs(s - amax / sp.MAXCODE[fmt]) <= (2.0 ** -23 * amax + 1.01 * fp32.max(-1)) / sp.MAXCODE[fmt]).all()
        u = sp.decode(codes[sl[st]].view(np.int8) if fmt == INT8 else codes[sl[st]], fmt)
        want = y / np.where(s > 0, s, 1)[..., None]
        # the code: half a step, and what FP32 may move the value across a border
        # (a product with M / amax: three roundings, 2^-22 of the value)
        slack = 1.01 * fp32 / np.where(s > 0, s, 1)[..., None] + 2.0 ** -21 * np.abs(want)
        step = 0.5 if fmt == INT8 else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
        assert np.isfinite(u).all()
        assert (np.abs(u - want) <= step + slack).all(), float((np.abs(u - want) - step - slack).max())
        assert (np.abs(u).max(-1)[amax > 0] == sp.MAXCODE[fmt]).all()   # the largest takes the last code


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("idx", range(len(WRITES)))
def test_quant_write(idx, fmt):
    T, Hq, Hkv, D, r, style, bs, strided = WRITES[idx]
    res = quantise(fmt, WRITES[idx], seed=200 + idx)
    check_quant(fmt, res, Hq, Hkv, r, style)
    yq, mq = sp.rotate(res["x"][:, :Hq].astype(np.float64), res["cos"], res["sin"], r, style)
    live = ~res["skip"]
    assert (res["q"][res["skip"]] == SENT).all()
    sp.check_f16(res["q"].view(np.float16)[live], yq[live], mq[live], "q_out")


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_quant_extremes(fmt):
    """Zero heads, subnormal heads, the largest FP16 values, infinities and NaN."""
    T, Hq, Hkv, D, r, style, bs = 9, 2, 2, 64, 32, NEOX, 4
    shape = (T, Hq, Hkv, D, r, style, bs, True)
    rng = np.random.Generator(np.random.PCG64(3))
    x = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float16)
    x[0, Hq:] = 0
    x[1, Hq:] = 2.0 ** -24 * rng.integers(-3, 4, (2 * Hkv, D))
    x[1, Hq:, 0] = 2.0 ** -24
    x[2, Hq:] = 65504.0 * np.sign(rng.standard_normal((2 * Hkv, D)))
    x[3, Hq:] = -0.0
    x[6, Hq, 40], x[6, Hq + 2, 1] = np.inf, -np.inf
    x[7, Hq + 1, 3], x[7, Hq + 3, 60] = np.nan, np.nan
    tiny = sp.table(61, r) * np.float32(2.0 ** -90)
    for tab in (None, tiny):
        res = quantise(fmt, shape, x=x, seed=5, tab=tab, bad=False)
        sl = res["slots"]
        bad = {(6, 0, 0), (6, 1, 0), (7, 0, 1), (7, 1, 1)}
        for t in range(T):
            for plane in (0, 1):
                for h in range(Hkv):
                    code, s = res["codes"][plane][sl[t], h], res["scales"][plane][sl[t], h]
                    if (t, plane, h) in bad:
                        assert np.isnan(s) and (code == 0).all(), (t, plane, h)
                    else:
                        assert np.isfinite(s) and s >= 0
                        if t in (0, 3):
                            assert s == 0 and not sp.decode(code.view(np.int8) if fmt == INT8 else code, fmt).any()
        if tab is None:
            ok = [t for t in range(T) if t not in (6, 7)]
            sub = {n: res[n][ok] for n in ("x", "cos", "sin", "slots", "stored", "skip")}
            keep = np.zeros(len(res["codes"][0]), bool)
            keep[sl[ok]] = True
            codes = tuple(np.where(keep[:, None, None], c, 0x55).astype(np.uint8) for c in res["codes"])
            scales = tuple(np.where(keep[:, None], s, np.float32(-3)) for s in res["scales"])
            check_quant(fmt, dict(sub, codes=codes, scales=scales), Hq, Hkv, r, style)


# ------------------------------------------------------------------ read --

READS = [
    # N, B, Hkv, D, tpp
    (1, 1, 1, 64, 1),
    (77, 3, 2, 64, 16),
    (300, 5, 3, 128, 7),
    (515, 9, 8, 128, 64),
    (100, 2, 1, 256, 100),
    (4097, 13, 5, 64, 32),
]


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("idx", range(len(READS)))
def test_read(idx, fmt):
    import rope_kv_cache_gb300 as rk
    N, B, Hkv, D, tpp = READS[idx]
    rng = np.random.Generator(np.random.PCG64(300 + idx))
    M = -(-(N // B + 9) // tpp)
    pages = B * M + 3
    tab = np.stack([rng.permutation(pages)[:B * M].reshape(B, M),
                    rng.permutation(pages)[:B * M].reshape(B, M) + pages], 1).astype(np.int32)
    if N > 50:
        tab[0, 0, 0], tab[1, 1, M - 1] = -1, pages - 1          # unmapped K; a K id in the V plane
        tab[1, 0, 0], tab[0, 1, M - 1] = pages, 2 * pages       # a V id in the K plane; past the pool
    seq = rng.integers(0, B, N).astype(np.int32)
    pos = rng.integers(0, M * tpp, N).astype(np.int32)
    if N > 50:
        pos[[3, 5]], seq[[7, 9]], pos[11] = (-1, M * tpp), (-1, B), 2 ** 31 - 1
    raw = rng.integers(0, 256, (2, pages, tpp, Hkv, D * (2 if fmt == F16 else 1))).astype(np.uint8)
    scales = None
    if fmt == F16:
        pool = raw.view(np.float16)
        pt = dev(pool)
    else:
        pool = raw.view(np.int8) if fmt == INT8 else raw
        pt = dev(pool) if fmt == INT8 else dev(raw).view(torch.float8_e4m3fn)
        scales = (2.0 ** rng.uniform(-30, 12, (2, pages, Hkv, tpp))).astype(np.float32)
        scales[0, 0, 0, 0] = np.nan
    ko, vo = sentinel((N, Hkv, D)), sentinel((N, Hkv, D))
    rk.paged_kv_read(pt, dev(tab), dev(pos), dev(seq), ko, vo,
                     kv_scales=None if scales is None else dev(scales))
    torch.cuda.synchronize()
    for plane, got in ((0, bits(ko)), (1, bits(vo))):
        want = np.full((N, Hkv, D), SENT, np.uint16)
        for t in range(N):
            if pos[t] < 0 or not 0 <= seq[t] < B or pos[t] // tpp >= M:
                continue
            i = int(tab[seq[t], plane, pos[t] // tpp]) - plane * pages
            if not 0 <= i < pages:
                continue
            row = pool[plane, i, pos[t] % tpp]
            if fmt == F16:
                want[t] = row.view(np.uint16)
            else:
                # code and scale are exact in FP32, their product is rounded there and once to FP16
                with np.errstate(over="ignore", invalid="ignore"):
                    want[t] = (sp.decode(row, fmt).astype(np.float32) * scales[plane, i, :, pos[t] % tpp][:, None]) \
                        .astype(np.float16).view(np.uint16)
        nan = np.isnan(want.view(np.float16)) & (want != SENT)
        assert fmt == F16 or np.isnan(got.view(np.float16)[nan]).all()
        keep = np.ones_like(nan) if fmt == F16 else ~nan
        assert np.array_equal(got[keep], want[keep]), plane


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_write_then_read(fmt):
    """The two as they are used: what the write stored comes back through the page table,
    each element within half a code step of the FP16 row."""
    import rope_kv_cache_gb300 as rk
    T, Hq, Hkv, D, r, bs = 333, 8, 2, 128, 64, 16
    rng, x, (q, k, v), blocks, _ = make(11, T, Hq, Hkv, D, bs, True)
    perm = rng.permutation(blocks)
    p = np.arange(T)
    slots = perm[p // bs] * bs + p % bs
    pool = torch.zeros(2, blocks, bs, Hkv, D, dtype=torch.uint8, device=DEV).view(
        torch.float8_e4m3fn if fmt == E4M3 else torch.int8)
    scales = torch.zeros(2, blocks, Hkv, bs, device=DEV)
    tab = sp.table(T, r)
    rk.rope_write_kv_slot_mapping_quant(dev(tab), dev(p), q, k, v, dev(slots), pool[0], pool[1],
                                        scales[0], scales[1], sentinel((T, Hq, D)), style=GPTJ)
    table = np.stack([perm, perm + blocks])[None].astype(np.int32)
    ko, vo = sentinel((T, Hkv, D)), sentinel((T, Hkv, D))
    rk.paged_kv_read(pool, dev(table), dev(p.astype(np.int32)), dev(np.zeros(T, np.int32)), ko, vo,
                     kv_scales=scales)
    torch.cuda.synchronize()
    xd = x.astype(np.float64)
    yk, _ = sp.rotate(xd[:, Hq:Hq + Hkv], tab[:, :r // 2].astype(np.float64),
                      tab[:, r // 2:].astype(np.float64), r, GPTJ)
    for got, y in ((ko, yk), (vo, xd[:, Hq + Hkv:])):
        s = np.abs(y).max(-1, keepdims=True) / sp.MAXCODE[fmt]
        step = 0.5 * s if fmt == INT8 else np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s)
        # half a code step, one FP16 rounding of a value that may lie that much higher, FP32 slack
        tol = step * (1 + 2.0 ** -10) + 2.0 ** -11 * np.abs(y) + 2.0 ** -20 * s * 448
        assert (np.abs(got.cpu().numpy().astype(np.float64) - y) <= tol).all()


def test_other_stream_and_graph():
    """The calls run on the given stream and replay from a graph with new inputs."""
    import rope_kv_cache_gb300 as rk
    T, Hq, Hkv, D, r, bs = 40, 4, 2, 64, 64, 16
    rng, x, (q, k, v), blocks, slots = make(21, T, Hq, Hkv, D, bs, False)
    tab, pos, sl = dev(sp.table(64, r)), dev(rng.integers(0, 64, T)), dev(slots)
    kc, vc = empty8(INT8, (blocks, bs, Hkv, D)), empty8(INT8, (blocks, bs, Hkv, D))
    ks, vs = torch.zeros(blocks, Hkv, bs, device=DEV), torch.zeros(blocks, Hkv, bs, device=DEV)
    qo = sentinel((T, Hq, D))

    def call(**kw):
        rk.rope_write_kv_slot_mapping_quant(tab, pos, q, k, v, sl, kc, vc, ks, vs, qo, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    first = (kc.clone(), ks.clone(), bits(qo))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    k2 = k * 2
    k.copy_(k2)
    g.replay()
    torch.cuda.synchronize()
    # twice the values: the same codes, twice the scale (both exact)
    stored = sorted(slots)
    assert torch.equal(kc.view(-1, Hkv, D)[stored], first[0].view(-1, Hkv, D)[stored])
    assert torch.equal(ks, first[1] * 2) and np.array_equal(bits(qo), first[2])
